// state_pool.cuh -- serving kernels over a pool of recurrent states
// [slots, H, d, e] (fp32): the gated delta rule's step for one token per
// sequence, and the copies that fork, move and clear slots.
#pragma once
#include "gdr_common.cuh"

namespace la2 {
namespace gdr {

constexpr int kStepThreads = 256;
constexpr int kStepRows = 16;  // rows of the state per thread, at most

// One token of row b, head h (gdr_common.cuh).  Both products with the old
// state, S^T k and S^T q, are taken in one pass while the state sits in
// registers; since S' = a S + k u^T, the output needs no second one:
//
//   u = beta (v - a S^T k),   o = a S^T q + (k . q) u,   S' = a S + k u^T.
//
// The state is read and written once (2 d e words of a few flops each: bound
// by memory bandwidth).  A CTA takes one (row, head) and up to 32 W columns
// (W = 4: 16-byte loads, e % 4 == 0; W = 1 otherwise); the threads of a group
// of cu hold one row's columns, the groups take rows in turn.
//
// slots[b] outside 0 .. n_slots - 1, or listed for an earlier row already:
// the row's output is zero and no state changes.
template <typename Tin, int W>
__global__ void __launch_bounds__(kStepThreads)
gdr_step(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
         const float* __restrict__ g, const float* __restrict__ beta, float* state,
         const int* __restrict__ slots, int n_slots, float* __restrict__ out, int Hk, int H, int d, int e) {
    __shared__ float ks[128], qs[128];
    __shared__ float part[2][kStepThreads * W];
    const int n = blockIdx.x, b = n / H, h = n % H, tid = threadIdx.x;
    const int col0 = blockIdx.y * 32 * W;
    const int cu = min(32, (e - col0) / W);  // column units of this CTA
    const int groups = kStepThreads / cu, rg = tid / cu, col = col0 + tid % cu * W;
    const int slot = slots ? slots[b] : b;
    bool live = slot >= 0 && slot < n_slots;
    float* S = state + ((static_cast<size_t>(live ? slot : 0)) * H + h) * d * e;
    float sv[kStepRows][W];
    if (live) {
#pragma unroll
        for (int r = 0; r < kStepRows; ++r) {
            const int i = rg + r * groups;
#pragma unroll
            for (int w = 0; w < W; ++w) sv[r][w] = 0.f;
            if (rg < groups && i < d) {
                const float* row = S + static_cast<size_t>(i) * e + col;
                if constexpr (W == 4) {
                    const float4 x = *reinterpret_cast<const float4*>(row);
                    sv[r][0] = x.x; sv[r][1] = x.y; sv[r][2] = x.z; sv[r][3] = x.w;
                } else {
                    sv[r][0] = row[0];
                }
            }
        }
    }
    const int hk = h / (H / Hk);
    if (tid < d) {
        const size_t at = (static_cast<size_t>(b) * Hk + hk) * d + tid;
        ks[tid] = to_float(k[at]);
        qs[tid] = to_float(q[at]);
    }
    int twice = 0;
    if (slots)
        for (int x = tid; x < b; x += kStepThreads) twice |= slots[x] == slot;
    live = !__syncthreads_or(twice) && live;
    float* on = out + static_cast<size_t>(n) * e;
    if (!live) {
        if (rg == 0)
#pragma unroll
            for (int w = 0; w < W; ++w) on[col + w] = 0.f;
        return;
    }
    const float a = g ? expf(g[n]) : 1.f, bt = beta[n];
    float pk[W], pq[W];
#pragma unroll
    for (int w = 0; w < W; ++w) pk[w] = pq[w] = 0.f;
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int i = rg + r * groups;
        if (rg < groups && i < d) {
            const float ki = ks[i], qi = qs[i];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                pk[w] = fmaf(sv[r][w], ki, pk[w]);
                pq[w] = fmaf(sv[r][w], qi, pq[w]);
            }
        }
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
        part[0][tid * W + w] = pk[w];
        part[1][tid * W + w] = pq[w];
    }
    float kq = 0.f;
    for (int i = tid & 31; i < d; i += 32) kq = fmaf(ks[i], qs[i], kq);
    for (int m = 16; m; m >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, m);
    __syncthreads();
    float u[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        float sk = 0.f, sq = 0.f;
        if (rg < groups)
            for (int y = 0; y < groups; ++y) {
                sk += part[0][(y * cu + tid % cu) * W + w];
                if (rg == 0) sq += part[1][(y * cu + tid % cu) * W + w];
            }
        const float vv = rg < groups ? to_float(v[static_cast<size_t>(n) * e + col + w]) : 0.f;
        u[w] = bt * (vv - a * sk);
        if (rg == 0) on[col + w] = fmaf(a, sq, kq * u[w]);
    }
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int i = rg + r * groups;
        if (rg < groups && i < d) {
            float* row = S + static_cast<size_t>(i) * e + col;
            const float ki = ks[i];
#pragma unroll
            for (int w = 0; w < W; ++w) sv[r][w] = fmaf(a, sv[r][w], ki * u[w]);
            if constexpr (W == 4) *reinterpret_cast<float4*>(row) = make_float4(sv[r][0], sv[r][1], sv[r][2], sv[r][3]);
            else row[0] = sv[r][0];
        }
    }
}

// Pool copies: for every pair i, slot dst[i] takes what slot src[i] held BEFORE
// the call (src[i] < 0: zeros); pairs that name a slot outside the pool do
// nothing; where a slot is the destination of several pairs the last one
// counts.  Sources may be destinations of other pairs, so a CTA reads its
// slice of every source into shared memory before it writes any: slices of
// different CTAs never meet, and no order between CTAs is needed.  Each place
// of a destination is written by one thread, in the pairs' order (all pairs of
// one slot have the same dst % writers).
constexpr int kPoolThreads = 256;
constexpr int kPoolMaxPairs = 4096;

// V: float4, or float where the page or the pool's address asks for it.
// `units` V's of a page per slice, a power of two of at most kPoolThreads.
template <typename V>
__global__ void __launch_bounds__(kPoolThreads)
pool_copy(V* pool, const int* __restrict__ src, const int* __restrict__ dst, int n,
          int n_slots, long long page, int units) {
    extern __shared__ unsigned char pool_raw[];
    V* buf = reinterpret_cast<V*>(pool_raw);                              // [n][units]
    int* ss = reinterpret_cast<int*>(buf + static_cast<size_t>(n) * units);  // [n]
    int* dd = ss + n;
    const int tid = threadIdx.x, u = tid % units, w = tid / units, writers = kPoolThreads / units;
    for (int i = tid; i < n; i += kPoolThreads) {
        ss[i] = src[i];
        dd[i] = dst[i];
    }
    __syncthreads();
    const long long at = static_cast<long long>(blockIdx.x) * units + u;
    const bool on = at < page;
    if (on) {
#pragma unroll 8
        for (int i = w; i < n; i += writers) {
            const int s = ss[i];
            V x{};
            if (s >= 0 && s < n_slots) x = pool[s * page + at];
            buf[i * units + u] = x;
        }
    }
    __syncthreads();
    if (on) {
        for (int i = 0; i < n; ++i) {
            const int t = dd[i];
            if (t >= 0 && t < n_slots && ss[i] < n_slots && t % writers == w) pool[t * page + at] = buf[i * units + u];
        }
    }
}

}  // namespace gdr
}  // namespace la2
