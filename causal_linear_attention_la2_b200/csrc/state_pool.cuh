// state_pool.cuh -- serving kernels over a pool of recurrent states
// [slots, H, d, e] (fp32): the gated delta rule's step for one token per
// sequence, and the copies that fork, move and clear slots.
#pragma once
#include "gdr_common.cuh"

namespace la2 {
namespace gdr {

constexpr int kStepThreads = 256;
constexpr int kStepUnits = 8;             // column units of a CTA
constexpr int kStepRows = 128 / 32;       // rows of the state per thread, at most

// One token of row b, head h (gdr_common.cuh).  Both products with the old
// state, S^T k and S^T q, are taken in one pass while the state sits in
// registers; since S' = a S + k u^T, the output needs no second one:
//
//   u = beta (v - a S^T k),   o = a S^T q + (k . q) u,   S' = a S + k u^T.
//
// The state is read and written once (2 d e words of a few flops each: bound by
// memory bandwidth), so what counts is how much of it is on its way: a CTA takes
// eight column units (W = 4 floats, 16-byte loads, where e % 4 == 0; W = 1
// otherwise) of one (row, head) with four rows per thread at d = 128, and eight
// CTAs share an SM.  64 x 40 states of 128 x 128: 116 us with whole states of 256
// threads (154 registers, one CTA per SM), 85 us with 512 threads.
//
// slots[b] outside 0 .. n_slots - 1, or listed for an earlier row already:
// the row's output is zero and no state changes.
template <typename Tin, int W>
__global__ void __launch_bounds__(kStepThreads)
gdr_step(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
         const float* __restrict__ g, const float* __restrict__ beta, float* state,
         const int* __restrict__ slots, int n_slots, float* __restrict__ out, int Hk, int H, int d, int e) {
    constexpr int kWarps = kStepThreads / 32;
    __shared__ float ks[128], qs[128];
    __shared__ __align__(16) float part[2][kWarps][kStepUnits * W];
    const int n = blockIdx.x, b = n / H, h = n % H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cl = lane % kStepUnits, col = (blockIdx.y * kStepUnits + cl) * W;
    const int i0 = 4 * warp + lane / kStepUnits;  // rows i0, i0 + 32, ..
    const bool on = col < e;
    const int slot = slots ? slots[b] : b;
    bool live = slot >= 0 && slot < n_slots;
    float* S = state + ((static_cast<size_t>(live ? slot : 0)) * H + h) * d * e + col;
    float sv[kStepRows][W];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int i = i0 + 32 * r;
#pragma unroll
        for (int w = 0; w < W; ++w) sv[r][w] = 0.f;
        if (live && on && i < d) {
            const float* row = S + static_cast<size_t>(i) * e;
            if constexpr (W == 4) {
                const float4 x = *reinterpret_cast<const float4*>(row);
                sv[r][0] = x.x; sv[r][1] = x.y; sv[r][2] = x.z; sv[r][3] = x.w;
            } else {
                sv[r][0] = row[0];
            }
        }
    }
    if (tid < d) {
        const size_t at = (static_cast<size_t>(b) * Hk + h / (H / Hk)) * d + tid;
        ks[tid] = to_float(k[at]);
        qs[tid] = to_float(q[at]);
    }
    const float a = g ? expf(g[n]) : 1.f, bt = beta[n];
    float vv[W];
#pragma unroll
    for (int w = 0; w < W; ++w) vv[w] = on ? to_float(v[static_cast<size_t>(n) * e + col + w]) : 0.f;
    int twice = 0;
    if (slots)
        for (int x = tid; x < b; x += kStepThreads) twice |= slots[x] == slot;
    live = !__syncthreads_or(twice) && live;
    float* to = out + static_cast<size_t>(n) * e + col;
    if (!live) {
        if (on && tid < kStepUnits)
#pragma unroll
            for (int w = 0; w < W; ++w) to[w] = 0.f;
        return;
    }
    float pk[W], pq[W], ki[kStepRows], kq = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) pk[w] = pq[w] = 0.f;
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int i = i0 + 32 * r;
        const float qi = i < d ? qs[i] : 0.f;
        ki[r] = i < d ? ks[i] : 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            pk[w] = fmaf(sv[r][w], ki[r], pk[w]);
            pq[w] = fmaf(sv[r][w], qi, pq[w]);
        }
    }
    for (int i = lane; i < d; i += 32) kq = fmaf(ks[i], qs[i], kq);
#pragma unroll
    for (int m = 16; m; m >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, m);
#pragma unroll
    for (int m = kStepUnits; m < 32; m <<= 1)
#pragma unroll
        for (int w = 0; w < W; ++w) {
            pk[w] += __shfl_xor_sync(0xffffffffu, pk[w], m);
            pq[w] += __shfl_xor_sync(0xffffffffu, pq[w], m);
        }
    if (lane < kStepUnits)
#pragma unroll
        for (int w = 0; w < W; ++w) {
            part[0][warp][cl * W + w] = pk[w];
            part[1][warp][cl * W + w] = pq[w];
        }
    __syncthreads();
    float u[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int y = 0; y < kWarps; ++y) {
            sk += part[0][y][cl * W + w];
            if (tid < kStepUnits) sq += part[1][y][cl * W + w];
        }
        u[w] = bt * (vv[w] - a * sk);
        if (on && tid < kStepUnits) to[w] = fmaf(a, sq, kq * u[w]);
    }
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int i = i0 + 32 * r;
        if (on && i < d) {
            float* row = S + static_cast<size_t>(i) * e;
#pragma unroll
            for (int w = 0; w < W; ++w) sv[r][w] = fmaf(a, sv[r][w], ki[r] * u[w]);
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
// different CTAs never meet, and no order between CTAs is needed.  Which pair is
// the last one of its destination a table of the slots says (pools of up to
// kPoolTable slots); in larger pools each place of a destination is written by one
// thread, in the pairs' order (all pairs of one slot have the same remainder by
// the number of writers, a power of two).
constexpr int kPoolThreads = 256;
constexpr int kPoolMaxPairs = 4096, kPoolTable = 4096;

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
    int* last = dd + n;  // [n_slots], where the pool is small enough
    const bool table = n_slots <= kPoolTable;
    const int tid = threadIdx.x, u = tid % units, w = tid / units, writers = kPoolThreads / units;
    for (int i = tid; i < n; i += kPoolThreads) {
        ss[i] = src[i];
        dd[i] = dst[i];
    }
    if (table)
        for (int i = tid; i < n_slots; i += kPoolThreads) last[i] = -1;
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
    if (table)
        for (int i = tid; i < n; i += kPoolThreads)
            if (dd[i] >= 0 && dd[i] < n_slots && ss[i] < n_slots) atomicMax(&last[dd[i]], i);
    __syncthreads();
    if (!on) return;
    if (table) {
#pragma unroll 4
        for (int i = w; i < n; i += writers) {
            const int t = dd[i];
            if (t >= 0 && t < n_slots && last[t] == i) pool[t * page + at] = buf[i * units + u];
        }
        return;
    }
    for (int i = 0; i < n; ++i) {
        const int t = dd[i];
        if (t >= 0 && t < n_slots && ss[i] < n_slots && (t & (writers - 1)) == w) pool[t * page + at] = buf[i * units + u];
    }
}

}  // namespace gdr
}  // namespace la2
