// state_pool.cuh -- serving kernels over a pool of recurrent states
// [slots, H, d, e] (fp32): the gated delta rule's step for one token per
// sequence, and the copies that fork, move and clear slots.
#pragma once
#include "gdr_common.cuh"
#include "ptx_sm100.cuh"

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
// otherwise) of one (row, head) with four rows per thread at d = 128, and four
// CTAs (64 registers a thread) share an SM.  64 x 40 states of 128 x 128: 116 us with whole states of 256
// threads (154 registers, one CTA per SM), 85 us with 512 threads.
//
// slots[b] outside 0 .. n_slots - 1, or listed for an earlier row already:
// the row's output is zero and no state changes.
template <typename Tin, int W>
__global__ void __launch_bounds__(kStepThreads, 4)
gdr_step(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
         const float* __restrict__ g, const float* __restrict__ beta, float* state,
         const int* __restrict__ slots, int n_slots, float* __restrict__ out, int Hk, int H, int d, int e) {
    constexpr int kWarps = kStepThreads / 32;
    __shared__ float ks[128], qs[128];
    __shared__ __align__(16) float part[2][kWarps][kStepUnits * W];
    const int blocks = (e + kStepUnits * W - 1) / (kStepUnits * W);  // column blocks of one state run side by side
    const int n = blockIdx.x / blocks, b = n / H, h = n % H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cl = lane % kStepUnits, col = (blockIdx.x % blocks * kStepUnits + cl) * W;
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

// The same step for many states: a CTA per SM whose threads form teams, as many
// as leave each thread at most 8 16-byte pieces of a state (one of 512 threads at
// 128 x 128, four at 64 x 64).  A team walks over its (row, head)s with three or
// more whole states in shared memory, one being worked on, one being stored, the
// others being loaded (bulk copies), so that the memory system always has 64 KB to
// bring and 64 KB to take per SM whatever the arithmetic in between waits for.  What
// a step reads besides (the slot and the rows before it that name it too, gates, k,
// q, v) is on its way a step ahead: read in the step itself, its latency is the
// step's.  States are 16-byte aligned, e a multiple of 4.  Each thread keeps its part
// of the state in registers between the two products and the update.
// 2560 states of 128 x 128: 63 us (84% of the copy rate), with what a step reads
// besides read in the step 79 us; of 64 x 64: 25 us, with one team of 512 49 us.
constexpr int kBulkThreads = 512;
constexpr int kBulkRows = 8;
constexpr int kBulkStages = 8;  // at most; at least three
constexpr int kBulkStates = 3 * 128 * 128;  // floats of all states of a CTA

template <int kTeam>
struct alignas(16) BulkSmem {  // one per team, one behind the other
    float part[2][kTeam * 4];
    float ks[2][128], qs[2][128];
    float u[128], kq;
    unsigned long long full[kBulkStages];
};

inline int bulk_team(int d, int e) {
    for (int team = 128; team < kBulkThreads; team *= 2)
        if (d <= kBulkRows * (team / (e / 4)) && d <= team && e <= team) return team;
    return kBulkThreads;
}

inline int bulk_stages(int d, int e) {
    const int fit = kBulkStates / (kBulkThreads / bulk_team(d, e) * d * e);
    return fit < kBulkStages ? fit : kBulkStages;
}

template <int kTeam>
constexpr size_t bulk_smem_bytes() {
    return (sizeof(BulkSmem<kTeam>) * (kBulkThreads / kTeam) + 127) / 128 * 128 + kBulkStates * sizeof(float);
}

// Barriers of one team
template <int kTeam>
struct Team {
    int id;  // hardware barrier
    __device__ __forceinline__ void sync() const {
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(kTeam) : "memory");
    }
    __device__ __forceinline__ bool any(bool x) const {
        int r;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\t"
            "selp.s32 %0, 1, 0, q;\n\t}"
            : "=r"(r) : "r"(static_cast<int>(x)), "r"(id), "n"(kTeam) : "memory");
        return r != 0;
    }
};

// Every wait is bounded; a team that gives up waits for its copies in flight before
// its shared memory can go to another CTA.  kHold (la2_gdr_selftest_timeout): the
// third state is announced and not loaded, and the bound is 20 ms.
template <typename Tin, int kTeam, bool kHold = false>
__global__ void __launch_bounds__(kBulkThreads, 1)
gdr_step_bulk(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
              const float* __restrict__ g, const float* __restrict__ beta, float* state,
              const int* __restrict__ slots, int n_slots, float* __restrict__ out, int total, int Hk, int H, int d,
              int e, int stages, int* status) {
    extern __shared__ __align__(128) unsigned char bulk_raw[];
    constexpr int kTeams = kBulkThreads / kTeam;
    const int team = threadIdx.x / kTeam, tid = threadIdx.x % kTeam, page = d * e;
    BulkSmem<kTeam>& sm = reinterpret_cast<BulkSmem<kTeam>*>(bulk_raw)[team];
    float* stage = reinterpret_cast<float*>(bulk_raw + (sizeof(BulkSmem<kTeam>) * kTeams + 127) / 128 * 128) +
                   static_cast<size_t>(team) * stages * page;
    const Team<kTeam> all{1 + team};
    const uint32_t bytes = static_cast<uint32_t>(page) * 4, full = smem_u32(sm.full);
    const int cu = e / 4, groups = kTeam / cu, rg = tid / cu, ju = tid % cu;
    const bool on = rg < groups;
    const int first = team * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    constexpr uint64_t kLimit = kHold ? 20000000ull : 2000000000ull;  // ns
    const int every = kTeams * static_cast<int>(gridDim.x);
    const int mine = first < total ? (total - 1 - first) / every + 1 : 0;
    const auto index = [&](int y) { return first + y * every; };
    const auto slot_of = [&](int y) {
        const int b = index(y) / H;
        return slots ? slots[b] : b;
    };
    const auto load = [&](int y, int slot) {  // one thread
        if (slot < 0 || slot >= n_slots) slot = 0;  // read and dropped: a pool without slots is not launched
        const uint32_t bar = full + 8 * (y % stages);
        mbar_arrive_expect_tx(bar, bytes);
        if (kHold && y == 2) return;
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         smem_u32(stage + static_cast<size_t>(y % stages) * page)),
                     "l"(state + (static_cast<size_t>(slot) * H + index(y) % H) * page), "r"(bytes), "r"(bar)
                     : "memory");
    };
    const auto keep = [&](int y, Tin kk, Tin qq) {
        if (tid < d) {
            sm.ks[y & 1][tid] = to_float(kk);
            sm.qs[y & 1][tid] = to_float(qq);
        }
    };
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(full + 8 * s, 1);
        fence_mbar_init();
        for (int y = 0; y + 1 < stages && y < mine; ++y) load(y, slot_of(y));
    }
    struct Step {  // what one step reads besides the state
        int slot, other;  // other: this thread's share of the rows before (their first kTeam)
        float g, bt;
        Tin k, q, v;  // converted when they are used: a conversion waits for the load
    };
    const auto fetch = [&](int y) {
        Step x = {-1, -1, 0.f, 0.f, Tin(0.f), Tin(0.f), Tin(0.f)};
        if (y < mine) {
            const int n = index(y), b = n / H;
            x.slot = slots ? slots[b] : b;
            if (slots && tid < b) x.other = slots[tid];
            if (tid < d) {
                const size_t at = (static_cast<size_t>(b) * Hk + (n - b * H) / (H / Hk)) * d + tid;
                x.k = k[at];
                x.q = q[at];
            }
            if (g) x.g = g[n];
            x.bt = beta[n];
            if (tid < e) x.v = v[static_cast<size_t>(n) * e + tid];
        }
        return x;
    };
    Step now = fetch(0);
    keep(0, now.k, now.q);
    all.sync();
    for (int y = 0, s = 0, turn = 0; y < mine; ++y) {
        const int n = index(y), b = n / H;
        const Step next = fetch(y + 1);
        const int ahead = y + stages - 1 < mine && tid == 0 ? slot_of(y + stages - 1) : 0;
        const int slot = now.slot;
        const float a = g ? expf(now.g) : 1.f, bt = now.bt;
        int twice = slots && tid < b && now.other == slot;
        if (slots)
            for (int x = tid + kTeam; x < b; x += kTeam) twice |= slots[x] == slot;
        const float vv = to_float(now.v);
        const bool ok = mbar_wait(full + 8 * s, turn, kLimit);
        if (all.any(!ok)) {
            if (tid == 0) {
                atomicCAS(status, 0, 5 | (230 << 8));
                for (int x = y; x < mine && x < y + stages - 1; ++x)  // loads in flight
                    mbar_wait(full + 8 * (x % stages), x / stages & 1, kLimit);
            }
            break;
        }
        float4* S = reinterpret_cast<float4*>(stage + static_cast<size_t>(s) * page);
        const float *ks = sm.ks[y & 1], *qs = sm.qs[y & 1];
        float4 sv[kBulkRows];
        float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
        for (int r = 0; r < kBulkRows; ++r) {
            const int i = rg + r * groups;
            if (on && i < d) {
                sv[r] = S[i * cu + ju];
                const float ki = ks[i], qi = qs[i];
                pk.x = fmaf(sv[r].x, ki, pk.x);
                pk.y = fmaf(sv[r].y, ki, pk.y);
                pk.z = fmaf(sv[r].z, ki, pk.z);
                pk.w = fmaf(sv[r].w, ki, pk.w);
                pq.x = fmaf(sv[r].x, qi, pq.x);
                pq.y = fmaf(sv[r].y, qi, pq.y);
                pq.z = fmaf(sv[r].z, qi, pq.z);
                pq.w = fmaf(sv[r].w, qi, pq.w);
            }
        }
        if (on) {
            reinterpret_cast<float4*>(sm.part[0])[tid] = pk;
            reinterpret_cast<float4*>(sm.part[1])[tid] = pq;
        }
        if (tid >= kTeam - 32) {  // k . q
            float kq = 0.f;
            for (int i = tid & 31; i < d; i += 32) kq = fmaf(ks[i], qs[i], kq);
#pragma unroll
            for (int m = 16; m; m >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, m);
            if (tid == kTeam - 1) sm.kq = kq;
        }
        const bool live = !all.any(twice) && slot >= 0 && slot < n_slots;
        if (tid < e) {
            float sk = 0.f, sq = 0.f;
            const float kq = sm.kq;
#pragma unroll 16
            for (int x = 0; x < groups; ++x) {
                sk += sm.part[0][x * e + tid];
                sq += sm.part[1][x * e + tid];
            }
            const float u = bt * (vv - a * sk);
            sm.u[tid] = u;
            out[static_cast<size_t>(n) * e + tid] = live ? fmaf(a, sq, kq * u) : 0.f;
        }
        keep(y + 1, next.k, next.q);
        all.sync();
        if (live && on) {
            const float4 u = reinterpret_cast<const float4*>(sm.u)[ju];
#pragma unroll
            for (int r = 0; r < kBulkRows; ++r) {
                const int i = rg + r * groups;
                if (i < d) {
                    const float ki = ks[i];
                    S[i * cu + ju] = make_float4(fmaf(a, sv[r].x, ki * u.x), fmaf(a, sv[r].y, ki * u.y),
                                                 fmaf(a, sv[r].z, ki * u.z), fmaf(a, sv[r].w, ki * u.w));
                }
            }
        }
        fence_proxy_async_smem();
        all.sync();
        if (tid == 0) {
            if (live)
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                 state + (static_cast<size_t>(slot) * H + n % H) * page),
                             "r"(smem_u32(S)), "r"(bytes)
                             : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            if (y + stages - 1 < mine) {
                // its stage is the one that was stored a step ago
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                load(y + stages - 1, ahead);
            }
        }
        now = next;
        if (++s == stages) {
            s = 0;
            turn ^= 1;
        }
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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
