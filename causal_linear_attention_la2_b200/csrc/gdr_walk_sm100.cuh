// gdr_walk_sm100.cuh -- the walks of gdr_chunk.cuh along a sequence for e = 128,
// on the tcgen05 tensor cores: one CTA per (batch entry, value head).
//
// Everything that is carried or formed has the 128 value columns on the TMEM
// lanes, as in gdr_chunk.cuh's register form: S^T [e][d] in fp32 (the MMAs
// accumulate onto it), its high and low bf16 parts as the TMEM A operand of the
// products with K and Q, and the 64 rows of the chunk as 64 columns.  A thread
// of the epilogue warps owns one value column, so nothing crosses lanes.
//
// Per chunk the chain is: S K^T -> (z) -> N -> (w, u) -> K -> (S), three MMA
// groups with an epilogue after each:
//   forward   D1 = S K^T;  Z = V - e^G D1;  W = Z - N (beta Z);  U = beta W;
//             S = e^{G_C} S + K^T (e^{G_C - G} U);  beside it D2 = S Q^T, D4 = P U,
//             o = e^G D2 + D4.
//   backward  D1 = dS K^T, D2 = P^T dO;  dU = e^{G_C - G} D1 + D2;
//             X = dU - N^T (beta dU);
//             dS = e^{G_C} dS + Q^T (e^G dO) - K^T (beta e^G X).
// e^{G_C} is multiplied in when the state is read to form its two parts, one
// chunk ahead, so the accumulation needs no extra pass.
//
// Warps (16): 0 loads (TMA tiles, bulk copies of what gdr_prep left), 1 issues
// the MMAs, 2 owns the TMEM allocation; 4-7 and 8-11 are the chain's epilogue,
// half of the columns each; 12-15 do what is off the chain (the output; the copy
// of the state for the backward; the operand e^G dO).
//
// Every wait is bounded (two seconds); a role that gives up raises the CTA's
// abort flag, all leave their loops, copies and MMAs in flight are waited for
// and TMEM is freed.
#pragma once
#include "gdr_chunk.cuh"
#include "ptx_sm100.cuh"

namespace la2 {
namespace gdr {
namespace walk {

constexpr int kE = 128;
constexpr int kThreads = 512;
constexpr int kChainWarps = 8, kSideWarps = 4;

enum Mode { kForward = 0, kSave = 1, kBackward = 2 };

template <int D>
struct Stage {  // 1024-byte aligned; tiles of 64 rows x 64 columns (128 bytes, swizzled)
    unsigned char k[D / 64][kC * 128], q[D / 64][kC * 128], v[kE / 64][kC * 128];
    unsigned char img[4][kC * kC * 2];  // N hi, N lo, P hi, P lo
    float eg[kC], rest[kC], beta[kC];
    unsigned char pad[1024 - 3 * kC * 4];
};

enum Bar { kFull = 0, kEmpty = 2, kD1 = 4, kZ, kW, kU, kS, kState, kD2, kD2Free, kO, kOFree, kSide, kSaved, kRaw, kEnd, kBars };

template <int D>
struct Smem {
    Stage<D> stage[2];
    unsigned long long bar[kBars];
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

struct Waiter {
    uint32_t bars;
    volatile int* abort;
    int* status;
    // Whole warp; false: this role or another one has given up
    __device__ __forceinline__ bool operator()(int bar, uint32_t parity) const {
        const uint32_t b = bars + 8 * bar;
        bool ok = mbar_try_wait(b, parity & 1);
        if (!__all_sync(0xffffffffu, ok)) ok = slow(b, parity & 1, bar);
        return __all_sync(0xffffffffu, ok);
    }
    __device__ __noinline__ bool slow(uint32_t b, uint32_t parity, int where) const {
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(b, parity)) {
            if (*abort) return false;
            if (global_ns() - t0 > 2000000000ull) {
                *abort = 1;
                atomicCAS(status, 0, 5 | ((200 + where) << 8));
                return false;
            }
        }
        return true;
    }
};

// Operand layout in TMEM, 32 columns (words) per 32 elements of K: 16 words of
// high parts, 16 of low parts.  Word offset of k step kk.
__device__ __forceinline__ uint32_t op_hi(int kk) { return 32 * (kk >> 1) + 8 * (kk & 1); }
__device__ __forceinline__ uint32_t op_lo(int kk) { return op_hi(kk) + 16; }

__device__ __forceinline__ void split32(const float (&x)[32], uint32_t (&w)[32]) {
#pragma unroll
    for (int y = 0; y < 16; ++y) split_pack2v(make_float2(x[2 * y], x[2 * y + 1]), w[y], w[16 + y]);
}

// 32 values of one column of a [64 rows][128 columns] bf16 tile pair: rows r0 ..
__device__ __forceinline__ float tile_at(uint32_t tile, int r, int c) {
    uint32_t x;
    const uint32_t a = tile + (c >> 6) * (kC * 128) + piece<128>(r, (c & 63) >> 3) + 2 * (c & 7);
    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(x) : "r"(a));
    return __uint_as_float(x << 16);
}

__device__ __forceinline__ void put_row(const Args& A, void* out, size_t at, float x) {
    if (A.out_bf16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
    else static_cast<float*>(out)[at] = x;
}

template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
gdr_walk(Args A, const ChunkWs* ws, Saved out, int chunks, const __grid_constant__ CUtensorMap mk,
         const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mv, int* status) {
    extern __shared__ unsigned char walk_tc_raw[];
    // the dynamic segment starts at a 1024-byte boundary or the tail of 1 KB makes it one
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(walk_tc_raw + ((1024 - (smem_addr(walk_tc_raw) & 1023)) & 1023));
    constexpr bool kRev = kMode == kBackward;
    constexpr uint32_t kTile = kC * 128;
    // TMEM columns
    constexpr uint32_t cS = 0, cB = D, cA = 2 * D, cW = cA + 64, cD2 = cW + 64, cD4 = cD2 + 64;
    const int n = blockIdx.x, b = n / A.H, h = n % A.H, hk = h / (A.H / A.Hk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = length_of(A, b), nc = (len + kC - 1) / kC;
    const size_t page = static_cast<size_t>(D) * kE;
    const ChunkWs* cw = ws + static_cast<size_t>(n) * chunks;
    const uint32_t bars = smem_addr(sm.bar);
    volatile int* abort = &sm.abort;
    const Waiter wait{bars, abort, status};
    const auto bar = [&](int i) { return bars + 8 * i; };

    if (tid == 0) {
        sm.abort = 0;
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kFull + s), 1);
            mbar_init(bar(kEmpty + s), 1 + kChainWarps + kSideWarps);
        }
        for (int i : {kD1, kW, kS, kD2, kO, kRaw, kEnd}) mbar_init(bar(i), 1);
        for (int i : {kZ, kU, kState}) mbar_init(bar(i), kChainWarps);
        for (int i : {kD2Free, kOFree, kSide, kSaved}) mbar_init(bar(i), kSideWarps);
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc(smem_addr(&sm.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        constexpr uint32_t kRows = (kMode == kSave ? D / 64 : 2 * (D / 64)) * kTile + (kE / 64) * kTile;
        constexpr uint32_t kImg = (kMode == kSave ? 2 : 4) * kC * kC * 2, kCoef = 3 * kC * 4;
        int issued = 0;
        for (int it = 0; it < nc; ++it) {
            const int s = it & 1, c = kRev ? nc - 1 - it : it, t0 = c * kC;
            if (it >= 2 && !wait(kEmpty + s, (it >> 1) - 1)) break;
            Stage<D>& st = sm.stage[s];
            const bool cut = t0 + kC > len && len < A.T;  // rows of this sequence's padding would be loaded
            const int on = cut ? kRaw : kFull + s;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(on), kRows + kImg + kCoef);
                const auto rows = [&](unsigned char* to, const CUtensorMap& m, int head, int tiles) {
                    for (int x = 0; x < tiles; ++x)
                        tma_load_4d(smem_addr(to) + x * kTile, &m, bar(on), 64 * x, A.bthd ? head : t0,
                                    A.bthd ? t0 : head, b);
                };
                rows(st.k[0], mk, hk, D / 64);
                if (kMode != kSave) rows(st.q[0], mq, hk, D / 64);
                rows(st.v[0], mv, h, kE / 64);
                bulk_load(smem_addr(st.img), cw[c].img, kImg, bar(on));
                bulk_load(smem_addr(st.eg), cw[c].eg, kCoef, bar(on));
            }
            issued = it + 1;
            if (cut) {
                if (!wait(kRaw, 0)) break;  // one chunk per sequence at most
                for (int r = len - t0; r < kC; ++r)
                    for (int x = lane; x < 8; x += 32) {
                        const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int y = 0; y < D / 64; ++y) {
                            *reinterpret_cast<uint4*>(st.k[y] + r * 128 + x * 16) = z;
                            if (kMode != kSave) *reinterpret_cast<uint4*>(st.q[y] + r * 128 + x * 16) = z;
                        }
#pragma unroll
                        for (int y = 0; y < kE / 64; ++y) *reinterpret_cast<uint4*>(st.v[y] + r * 128 + x * 16) = z;
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive(bar(kFull + s));
            }
        }
        // the copies in flight have landed before the CTA's shared memory goes
        for (int it = max(0, issued - 2); it < issued; ++it) {
            const int c = kRev ? nc - 1 - it : it;
            const bool cut = c * kC + kC > len && len < A.T;
            mbar_wait(cut ? bar(kRaw) : bar(kFull + (it & 1)), cut ? 0 : (it >> 1) & 1);
        }
    } else if (warp == 1) {
        // ----------------------------------------------------------------- MMAs
        const uint32_t lead = lane == 0;
        constexpr uint32_t kId = idesc_bf16_f32(kE, 64, 0, 0);    // B [64 rows][k]
        constexpr uint32_t kIdT = idesc_bf16_f32(kE, 64, 0, 1);   // B from rows [k][64]
        constexpr uint32_t kIdTT = idesc_bf16_f32(kE, 64, 1, 1);  // A from rows [k][128] as well
        constexpr uint32_t kIdS = idesc_bf16_f32(kE, D, 0, 1);    // B from rows [k][d]
        for (int it = 0; it < nc; ++it) {
            const int s = it & 1;
            Stage<D>& st = sm.stage[s];
            if (!wait(kFull + s, it >> 1)) break;
            const uint64_t dk = sdesc_sw128(smem_addr(st.k), 16, 1024), dq = sdesc_sw128(smem_addr(st.q), 16, 1024);
            const uint64_t tk = sdesc_sw128(smem_addr(st.k), kTile, 1024), tq = sdesc_sw128(smem_addr(st.q), kTile, 1024);
            const uint32_t img = smem_addr(st.img);
            if (kRev) {
                // P^T dO: free of the chain (z of the chunk before has read it out)
                const uint64_t td = sdesc_sw128(smem_addr(st.v), kTile, 1024);
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ss_w(tm + cD2, desc_add(td, kk * 2048),
                                      sdesc_sw128(img + (2 + x) * kTile + kk * 2048, kTile, 1024), kIdTT, x + kk > 0, lead);
            }
            if (!wait(kState, it)) break;
            if (!kRev && kMode == kForward && it > 0 && !wait(kO, it - 1)) break;  // P U has read its operand
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t bd = desc_add(dk, (kk >> 2) * kTile + (kk & 3) * 32);
                mma_bf16_ts_w(tm + cA, tm + cB + op_hi(kk), bd, kId, kk > 0, lead);
                mma_bf16_ts_w(tm + cA, tm + cB + op_lo(kk), bd, kId, 1, lead);
            }
            mma_commit_w(bar(kD1), lead);
            if (kMode == kForward) {
                if (it > 0 && !wait(kD2Free, it - 1)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint64_t bd = desc_add(dq, (kk >> 2) * kTile + (kk & 3) * 32);
                    mma_bf16_ts_w(tm + cD2, tm + cB + op_hi(kk), bd, kId, kk > 0, lead);
                    mma_bf16_ts_w(tm + cD2, tm + cB + op_lo(kk), bd, kId, 1, lead);
                }
                mma_commit_w(bar(kD2), lead);
            }
            if (kRev) {
                if (!wait(kSide, it)) break;  // e^G dO
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_bf16_ts_w(tm + cS, tm + cD4 + op_hi(kk), desc_add(tq, kk * 2048), kIdS, 1, lead);
                    mma_bf16_ts_w(tm + cS, tm + cD4 + op_lo(kk), desc_add(tq, kk * 2048), kIdS, 1, lead);
                }
            }
            if (!wait(kZ, it)) break;
            tc_fence_after();
            {
                const uint32_t id = kRev ? kIdT : kId;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t o = kRev ? kk * 2048 : kk * 32;
                    const uint64_t bh = sdesc_sw128(img + o, kRev ? kTile : 16, 1024);
                    const uint64_t bl = sdesc_sw128(img + kTile + o, kRev ? kTile : 16, 1024);
                    mma_bf16_ts_w(tm + cW, tm + cA + op_hi(kk), bh, id, 1, lead);
                    mma_bf16_ts_w(tm + cW, tm + cA + op_lo(kk), bh, id, 1, lead);
                    mma_bf16_ts_w(tm + cW, tm + cA + op_hi(kk), bl, id, 1, lead);
                }
            }
            mma_commit_w(bar(kW), lead);
            if (!wait(kU, it)) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                mma_bf16_ts_w(tm + cS, tm + cW + op_hi(kk), desc_add(tk, kk * 2048), kIdS, 1, lead);
                mma_bf16_ts_w(tm + cS, tm + cW + op_lo(kk), desc_add(tk, kk * 2048), kIdS, 1, lead);
            }
            mma_commit_w(bar(kS), lead);
            if (kMode == kForward) {
                if (it > 0 && !wait(kOFree, it - 1)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t bh = sdesc_sw128(img + 2 * kTile + kk * 32, 16, 1024);
                    const uint64_t bl = sdesc_sw128(img + 3 * kTile + kk * 32, 16, 1024);
                    mma_bf16_ts_w(tm + cD4, tm + cA + op_hi(kk), bh, kId, kk > 0, lead);
                    mma_bf16_ts_w(tm + cD4, tm + cA + op_lo(kk), bh, kId, 1, lead);
                    mma_bf16_ts_w(tm + cD4, tm + cA + op_hi(kk), bl, kId, 1, lead);
                }
                mma_commit_w(bar(kO), lead);
            }
            mma_commit_w(bar(kEmpty + s), lead);
        }
    } else if (warp >= 4 && warp < 12) {
        // ------------------------------------------------------ the chain's epilogue
        const int half = (warp - 4) >> 2, e = 32 * (warp & 3) + lane;
        const uint32_t row = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        constexpr int kGroups = D / 64;  // groups of 32 state columns of this half
        const auto state = [&](const float* p, int i) { return p ? p[static_cast<size_t>(i) * kE + e] : 0.f; };
        const float* first = kRev ? A.dfinal : A.init;
        if (first) first += n * page;
        float* last = kRev ? A.dinit : A.fin;
        if (kMode == kSave) last = nullptr;
        if (last) last += n * page;
        const int r0 = 32 * half;
        const auto publish = [&](float (&S)[32], int q, float ec) {  // two parts, and e^{G_C} S to accumulate onto
            uint32_t w[32];
            split32(S, w);
            tmem_st32u(row + cB + 32 * q, w);
#pragma unroll
            for (int y = 0; y < 32; ++y) S[y] *= ec;
            tmem_st32(row + cS + 32 * q, S);
        };
        const auto done = [&](int i) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(bar(i));
        };
        bool ok = nc > 0 && wait(kFull, 0);
        if (ok || nc == 0) {
            const float ec = nc > 0 ? sm.stage[0].eg[kC - 1] : 1.f;
#pragma unroll 1
            for (int y = 0; y < kGroups; ++y) {
                const int q = half * kGroups + y;
                float S[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) S[i] = state(first, 32 * q + i);
                if (nc > 0) publish(S, q, ec);
                else if (last)
#pragma unroll
                    for (int i = 0; i < 32; ++i) last[static_cast<size_t>(32 * q + i) * kE + e] = S[i];
            }
        }
        if (ok) done(kState);
        for (int it = 0; ok && it < nc; ++it) {
            const int s = it & 1, c = kRev ? nc - 1 - it : it;
            Stage<D>& st = sm.stage[s];
            if (!(ok = wait(kD1, it))) break;
            tc_fence_after();
            {
                float x[32], y[32];
                uint32_t w[32];
                tmem_ld32(row + cA + r0, x);
                if (kRev) {
                    tmem_ld32(row + cD2 + r0, y);
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = fmaf(st.rest[r0 + i], x[i], y[i]);
                } else {
                    const uint32_t vt = smem_addr(st.v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = fmaf(-st.eg[r0 + i], x[i], tile_at(vt, r0 + i, e));
                }
                tmem_st32(row + cW + r0, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= -st.beta[r0 + i];
                split32(x, w);
                tmem_st32u(row + cA + r0, w);
            }
            done(kZ);
            if (!(ok = wait(kW, it))) break;
            tc_fence_after();
            {
                float x[32];
                uint32_t w[32];
                tmem_ld32(row + cW + r0, x);
                if (kMode != kForward) {  // rows w or x for the gradients
                    float* to = (kRev ? out.X : out.W) + (static_cast<size_t>(n) * A.T + c * kC + r0) * kE + e;
                    const int left = len - c * kC - r0;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < left) to[static_cast<size_t>(i) * kE] = x[i];
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= st.beta[r0 + i];
                if (kMode == kForward) {
                    split32(x, w);
                    tmem_st32u(row + cA + r0, w);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= kRev ? -st.eg[r0 + i] : st.rest[r0 + i];
                split32(x, w);
                tmem_st32u(row + cW + r0, w);
            }
            __syncwarp();
            if (lane == 0) arrive(bar(kEmpty + s));  // this stage's rows and coefficients are read out
            done(kU);
            float ec = 1.f;
            if (it + 1 < nc) {
                if (!(ok = wait(kFull + (s ^ 1), (it + 1) >> 1))) break;
                ec = sm.stage[s ^ 1].eg[kC - 1];
            }
            if (kMode != kForward && !(ok = wait(kSaved, it))) break;
            if (!(ok = wait(kS, it))) break;
            tc_fence_after();
            if (it + 1 < nc) {
#pragma unroll 1
                for (int y = 0; y < kGroups; ++y) {
                    const int q = half * kGroups + y;
                    float S[32];
                    tmem_ld32(row + cS + 32 * q, S);
                    publish(S, q, ec);
                }
                done(kState);
            } else if (last) {
#pragma unroll 1
                for (int y = 0; y < kGroups; ++y) {
                    const int q = half * kGroups + y;
                    float S[32];
                    tmem_ld32(row + cS + 32 * q, S);
#pragma unroll
                    for (int i = 0; i < 32; ++i) last[static_cast<size_t>(32 * q + i) * kE + e] = S[i];
                }
            }
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------ off the chain
        const int e = 32 * (warp & 3) + lane;
        const uint32_t row = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        for (int it = 0; it < nc; ++it) {
            const int s = it & 1, c = kRev ? nc - 1 - it : it, t0 = c * kC;
            Stage<D>& st = sm.stage[s];
            if (!wait(kFull + s, it >> 1)) break;
            if (kMode == kForward) {
                float o[2][32];
                if (!wait(kD2, it)) break;
                tc_fence_after();
                tmem_ld32(row + cD2, o[0]);
                tmem_ld32(row + cD2 + 32, o[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(bar(kD2Free));
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[x][i] *= st.eg[32 * x + i];
                __syncwarp();
                if (lane == 0) arrive(bar(kEmpty + s));
                if (!wait(kO, it)) break;
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float y[32];
                    tmem_ld32(row + cD4 + 32 * x, y);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[x][i] += y[i];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(bar(kOFree));
                const size_t step = row_at(A, 0, 0, A.H, 1, kE) - row_at(A, 0, 0, A.H, 0, kE);
                const size_t at = row_at(A, b, h, A.H, t0, kE) + e;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (t0 + 32 * x + i < len) put_row(A, A.o, at + (32 * x + i) * step, o[x][i]);
                continue;
            }
            if (kRev) {
                if (it > 0 && !wait(kS, it - 1)) break;  // the operand of the chunk before is read out
                tc_fence_after();
                const uint32_t dt = smem_addr(st.v);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float y[32];
                    uint32_t w[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[i] = st.eg[32 * x + i] * tile_at(dt, 32 * x + i, e);
                    split32(y, w);
                    tmem_st32u(row + cD4 + 32 * x, w);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(bar(kSide));
            }
            __syncwarp();
            if (lane == 0) arrive(bar(kEmpty + s));
            // the state (forward: before the chunk, backward: the gradient after it) to memory, [2][e][d]
            if (!wait(kState, it)) break;
            tc_fence_after();
            uint32_t* hi = reinterpret_cast<uint32_t*>((kRev ? out.dS1 : out.S0) +
                                                       (static_cast<size_t>(n) * chunks + c) * 2 * page) + e * (D / 2);
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                float w[32];
                tmem_ld32(row + cB + 32 * q, w);
#pragma unroll
                for (int x = 0; x < 32; x += 4) {
                    uint4 y = make_uint4(__float_as_uint(w[x]), __float_as_uint(w[x + 1]), __float_as_uint(w[x + 2]),
                                         __float_as_uint(w[x + 3]));
                    *reinterpret_cast<uint4*>(hi + (x >> 4) * (page / 2) + 16 * q + (x & 15)) = y;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(bar(kSaved));
        }
    }
    __syncwarp();
    // MMAs in flight end before TMEM goes: the issuer's last commit is waited for
    if (warp == 1) {
        mma_commit_w(bar(kEnd), lane == 0);
        mbar_wait(bar(kEnd), 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tm, 512);
}

}  // namespace walk
}  // namespace gdr
}  // namespace la2
