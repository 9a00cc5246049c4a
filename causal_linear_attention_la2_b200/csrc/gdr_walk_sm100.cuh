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
// e^{G_C} is multiplied in one chunk ahead, when the two parts of the state are
// already handed to the next product.  S K^T and S Q^T are one product of 128 columns:
// half as many instructions to issue, which is done inside elect.sync (about 20
// cycles each; 78 under a test of the lane).  Each round from one product's
// commit to the next one's issue costs some 1800 cycles, of which the MMAs are a
// fraction: three of them bound the walk, 2.9 us a chunk (80 sequences of 96 chunks
// of d = 128: 287 us; 28 warps instead of 16 took 338 us).
//
// Warps (16): 0 loads (TMA tiles, bulk copies of what gdr_prep left), 1 issues
// the MMAs, 2 owns the TMEM allocation; 4-7 and 8-11 are the chain's epilogue,
// half of the columns each; 12-15 do what is off the chain (the output; the operand
// e^G dO).
//
// Every wait is bounded (two seconds); a role that gives up raises the CTA's
// abort flag, all leave their loops, copies and MMAs in flight are waited for
// and TMEM is freed.
#pragma once
#include <type_traits>

#include "gdr_chunk.cuh"
#include "ptx_sm100.cuh"

namespace la2 {
namespace gdr {
namespace walk {

constexpr int kE = 128;
constexpr int kThreads = 512;
constexpr int kChainWarps = 8, kSideWarps = 4;

enum Mode { kForward = 0, kSave = 1, kBackward = 2, kTransfer = 3 };

// Few sequences: each is cut into `segs` segments of `per` chunks that are walked
// at the same time.  What a segment does to the state that enters it is
// S -> M S + B; kTransfer walks all segments but the first and the last twice,
// from zero for B and from the identity with v = 0 for M (d columns), the first
// one once, from where it starts; gdr_join applies them in turn, and the forward
// walk of each segment starts from its result.
struct Segments {
    int segs, per;  // 1: whole sequences
    float* pages;   // [segs - 1][B*H][3][d][128]: B, M, the state that enters segment s + 1
};

template <int D>
struct Stage {  // 1024-byte aligned; tiles of 64 rows x 64 columns (128 bytes, swizzled)
    unsigned char kq[D / 64][2][kC * 128];  // K and Q of 64 columns side by side: one operand of 128 rows
    unsigned char v[kE / 64][kC * 128];
    unsigned char img[4][kC * kC * 2];  // N hi, N lo, P hi, P lo
    float eg[kC], rest[kC], beta[kC], neg_eg[kC], neg_beta[kC], rest_beta[kC], neg_beta_eg[kC];
    unsigned char pad[2048 - kCoefs * kC * 4];
};

enum Bar { kFull = 0, kEmpty = 2, kState = 4, kFullP = 6, kEmptyP = 8, kD1 = 10, kZ, kW, kU, kUp, kS, kScaled, kD2Free, kO, kOFree, kSide, kRaw, kEnd, kBars };

template <int D>
struct Smem {
    Stage<D> stage[2];
    unsigned char u[2][kE * 128];  // forward: U^T [e][64 rows], high and low, the operand of P U
    unsigned char o[kSideWarps][kC * 64];  // forward: bf16 output rows of 32 value columns per warp
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

// One lane of the warp, always the same one.  MMAs are issued inside a branch on
// it: under any other condition the compiler has to allow for several lanes.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// D[tmem] (+)= A[tmem] B[smem]; one thread
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
}

// Bounds of the waits in ns; the second one for kernels that la2_gdr_selftest_timeout
// holds (kHold: one copy of the second chunk is announced and not issued).
template <bool kHold>
constexpr uint64_t kWaitNs = kHold ? 20000000ull : 2000000000ull;

// The timer is read every 64 tries only: reading it takes longer than most waits.
template <bool kHold>
__device__ __noinline__ bool wait_slow(uint32_t b, uint32_t parity, int where, volatile int* abort, int* status) {
    uint64_t t0 = 0;
    for (uint32_t tries = 1;; ++tries) {
        if (mbar_try_wait(b, parity)) return true;
        if (tries % 64) continue;
        if (*abort) return false;
        if (!t0) t0 = global_ns();
        if (global_ns() - t0 > kWaitNs<kHold>) {
            *abort = 1;
            atomicCAS(status, 0, 5 | ((200 + where) << 8));
            return false;
        }
    }
}

template <bool kHold>
struct Waiter {
    uint32_t bars;
    volatile int* abort;
    int* status;
    // Whole warp; false: this role or another one has given up
    __device__ __forceinline__ bool operator()(int bar, uint32_t parity) const {
        const uint32_t b = bars + 8 * bar;
        bool ok = mbar_try_wait(b, parity & 1);
        if (!__all_sync(0xffffffffu, ok)) ok = wait_slow<kHold>(b, parity & 1, bar, abort, status);
        return __all_sync(0xffffffffu, ok);
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

// Row r, column c of a [64 rows][128 columns] bf16 tile pair
__device__ __forceinline__ uint32_t tile_bits(uint32_t tile, int r, int c) {
    unsigned short x;
    const uint32_t a = tile + (c >> 6) * (kC * 128) + piece<128>(r, (c & 63) >> 3) + 2 * (c & 7);
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ float tile_at(uint32_t tile, int r, int c) { return __uint_as_float(tile_bits(tile, r, c) << 16); }

// The walk of CTA `block` of seqs x parts
template <int D, int kMode, bool kHold = false>
__device__ __forceinline__ void walk_along(const Args& A, const ChunkWs* ws, const Saved& out, const Segments& sg, int chunks,
                                           const CUtensorMap& mk, const CUtensorMap& mq, const CUtensorMap& mv, int* status,
                                           int block) {
    extern __shared__ __align__(1024) unsigned char walk_tc_raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(walk_tc_raw);
    constexpr bool kRev = kMode == kBackward;
    constexpr uint32_t kTile = kC * 128;
    // TMEM columns
    constexpr uint32_t cS = 0, cB = D, cA = 2 * D, cD2 = cA + 64, cW = cD2 + 64, cD4 = cW + 64;
    // kForward: segment by segment; kTransfer: B of the first one, B and M of the others
    const int seqs = A.B * A.H, n = block % seqs, part = block / seqs;
    const int seg = kMode == kTransfer ? (part + 1) >> 1 : kMode == kForward ? part : 0;
    const bool unit = kMode == kTransfer && part > 0 && !(part & 1);  // from the identity, with v = 0
    const int b = n / A.H, h = n % A.H, hk = h / (A.H / A.Hk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = length_of(A, b), all = (len + kC - 1) / kC;
    // chunks c0 .. c0 + nc - 1 of the sequence
    const int c0 = (kMode == kForward || kMode == kTransfer) && sg.segs > 1 ? seg * sg.per : 0;
    const int nc = sg.segs > 1 ? max(0, min(sg.per, all - c0)) : all;
    const size_t page = static_cast<size_t>(D) * kE;
    const auto pages = [&](int s, int which) { return sg.pages + ((static_cast<size_t>(s) * seqs + n) * 3 + which) * page; };
    const ChunkWs* cw = ws + static_cast<size_t>(n) * chunks;
    const uint32_t bars = smem_addr(sm.bar);
    volatile int* abort = &sm.abort;
    const Waiter<kHold> wait{bars, abort, status};
    const auto drain = [&](int i, int parity) { mbar_wait(bars + 8 * i, parity & 1, kWaitNs<kHold>); };
    const auto bar = [&](int i) { return bars + 8 * i; };

    if (tid == 0) {
        sm.abort = 0;
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kFull + s), 1);
            mbar_init(bar(kEmpty + s), 1 + kChainWarps + kSideWarps);
            mbar_init(bar(kFullP + s), 1);
            mbar_init(bar(kEmptyP + s), 1);
        }
        for (int i : {kD1, kW, kS, kO, kRaw, kEnd}) mbar_init(bar(i), 1);
        for (int i : {kState + 0, kState + 1, int(kZ), int(kU), int(kUp), int(kScaled)}) mbar_init(bar(i), kChainWarps);
        for (int i : {kD2Free, kOFree, kSide}) mbar_init(bar(i), kSideWarps);
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
    if (tm != 0) {  // not seen: an allocation of every column starts at the first
        if (tid == 0) atomicCAS(status, 0, 5 | (199 << 8));
        __syncthreads();
        if (warp == 2) tmem_dealloc(tm, 512);
        return;
    }

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        constexpr bool kNoQ = kMode == kSave || kMode == kTransfer;
        constexpr uint32_t kRows = (kNoQ ? D / 64 : 2 * (D / 64)) * kTile + (kE / 64) * kTile;
        constexpr uint32_t kImg = (kRev ? 4 : 2) * kC * kC * 2, kCoef = kCoefs * kC * 4;
        int issued = 0;
        for (int it = 0; it < nc; ++it) {
            const int s = it & 1, c = kRev ? nc - 1 - it : c0 + it, t0 = c * kC;
            if (it >= 2 && !wait(kEmpty + s, (it >> 1) - 1)) break;
            Stage<D>& st = sm.stage[s];
            const bool cut = t0 + kC > len && len < A.T;  // rows of this sequence's padding would be loaded
            const int on = cut ? kRaw : kFull + s;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(on), kRows + kImg + kCoef);
                const auto rows = [&](unsigned char* to, const CUtensorMap& m, int head, int x) {
                    tma_load_4d(smem_addr(to), &m, bar(on), 64 * x, A.bthd ? head : t0, A.bthd ? t0 : head, b);
                };
                for (int x = 0; x < D / 64; ++x) {
                    if (!(kHold && it == 1 && x == 0)) rows(st.kq[x][0], mk, hk, x);
                    if (!kNoQ) rows(st.kq[x][1], mq, hk, x);
                }
                for (int x = 0; x < kE / 64; ++x) rows(st.v[x], mv, h, x);
                bulk_load(smem_addr(st.img), cw[c].img, kImg, bar(on));
                bulk_load(smem_addr(st.eg), cw[c].eg, kCoef, bar(on));
            }
            if (kMode == kForward) {  // P, which is read a chunk later than the rest, has barriers of its own
                if (it >= 2 && !wait(kEmptyP + s, (it >> 1) - 1)) {
                    ++issued;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(kFullP + s), 2 * kC * kC * 2);
                    bulk_load(smem_addr(st.img[2]), cw[c].img[2], 2 * kC * kC * 2, bar(kFullP + s));
                }
            }
            issued = it + 1;
            if (cut) {
                if (!wait(kRaw, 0)) break;  // one chunk per sequence at most
                for (int r = len - t0; r < kC; ++r)
                    for (int x = lane; x < 8; x += 32) {
                        const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int y = 0; y < D / 64; ++y) {
                            *reinterpret_cast<uint4*>(st.kq[y][0] + r * 128 + x * 16) = z;
                            if (!kNoQ) *reinterpret_cast<uint4*>(st.kq[y][1] + r * 128 + x * 16) = z;
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
            const int c = kRev ? nc - 1 - it : c0 + it;
            const bool cut = c * kC + kC > len && len < A.T;
            drain(cut ? kRaw : kFull + (it & 1), cut ? 0 : it >> 1);
            // (a P that was never asked for, after an abort, costs this wait its whole bound)
            if (kMode == kForward) drain(kFullP + (it & 1), it >> 1);
        }
    } else if (warp == 1) {
        // ----------------------------------------------------------------- MMAs
        constexpr uint32_t kId = idesc_bf16_f32(kE, 64, 0, 0);    // B [64 rows][k]
        constexpr uint32_t kIdQ = idesc_bf16_f32(kE, 128, 0, 0);  // B [128 rows][k]
        constexpr uint32_t kIdT = idesc_bf16_f32(kE, 64, 0, 1);   // B from rows [k][64]
        constexpr uint32_t kIdTT = idesc_bf16_f32(kE, 64, 1, 1);  // A from rows [k][128] as well
        constexpr uint32_t kIdS = idesc_bf16_f32(kE, D, 0, 1);    // B from rows [k][d]
        constexpr int kGroups = D / 64;
        // All of TMEM is this CTA's, so its first column is 0 (checked above); with the
        // stage known at compile time too, every address below is a constant, and
        // an MMA is issued in a few cycles (78 with the addresses in registers).
        constexpr uint32_t tm = 0;
        // P U of chunk `it`, issued behind S K^T of the next chunk: the tensor cores
        // would idle there, and the chain does not wait for it.
        const auto output = [&](int it, auto stage) -> bool {
            constexpr int s = decltype(stage)::value;
            if (!(wait(kUp, it) && wait(kFullP + s, it >> 1) && (it == 0 || wait(kOFree, it - 1)))) return false;
            tc_fence_after();
            if (elect()) {
                const uint32_t img = smem_addr(sm.stage[s].img);
                const uint64_t uh = sdesc_sw128(smem_addr(sm.u[0]), 16, 1024), ul = sdesc_sw128(smem_addr(sm.u[1]), 16, 1024);
                const uint64_t ph = sdesc_sw128(img + 2 * kTile, 16, 1024), pl = sdesc_sw128(img + 3 * kTile, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_bf16_ss(tm + cD4, desc_add(uh, kk * 32), desc_add(ph, kk * 32), kId, kk > 0);
                    mma_bf16_ss(tm + cD4, desc_add(ul, kk * 32), desc_add(ph, kk * 32), kId, 1);
                    mma_bf16_ss(tm + cD4, desc_add(uh, kk * 32), desc_add(pl, kk * 32), kId, 1);
                }
                mma_commit(bar(kO));
                mma_commit(bar(kEmptyP + s));
            }
            return true;
        };
        const auto chunk = [&](int it, auto stage) -> bool {
            constexpr int s = decltype(stage)::value;
            Stage<D>& st = sm.stage[s];
            if (!wait(kFull + s, it >> 1)) return false;
            const uint32_t kq = smem_addr(st.kq), img = smem_addr(st.img);
            const uint64_t dk = sdesc_sw128(kq, 16, 1024);
            const uint64_t tk = sdesc_sw128(kq, 2 * kTile, 1024), tq = sdesc_sw128(kq + kTile, 2 * kTile, 1024);
            if (kRev) {
                // P^T dO: free of the chain (z of the chunk before has read it out)
                const uint64_t td = sdesc_sw128(smem_addr(st.v), kTile, 1024);
                tc_fence_after();
                if (elect())
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ss(tm + cD2, desc_add(td, kk * 2048),
                                      sdesc_sw128(img + (2 + x) * kTile + kk * 2048, kTile, 1024), kIdTT, x + kk > 0);
            }
            // the output warps have read what S Q^T overwrites
            if (kMode == kForward && it > 0 && !wait(kD2Free, it - 1)) return false;
#pragma unroll
            for (int y = 0; y < kGroups; ++y) {
                if (!wait(kState + y, it)) return false;
                tc_fence_after();
                if (elect()) {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int kk = 2 * ((z >> 1) * kGroups + y) + (z & 1);
                    const uint64_t bd = desc_add(dk, (kk >> 2) * 2 * kTile + (kk & 3) * 32);
                    const uint32_t id = kMode == kForward ? kIdQ : kId;
                    mma_ts(tm + cA, tm + cB + op_hi(kk), bd, id, y + z > 0);
                    mma_ts(tm + cA, tm + cB + op_lo(kk), bd, id, 1);
                }
                if (y == kGroups - 1) mma_commit(bar(kD1));
                }
            }
            if (kMode == kForward && it > 0 && !output(it - 1, std::integral_constant<int, s ^ 1>())) return false;
            if (kRev) {
                if (!(wait(kSide, it) && wait(kScaled, it))) return false;  // e^G dO
                tc_fence_after();
                if (elect())
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_ts(tm + cS, tm + cD4 + op_hi(kk), desc_add(tq, kk * 2048), kIdS, 1);
                    mma_ts(tm + cS, tm + cD4 + op_lo(kk), desc_add(tq, kk * 2048), kIdS, 1);
                }
            }
            if (!wait(kZ, it)) return false;
            tc_fence_after();
            if (elect()) {
                const uint32_t id = kRev ? kIdT : kId;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t o = kRev ? kk * 2048 : kk * 32;
                    const uint64_t bh = sdesc_sw128(img + o, kRev ? kTile : 16, 1024);
                    const uint64_t bl = sdesc_sw128(img + kTile + o, kRev ? kTile : 16, 1024);
                    mma_ts(tm + cW, tm + cA + op_hi(kk), bh, id, 1);
                    mma_ts(tm + cW, tm + cA + op_lo(kk), bh, id, 1);
                    mma_ts(tm + cW, tm + cA + op_hi(kk), bl, id, 1);
                }
                mma_commit(bar(kW));
            }
            if (!(wait(kScaled, it) && wait(kU, it))) return false;
            tc_fence_after();
            if (elect()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                mma_ts(tm + cS, tm + cW + op_hi(kk), desc_add(tk, kk * 2048), kIdS, 1);
                mma_ts(tm + cS, tm + cW + op_lo(kk), desc_add(tk, kk * 2048), kIdS, 1);
            }
            mma_commit(bar(kS));
            }
            if (elect()) mma_commit(bar(kEmpty + s));
            return true;
        };
        for (int it = 0; it < nc; it += 2) {
            if (!chunk(it, std::integral_constant<int, 0>())) break;
            if (it + 1 < nc && !chunk(it + 1, std::integral_constant<int, 1>())) break;
        }
        if (kMode == kForward && nc > 0 && !sm.abort) {
            if (nc & 1) output(nc - 1, std::integral_constant<int, 0>());
            else output(nc - 1, std::integral_constant<int, 1>());
        }
    } else if (warp >= 4 && warp < 12) {
        // ------------------------------------------------------ the chain's epilogue
        const int half = (warp - 4) >> 2, e = 32 * (warp & 3) + lane;
        const uint32_t row = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        constexpr int kGroups = D / 64;  // groups of 32 state columns of this half
        const auto state = [&](const float* p, int i) {
            if (unit) return e == i ? 1.f : 0.f;
            return p ? p[static_cast<size_t>(i) * kE + e] : 0.f;
        };
        const float* first = kRev ? A.dfinal : A.init;
        if (first) first += n * page;
        float* last = kRev ? A.dinit : A.fin;
        if (kMode == kSave) last = nullptr;
        if (last) last += n * page;
        if (kMode == kForward && sg.segs > 1) {
            if (seg > 0) first = pages(seg - 1, 2);
            // the final state is that of the segment with the sequence's last row (the first one of an empty sequence)
            if (all > 0 ? c0 >= all || c0 + nc < all : seg > 0) last = nullptr;
        }
        if (kMode == kTransfer) {
            if (seg > 0) first = nullptr;
            last = pages(seg, unit ? 1 : 0);
        }
        const int r0 = 32 * half;
        const auto done = [&](int i) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(bar(i));
        };
        // x *= f, f 32 consecutive floats of shared memory (the same for the whole warp)
        const auto times = [](float (&x)[32], const float* f) {
#pragma unroll
            for (int y = 0; y < 32; y += 4) {
                const float4 m = *reinterpret_cast<const float4*>(f + y);
                const float2 p = mul2(make_float2(m.x, m.y), make_float2(x[y], x[y + 1]));
                const float2 r = mul2(make_float2(m.z, m.w), make_float2(x[y + 2], x[y + 3]));
                x[y] = p.x;
                x[y + 1] = p.y;
                x[y + 2] = r.x;
                x[y + 3] = r.y;
            }
        };
        const auto scale = [&](float ec) {  // S -> e^{G_C} S, to accumulate onto
#pragma unroll 1
            for (int y = 0; y < kGroups; ++y) {
                const uint32_t at = row + cS + 32 * (half * kGroups + y);
                float S[32];
                tmem_ld32(at, S);
#pragma unroll
                for (int i = 0; i < 32; ++i) S[i] *= ec;
                tmem_st32(at, S);
            }
            done(kScaled);
        };
        // 32 columns of d of the state (its two parts) to memory, in Saved's layout: each lane's 16 bytes next to the
        // neighbouring lanes'.  `at`: forward, the chunk that the state enters; backward, the one whose dS1 it is.
        const auto keep = [&](const uint32_t (&w)[32], int q, int at) {
            __nv_bfloat16* to = (kRev ? out.dS1 + (static_cast<size_t>(n) * chunks + at) * 2 * page
                                      : out.S0 + (static_cast<size_t>(n) * chunks + at) * 2 * page) + e * 8;
#pragma unroll
            for (int x = 0; x < 32; x += 4)
                *reinterpret_cast<uint4*>(to + (x >> 4) * page + (4 * q + (x & 15) / 4) * (kE * 8)) =
                    make_uint4(w[x], w[x + 1], w[x + 2], w[x + 3]);
        };
        bool ok = nc > 0;
#pragma unroll 1
        for (int y = 0; y < kGroups; ++y) {
            const int q = half * kGroups + y;
            float S[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = state(first, 32 * q + i);
            if (nc > 0) {
                uint32_t w[32];
                tmem_st32(row + cS + 32 * q, S);
                split32(S, w);
                tmem_st32u(row + cB + 32 * q, w);
                done(kState + y);
                if (kMode == kSave || kRev) keep(w, q, kRev ? nc - 1 : 0);
            } else if (last) {
#pragma unroll
                for (int i = 0; i < 32; ++i) last[static_cast<size_t>(32 * q + i) * kE + e] = S[i];
            }
        }
        for (int it = 0; ok && it < nc; ++it) {
            const int s = it & 1, c = kRev ? nc - 1 - it : c0 + it;
            Stage<D>& st = sm.stage[s];
            if (!(ok = wait(kFull + s, it >> 1))) break;
            scale(st.eg[kC - 1]);
            uint32_t v[16];  // this column of 32 rows of V, in pairs: read before the product is waited for
            if (!kRev) {
                const uint32_t vt = smem_addr(st.v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] = unit ? 0u : tile_bits(vt, r0 + 2 * i, e) | tile_bits(vt, r0 + 2 * i + 1, e) << 16;
            }
            if (!(ok = wait(kD1, it))) break;
            tc_fence_after();
            {
                float x[32];
                uint32_t w[32];
                tmem_ld32(row + cA + r0, x);
                if (kRev) {
                    float y[32];
                    tmem_ld32(row + cD2 + r0, y);
                    times(x, st.rest + r0);
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] += y[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(st.neg_eg + r0 + i);
                        const uint32_t v0 = v[i / 2], v1 = v[i / 2 + 1];
                        const float2 p = fma2(make_float2(m.x, m.y), make_float2(x[i], x[i + 1]),
                                              make_float2(low_of(v0), high_of(v0)));
                        const float2 r = fma2(make_float2(m.z, m.w), make_float2(x[i + 2], x[i + 3]),
                                              make_float2(low_of(v1), high_of(v1)));
                        x[i] = p.x;
                        x[i + 1] = p.y;
                        x[i + 2] = r.x;
                        x[i + 3] = r.y;
                    }
                }
                tmem_st32(row + cW + r0, x);
                times(x, st.neg_beta + r0);
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
                {
                    float u[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) u[i] = x[i];
                    times(u, (kRev ? st.neg_beta_eg : st.rest_beta) + r0);
                    split32(u, w);
                    tmem_st32u(row + cW + r0, w);
                }
                done(kU);
                if (kMode == kForward) {
                    times(x, st.beta + r0);
                    split32(x, w);
                    if (it > 0 && !(ok = wait(kO, it - 1))) break;  // P U of the chunk before has read its operand
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        st_shared_v4(smem_addr(sm.u[y >> 2]) + piece<128>(e, 4 * half + (y & 3)), w[4 * y], w[4 * y + 1],
                                     w[4 * y + 2], w[4 * y + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive(bar(kUp));
                } else if (kMode != kTransfer) {  // rows w or x for the gradients
                    float* to = (kRev ? out.X : out.W) + (static_cast<size_t>(n) * A.T + c * kC + r0) * kE + e;
                    const int left = len - c * kC - r0;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < left) to[static_cast<size_t>(i) * kE] = x[i];
                }
            }
            __syncwarp();
            if (lane == 0) arrive(bar(kEmpty + s));  // this stage's rows and factors are read out
            if (!(ok = wait(kS, it))) break;
            tc_fence_after();
            if (it + 1 < nc) {
#pragma unroll 1
                for (int y = 0; y < kGroups; ++y) {
                    const int q = half * kGroups + y;
                    float S[32];
                    uint32_t w[32];
                    tmem_ld32(row + cS + 32 * q, S);
                    split32(S, w);
                    tmem_st32u(row + cB + 32 * q, w);
                    done(kState + y);
                    if (kMode == kSave || kRev) keep(w, q, kRev ? c - 1 : c + 1);
                }
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
            const int s = it & 1, c = kRev ? nc - 1 - it : c0 + it, t0 = c * kC;
            Stage<D>& st = sm.stage[s];
            if (!wait(kFull + s, it >> 1)) break;
            if (kMode == kForward) {
                // Accumulator fragments (ptx_sm100.cuh): o[x][4 j + y] is row 32 x + 8 j + 2 i + (y & 1) of
                // value column g + 8 (y >> 1), o[x][16 + ..] of column 16 further.
                float o[2][32];
                const int g = lane >> 2, i = lane & 3;
                if (!wait(kD1, it)) break;
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    tmem_ld16x256b_x4_pair(row + cD2 + 32 * x, row + cD2 + 32 * x + (16u << 16), o[x]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(bar(kD2Free));
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 m = *reinterpret_cast<const float2*>(st.eg + 32 * x + 8 * j + 2 * i);
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int z = 0; z < 4; z += 2) {
                                o[x][16 * y + 4 * j + z] *= m.x;
                                o[x][16 * y + 4 * j + z + 1] *= m.y;
                            }
                    }
                __syncwarp();
                if (lane == 0) arrive(bar(kEmpty + s));
                if (!wait(kO, it)) break;
                tc_fence_after();
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float y[32];
                    tmem_ld16x256b_x4_pair(row + cD4 + 32 * x, row + cD4 + 32 * x + (16u << 16), y);
#pragma unroll
                    for (int z = 0; z < 32; ++z) o[x][z] += y[z];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(bar(kOFree));
                const size_t step = A.bthd ? static_cast<size_t>(A.H) * kE : kE;
                const size_t at = row_at(A, b, h, A.H, t0, kE) + 32 * (warp & 3);
                const int left = len - t0;
                if (A.out_bf16) {
                    // through shared memory: rows of 64 bytes, their pieces permuted by the row
                    unsigned char* mine = sm.o[warp & 3];
                    const uint32_t base = smem_addr(mine);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int t = 32 * x + 8 * j + (lane & 7);
                            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(
                                             base + t * 64 + (((lane >> 3) ^ ((t >> 1) & 3)) << 4)),
                                         "r"(pack(o[x][4 * j], o[x][4 * j + 1])),
                                         "r"(pack(o[x][4 * j + 2], o[x][4 * j + 3])),
                                         "r"(pack(o[x][16 + 4 * j], o[x][16 + 4 * j + 1])),
                                         "r"(pack(o[x][16 + 4 * j + 2], o[x][16 + 4 * j + 3]))
                                         : "memory");
                        }
                    __syncwarp();
                    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(A.o) + at + 8 * i;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int t = 8 * y + g;
                        if (t < left)
                            *reinterpret_cast<uint4*>(p + t * step) =
                                *reinterpret_cast<const uint4*>(mine + t * 64 + ((i ^ ((t >> 1) & 3)) << 4));
                    }
                    __syncwarp();
                } else {
                    float* p = static_cast<float*>(A.o) + at + g;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int z = 0; z < 32; ++z) {
                            const int t = 32 * x + 8 * (z / 4 % 4) + 2 * i + (z & 1);
                            if (t < left) p[t * step + 16 * (z >> 4) + 8 * (z >> 1 & 1)] = o[x][z];
                        }
                }
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
        }
    }
    __syncwarp();
    // MMAs in flight end before TMEM goes: the issuer's last commit is waited for
    if (warp == 1) {
        if (elect()) mma_commit(bar(kEnd));
        drain(kEnd, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tm, 512);
}

template <int D, int kMode, bool kHold = false>
__global__ void __launch_bounds__(kThreads, 1)
gdr_walk(Args A, const ChunkWs* ws, Segments sg, int chunks, const __grid_constant__ CUtensorMap mk,
         const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mv, int* status) {
    walk_along<D, kMode, kHold>(A, ws, Saved{}, sg, chunks, mk, mq, mv, status, blockIdx.x);
}

// Both walks of a backward: the gradient of the state needs nothing of the forward
// walk, so they run side by side where the SMs suffice, the longer one's CTAs first.
// 80 sequences of 96 chunks, d = 128: 649 us (12 CTAs find no SM at first), one after
// the other 319 + 338 us.
template <int D, bool kHold = false>
__global__ void __launch_bounds__(kThreads, 1)
gdr_walks(Args A, const ChunkWs* ws, Saved out, int chunks, const __grid_constant__ CUtensorMap mk,
          const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mv,
          const __grid_constant__ CUtensorMap md, int* status) {
    const int seqs = gridDim.x / 2, block = blockIdx.x;
    const Segments whole = {1, chunks, nullptr};
    if (block < seqs) walk_along<D, kBackward, kHold>(A, ws, out, whole, chunks, mk, mq, md, status, block);
    else walk_along<D, kSave, kHold>(A, ws, out, whole, chunks, mk, mq, mv, status, block - seqs);
}

// The states that enter segments 1, 2, ..: S_{s+1} = M_s S_s + B_s in fp32, 32
// value columns per CTA (a lane each), d / 8 rows per warp; the next segment's M is
// on its way (each warp its own rows) while this one's is used.
constexpr int kJoinThreads = 256;

template <int D>
struct JoinSmem {
    float M[2][D][kE];
    float S[D][32];
};

template <int D>
__global__ void __launch_bounds__(kJoinThreads)
gdr_join(Args A, Segments sg) {
    extern __shared__ __align__(128) unsigned char join_raw[];
    JoinSmem<D>& sm = *reinterpret_cast<JoinSmem<D>*>(join_raw);
    const int seqs = A.B * A.H, n = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = 32 * blockIdx.y + lane;
    constexpr int kRows = D / (kJoinThreads / 32);
    const size_t page = static_cast<size_t>(D) * kE;
    const auto pages = [&](int s) { return sg.pages + (static_cast<size_t>(s) * seqs + n) * 3 * page; };
    const auto fetch = [&](int s) {  // M of segment s: this warp's rows
        if (s > 0 && s + 1 < sg.segs)
            for (int r = warp * kRows; r < (warp + 1) * kRows; ++r)
                cp16(smem_addr(&sm.M[s & 1][r][4 * lane]), pages(s) + page + static_cast<size_t>(r) * kE + 4 * lane, true);
        cp_commit();
    };
    fetch(0);
    for (int s = 0; s + 1 < sg.segs; ++s) {
        fetch(s + 1);
        float* at = pages(s);
        float acc[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) acc[r] = at[static_cast<size_t>(warp * kRows + r) * kE + e];
        cp_wait<1>();
        __syncthreads();
        if (s > 0) {  // the first segment's walk began with the initial state
        const float(*M)[kE] = &sm.M[s & 1][warp * kRows];
#pragma unroll 4
        for (int k = 0; k < D; k += 4) {
            const float s0 = sm.S[k][lane], s1 = sm.S[k + 1][lane], s2 = sm.S[k + 2][lane], s3 = sm.S[k + 3][lane];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float4 m = *reinterpret_cast<const float4*>(&M[r][k]);
                acc[r] = fmaf(m.x, s0, fmaf(m.y, s1, fmaf(m.z, s2, fmaf(m.w, s3, acc[r]))));
            }
        }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            sm.S[warp * kRows + r][lane] = acc[r];
            at[2 * page + static_cast<size_t>(warp * kRows + r) * kE + e] = acc[r];
        }
    }
}

}  // namespace walk
}  // namespace gdr
}  // namespace la2
