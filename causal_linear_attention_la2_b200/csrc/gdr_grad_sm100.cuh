// gdr_grad_sm100.cuh -- dq, dk, dv, dg and dbeta of the gated delta rule for d, e
// in {64, 128} on the tcgen05 tensor cores, all chunks independently, from what the
// walks left (gdr_walk_sm100.cuh, gdr_chunk.cuh): per chunk the state S0 before it, the gradient
// dS1 of the state after it, and the rows w and x.  With U = beta W:
//
//   dP = M o (dO U^T),   E_ts = -beta_t M_ts (x_t . u_s)  (s < t)
//   dq^T = S0 dO^T diag(e^G) + K^T dP^T
//   dk^T = -S0 X^T diag(beta e^G) + K^T E^T + K^T E + Q^T dP + dS1 U^T diag(e^{G_C - G})
//   dv = beta x,   dbeta_t = x_t . w_t
//   dL/dG_t = q_t . dq_t + k_t . row_t - k_t . col_t, row the first two terms of dk, col the
//   others, and <dS1, S1> more in the chunk's last row; dg: sums of dL/dG from a row to the chunk's end.
//   Most of it cancels (a pair of rows that are both summed does), so both sides are made of the
//   same operands: row from E, like col (from x and w, k_t . row_t = beta_t x_t . (w_t - v_t), what the
//   parts of E are off by stays), and with c_t = k_t . dS1 u_t e^{G_C - G_t}, the last term of
//   k_t . col_t, <dS1, S1> = e^{G_C} <dS1, S0> + sum of c_t.  (From the saved S1, whose two parts
//   are off by up to 2^-17 of a number, dg was off by up to 1e-4 of its norm where the gates close and what a chunk
//   writes is all of S1.)
//
// The products run with d on the TMEM lanes (M = d; 128 rows for dP and E, which
// are made together as [dO; X] U^T).  The scales of single rows are applied when
// the accumulators are read.  Every formed operand is a high and a low bf16 part.
//
// One persistent CTA per SM walks over (chunk, key head, value head) items.  Per
// item it reads 2 x 64 KB of states (dS1 and S0 once more, out of L2), 64 KB of w and x
// and 48 KB of rows and writes 80 KB (d = 128); the conversions of w and x and the ring of
// the state parts, one after the other, bound it.  80 sequences of 96 chunks, d = e = 128:
// 535 us; 128 of 32 chunks, d = e = 64: 165 us.  The value heads of a key head follow one
// another in one CTA, so that dq and dk are summed in their order without atomics; with
// few chunks and one key head most SMs are idle (256 rows, 16 value heads, d = e = 128,
// the whole backward: 179 us on one key head, 58 us on 16).  Warps:
//   0      loads: dO and factors, K and Q, the four state parts through a ring
//   1      MMAs
//   2      TMEM allocation;  3  dg, dbeta
//   4-19   epilogues: dP and E as operands; <dS1, S0>; dq, dk, q . dq (16 columns a warp: what a
//          warp does to an item is one long dependent chain, and 8 warps of 32
//          columns took 650 us where these took 592 us, on 80 sequences of 96 chunks)
//   20-23  w, x -> operands U, X; dv, and dbeta
// Waits are bounded as in gdr_walk_sm100.cuh.
#pragma once
#include "gdr_walk_sm100.cuh"

namespace la2 {
namespace gdr {
namespace grad {

using walk::arrive;
using walk::bulk_load;
using walk::elect;
using walk::Waiter;

constexpr int kThreads = 768;
constexpr int kEpiWarps = 16, kRowWarps = 4, kRowWarp0 = 4 + kEpiWarps;
constexpr int kFactors = 9;  // eg .. gl of ChunkWs

enum Bar { kRows = 0, kRowsFree, kKQ, kKQFree, kXU, kXUFree, kRing, kRingFree = kRing + 2, kPE = kRingFree + 2,
           kPEFull, kDone, kFree, kSums, kSumsFree = kSums + 2, kPart = kSumsFree + 2, kRaw = kPart + 2, kEpi, kEnd, kBars };

template <int D, int E>
struct Smem {
    // 64 columns of e: rows of dO, X hi, X lo (the operand [dO; X hi] and, one tile on, [X hi; X lo])
    unsigned char dx[E / 64][3][kC * 128];
    unsigned char u[E / 64][2][kC * 128];   // U hi, U lo
    unsigned char k[D / 64][kC * 128], q[D / 64][kC * 128];
    unsigned char pe[2][2][kC * 128];        // hi, lo: rows of dP, rows of E
    unsigned char ring[2][D * E * 2];       // one part of a state: [d / 8][e][8]
    float f[2][kFactors][kC];                // factors, by item parity
    float dbeta[2][kC];                      // row sums, by item parity
    float part[2][4][kC];                    // q . dq + k . (row - col) of a quadrant's rows of d, by item parity
    float dot[2][kEpiWarps];                 // <dS1, S1> in parts, by item parity
    unsigned long long bar[kBars];
    uint32_t tmem;
    int abort;
};

// Shared-memory descriptor of an operand stored as blocks of 8 M/N elements
// (16 bytes) x k, k consecutive, without a swizzle: `mn` bytes from one block of
// M/N to the next, 128 bytes from 8 k to the next 8.
__device__ __forceinline__ uint64_t sdesc_blocks(uint32_t addr, uint32_t mn) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(128 >> 4) << 16;
    d |= static_cast<uint64_t>((mn >> 4) & 0x3FFFu) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}

// 16 lanes x 16 columns of TMEM as fragments (v[4 j ..]: columns 8 j .., as in
// ptx_sm100.cuh's pair of such loads), waited for in the same statement
__device__ __forceinline__ void tmem_frag(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// kHold: la2_gdr_selftest_timeout; a tile of K of the CTA's second item is announced and not loaded
template <int D, int E, bool kHold = false>
__global__ void __launch_bounds__(kThreads, 1)
gdr_grad_tc(Args A, const ChunkWs* ws, Saved in, int chunks, int items, const __grid_constant__ CUtensorMap mk,
            const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap md, int* status) {
    extern __shared__ __align__(1024) unsigned char grad_tc_raw[];
    Smem<D, E>& sm = *reinterpret_cast<Smem<D, E>*>(grad_tc_raw);
    constexpr uint32_t kTile = kC * 128, kPiece = D * E * 2;
    constexpr uint32_t cPE = 0, cA = 128, cB = 256, cC = 384;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rep = A.H / A.Hk;
    const uint32_t bars = smem_addr(sm.bar);
    const auto bar = [&](int i) { return bars + 8 * i; };
    const Waiter<kHold> wait{bars, &sm.abort, status};
    const auto drain = [&](int i, int parity) { mbar_wait(bar(i), parity & 1, walk::kWaitNs<kHold>); };

    if (tid == 0) {
        sm.abort = 0;
        for (int i : {int(kRows), int(kKQ), kRing + 0, kRing + 1, kRingFree + 0, kRingFree + 1, int(kRowsFree), int(kXUFree),
                      int(kPE), int(kDone), int(kRaw), int(kEnd)})
            mbar_init(bar(i), 1);
        mbar_init(bar(kKQFree), kEpiWarps);
        mbar_init(bar(kXU), kRowWarps);
        mbar_init(bar(kSums), kRowWarps);
        mbar_init(bar(kSums + 1), kRowWarps);
        mbar_init(bar(kSumsFree), 1);
        mbar_init(bar(kSumsFree + 1), 1);
        mbar_init(bar(kPart), kEpiWarps);
        mbar_init(bar(kPart + 1), kEpiWarps);
        mbar_init(bar(kPEFull), kEpiWarps);
        mbar_init(bar(kFree), kEpiWarps);
        mbar_init(bar(kEpi), kEpiWarps);
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc(smem_addr(&sm.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sm.tmem != 0) {  // not seen: an allocation of every column starts at the first
        if (tid == 0) atomicCAS(status, 0, 5 | (198 << 8));
        __syncthreads();
        if (warp == 2) tmem_dealloc(sm.tmem, 512);
        return;
    }

    // Item -> chunk of a key head (consecutive items of a CTA step through the value heads of one)
    struct Item {
        int b, hk, h, c, hh, len, u;
    };
    const int units = items / rep;
    const int mine = (units - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    const auto item_at = [&](int unit, int hh) {
        Item x;
        const int u = static_cast<int>(blockIdx.x) + unit * static_cast<int>(gridDim.x);
        x.c = u % chunks;
        x.hk = u / chunks % A.Hk;
        x.b = u / chunks / A.Hk;
        x.hh = hh;
        x.u = unit;
        x.h = x.hk * rep + hh;
        x.len = length_of(A, x.b);
        return x;
    };
    // Runs body(item, its number) over this CTA's items; chunks behind a sequence's end are passed over
    const auto each = [&](auto body) {
        int y = 0;
        for (int u = 0; u < mine; ++u) {
            if (item_at(u, 0).c * kC >= item_at(u, 0).len) continue;
            for (int hh = 0; hh < rep; ++hh, ++y)
                if (!body(item_at(u, hh), y)) return y;
        }
        return y;
    };

    if (warp == 0) {
        int cuts = 0, rows = 0, kqs = 0, pieces = 0;
        each([&](const Item& x, int y) {
            const int t0 = x.c * kC;
            const size_t seq = static_cast<size_t>(x.b) * A.H + x.h, cn = seq * chunks + x.c;
            const auto tile = [&](unsigned char* to, const CUtensorMap& m, int head, int col, int on) {
                tma_load_4d(smem_addr(to), &m, bar(on), 64 * col, A.bthd ? head : t0, A.bthd ? t0 : head, x.b);
            };
            if (y > 0 && !wait(kRowsFree, y - 1)) return false;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(kRows), (E / 64) * kTile);
                for (int z = 0; z < E / 64; ++z) tile(sm.dx[z][0], md, x.h, z, kRows);
            }
            rows = y + 1;
            const size_t page = static_cast<size_t>(D) * E;
            const auto piece_in = [&](int z) {
                const int s = z & 1, p = 4 * y + z;
                if (p >= 2 && !wait(kRingFree + s, (p >> 1) - 1)) return false;
                const __nv_bfloat16* from = z < 2 ? in.S0 + cn * 2 * page + z * page
                                                  : in.dS1 + cn * 2 * page + (z - 2) * page;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(kRing + s), kPiece);
                    bulk_load(smem_addr(sm.ring[s]), from, kPiece, bar(kRing + s));
                }
                pieces = p + 1;
                return true;
            };
            if (!piece_in(0) || !piece_in(1)) return false;
            // K and Q, needed last
            if (y > 0 && !wait(kKQFree, y - 1)) return false;
            const bool cut = t0 + kC > x.len && x.len < A.T;  // rows of padding would be summed over
            if (lane == 0) {
                const int on = cut ? kRaw : kKQ;
                mbar_arrive_expect_tx(bar(on), 2 * (D / 64) * kTile);
                for (int z = 0; z < D / 64; ++z) {
                    if (!(kHold && y == 1 && z == 0)) tile(sm.k[z], mk, x.hk, z, on);
                    tile(sm.q[z], mq, x.hk, z, on);
                }
            }
            if (cut) {
                if (!wait(kRaw, cuts++)) return false;
                for (int r = x.len - t0; r < kC; ++r)
                    if (lane < 8)
#pragma unroll
                        for (int z = 0; z < D / 64; ++z) {
                            *reinterpret_cast<uint4*>(sm.k[z] + r * 128 + lane * 16) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4*>(sm.q[z] + r * 128 + lane * 16) = make_uint4(0, 0, 0, 0);
                        }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive(bar(kKQ));
            }
            kqs = y + 1;
            return piece_in(2) && piece_in(3);
        });
        // the copies in flight have landed before shared memory goes
        if (rows) drain(kRows, rows - 1);
        if (kqs) drain(kKQ, kqs - 1);
        if (cuts) drain(kRaw, cuts - 1);  // (no arrival at kKQ follows where this role gave up on them)
        for (int p = max(0, pieces - 2); p < pieces; ++p) drain(kRing + (p & 1), p >> 1);
    } else if (warp == 1) {
        constexpr uint32_t kIdPE = idesc_bf16_f32(128, 128, 0, 0), kIdPE2 = idesc_bf16_f32(128, 64, 0, 0);
        constexpr uint32_t kIdS = idesc_bf16_f32(D, 64, 1, 0), kIdSU = idesc_bf16_f32(D, 128, 1, 0);
        constexpr uint32_t kIdKT = idesc_bf16_f32(D, 64, 1, 1);
        constexpr uint32_t kDx = 3 * kTile, kU = 2 * kTile;  // strides from 64 columns of e to the next
        const uint32_t dx = smem_addr(sm.dx), u = smem_addr(sm.u);
        const uint64_t dO = sdesc_sw128(dx, 16, 1024), xh = desc_add(dO, kTile), xl = desc_add(dO, 2 * kTile);
        const uint64_t uh = sdesc_sw128(u, 16, 1024);
        each([&](const Item&, int y) {
            if (!(wait(kRows, y) && wait(kXU, y) && (y == 0 || wait(kFree, y - 1)))) return false;
            tc_fence_after();
            if (elect()) {
#pragma unroll
                for (int kk = 0; kk < E / 16; ++kk) {
                    const uint32_t a = (kk >> 2) * kDx + (kk & 3) * 32, b = (kk >> 2) * kU + (kk & 3) * 32;
                    mma_bf16_ss(cPE, desc_add(dO, a), desc_add(uh, b), kIdPE, kk > 0);
                }
#pragma unroll
                for (int kk = 0; kk < E / 16; ++kk) {
                    const uint32_t a = (kk >> 2) * kDx + (kk & 3) * 32, b = (kk >> 2) * kU + (kk & 3) * 32;
                    mma_bf16_ss(cB, desc_add(xh, a), desc_add(uh, b), kIdPE2, kk > 0);  // rows 64 ..: X lo U hi
                }
                mma_commit(bar(kPE));
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {  // S0
                const int s = z & 1, p = 4 * y + z;
                if (!wait(kRing + s, p >> 1)) return false;
                tc_fence_after();
                if (elect()) {
                    const uint64_t st = sdesc_blocks(smem_addr(sm.ring[s]), E * 16);
#pragma unroll
                    for (int kk = 0; kk < E / 16; ++kk) {
                        const uint32_t b = (kk >> 2) * kDx + (kk & 3) * 32;
                        const uint64_t a = desc_add(st, kk * 256);
                        mma_bf16_ss(cA, a, desc_add(dO, b), kIdS, z + kk > 0);
                        mma_bf16_ss(cA + 64, a, desc_add(xh, b), kIdS, z + kk > 0);
                        if (z == 0) mma_bf16_ss(cA + 64, a, desc_add(xl, b), kIdS, 1);
                    }
                    mma_commit(bar(kRingFree + s));
                }
            }
            if (elect()) mma_commit(bar(kRowsFree));  // dO is read out (X and the factors have barriers of their own)
#pragma unroll
            for (int z = 2; z < 4; ++z) {  // dS1
                const int s = z & 1, p = 4 * y + z;
                if (!wait(kRing + s, p >> 1)) return false;
                tc_fence_after();
                if (elect()) {
                    const uint64_t st = sdesc_blocks(smem_addr(sm.ring[s]), E * 16);
#pragma unroll
                    for (int kk = 0; kk < E / 16; ++kk)
                        mma_bf16_ss(cC, desc_add(st, kk * 256), desc_add(uh, (kk >> 2) * kU + (kk & 3) * 32), kIdSU,
                                    z > 2 || kk > 0);
                    mma_commit(bar(kRingFree + s));
                }
            }
            if (elect()) mma_commit(bar(kXUFree));
            if (!(wait(kKQ, y) && wait(kPEFull, y))) return false;
            tc_fence_after();
            if (elect()) {
                const uint64_t kt = sdesc_sw128(smem_addr(sm.k), kTile, 1024), qt = sdesc_sw128(smem_addr(sm.q), kTile, 1024);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const uint64_t p0 = sdesc_sw128(smem_addr(sm.pe[z]), 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)  // rows of dP and E are one operand of 128 rows
                        mma_bf16_ss(cB, desc_add(kt, kk * 2048), desc_add(p0, kk * 32), kIdSU, z + kk > 0);
                }
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const uint32_t pe = smem_addr(sm.pe[z]);
                    const uint64_t pt = sdesc_sw128(pe, kTile, 1024), et = sdesc_sw128(pe + kTile, kTile, 1024);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        mma_bf16_ss(cPE, desc_add(kt, kk * 2048), desc_add(et, kk * 2048), kIdKT, z + kk > 0);
                        mma_bf16_ss(cPE, desc_add(qt, kk * 2048), desc_add(pt, kk * 2048), kIdKT, 1);
                    }
                }
                mma_commit(bar(kDone));
            }
            return true;
        });
        if (elect()) mma_commit(bar(kEnd));
        drain(kEnd, 0);
    } else if (warp < 4) {
        if (warp == 3) each([&](const Item& x, int y) {
            const int t0 = x.c * kC, t = 2 * lane;
            if (!(wait(kPart + (y & 1), y >> 1) && wait(kSums + (y & 1), y >> 1))) return false;
            // sums of dL/dG from each row to the chunk's end: two rows per lane
            const float(*part)[kC] = sm.part[y & 1];
            float y0 = part[0][t] + part[1][t] + part[2][t] + part[3][t];
            float y1 = part[0][t + 1] + part[1][t + 1] + part[2][t + 1] + part[3][t + 1];
            // (the rows of dO behind the end are whatever lies there)
            if (t0 + t >= x.len) y0 = 0.f;
            if (t0 + t + 1 >= x.len) y1 = 0.f;
            if (lane == 31)
                for (int w = 0; w < kEpiWarps; ++w) y1 += sm.dot[y & 1][w];
            float s = y0 + y1;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const float z = __shfl_down_sync(0xffffffffu, s, m);
                if (lane + m < 32) s += z;
            }
            const float db0 = sm.dbeta[y & 1][t], db1 = sm.dbeta[y & 1][t + 1];
            __syncwarp();
            if (lane == 0) arrive(bar(kSumsFree + (y & 1)));
            const size_t at = row_at(A, x.b, x.h, A.H, t0 + t, 1), next = at + (A.bthd ? A.H : 1);
            if (t0 + t < x.len) {
                if (A.dg) A.dg[at] = s;
                A.dbeta[at] = db0;
            }
            if (t0 + t + 1 < x.len) {
                if (A.dg) A.dg[next] = s - y0;
                A.dbeta[next] = db1;
            }
            return true;
        });
    } else if (warp < kRowWarp0) {
        const int quad = warp & 3, part = (warp - 4) >> 2, g = lane >> 2, i = lane & 3;
        const uint32_t row = static_cast<uint32_t>(32 * quad) << 16;
        constexpr int kHalves = D / 64;  // groups of 16 rows of d in this warp's 32 lanes
        const int r0 = 16 * part;  // this warp's columns
        int met = 0;
        const auto meet = [&] {  // all epilogue warps, with a bounded wait
            __syncwarp();
            if (lane == 0) arrive(bar(kEpi));
            return wait(kEpi, met++);
        };
        // sums over the value heads of a key head, between two of its items: this thread's dq and dk, a value per 256
        float* sums = in.sums + static_cast<size_t>(blockIdx.x) * (2 * kHalves * 8 * 32 * kEpiWarps) + (tid - 128);
        // factors of the item that begins at or behind (u, hh), into registers and from there into f[y & 1]
        float fac[2];
        const auto fetch = [&](int u, int hh) {
            while (u < mine && item_at(u, 0).c * kC >= item_at(u, 0).len) ++u;
            if (u >= mine) return;
            const Item x = item_at(u, hh);
            const float* from = ws[(static_cast<size_t>(x.b) * A.H + x.h) * chunks + x.c].eg;
#pragma unroll
            for (int z = 0; z < 2; ++z)
                if (tid - 128 + z * 32 * kEpiWarps < kFactors * kC) fac[z] = from[tid - 128 + z * 32 * kEpiWarps];
        };
        const auto store = [&](int y) {
#pragma unroll
            for (int z = 0; z < 2; ++z)
                if (tid - 128 + z * 32 * kEpiWarps < kFactors * kC) sm.f[y & 1][0][tid - 128 + z * 32 * kEpiWarps] = fac[z];
        };
        fetch(0, 0);
        store(0);
        if (meet()) each([&](const Item& x, int y) {
            const int t0 = x.c * kC;
            const float(*f)[kC] = sm.f[y & 1];
            const float *eg = f[0], *rest = f[1], *neg_beta = f[4], *neg_beta_eg = f[6], *G = f[7], *Gl = f[8];
            if (x.hh + 1 < rep) fetch(x.u, x.hh + 1);
            else fetch(x.u + 1, 0);
            if (!wait(kPE, y)) return false;
            tc_fence_after();
            {  // rows 0 .. 63: dP, 64 .. 127: E; this thread's row, columns r0 ..
                const int r = 32 * quad + lane, t = r & 63;
                const bool isE = r >= 64;
                float v[16], z[16];
                uint32_t w[16];
                tmem_ld16(row + cPE + r0, v);
                tmem_ld16(row + cPE + 64 + r0, z);
#pragma unroll
                for (int s = 0; s < 16; ++s) v[s] += z[s];
                if (quad >= 2) {
                    tmem_ld16(row + cB + r0, z);
#pragma unroll
                    for (int s = 0; s < 16; ++s) v[s] += z[s];
                }
                const float gt = G[t], gtl = Gl[t], m = isE ? neg_beta[t] : 1.f;
                const int last = t0 + t < x.len ? (isE ? t - 1 : t) : -1;  // columns 0 .. last are below the diagonal
#pragma unroll
                for (int s = 0; s < 16; s += 4) {
                    const float4 gs = *reinterpret_cast<const float4*>(G + r0 + s);
                    const float4 gl = *reinterpret_cast<const float4*>(Gl + r0 + s);
                    const float e4[4] = {(gt - gs.x) + (gtl - gl.x), (gt - gs.y) + (gtl - gl.y), (gt - gs.z) + (gtl - gl.z),
                                         (gt - gs.w) + (gtl - gl.w)};
#pragma unroll
                    for (int y4 = 0; y4 < 4; ++y4) {
                        // (above the diagonal the power may be infinite, and is not used)
                        const float on = v[s + y4] * (m * exp2_flat(e4[y4]));
                        v[s + y4] = r0 + s + y4 <= last ? on : 0.f;
                    }
                }
#pragma unroll
                for (int y2 = 0; y2 < 8; ++y2) split_pack2v(make_float2(v[2 * y2], v[2 * y2 + 1]), w[y2], w[8 + y2]);
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    st_shared_v4(smem_addr(sm.pe[p >> 1][isE]) + piece<128>(t, 2 * part + (p & 1)), w[4 * p], w[4 * p + 1],
                                 w[4 * p + 2], w[4 * p + 3]);
            }
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(bar(kPEFull));
            // <dS1, S0> out of L2 while the last products run: a share of the 16-byte pieces per thread
            float dot;
            {
                const size_t seq = static_cast<size_t>(x.b) * A.H + x.h, page = static_cast<size_t>(D) * E;
                const uint4* s0 = reinterpret_cast<const uint4*>(in.S0 + (seq * chunks + x.c) * 2 * page);
                const uint4* d1 = reinterpret_cast<const uint4*>(in.dS1 + (seq * chunks + x.c) * 2 * page);
                constexpr int kPieces = D * E / 8, kStep = 32 * kEpiWarps;  // of one part
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int z0 = 0; z0 < kPieces; z0 += 2 * kStep) {
                    uint4 v[2][4];
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (z0 + r * kStep < kPieces) {
                            const int z = z0 + r * kStep + tid - 128;
                            v[r][0] = s0[z];
                            v[r][1] = s0[z + kPieces];
                            v[r][2] = d1[z];
                            v[r][3] = d1[z + kPieces];
                        }
                    const auto take = [&](uint32_t sh, uint32_t sl, uint32_t dh, uint32_t dl) {
                        const float2 s2 = make_float2(low_of(sh) + low_of(sl), high_of(sh) + high_of(sl));
                        const float2 d2 = make_float2(low_of(dh) + low_of(dl), high_of(dh) + high_of(dl));
                        sum = fma2(s2, d2, sum);
                    };
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (z0 + r * kStep < kPieces) {
                            take(v[r][0].x, v[r][1].x, v[r][2].x, v[r][3].x);
                            take(v[r][0].y, v[r][1].y, v[r][2].y, v[r][3].y);
                            take(v[r][0].z, v[r][1].z, v[r][2].z, v[r][3].z);
                            take(v[r][0].w, v[r][1].w, v[r][2].w, v[r][3].w);
                        }
                }
                dot = eg[kC - 1] * (sum.x + sum.y);
            }
            if (!(wait(kDone, y) && wait(kKQ, y) && (y < 2 || wait(kSumsFree + (y & 1), (y >> 1) - 1)))) return false;
            tc_fence_after();
            // dq and dk of this item: rows 16 hb + g (+ 8) of d in this quadrant, columns 8 j + 2 i (+ 1) of this half
            // (D = 64: M = 64 puts 16 rows into each quadrant)
            // of += (factor of the column) accumulator, column block `col`
            const auto add = [&](uint32_t col, float (&of)[kHalves * 8], const float* f2) {
#pragma unroll
                for (int hb = 0; hb < kHalves; ++hb) {
                    float a[8];
                    tmem_frag(row + col + r0 + (static_cast<uint32_t>(16 * hb) << 16), a);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float2 m = make_float2(1.f, 1.f);
                        if (f2) m = *reinterpret_cast<const float2*>(f2 + r0 + 8 * j + 2 * i);
#pragma unroll
                        for (int z = 4 * j; z < 4 * j + 4; z += 2) {
                            of[8 * hb + z] = fmaf(a[z], m.x, of[8 * hb + z]);
                            of[8 * hb + z + 1] = fmaf(a[z + 1], m.y, of[8 * hb + z + 1]);
                        }
                    }
                }
            };
            const bool first = x.hh == 0, last_head = x.hh == rep - 1;
            const size_t step = A.bthd ? static_cast<size_t>(A.Hk) * D : D;
            const int d_at = (D / 4) * quad, left = x.len - t0;
            const size_t out_at = row_at(A, x.b, x.hk, A.Hk, t0, D) + d_at;
            float nq[kHalves * 8] = {}, nk[kHalves * 8] = {};  // dq and dk of this item
            // dq (o = 0) or dk (o = 1) added to the heads before, and kept or written out
            const auto finish = [&](float (&now)[kHalves * 8], int o, void* out) {
                float* sum = sums + o * (kHalves * 8 * 32 * kEpiWarps);
                if (!first)
#pragma unroll
                    for (int z = 0; z < kHalves * 8; ++z) now[z] += sum[z * 32 * kEpiWarps];
                if (!last_head) {
#pragma unroll
                    for (int z = 0; z < kHalves * 8; ++z) sum[z * 32 * kEpiWarps] = now[z];
                } else if (A.out_bf16) {
                    // through this warp's part of the dP, E operand, which the MMAs have read: [16 rows][16 or 32 columns]
                    constexpr int kRow = 2 * (D / 4), kPc = kRow / 16;  // bytes and pieces of a row
                    unsigned char* to = sm.pe[0][0] + (2 * (warp - 4) + o) * (2 * kC * 128 / kEpiWarps);
#pragma unroll
                    for (int hb = 0; hb < kHalves; ++hb) {
                        const int m = lane >> 3, t = 8 * (m >> 1) + (lane & 7), p = 2 * hb + (m & 1), z = 8 * hb;
                        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(
                                         smem_addr(to) + t * kRow + ((p ^ ((t >> 1) & (kPc - 1))) << 4)),
                                     "r"(pack(now[z], now[z + 1])), "r"(pack(now[z + 2], now[z + 3])),
                                     "r"(pack(now[z + 4], now[z + 5])), "r"(pack(now[z + 6], now[z + 7]))
                                     : "memory");
                    }
                    __syncwarp();
                    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(out) + out_at;
#pragma unroll
                    for (int z = lane; z < 16 * kPc; z += 32) {
                        const int t = z / kPc, c = z % kPc;
                        if (r0 + t < left)
                            *reinterpret_cast<uint4*>(p + (r0 + t) * step + 8 * c) =
                                *reinterpret_cast<const uint4*>(to + t * kRow + ((c ^ ((t >> 1) & (kPc - 1))) << 4));
                    }
                } else {
                    float* p = static_cast<float*>(out) + out_at;
#pragma unroll
                    for (int z = 0; z < kHalves * 8; ++z) {
                        const int t = r0 + 8 * (z / 4 % 2) + 2 * i + (z & 1);
                        if (t < left) p[t * step + g + 16 * (z >> 3) + 8 * (z >> 1 & 1)] = now[z];
                    }
                }
            };
            add(cC, nk, rest);
            add(cC + 64, nk, rest);
            float s[4] = {};  // of columns 8 (j / 2) + 2 i + j % 2: this warp's rows of d of q . dq + k . (row - col)
            const auto along = [&](const unsigned char (*rows)[kC * 128], const float (&of)[kHalves * 8], float sign) {
#pragma unroll
                for (int hb = 0; hb < kHalves; ++hb) {
                    // fragments of the transposed tile: rows of d, columns t, of the two tiles of this warp's columns
                    const int d0 = d_at + 16 * hb, m = lane >> 3;
                    uint32_t qq[4];
                    ldsm_t(qq, smem_addr(rows[d0 >> 6]) +
                                   piece<128>(r0 + 8 * (m >> 1) + (lane & 7), ((d0 & 63) >> 3) + (m & 1)));
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int at = 8 * hb + 4 * z, j = 2 * z;
                        s[j] = fmaf(sign * low_of(qq[2 * z]), of[at], fmaf(sign * low_of(qq[2 * z + 1]), of[at + 2], s[j]));
                        s[j + 1] = fmaf(sign * high_of(qq[2 * z]), of[at + 1],
                                        fmaf(sign * high_of(qq[2 * z + 1]), of[at + 3], s[j + 1]));
                    }
                }
            };
            along(sm.k, nk, 1.f);
            dot += (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
            for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = 0.f;
            add(cPE, nk, nullptr);
            along(sm.k, nk, -2.f);
            add(cA + 64, nk, neg_beta_eg);
            add(cB + 64, nk, nullptr);
            along(sm.k, nk, 1.f);  // row + col - 2 col
            add(cA, nq, eg);
            add(cB, nq, nullptr);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(bar(kFree));  // the accumulators are read out: the next item's products may begin
            {
                along(sm.q, nq, 1.f);
                // 4 sums over the 8 lanes of equal i, halving what a lane holds: lanes of g / 2 = j end with sum j
#pragma unroll
                for (int m = 16, held = 2; m >= 8; m >>= 1, held >>= 1)
#pragma unroll
                    for (int z = 0; z < 2; ++z)
                        if (z < held) {
                            const bool up = lane & m;
                            const float give = up ? s[z] : s[held + z], keep = up ? s[held + z] : s[z];
                            s[z] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                        }
                s[0] += __shfl_xor_sync(0xffffffffu, s[0], 4);
                if (!(g & 1)) sm.part[y & 1][quad][r0 + 8 * (g >> 2) + 2 * i + (g >> 1 & 1)] = s[0];
            }
            if (lane == 0) sm.dot[y & 1][warp - 4] = dot;
            __syncwarp();
            if (lane == 0) {
                arrive(bar(kPart + (y & 1)));
                arrive(bar(kKQFree));
            }
            finish(nq, 0, A.dq);
            finish(nk, 1, A.dk);
            store(y + 1);
            // what was staged in the place of dP and E is read out, and the next item's factors are there
            return meet();
        });
    } else {
        each([&](const Item& x, int y) {
            // E / 4 lanes hold a row, four columns each: a slot is one row (E = 128) or two (E = 64)
            constexpr int kLanes = E / 4, kPer = 32 / kLanes;
            const int t0 = x.c * kC, col = 4 * (lane % kLanes);
            const size_t seq = static_cast<size_t>(x.b) * A.H + x.h;
            const ChunkWs& cw = ws[seq * chunks + x.c];
            const size_t step = A.bthd ? static_cast<size_t>(A.H) * E : E;
#pragma unroll 1
            for (int z = 0; z < 4 / kPer; ++z) {  // 4 slots at a time, all loads first
                const int row0 = 16 * (warp - kRowWarp0) + 4 * kPer * z + lane / kLanes;  // of slot 0; slot r: kPer r further
                const int left = x.len - t0 - row0;
                const size_t io = row_at(A, x.b, x.h, A.H, t0 + row0, E) + col;
                float4 w[4], xx[4];
                float bt[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    w[r] = xx[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                    bt[r] = 0.f;
                    if (kPer * r < left) {
                        const size_t at = (seq * A.T + t0 + row0 + kPer * r) * E + col;
                        w[r] = *reinterpret_cast<const float4*>(in.W + at);
                        xx[r] = *reinterpret_cast<const float4*>(in.X + at);
                        bt[r] = cw.beta[row0 + kPer * r];
                    }
                }
                // the MMAs have read the operands of the item before, warp 3 the row sums of the one before that
                if (z == 0 && y > 0 && !wait(kXUFree, y - 1)) return false;
                if (z == 0 && y > 1 && !wait(kSumsFree + (y & 1), (y >> 1) - 1)) return false;
                float sum[4];  // of each slot: x . w
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t at = piece<128>(row0 + kPer * r, (col & 63) >> 3) + 2 * (col & 7);
                    uint32_t h0, h1, l0, l1;
                    split(bt[r] * w[r].x, bt[r] * w[r].y, h0, l0);
                    split(bt[r] * w[r].z, bt[r] * w[r].w, h1, l1);
                    *reinterpret_cast<uint2*>(sm.u[col >> 6][0] + at) = make_uint2(h0, h1);
                    *reinterpret_cast<uint2*>(sm.u[col >> 6][1] + at) = make_uint2(l0, l1);
                    split(xx[r].x, xx[r].y, h0, l0);
                    split(xx[r].z, xx[r].w, h1, l1);
                    *reinterpret_cast<uint2*>(sm.dx[col >> 6][1] + at) = make_uint2(h0, h1);
                    *reinterpret_cast<uint2*>(sm.dx[col >> 6][2] + at) = make_uint2(l0, l1);
                    sum[r] = fmaf(xx[r].x, w[r].x, fmaf(xx[r].y, w[r].y, fmaf(xx[r].z, w[r].z, xx[r].w * w[r].w)));
                }
                // 4 sums over the lanes of a row, halving what a lane holds with each exchange
#pragma unroll
                for (int m = kLanes / 2, held = 2; held > 0; m >>= 1, held >>= 1)
#pragma unroll
                    for (int y2 = 0; y2 < 2; ++y2)
                        if (y2 < held) {
                            const bool up = lane & m;
                            const float give = up ? sum[y2] : sum[held + y2], keep = up ? sum[held + y2] : sum[y2];
                            sum[y2] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                        }
#pragma unroll
                for (int m = kLanes / 8; m; m >>= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], m);
                const int mine_ = lane % kLanes / (kLanes / 4);  // which sum this lane ended with
                if (lane % (kLanes / 4) == 0) sm.dbeta[y & 1][row0 + kPer * mine_] = sum[0];
                if (A.out_bf16) {
                    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(A.dv) + io;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (kPer * r < left)
                            *reinterpret_cast<uint2*>(p + kPer * r * step) = make_uint2(
                                pack(bt[r] * xx[r].x, bt[r] * xx[r].y), pack(bt[r] * xx[r].z, bt[r] * xx[r].w));
                } else {
                    float* p = static_cast<float*>(A.dv) + io;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (kPer * r < left)
                            *reinterpret_cast<float4*>(p + kPer * r * step) =
                                make_float4(bt[r] * xx[r].x, bt[r] * xx[r].y, bt[r] * xx[r].z, bt[r] * xx[r].w);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                arrive(bar(kSums + (y & 1)));
                arrive(bar(kXU));
            }
            return true;
        });
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(sm.tmem, 512);
}

}  // namespace grad
}  // namespace gdr
}  // namespace la2
