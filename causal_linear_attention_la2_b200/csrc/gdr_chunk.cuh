// gdr_chunk.cuh -- the gated delta rule by chunks of C = 64 rows on the tensor
// cores, for bf16 inputs with d, e in {64, 128}.
//
// With G_t the cumulative gates of a chunk, S0 the state before it and
// Ah_ts = e^{G_t - G_s} (k_t . k_s) (s < t), P_ts = e^{G_t - G_s} (q_t . k_s) (s <= t),
// the rows w_t of the chunk solve (I + Ah diag(beta)) W = Z, Z = V - diag(e^G) K S0.
// With N = (I + Ah diag(beta))^{-1} Ah (strictly lower) both inverses that the two directions need are plain:
//
//   (I + Ah diag(beta))^{-1} = I - N diag(beta),  (I + diag(beta) Ah)^{-1} = I - diag(beta) N,
//
// without dividing by beta (which may be 0).  So
//
//   W = Z - N (beta Z),   U = beta W,
//   O = diag(e^G) Q S0 + P U,   S1 = e^{G_C} S0 + K^T (e^{G_C - G} U),
//
// and backward, with dS1 the gradient of the state after the chunk,
//
//   dU = P^T dO + e^{G_C - G} K dS1,   X = dU - N^T (beta dU),   dV = beta X,
//   dS0 = e^{G_C} dS1 + Q^T (e^G dO) - K^T (beta e^G X).
//
// gdr_prep makes N and P of all chunks at once; gdr_chain and gdr_chains walk
// the chunks of a sequence for e = 64 (gdr_walk_sm100.cuh for e = 128);
// gdr_grad_tc (gdr_grad_sm100.cuh), again for all chunks at once, makes dq, dk,
// dv, dg and dbeta.
//
// Precision: q, k, v, dO enter the products as they are (bf16, exact); every
// operand that is formed here (states, N, P, W, X, dP, E) is split into a high
// and a low bf16 part, at most 2^-17 of the value being lost (half a step of the
// low part, which is at most 2^-8 of the value), and the product of two low parts, at
// most 2^-16 of a product, is dropped.  That leaves fp32 results 3e-6 to 9e-6 of their
// norm off (fp32 throughout: 1e-7 to 5e-7), far below the rounding of bf16 outputs
// (2^-8 of a value); a third part would take the products of each operand from two to
// three and the states on the chunk borders from 4 to 6 bytes a number.  Sums, the
// states that are carried and exponentials are fp32; cumulative gates are fp64 sums
// kept as two floats.
//
// The walks run transposed, S^T [e][d] with 16 rows (value columns of the
// state, which do not interact) per warp: the accumulator fragment of one
// product is the A fragment of the next (the 16 x 8 accumulator of two
// neighbouring tiles is the 16 x 16 operand), so the state and everything formed
// from it stay in the registers of one warp from the first row to the last,
// and the warps of a CTA share only the tiles of K, Q, N and P.
#pragma once
#include <type_traits>

#include "gdr_common.cuh"
#include "ptx_sm100.cuh"

namespace la2 {
namespace gdr {

constexpr int kC = 64;

// Workspace of one chunk of one value head: N and P, each as a high and a low
// 64 x 64 bf16 image (row t of 128 bytes, 16-byte pieces permuted by t % 8, as
// they lie in shared memory), and the factors of each row: e^G, e^{G_C - G}, beta
// and what the walks multiply by, and G / ln 2 as two floats.
struct ChunkWs {
    unsigned char img[4][kC * kC * 2];  // N hi, N lo, P hi, P lo
    float eg[kC], rest[kC], beta[kC];
    float neg_eg[kC], neg_beta[kC], rest_beta[kC], neg_beta_eg[kC];
    float g[kC], gl[kC];
};
constexpr int kCoefs = 7;  // eg .. neg_beta_eg
static_assert(sizeof(ChunkWs) % 256 == 0, "chunks stay 256-byte aligned");

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
    const int n = ok ? 16 : 0;  // 0: zeros, src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack(float x, float y) {  // x in the low half
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}
__device__ __forceinline__ float low_of(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float high_of(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// (x, y) as a high and a low pair of bf16
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack(x, y);
    lo = pack(x - low_of(hi), y - high_of(hi));
}

// The A fragments of columns 16 kk .. 16 kk + 15 of an accumulator
__device__ __forceinline__ void frag_split(const float (&c0)[4], const float (&c1)[4], uint32_t (&h)[4],
                                           uint32_t (&l)[4]) {
    split(c0[0], c0[1], h[0], l[0]);
    split(c0[2], c0[3], h[1], l[1]);
    split(c1[0], c1[1], h[2], l[2]);
    split(c1[2], c1[3], h[3], l[3]);
}

// Byte offset of 16-byte piece `p` of row `r` in a tile of rows of `kBytes`
// bytes, the pieces permuted so that eight rows' equal pieces fall into
// different banks.
template <int kBytes>
__device__ __forceinline__ uint32_t piece(int r, int p) {
    return static_cast<uint32_t>(r * kBytes + ((p ^ (r & 7)) << 4));
}

// The four fragment addressings of ldmatrix; rows of kBytes bytes.
// rows [n][k]: B fragments of n tiles 2 jp, 2 jp + 1 (b[0..1], b[2..3]), k step kk
template <int kBytes>
__device__ __forceinline__ void ld_b(uint32_t (&b)[4], uint32_t tile, int jp, int kk, int lane) {
    const int m = lane >> 3, r = lane & 7;
    ldsm(b, tile + piece<kBytes>(8 * (2 * jp + (m >> 1)) + r, 2 * kk + (m & 1)));
}
// rows [k][n]: the same fragments from the transposed tile
template <int kBytes>
__device__ __forceinline__ void ld_bt(uint32_t (&b)[4], uint32_t tile, int jp, int kk, int lane) {
    const int m = lane >> 3, r = lane & 7;
    ldsm_t(b, tile + piece<kBytes>(16 * kk + (m & 1) * 8 + r, 2 * jp + (m >> 1)));
}
// rows [m][k]: A fragment of rows 16 mi .., k step kk
template <int kBytes>
__device__ __forceinline__ void ld_a(uint32_t (&a)[4], uint32_t tile, int mi, int kk, int lane) {
    const int m = lane >> 3, r = lane & 7;
    ldsm(a, tile + piece<kBytes>(16 * mi + (m & 1) * 8 + r, 2 * kk + (m >> 1)));
}
// rows [k][m]: the same fragment from the transposed tile; as accumulator
// values: a[0], a[1] tile 2 kk (rows g, g + 8), a[2], a[3] tile 2 kk + 1
template <int kBytes>
__device__ __forceinline__ void ld_at(uint32_t (&a)[4], uint32_t tile, int mi, int kk, int lane) {
    const int m = lane >> 3, r = lane & 7;
    ldsm_t(a, tile + piece<kBytes>(16 * kk + (m >> 1) * 8 + r, 2 * mi + (m & 1)));
}

__device__ __forceinline__ void mma2(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[4], const uint32_t (&b)[4]) {
    mma(c0, a, b[0], b[1]);
    mma(c1, a, b[2], b[3]);
}

// Rows t0 .. t0 + 63 (those behind `len` as zeros) of W columns from column c0
// of a bf16 tensor of `width` columns into a tile of rows of 2 W bytes.
template <int W, int kThreads>
__device__ __forceinline__ void load_tile(uint32_t tile, const Args& A, const void* src, int b, int h, int nh,
                                          int width, int c0, int t0, int len) {
    constexpr int kPieces = W / 8, kStep = kThreads / kPieces;
    static_assert(kThreads % kPieces == 0 && kC % kStep == 0 && kStep % 8 == 0, "whole rows, one permutation per thread");
    const int r = threadIdx.x / kPieces, c = threadIdx.x % kPieces;
    const size_t step = static_cast<size_t>(kStep) * width * (A.bthd ? nh : 1);
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(src);
    const __nv_bfloat16* p = base + row_at(A, b, h, nh, t0 + r, width) + c0 + 8 * c;
    const uint32_t to = tile + piece<2 * W>(r, c);
#pragma unroll
    for (int x = 0; x < kC / kStep; ++x, p += step) {
        const bool ok = t0 + r + x * kStep < len;
        cp16(to + x * kStep * 2 * W, ok ? p : base, ok);
    }
}

template <int kThreads>
__device__ __forceinline__ void load_bytes(uint32_t dst, const void* src, int bytes) {
    for (int x = threadIdx.x * 16; x < bytes; x += kThreads * 16)
        cp16(dst + x, static_cast<const char*>(src) + x, true);
}

// ------------------------------------------------------------------ gdr_prep

constexpr int kPrepThreads = 256;
constexpr int kPitchA = kC + 8, kPitchN = kC + 4;  // floats per row in shared memory

template <int D>
struct PrepSmem {  // four CTAs per SM
    union {
        unsigned char kq[2][kC * D * 2];
        struct {
            union {
                float a[kC][kPitchA];                // Ah
                unsigned char nimg[2][kC * kC * 2];  // N as two images, when Ah is read out
            };
            float n[kC][kPitchN];  // N
        };
    };
    unsigned char pimg[2][kC * kC * 2];
    struct {
        float eg[kC], rest[kC], beta[kC];
        float neg_eg[kC], neg_beta[kC], rest_beta[kC], neg_beta_eg[kC];
        float g[kC], gl[kC];
    } out;  // as at the end of ChunkWs
};

// (x, y) as three pairs of bf16: all 24 bits of the significand
__device__ __forceinline__ void split3(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
    h = pack(x, y);
    x -= low_of(h);
    y -= high_of(h);
    split(x, y, m, l);
}

// acc (rows tr .., columns sc .. of a 16 x 8 tile) -= M diag(beta) n over r0 ..
// r0 + 16 kSteps, M and n fp32 in shared memory.  Both are split into three bf16
// parts (2^-24 is lost, as in fp32): where keys repeat the terms cancel, and what
// two parts lose of them shows in N.
template <int kSteps, int kPitchM>
__device__ __forceinline__ void take(float (&acc)[4], const float (*M)[kPitchM], const float (*n)[kPitchN],
                                     const float* beta, int tr, int sc, int r0, int lane) {
    const int g = lane >> 2, i = lane & 3;
#pragma unroll
    for (int kk = 0; kk < kSteps; ++kk) {
        uint32_t ah[4], am[4], al[4], bh[2], bm[2], bl[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = r0 + 16 * kk + 8 * x + 2 * i;
            const float2 b2 = *reinterpret_cast<const float2*>(beta + r);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float2 m = *reinterpret_cast<const float2*>(&M[tr + g + 8 * y][r]);
                split3(-b2.x * m.x, -b2.y * m.y, ah[2 * x + y], am[2 * x + y], al[2 * x + y]);
            }
            split3(n[r][sc + g], n[r + 1][sc + g], bh[x], bm[x], bl[x]);
        }
        mma(acc, al, bh[0], bh[1]);
        mma(acc, am, bm[0], bm[1]);
        mma(acc, ah, bl[0], bl[1]);
        mma(acc, am, bh[0], bh[1]);
        mma(acc, ah, bm[0], bm[1]);
        mma(acc, ah, bh[0], bh[1]);
    }
}

// Shared memory to global memory past the registers; what was written has been fenced
__device__ __forceinline__ void store_bulk(void* to, const void* from, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(smem_addr(from)), "r"(bytes)
                 : "memory");
}

// N and P of one chunk: warps 0-3 make 16 rows of K K^T each, warps 4-7 of Q K^T.
//
// N = (I + Ah diag(beta))^{-1} Ah by halves: with the blocks of the first and
// second half of the rows,
//   N11, N22 as for a chunk of half the length,
//   Y = Ah21 - Ah21 diag(beta1) N11,   N21 = Y - N22 diag(beta2) Y,
// four blocks of 16 by forward substitution in fp32 (a thread per column,
// N_ts = Ah_ts - sum_{s < r < t} Ah_tr beta_r N_rs), then 16 -> 32 -> 64 on the
// tensor cores.  A substitution over all 64 rows is a chain four
// times as long with most threads idle (7680 chunks of d = 128: 355 us, 257 us
// with the joins on the SIMT cores, 158 us as it is).  What is left is a row of short
// phases with a barrier between them, four CTAs per SM in different ones: 11 us a
// chunk, against 77 us for the bytes.
template <int D>
__global__ void __launch_bounds__(kPrepThreads, 4)
gdr_prep(Args A, ChunkWs* ws, int chunks) {
    extern __shared__ __align__(128) unsigned char prep_raw[];
    PrepSmem<D>& sm = *reinterpret_cast<PrepSmem<D>*>(prep_raw);
    const int c = blockIdx.x % chunks, n = blockIdx.x / chunks, b = n / A.H, h = n % A.H;
    const int len = length_of(A, b), t0 = c * kC;
    if (t0 >= len) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hk = h / (A.H / A.Hk);
    const uint32_t kt = smem_addr(sm.kq[0]), qt = smem_addr(sm.kq[1]);
    load_tile<D, kPrepThreads>(kt, A, A.k, b, hk, A.Hk, A.d, 0, t0, len);
    load_tile<D, kPrepThreads>(qt, A, A.q, b, hk, A.Hk, A.d, 0, t0, len);
    cp_commit();
    if (warp == 0) {  // gates: two rows per lane, rows behind the end keep everything and write nothing
        const int t = 2 * lane;
        double g0 = 0.0, g1 = 0.0;
        float b0 = 0.f, b1 = 0.f;
        if (t0 + t < len) {
            const size_t at = row_at(A, b, h, A.H, t0 + t, 1);
            g0 = gate_at(A, at);
            b0 = A.beta[at];
        }
        if (t0 + t + 1 < len) {
            const size_t at = row_at(A, b, h, A.H, t0 + t + 1, 1);
            g1 = gate_at(A, at);
            b1 = A.beta[at];
        }
        double s = g0 + g1;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, s, m);
            if (lane >= m) s += y;
        }
        s *= 1.4426950408889634;  // in powers of two from here on
        g1 *= 1.4426950408889634;
        const double all = __shfl_sync(0xffffffffu, s, 31), first = s - g1;
        sm.out.g[t] = static_cast<float>(first);
        sm.out.g[t + 1] = static_cast<float>(s);
        sm.out.gl[t] = static_cast<float>(first - sm.out.g[t]);
        sm.out.gl[t + 1] = static_cast<float>(s - sm.out.g[t + 1]);
        sm.out.eg[t] = exp2f(sm.out.g[t]) * (1.f + 0.6931472f * sm.out.gl[t]);
        sm.out.eg[t + 1] = exp2f(sm.out.g[t + 1]) * (1.f + 0.6931472f * sm.out.gl[t + 1]);
        sm.out.rest[t] = exp2f(static_cast<float>(all - first));
        sm.out.rest[t + 1] = exp2f(static_cast<float>(all - s));
        sm.out.beta[t] = b0;
        sm.out.beta[t + 1] = b1;
#pragma unroll
        for (int y = t; y < t + 2; ++y) {
            const float bt = sm.out.beta[y];
            sm.out.neg_eg[y] = -sm.out.eg[y];
            sm.out.neg_beta[y] = -bt;
            sm.out.rest_beta[y] = sm.out.rest[y] * bt;
            sm.out.neg_beta_eg[y] = -bt * sm.out.eg[y];
        }
        fence_proxy_async_smem();
    }
    cp_wait<0>();
    __syncthreads();
    const int g = lane >> 2, i = lane & 3, rt = warp & 3;
    const bool isq = warp >= 4;
    float acc[8][4] = {};
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t aa[4], bb[4];
        ld_a<2 * D>(aa, isq ? qt : kt, rt, kk, lane);
#pragma unroll
        for (int jp = 0; jp < 4; ++jp) {
            if (jp <= rt) {
                ld_b<2 * D>(bb, kt, jp, kk, lane);
                mma2(acc[2 * jp], acc[2 * jp + 1], aa, bb);
            }
        }
    }
    __syncthreads();  // K and Q are read out: a and n take their place
    const float* beta = sm.out.beta;
    const float gt[2] = {sm.out.g[16 * rt + g], sm.out.g[16 * rt + g + 8]};
    const float gtl[2] = {sm.out.gl[16 * rt + g], sm.out.gl[16 * rt + g + 8]};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 gs = *reinterpret_cast<const float2*>(&sm.out.g[8 * j + 2 * i]);
        const float2 gsl = *reinterpret_cast<const float2*>(&sm.out.gl[8 * j + 2 * i]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = 16 * rt + g + 8 * half, s = 8 * j + 2 * i;
            float x[2] = {0.f, 0.f};
            if (j <= 2 * rt + 1) {
                const int last = isq ? t : t - 1;  // P has its diagonal, Ah has not
                const float m0 = exp2_flat((gt[half] - gs.x) + (gtl[half] - gsl.x));
                const float m1 = exp2_flat((gt[half] - gs.y) + (gtl[half] - gsl.y));
                x[0] = s <= last ? acc[j][2 * half] * m0 : 0.f;  // (above the diagonal m may be infinite)
                x[1] = s + 1 <= last ? acc[j][2 * half + 1] * m1 : 0.f;
            }
            if (isq) {
                uint32_t hi, lo;
                split(x[0], x[1], hi, lo);
                const uint32_t at = piece<128>(t, j) + 4 * i;
                *reinterpret_cast<uint32_t*>(sm.pimg[0] + at) = hi;
                *reinterpret_cast<uint32_t*>(sm.pimg[1] + at) = lo;
            } else {
                *reinterpret_cast<float2*>(&sm.a[t][s]) = make_float2(x[0], x[1]);
            }
        }
    }
    if (isq) fence_proxy_async_smem();
    __syncthreads();
    ChunkWs& to = ws[static_cast<size_t>(n) * chunks + c];
    const bool storer = tid == kPrepThreads - 1;
    if (storer) {
        store_bulk(to.img[2], sm.pimg, sizeof(sm.pimg));
        store_bulk(to.eg, &sm.out, sizeof(sm.out));
    }
    if (tid < kC) {  // blocks of 16: column tid
        const int r0 = tid & ~15, sl = tid & 15;
        float bN[16];
        bN[0] = 0.f;
        sm.n[r0][tid] = 0.f;
#pragma unroll
        for (int t = 1; t < 16; ++t) {
            float x0 = sm.a[r0 + t][tid], x1 = 0.f;
#pragma unroll
            for (int r = 0; r < t; r += 4) {
                const float4 y = *reinterpret_cast<const float4*>(&sm.a[r0 + t][r0 + r]);
                x0 = fmaf(-y.x, bN[r], x0);
                if (r + 1 < t) x1 = fmaf(-y.y, bN[r + 1], x1);
                if (r + 2 < t) x0 = fmaf(-y.z, bN[r + 2], x0);
                if (r + 3 < t) x1 = fmaf(-y.w, bN[r + 3], x1);
            }
            const float x = t > sl ? x0 + x1 : 0.f;
            sm.n[r0 + t][tid] = x;
            bN[t] = beta[r0 + t] * x;
        }
    } else if (tid < 2 * kC) {  // the blocks right of the diagonal that the last join reads
        const int r0 = (tid >> 5 & 1) * 32, t = r0 + (tid >> 1 & 15), s = r0 + 16 + 8 * (tid & 1);
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(&sm.n[t][s]) = z;
        *reinterpret_cast<float4*>(&sm.n[t][s + 4]) = z;
    }
    __syncthreads();
    const auto join = [&](auto steps, int r0, int tr, int sc, bool on) {  // halves of `half` rows from r0
        constexpr int half = 16 * decltype(steps)::value;
        float y[4] = {};
        const auto put = [&] {
            if (on) {
                *reinterpret_cast<float2*>(&sm.n[tr + g][sc + 2 * i]) = make_float2(y[0], y[1]);
                *reinterpret_cast<float2*>(&sm.n[tr + g + 8][sc + 2 * i]) = make_float2(y[2], y[3]);
            }
            __syncthreads();
        };
        if (on) {
            const float2 y0 = *reinterpret_cast<const float2*>(&sm.a[tr + g][sc + 2 * i]);
            const float2 y1 = *reinterpret_cast<const float2*>(&sm.a[tr + g + 8][sc + 2 * i]);
            y[0] = y0.x;
            y[1] = y0.y;
            y[2] = y1.x;
            y[3] = y1.y;
            take<half / 16>(y, sm.a, sm.n, beta, tr, sc, r0, lane);
        }
        put();
        if (on) take<half / 16>(y, sm.n, sm.n, beta, tr, sc, r0 + half, lane);
        __syncthreads();
        put();
    };
    join(std::integral_constant<int, 1>(), 32 * (warp & 1), 32 * (warp & 1) + 16, 32 * (warp & 1) + 8 * (warp >> 1 & 1),
         warp < 4);
    join(std::integral_constant<int, 2>(), 0, 32 + 16 * (warp & 1), 8 * (warp >> 1), true);
    {  // N as two images: two pieces of a row per thread, zeros above the blocks of 16 on the diagonal
        const int t = tid >> 2, p0 = 2 * (tid & 3);
#pragma unroll
        for (int p = p0; p < p0 + 2; ++p) {
            uint32_t w[8] = {};
            if (p0 / 2 <= t / 16) {
                const float4 x = *reinterpret_cast<const float4*>(&sm.n[t][8 * p]);
                const float4 y = *reinterpret_cast<const float4*>(&sm.n[t][8 * p + 4]);
                split(x.x, x.y, w[0], w[4]);
                split(x.z, x.w, w[1], w[5]);
                split(y.x, y.y, w[2], w[6]);
                split(y.z, y.w, w[3], w[7]);
            }
            *reinterpret_cast<uint4*>(sm.nimg[0] + piece<128>(t, p)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(sm.nimg[1] + piece<128>(t, p)) = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (storer) {
        store_bulk(to.img[0], sm.nimg, sizeof(sm.nimg));
        asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
    }
}

// ----------------------------------------------------------------- gdr_chain

constexpr int kWalkThreads = 128;  // 4 warps of 16 value columns
constexpr int kWalkCols = 64;

// What the walks leave for gdr_grad_tc, per chunk: the state before it (forward)
// and the gradient of the state after it (backward), in a high and a low part of
// d / 8 blocks of [e][8] (one value column's 16 bytes next to the next one's);
// the rows w and x as fp32 [B*H][T][e].
struct Saved {
    __nv_bfloat16 *S0;   // [B*H][chunks][2][d / 8][e][8]
    __nv_bfloat16 *dS1;  // [B*H][chunks][2][d / 8][e][8]
    float *W, *X;
    float* sums;         // gdr_grad_tc's sums over the value heads of a key head, 64 KB per CTA
};

template <int D>
__device__ __forceinline__ void save_state(const float (&S)[D / 8][4], __nv_bfloat16* to, int e, int row, int lane) {
    const int i = lane & 3;
    uint32_t* hi = reinterpret_cast<uint32_t*>(to);
    uint32_t* lo = hi + static_cast<size_t>(e) * D / 2;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t h, l;
            split(S[j][2 * half], S[j][2 * half + 1], h, l);
            const int at = (j * e + row + 8 * half) * 4 + i;
            hi[at] = h;
            lo[at] = l;
        }
    }
}

template <int D>
struct WalkSmem {  // two CTAs per SM at D = 128
    unsigned char k[2][kC * D * 2], q[2][kC * D * 2], v[2][kC * kWalkCols * 2];
    unsigned char np[4][kC * kC * 2];
    float coef[2][3][kC];  // e^G, e^{G_C - G}, beta
};

// Rows [t][16 columns of this warp] of an accumulator to global memory
__device__ __forceinline__ void store_rows(const Args& A, void* out, int bf16, const float (&o)[8][4], int b, int h,
                                           int t0, int len, int col, unsigned char* stage, int wcol, int lane) {
    const int g = lane >> 2, i = lane & 3;
    if (!bf16) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int t = t0 + 8 * j + 2 * i + x;
                if (t < len) {
                    float* p = static_cast<float*>(out) + row_at(A, b, h, A.H, t, A.e) + col;
                    p[g] = o[j][x];
                    p[g + 8] = o[j][2 + x];
                }
            }
        return;
    }
    // through this warp's own columns of a [64][64] tile that it has read out
    __syncwarp();
    const uint32_t base = smem_addr(stage);
#pragma unroll
    for (int jp = 0; jp < 4; ++jp) {
        const int m = lane >> 3, r = lane & 7;
        const uint32_t a = base + piece<128>(8 * (2 * jp + (m >> 1)) + r, wcol / 8 + (m & 1));
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a),
                     "r"(pack(o[2 * jp][0], o[2 * jp][1])), "r"(pack(o[2 * jp][2], o[2 * jp][3])),
                     "r"(pack(o[2 * jp + 1][0], o[2 * jp + 1][1])), "r"(pack(o[2 * jp + 1][2], o[2 * jp + 1][3]))
                     : "memory");
    }
    __syncwarp();
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const int r = 16 * y + (lane >> 1), p = lane & 1;
        if (t0 + r < len) {
            const uint4 x = *reinterpret_cast<const uint4*>(stage + piece<128>(r, wcol / 8 + p));
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + row_at(A, b, h, A.H, t0 + r, A.e) + col +
                                      8 * p) = x;
        }
    }
}

// The state of 16 value columns from memory [d][e] (or zero) and back
template <int D>
__device__ __forceinline__ void state_in(float (&S)[D / 8][4], const float* from, int e, int col, int lane) {
    const int g = lane >> 2, i = lane & 3;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            S[j][x] = from ? from[static_cast<size_t>(8 * j + 2 * i + (x & 1)) * e + col + g + 8 * (x >> 1)] : 0.f;
}
template <int D>
__device__ __forceinline__ void state_out(const float (&S)[D / 8][4], float* to, int e, int col, int lane) {
    const int g = lane >> 2, i = lane & 3;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            to[static_cast<size_t>(8 * j + 2 * i + (x & 1)) * e + col + g + 8 * (x >> 1)] = S[j][x];
}

// Forward walk over the chunks of one sequence, 64 value columns per CTA.
// kSave: no output; states and rows w for the backward.
template <int D, bool kSave>
__device__ __forceinline__ void chain(const Args& A, const ChunkWs* ws, const Saved& out, int chunks, int block) {
    extern __shared__ __align__(128) unsigned char walk_raw[];
    WalkSmem<D>& sm = *reinterpret_cast<WalkSmem<D>*>(walk_raw);
    const int slices = A.e / kWalkCols;
    const int n = block / slices, b = n / A.H, h = n % A.H, hk = h / (A.H / A.Hk);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, i = lane & 3;
    const int cta0 = block % slices * kWalkCols, wcol = 16 * warp, col = cta0 + wcol;
    const int len = length_of(A, b), nc = (len + kC - 1) / kC;
    const size_t page = static_cast<size_t>(A.d) * A.e;
    const ChunkWs* cw = ws + static_cast<size_t>(n) * chunks;
    float S[D / 8][4];
    state_in<D>(S, A.init ? A.init + n * page : nullptr, A.e, col, lane);

    const auto load_rows = [&](int c) {
        const int s = c & 1;
        load_tile<D, kWalkThreads>(smem_addr(sm.k[s]), A, A.k, b, hk, A.Hk, D, 0, c * kC, len);
        if (!kSave) load_tile<D, kWalkThreads>(smem_addr(sm.q[s]), A, A.q, b, hk, A.Hk, D, 0, c * kC, len);
        load_tile<kWalkCols, kWalkThreads>(smem_addr(sm.v[s]), A, A.v, b, h, A.H, A.e, cta0, c * kC, len);
        load_bytes<kWalkThreads>(smem_addr(sm.coef[s]), cw[c].eg, 3 * kC * 4);
        cp_commit();
    };
    const auto load_mats = [&](int c) {
        load_bytes<kWalkThreads>(smem_addr(sm.np), cw[c].img, (kSave ? 2 : 4) * kC * kC * 2);
        cp_commit();
    };
    if (nc > 0) {
        load_rows(0);
        load_mats(0);
    }
    for (int c = 0; c < nc; ++c) {
        const int s = c & 1;
        if (c + 1 < nc) load_rows(c + 1);
        else cp_commit();
        cp_wait<2>();
        __syncthreads();
        const uint32_t kt = smem_addr(sm.k[s]), qt = smem_addr(sm.q[s]), vt = smem_addr(sm.v[s]);
        const float *eg = sm.coef[s][0], *rest = sm.coef[s][1], *beta = sm.coef[s][2];
        float z[8][4] = {}, o[8][4] = {};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t ah[4], al[4], bb[4][4];
            frag_split(S[2 * kk], S[2 * kk + 1], ah, al);
            // a tile's products lie eight MMAs apart, so that none waits for the one before it
#pragma unroll
            for (int jp = 0; jp < 4; ++jp) ld_b<2 * D>(bb[jp], kt, jp, kk, lane);
#pragma unroll
            for (int jp = 0; jp < 4; ++jp) mma2(z[2 * jp], z[2 * jp + 1], ah, bb[jp]);
#pragma unroll
            for (int jp = 0; jp < 4; ++jp) mma2(z[2 * jp], z[2 * jp + 1], al, bb[jp]);
            if (!kSave) {
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) ld_b<2 * D>(bb[jp], qt, jp, kk, lane);
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) mma2(o[2 * jp], o[2 * jp + 1], ah, bb[jp]);
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) mma2(o[2 * jp], o[2 * jp + 1], al, bb[jp]);
            }
        }
        if (kSave) save_state<D>(S, out.S0 + (static_cast<size_t>(n) * chunks + c) * 2 * page, A.e, col + g, lane);
        // Z = V - e^G (K S0), then -beta Z as the operand of N
        uint32_t fh[4][4], fl[4][4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint32_t vv[4];
            ld_at<128>(vv, vt, warp, kk, lane);
            float y[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int j = 2 * kk + x;
                const float2 e2 = *reinterpret_cast<const float2*>(eg + 8 * j + 2 * i);
                const float2 b2 = *reinterpret_cast<const float2*>(beta + 8 * j + 2 * i);
                z[j][0] = fmaf(-e2.x, z[j][0], low_of(vv[2 * x]));
                z[j][1] = fmaf(-e2.y, z[j][1], high_of(vv[2 * x]));
                z[j][2] = fmaf(-e2.x, z[j][2], low_of(vv[2 * x + 1]));
                z[j][3] = fmaf(-e2.y, z[j][3], high_of(vv[2 * x + 1]));
                y[x][0] = -b2.x * z[j][0];
                y[x][1] = -b2.y * z[j][1];
                y[x][2] = -b2.x * z[j][2];
                y[x][3] = -b2.y * z[j][3];
                if (!kSave) {
                    o[j][0] *= e2.x;
                    o[j][1] *= e2.y;
                    o[j][2] *= e2.x;
                    o[j][3] *= e2.y;
                }
            }
            frag_split(y[0], y[1], fh[kk], fl[kk]);
        }
        cp_wait<1>();
        __syncthreads();
        const uint32_t nh = smem_addr(sm.np[0]), nl = smem_addr(sm.np[1]);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint32_t bb[4][4];
#pragma unroll
            for (int jp = kk; jp < 4; ++jp) ld_b<128>(bb[jp], nh, jp, kk, lane);
#pragma unroll
            for (int jp = kk; jp < 4; ++jp) mma2(z[2 * jp], z[2 * jp + 1], fh[kk], bb[jp]);
#pragma unroll
            for (int jp = kk; jp < 4; ++jp) mma2(z[2 * jp], z[2 * jp + 1], fl[kk], bb[jp]);
#pragma unroll
            for (int jp = kk; jp < 4; ++jp) ld_b<128>(bb[jp], nl, jp, kk, lane);
#pragma unroll
            for (int jp = kk; jp < 4; ++jp) mma2(z[2 * jp], z[2 * jp + 1], fh[kk], bb[jp]);
        }
        if (kSave) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int t = c * kC + 8 * j + 2 * i + x;
                    if (t < len) {
                        float* p = out.W + (static_cast<size_t>(n) * A.T + t) * A.e + col;
                        p[g] = z[j][x];
                        p[g + 8] = z[j][2 + x];
                    }
                }
        }
        // U = beta W
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 b2 = *reinterpret_cast<const float2*>(beta + 8 * j + 2 * i);
            z[j][0] *= b2.x;
            z[j][1] *= b2.y;
            z[j][2] *= b2.x;
            z[j][3] *= b2.y;
        }
        if (!kSave) {
            const uint32_t ph = smem_addr(sm.np[2]), pl = smem_addr(sm.np[3]);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t uh[4], ul[4];
                frag_split(z[2 * kk], z[2 * kk + 1], uh, ul);
                uint32_t bb[4][4];
#pragma unroll
                for (int jp = kk; jp < 4; ++jp) ld_b<128>(bb[jp], ph, jp, kk, lane);
#pragma unroll
                for (int jp = kk; jp < 4; ++jp) mma2(o[2 * jp], o[2 * jp + 1], uh, bb[jp]);
#pragma unroll
                for (int jp = kk; jp < 4; ++jp) mma2(o[2 * jp], o[2 * jp + 1], ul, bb[jp]);
#pragma unroll
                for (int jp = kk; jp < 4; ++jp) ld_b<128>(bb[jp], pl, jp, kk, lane);
#pragma unroll
                for (int jp = kk; jp < 4; ++jp) mma2(o[2 * jp], o[2 * jp + 1], uh, bb[jp]);
            }
            store_rows(A, A.o, A.out_bf16, o, b, h, c * kC, len, col, sm.v[s], wcol, lane);
        }
        __syncthreads();
        if (c + 1 < nc) load_mats(c + 1);
        else cp_commit();
        const float ec = eg[kC - 1];
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) S[j][x] *= ec;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            float y[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int j = 2 * kk + x;
                const float2 r2 = *reinterpret_cast<const float2*>(rest + 8 * j + 2 * i);
                y[x][0] = r2.x * z[j][0];
                y[x][1] = r2.y * z[j][1];
                y[x][2] = r2.x * z[j][2];
                y[x][3] = r2.y * z[j][3];
            }
            uint32_t uh[4], ul[4];
            frag_split(y[0], y[1], uh, ul);
#pragma unroll
            for (int j4 = 0; j4 < D / 16; j4 += 4) {
                uint32_t bb[4][4];
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) ld_bt<2 * D>(bb[jp], kt, j4 + jp, kk, lane);
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) mma2(S[2 * (j4 + jp)], S[2 * (j4 + jp) + 1], uh, bb[jp]);
#pragma unroll
                for (int jp = 0; jp < 4; ++jp) mma2(S[2 * (j4 + jp)], S[2 * (j4 + jp) + 1], ul, bb[jp]);
            }
        }
        __syncthreads();
    }
    if (!kSave && A.fin) state_out<D>(S, A.fin + n * page, A.e, col, lane);
}

// Backward walk: the gradient of the state from the last chunk to the first.
template <int D>
__device__ __forceinline__ void chain_rev(const Args& A, const ChunkWs* ws, const Saved& out, int chunks, int block) {
    extern __shared__ __align__(128) unsigned char walk_raw[];
    WalkSmem<D>& sm = *reinterpret_cast<WalkSmem<D>*>(walk_raw);
    const int slices = A.e / kWalkCols;
    const int n = block / slices, b = n / A.H, h = n % A.H, hk = h / (A.H / A.Hk);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, i = lane & 3;
    const int cta0 = block % slices * kWalkCols, wcol = 16 * warp, col = cta0 + wcol;
    const int len = length_of(A, b), nc = (len + kC - 1) / kC;
    const size_t page = static_cast<size_t>(A.d) * A.e;
    const ChunkWs* cw = ws + static_cast<size_t>(n) * chunks;
    float S[D / 8][4];  // the gradient
    state_in<D>(S, A.dfinal ? A.dfinal + n * page : nullptr, A.e, col, lane);

    const auto load_rows = [&](int c) {
        const int s = c & 1;
        load_tile<D, kWalkThreads>(smem_addr(sm.k[s]), A, A.k, b, hk, A.Hk, D, 0, c * kC, len);
        load_tile<D, kWalkThreads>(smem_addr(sm.q[s]), A, A.q, b, hk, A.Hk, D, 0, c * kC, len);
        load_tile<kWalkCols, kWalkThreads>(smem_addr(sm.v[s]), A, A.dout, b, h, A.H, A.e, cta0, c * kC, len);
        load_bytes<kWalkThreads>(smem_addr(sm.coef[s]), cw[c].eg, 3 * kC * 4);
        cp_commit();
    };
    const auto load_mats = [&](int c) {
        load_bytes<kWalkThreads>(smem_addr(sm.np), cw[c].img, 4 * kC * kC * 2);
        cp_commit();
    };
    if (nc > 0) {
        load_rows(nc - 1);
        load_mats(nc - 1);
    }
    for (int c = nc - 1; c >= 0; --c) {
        const int s = c & 1;
        if (c > 0) load_rows(c - 1);
        else cp_commit();
        cp_wait<2>();
        __syncthreads();
        const uint32_t kt = smem_addr(sm.k[s]), qt = smem_addr(sm.q[s]), vt = smem_addr(sm.v[s]);
        const float *eg = sm.coef[s][0], *rest = sm.coef[s][1], *beta = sm.coef[s][2];
        save_state<D>(S, out.dS1 + (static_cast<size_t>(n) * chunks + c) * 2 * page, A.e, col + g, lane);
        float x[8][4] = {};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t ah[4], al[4], bb[4][4];
            frag_split(S[2 * kk], S[2 * kk + 1], ah, al);
#pragma unroll
            for (int jp = 0; jp < 4; ++jp) ld_b<2 * D>(bb[jp], kt, jp, kk, lane);
#pragma unroll
            for (int jp = 0; jp < 4; ++jp) mma2(x[2 * jp], x[2 * jp + 1], ah, bb[jp]);
#pragma unroll
            for (int jp = 0; jp < 4; ++jp) mma2(x[2 * jp], x[2 * jp + 1], al, bb[jp]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 r2 = *reinterpret_cast<const float2*>(rest + 8 * j + 2 * i);
            x[j][0] *= r2.x;
            x[j][1] *= r2.y;
            x[j][2] *= r2.x;
            x[j][3] *= r2.y;
        }
        cp_wait<1>();
        __syncthreads();
        const uint32_t nh = smem_addr(sm.np[0]), nl = smem_addr(sm.np[1]);
        const uint32_t ph = smem_addr(sm.np[2]), pl = smem_addr(sm.np[3]);
        // + P^T dO
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint32_t da[4];
            ld_at<128>(da, vt, warp, kk, lane);
            uint32_t bb[4][4];
#pragma unroll
            for (int jp = 0; jp <= kk; ++jp) ld_bt<128>(bb[jp], ph, jp, kk, lane);
#pragma unroll
            for (int jp = 0; jp <= kk; ++jp) mma2(x[2 * jp], x[2 * jp + 1], da, bb[jp]);
#pragma unroll
            for (int jp = 0; jp <= kk; ++jp) ld_bt<128>(bb[jp], pl, jp, kk, lane);
#pragma unroll
            for (int jp = 0; jp <= kk; ++jp) mma2(x[2 * jp], x[2 * jp + 1], da, bb[jp]);
        }
        // X = dU - N^T (beta dU)
        {
            uint32_t fh[4][4], fl[4][4];
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                float y[2][4];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int j = 2 * kk + w;
                    const float2 b2 = *reinterpret_cast<const float2*>(beta + 8 * j + 2 * i);
                    y[w][0] = -b2.x * x[j][0];
                    y[w][1] = -b2.y * x[j][1];
                    y[w][2] = -b2.x * x[j][2];
                    y[w][3] = -b2.y * x[j][3];
                }
                frag_split(y[0], y[1], fh[kk], fl[kk]);
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t bb[4][4];
#pragma unroll
                for (int jp = 0; jp <= kk; ++jp) ld_bt<128>(bb[jp], nh, jp, kk, lane);
#pragma unroll
                for (int jp = 0; jp <= kk; ++jp) mma2(x[2 * jp], x[2 * jp + 1], fh[kk], bb[jp]);
#pragma unroll
                for (int jp = 0; jp <= kk; ++jp) mma2(x[2 * jp], x[2 * jp + 1], fl[kk], bb[jp]);
#pragma unroll
                for (int jp = 0; jp <= kk; ++jp) ld_bt<128>(bb[jp], nl, jp, kk, lane);
#pragma unroll
                for (int jp = 0; jp <= kk; ++jp) mma2(x[2 * jp], x[2 * jp + 1], fh[kk], bb[jp]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int t = c * kC + 8 * j + 2 * i + w;
                if (t < len) {
                    float* p = out.X + (static_cast<size_t>(n) * A.T + t) * A.e + col;
                    p[g] = x[j][w];
                    p[g + 8] = x[j][2 + w];
                }
            }
        // dS = e^{G_C} dS + Q^T (e^G dO) - K^T (beta e^G X)
        const float ec = eg[kC - 1];
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int w = 0; w < 4; ++w) S[j][w] *= ec;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 b2 = *reinterpret_cast<const float2*>(beta + 8 * j + 2 * i);
            x[j][0] *= b2.x;
            x[j][1] *= b2.y;
            x[j][2] *= b2.x;
            x[j][3] *= b2.y;
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint32_t da[4], h1[4], l1[4], h2[4], l2[4];
            ld_at<128>(da, vt, warp, kk, lane);
            float y[2][4], u[2][4];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int j = 2 * kk + w;
                const float2 e2 = *reinterpret_cast<const float2*>(eg + 8 * j + 2 * i);
                y[w][0] = e2.x * low_of(da[2 * w]);
                y[w][1] = e2.y * high_of(da[2 * w]);
                y[w][2] = e2.x * low_of(da[2 * w + 1]);
                y[w][3] = e2.y * high_of(da[2 * w + 1]);
                u[w][0] = -e2.x * x[j][0];
                u[w][1] = -e2.y * x[j][1];
                u[w][2] = -e2.x * x[j][2];
                u[w][3] = -e2.y * x[j][3];
            }
            frag_split(y[0], y[1], h1, l1);
            frag_split(u[0], u[1], h2, l2);
#pragma unroll
            for (int j4 = 0; j4 < D / 16; j4 += 4) {
                uint32_t bb[4][4];
                const auto both = [&](uint32_t tile, const uint32_t (&h)[4], const uint32_t (&l)[4]) {
#pragma unroll
                    for (int jp = 0; jp < 4; ++jp) ld_bt<2 * D>(bb[jp], tile, j4 + jp, kk, lane);
#pragma unroll
                    for (int jp = 0; jp < 4; ++jp) mma2(S[2 * (j4 + jp)], S[2 * (j4 + jp) + 1], h, bb[jp]);
#pragma unroll
                    for (int jp = 0; jp < 4; ++jp) mma2(S[2 * (j4 + jp)], S[2 * (j4 + jp) + 1], l, bb[jp]);
                };
                both(qt, h1, l1);
                both(kt, h2, l2);
            }
        }
        __syncthreads();
        if (c > 0) load_mats(c - 1);
        else cp_commit();
    }
    if (A.dinit) state_out<D>(S, A.dinit + n * page, A.e, col, lane);
}

template <int D>
__global__ void __launch_bounds__(kWalkThreads, 2)
gdr_chain(Args A, const ChunkWs* ws, int chunks) {
    chain<D, false>(A, ws, Saved{}, chunks, blockIdx.x);
}

// Both walks of a backward: the gradient of the state needs nothing of the forward
// walk, so they run side by side, the longer one's CTAs first.  128 sequences of
// 2048 rows, d = e = 64: 153 us, one after the other 89 + 112 us.
template <int D>
__global__ void __launch_bounds__(kWalkThreads, 2)
gdr_chains(Args A, const ChunkWs* ws, Saved out, int chunks) {
    const int half = gridDim.x / 2, block = blockIdx.x;
    if (block < half) chain_rev<D>(A, ws, out, chunks, block);
    else chain<D, true>(A, ws, out, chunks, block - half);
}

}  // namespace gdr
}  // namespace la2
