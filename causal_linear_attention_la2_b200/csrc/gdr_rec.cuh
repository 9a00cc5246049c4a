// gdr_rec.cuh -- the gated delta rule token by token in fp32 on the SIMT cores:
// every 1 <= d, e <= 128 and both input types (the bf16 sizes 64 and 128 have
// tensor-core kernels of their own).
//
// The columns of the state do not interact: column j of S needs k, q, beta, g
// and v_j alone.  So eight lanes hold one column (16 rows each at d = 128) in
// registers for the whole sequence, a token costs three multiply-adds a row and
// two sums over eight lanes, and the state never leaves the registers.  The
// backward runs the same recurrence for dS from the last row to the first,
//
//   dS += q do^T,  x = dS^T k,  dv = beta x,  dS = a (dS - k (beta x)^T),
//
// and a third kernel, parallel over 32-row chunks, makes dq, dk, dg and dbeta
// from the states on the chunk borders, the rows w and the rows x (gdr_grad_rec).
#pragma once
#include "gdr_common.cuh"

namespace la2 {
namespace gdr {

constexpr int kMaxDim = 128;
constexpr int kRecThreads = 128;  // 4 warps of 4 columns
constexpr int kRecCols = 16;
constexpr int kRecStep = 16;      // tokens staged in shared memory at a time
constexpr int kRecChunk = 32;     // chunk length of gdr_grad_rec

struct RecSmem {
    float k[kRecStep][kMaxDim + 4];
    float q[kRecStep][kMaxDim + 4];
    float v[kRecStep][kRecCols];
    float a[kRecStep];
    float b[kRecStep];
};

// Rows t0 .. t0 + n - 1 of k, q and 16 columns of `vals` (v or dout) on their way
// to shared memory (rows i >= d are zero): a thread's column of k and q, loaded
// while the rows before are worked on.
static_assert(kRecThreads == kMaxDim, "a thread per column of k and q");

template <typename Tin>
struct RecRows {
    Tin k[kRecStep], q[kRecStep], v[2];  // as loaded: a conversion would wait for them
    float g, b;

    __device__ __forceinline__ void load(const Args& A, const Tin* vals, int b0, int h, int t0, int n, int col0) {
        const int tid = threadIdx.x, hk = h / (A.H / A.Hk);
        const Tin* kp = static_cast<const Tin*>(A.k);
        const Tin* qp = static_cast<const Tin*>(A.q);
        const size_t at = row_at(A, b0, hk, A.Hk, t0, A.d) + tid, step = A.bthd ? static_cast<size_t>(A.Hk) * A.d : A.d;
        kp += at;
        qp += at;
        const int rows = tid < A.d ? n : 0;
#pragma unroll
        for (int r = 0; r < kRecStep; ++r) {
            k[r] = q[r] = Tin(0.f);
            if (r < rows) {
                k[r] = kp[r * step];
                q[r] = qp[r * step];
            }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int r = (tid + y * kRecThreads) / kRecCols, j = col0 + tid % kRecCols;
            v[y] = r < n && j < A.e ? vals[row_at(A, b0, h, A.H, t0 + r, A.e) + j] : Tin(0.f);
        }
        g = b = 0.f;
        if (tid < n) {
            const size_t at = row_at(A, b0, h, A.H, t0 + tid, 1);
            if (A.g) g = A.g[at];
            b = A.beta[at];
        }
    }
    __device__ __forceinline__ void store(RecSmem& sm) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int r = 0; r < kRecStep; ++r) {
            sm.k[r][tid] = to_float(k[r]);
            sm.q[r][tid] = to_float(q[r]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) sm.v[(tid + y * kRecThreads) / kRecCols][tid % kRecCols] = to_float(v[y]);
        if (tid < kRecStep) {
            sm.a[tid] = expf(bounded_gate(g));
            sm.b[tid] = b;
        }
    }
};

__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    return x;
}

// Lane r of the eight has rows 32 (m / 4) + 4 r + m % 4, m = 0 .. kRows - 1: 16 bytes next to its neighbours'
__device__ __forceinline__ int rec_row(int r, int m) { return 32 * (m >> 2) + 4 * r + (m & 3); }

template <int kRows>
__device__ __forceinline__ void rec_load(const float* p, int r, float (&x)[kRows]) {
#pragma unroll
    for (int m = 0; m < kRows; m += 4) {
        const float4 y = *reinterpret_cast<const float4*>(p + rec_row(r, m));
        x[m] = y.x;
        x[m + 1] = y.y;
        x[m + 2] = y.z;
        x[m + 3] = y.w;
    }
}

// Forward.  kRecRows: rows of the state per lane, 8 (d <= 64) or 16.  kSave: no output; the state entering each chunk goes to S0
// [B*H][chunks][d][e] and the rows w to W [B*H][T][e], for the backward.
template <typename Tin, bool kSave, int kRecRows>
__device__ __forceinline__ void rec_fwd(const Args& A, float* S0, float* W, RecSmem& sm, int cols) {
    const int n = blockIdx.x, b = n / A.H, h = n % A.H;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane & 7, lc = warp * 4 + (lane >> 3), col0 = cols * kRecCols;
    const int j = col0 + lc;
    const bool on = j < A.e;
    const int len = length_of(A, b);
    const int chunks = (A.T + kRecChunk - 1) / kRecChunk;
    const size_t page = static_cast<size_t>(A.d) * A.e;
    float S[kRecRows];
#pragma unroll
    for (int m = 0; m < kRecRows; ++m) {
        const int i = rec_row(r, m);
        S[m] = A.init && on && i < A.d ? A.init[n * page + static_cast<size_t>(i) * A.e + j] : 0.f;
    }
    const size_t step = A.bthd ? static_cast<size_t>(A.H) * A.e : A.e;  // from one row of v, out, dv to the next
    const size_t row0 = row_at(A, b, h, A.H, 0, A.e) + j;
    RecRows<Tin> next;
    if (len > 0) next.load(A, static_cast<const Tin*>(A.v), b, h, 0, min(kRecStep, len), col0);
    for (int t0 = 0; t0 < len; t0 += kRecStep) {
        const int m16 = min(kRecStep, len - t0);
        __syncthreads();
        next.store(sm);
        __syncthreads();
        if (t0 + kRecStep < len)
            next.load(A, static_cast<const Tin*>(A.v), b, h, t0 + kRecStep, min(kRecStep, len - t0 - kRecStep), col0);
        if (kSave && t0 % kRecChunk == 0 && on) {
            float* to = S0 + (static_cast<size_t>(n) * chunks + t0 / kRecChunk) * page + j;
#pragma unroll
            for (int m = 0; m < kRecRows; ++m)
                if (rec_row(r, m) < A.d) to[static_cast<size_t>(rec_row(r, m)) * A.e] = S[m];
        }
        float kn[kRecRows], qn[kRecRows];  // of the token to come
        rec_load(sm.k[0], r, kn);
        if (!kSave) rec_load(sm.q[0], r, qn);
        float an = sm.a[0], bn = sm.b[0], vn = sm.v[0][lc];
#pragma unroll 2
        for (int t = 0; t < m16; ++t) {
            float kk[kRecRows], qq[kRecRows];
#pragma unroll
            for (int m = 0; m < kRecRows; ++m) {
                kk[m] = kn[m];
                qq[m] = qn[m];
            }
            const float a = an, bt = bn, vt = vn;
            const int t1 = min(t + 1, kRecStep - 1);
            rec_load(sm.k[t1], r, kn);
            if (!kSave) rec_load(sm.q[t1], r, qn);
            an = sm.a[t1];
            bn = sm.b[t1];
            vn = sm.v[t1][lc];
            float p[4] = {};
#pragma unroll
            for (int m = 0; m < kRecRows; ++m) {
                S[m] *= a;
                p[m & 3] = fmaf(S[m], kk[m], p[m & 3]);
            }
            const float w = vt - sum8((p[0] + p[1]) + (p[2] + p[3]));
            const float u = bt * w;
            float o4[4] = {};
#pragma unroll
            for (int m = 0; m < kRecRows; ++m) {
                S[m] = fmaf(kk[m], u, S[m]);
                if (!kSave) o4[m & 3] = fmaf(S[m], qq[m], o4[m & 3]);
            }
            float o = (o4[0] + o4[1]) + (o4[2] + o4[3]);
            if (kSave) {
                if (on && r == 0) W[(static_cast<size_t>(n) * A.T + t0 + t) * A.e + j] = w;
            } else {
                o = sum8(o);
                if (on && r == 0) put(A.o, row0 + (t0 + t) * step, o, A.out_bf16);
            }
        }
    }
    if (!kSave && A.fin && on) {
#pragma unroll
        for (int m = 0; m < kRecRows; ++m)
            if (rec_row(r, m) < A.d) A.fin[n * page + static_cast<size_t>(rec_row(r, m)) * A.e + j] = S[m];
    }
}

// Backward in time: dv, d_init_state, the rows x to X [B*H][T][e] and the
// gradient of the state after each chunk to dS1 [B*H][chunks][d][e].
template <typename Tin, int kRecRows>
__device__ __forceinline__ void rec_rev(const Args& A, float* dS1, float* X, RecSmem& sm, int cols) {
    const int n = blockIdx.x, b = n / A.H, h = n % A.H;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane & 7, lc = warp * 4 + (lane >> 3), col0 = cols * kRecCols;
    const int j = col0 + lc;
    const bool on = j < A.e;
    const int len = length_of(A, b);
    const int chunks = (A.T + kRecChunk - 1) / kRecChunk;
    const size_t page = static_cast<size_t>(A.d) * A.e;
    float D[kRecRows];
#pragma unroll
    for (int m = 0; m < kRecRows; ++m) {
        const int i = rec_row(r, m);
        D[m] = A.dfinal && on && i < A.d ? A.dfinal[n * page + static_cast<size_t>(i) * A.e + j] : 0.f;
    }
    const size_t step = A.bthd ? static_cast<size_t>(A.H) * A.e : A.e;
    const size_t row0 = row_at(A, b, h, A.H, 0, A.e) + j;
    RecRows<Tin> next;
    const int tail = len > 0 ? (len - 1) / kRecStep * kRecStep : -1;
    if (len > 0) next.load(A, static_cast<const Tin*>(A.dout), b, h, tail, len - tail, col0);
    for (int t0 = tail; t0 >= 0; t0 -= kRecStep) {
        const int m16 = min(kRecStep, len - t0);
        __syncthreads();
        next.store(sm);
        __syncthreads();
        if (t0 > 0) next.load(A, static_cast<const Tin*>(A.dout), b, h, t0 - kRecStep, kRecStep, col0);
        // the last rows of a chunk: its dS1 is what arrives here
        if (on && ((t0 + kRecStep) % kRecChunk == 0 || t0 + m16 == len)) {
            float* to = dS1 + (static_cast<size_t>(n) * chunks + t0 / kRecChunk) * page + j;
#pragma unroll
            for (int m = 0; m < kRecRows; ++m)
                if (rec_row(r, m) < A.d) to[static_cast<size_t>(rec_row(r, m)) * A.e] = D[m];
        }
        float kn[kRecRows], qn[kRecRows];  // of the token to come
        rec_load(sm.k[m16 - 1], r, kn);
        rec_load(sm.q[m16 - 1], r, qn);
        float an = sm.a[m16 - 1], bn = sm.b[m16 - 1], vn = sm.v[m16 - 1][lc];
#pragma unroll 2
        for (int t = m16 - 1; t >= 0; --t) {
            float kk[kRecRows], qq[kRecRows];
#pragma unroll
            for (int m = 0; m < kRecRows; ++m) {
                kk[m] = kn[m];
                qq[m] = qn[m];
            }
            const float a = an, bt = bn, dout = vn;
            const int t1 = max(t - 1, 0);
            rec_load(sm.k[t1], r, kn);
            rec_load(sm.q[t1], r, qn);
            an = sm.a[t1];
            bn = sm.b[t1];
            vn = sm.v[t1][lc];
            float p[4] = {};
#pragma unroll
            for (int m = 0; m < kRecRows; ++m) {
                D[m] = fmaf(qq[m], dout, D[m]);
                p[m & 3] = fmaf(D[m], kk[m], p[m & 3]);
            }
            const float x = sum8((p[0] + p[1]) + (p[2] + p[3])), dw = bt * x;
#pragma unroll
            for (int m = 0; m < kRecRows; ++m) D[m] = a * fmaf(-kk[m], dw, D[m]);
            if (on && r == 0) {
                X[(static_cast<size_t>(n) * A.T + t0 + t) * A.e + j] = x;
                put(A.dv, row0 + (t0 + t) * step, dw, A.out_bf16);
            }
        }
    }
    if (A.dinit && on) {
#pragma unroll
        for (int m = 0; m < kRecRows; ++m)
            if (rec_row(r, m) < A.d) A.dinit[n * page + static_cast<size_t>(rec_row(r, m)) * A.e + j] = D[m];
    }
}

template <typename Tin, int kRecRows>
__global__ void __launch_bounds__(kRecThreads)
gdr_rec_fwd(Args A) {
    __shared__ RecSmem sm;
    rec_fwd<Tin, false, kRecRows>(A, nullptr, nullptr, sm, blockIdx.y);
}

// Both walks of a backward: the gradient of the state needs nothing of the forward
// walk, so they run side by side, the longer one's CTAs first.  4 sequences of up to
// 517 rows, d = e = 64, fp32: 149 us, one after the other 124 + 149 us; 130 us since
// the next token's rows are read ahead.
template <typename Tin, int kRecRows>
__global__ void __launch_bounds__(kRecThreads, 4)
gdr_rec_walks(Args A, float* S0, float* dS1, float* W, float* X) {
    __shared__ RecSmem sm;
    const int half = gridDim.y / 2, cols = blockIdx.y;
    if (cols < half) rec_rev<Tin, kRecRows>(A, dS1, X, sm, cols);
    else rec_fwd<Tin, true, kRecRows>(A, S0, W, sm, cols - half);
}

// dq, dk, dg, dbeta of one chunk of C = 32 rows of key head hk, summed over the
// value heads that share it in their order.  With G the cumulative gates of the
// chunk, S0 the state before it, dS1 the gradient of the state after it,
// U = beta W, M_ts = exp(G_t - G_s) (s <= t):
//
//   dP = M o (dO U^T),   E_ts = -beta_t M_ts (x_t . u_s)  (s < t)
//   dq_t  = e^{G_t} S0 do_t + sum_s dP_ts k_s
//   row_t = sum_s E_ts k_s - beta_t e^{G_t} S0 x_t             (k_t read as a query of the state)
//   col_s = sum_t (E_ts k_t + dP_ts q_t) + e^{G_C - G_s} dS1 u_s   (k_s written into the state)
//   dk = row + col,   dbeta_t = x_t . w_t
//   dL/dG_t = q_t . dq_t + k_t . row_t - k_t . col_t, and <dS1, S1> more at the chunk's end,
//   with k_t . row_t = beta_t x_t . (w_t - v_t) (the rows' definition, so no product is needed);
//   dg = sums of dL/dG from a row to the chunk's end.
//
// A thread makes column i of 16 rows (8 where d <= 64).  In each product one factor is the same for
// all lanes and is read four numbers at a time, and one differs (a row of S per
// lane); read one by one, the loads took five times as long as the multiply-adds
// (2048 chunks of d = e = 128: 1245 us, 670 us now, the loads of a chunk among them).
struct GradSmem {
    static constexpr int C = kRecChunk, P = kMaxDim + 1, P4 = kMaxDim + 4, CP = C + 4;
    float dout[C][P4], u[C][P4], x[C][P4];  // zero behind e
    float dp[C][CP], E[C][CP];
    float q[C][P], k[C][P];
    float S[kMaxDim][P];                    // zero behind e
    float G[C], Gl[C], b[C], db[C], xr[C], dG[C];
    float part[8][C];
    float red[8];
};

constexpr int kGradThreads = 256;

// kCols: columns i of dq and dk that are worked on side by side, 64 (d <= 64) or 128
template <typename Tin, int kCols>
__global__ void __launch_bounds__(kGradThreads, 1)
gdr_grad_rec(Args A, const float* S0, const float* dS1, const float* W, const float* X) {
    constexpr int C = kRecChunk;
    extern __shared__ __align__(16) float gsm_raw[];
    GradSmem& sm = *reinterpret_cast<GradSmem*>(gsm_raw);
    const int chunks = (A.T + C - 1) / C;
    const int c = blockIdx.x % chunks, hk = blockIdx.x / chunks % A.Hk;
    const int b = blockIdx.x / chunks / A.Hk;
    const int len = length_of(A, b), t0 = c * C;
    if (t0 >= len) return;
    const int n = min(C, len - t0), rep = A.H / A.Hk, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    constexpr int kRows = C * kCols / kGradThreads, kWarps = kCols / 32;
    const int i = tid % kCols, r0 = tid / kCols * kRows;  // column i of dq and dk, rows r0 ..
    const size_t page = static_cast<size_t>(A.d) * A.e;
    const Tin* q = static_cast<const Tin*>(A.q);
    const Tin* k = static_cast<const Tin*>(A.k);
    const Tin* v = static_cast<const Tin*>(A.v);
    const Tin* dout = static_cast<const Tin*>(A.dout);
#pragma unroll 8
    for (int y = tid; y < C * kMaxDim; y += kGradThreads) {
        const int t = y / kMaxDim, m = y % kMaxDim;
        const bool ok = t < n && m < A.d;
        const size_t at = ok ? row_at(A, b, hk, A.Hk, t0 + t, A.d) + m : 0;
        sm.q[t][m] = ok ? to_float(q[at]) : 0.f;
        sm.k[t][m] = ok ? to_float(k[at]) : 0.f;
    }
    float accq[kRows], acck[kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m) accq[m] = acck[m] = 0.f;
    for (int hh = 0; hh < rep; ++hh) {
        const int h = hk * rep + hh;
        const size_t seq = static_cast<size_t>(b) * A.H + h;
        const float* S0c = S0 + (seq * chunks + c) * page;
        const float* dS1c = dS1 + (seq * chunks + c) * page;
        __syncthreads();
        if (tid < C) {  // cumulative gates, as two floats: a difference of two large ones keeps its digits
            double s = tid < n ? static_cast<double>(gate_at(A, row_at(A, b, h, A.H, t0 + tid, 1))) : 0.0;
#pragma unroll
            for (int m = 1; m < C; m <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, s, m);
                if (lane >= m) s += y;
            }
            sm.G[tid] = static_cast<float>(s);
            sm.Gl[tid] = static_cast<float>(s - sm.G[tid]);
            sm.b[tid] = tid < n ? A.beta[row_at(A, b, h, A.H, t0 + tid, 1)] : 0.f;
        }
        __syncthreads();
        // a warp takes rows warp, warp + 8, ..: u, x, dout and the row sums
#pragma unroll
        for (int t = warp; t < C; t += 8) {
            float db = 0.f, xr = 0.f;
#pragma unroll
            for (int j = lane; j < kMaxDim; j += 32) {
                float w = 0.f, x = 0.f, dd = 0.f, vv = 0.f;
                if (t < n && j < A.e) {
                    const size_t at = (seq * A.T + t0 + t) * A.e + j;
                    const size_t io = row_at(A, b, h, A.H, t0 + t, A.e) + j;
                    w = W[at];
                    x = X[at];
                    dd = to_float(dout[io]);
                    vv = to_float(v[io]);
                }
                sm.u[t][j] = sm.b[t] * w;
                sm.x[t][j] = x;
                sm.dout[t][j] = dd;
                db = fmaf(x, w, db);
                xr = fmaf(x, w - vv, xr);
            }
            for (int m = 16; m; m >>= 1) {
                db += __shfl_xor_sync(0xffffffffu, db, m);
                xr += __shfl_xor_sync(0xffffffffu, xr, m);
            }
            if (lane == 0) {
                sm.db[t] = db;
                sm.xr[t] = sm.b[t] * xr;
            }
        }
#pragma unroll 4
        for (int r = warp; r < A.d; r += 8)
#pragma unroll
            for (int j = lane; j < kMaxDim; j += 32) sm.S[r][j] = j < A.e ? S0c[static_cast<size_t>(r) * A.e + j] : 0.f;
        __syncthreads();
        const auto dot4 = [](const float4& a, const float4& x, float y) {
            return fmaf(a.x, x.x, fmaf(a.y, x.y, fmaf(a.z, x.z, fmaf(a.w, x.w, y))));
        };
        const auto at4 = [](const float* p) { return *reinterpret_cast<const float4*>(p); };
        for (int y = tid; y < C * C; y += kGradThreads) {
            const int t = y / C, s = y % C;
            float p = 0.f, x = 0.f;
            if (s <= t) {
                for (int j = 0; j < A.e; j += 4) {
                    const float4 us = at4(&sm.u[s][j]);
                    p = dot4(at4(&sm.dout[t][j]), us, p);
                    x = dot4(at4(&sm.x[t][j]), us, x);
                }
                const float M = expf((sm.G[t] - sm.G[s]) + (sm.Gl[t] - sm.Gl[s]));
                p *= M;
                x = s < t ? -x * M * sm.b[t] : 0.f;
            }
            sm.dp[t][s] = p;
            sm.E[t][s] = x;
        }
        __syncthreads();
        float fq[kRows], row[kRows], col[kRows], colS[kRows];
#pragma unroll
        for (int m = 0; m < kRows; ++m) fq[m] = row[m] = col[m] = colS[m] = 0.f;
        if (i < A.d) {
            for (int j = 0; j < A.e; j += 4) {
                const float4 s = make_float4(sm.S[i][j], sm.S[i][j + 1], sm.S[i][j + 2], sm.S[i][j + 3]);
#pragma unroll
                for (int m = 0; m < kRows; ++m) {
                    fq[m] = dot4(at4(&sm.dout[r0 + m][j]), s, fq[m]);
                    row[m] = dot4(at4(&sm.x[r0 + m][j]), s, row[m]);
                }
            }
#pragma unroll
            for (int m = 0; m < kRows; ++m) {
                const int t = r0 + m;
                const float eg = expf(sm.G[t]) * (1.f + sm.Gl[t]);
                fq[m] *= eg;
                row[m] *= -sm.b[t] * eg;
            }
#pragma unroll 1
            for (int s = 0; s < C; s += 4) {
                const float4 ks = make_float4(sm.k[s][i], sm.k[s + 1][i], sm.k[s + 2][i], sm.k[s + 3][i]);
                const float4 qs = make_float4(sm.q[s][i], sm.q[s + 1][i], sm.q[s + 2][i], sm.q[s + 3][i]);
#pragma unroll
                for (int m = 0; m < kRows; ++m) {
                    fq[m] = dot4(at4(&sm.dp[r0 + m][s]), ks, fq[m]);
                    row[m] = dot4(at4(&sm.E[r0 + m][s]), ks, row[m]);
                }
                const auto across = [&](int y, float kk, float qq) {  // row s + y of E and dP, columns r0 ..
#pragma unroll
                    for (int m = 0; m < kRows; m += 4) {
                        const float4 ee = at4(&sm.E[s + y][r0 + m]), pp = at4(&sm.dp[s + y][r0 + m]);
                        col[m] = fmaf(ee.x, kk, fmaf(pp.x, qq, col[m]));
                        col[m + 1] = fmaf(ee.y, kk, fmaf(pp.y, qq, col[m + 1]));
                        col[m + 2] = fmaf(ee.z, kk, fmaf(pp.z, qq, col[m + 2]));
                        col[m + 3] = fmaf(ee.w, kk, fmaf(pp.w, qq, col[m + 3]));
                    }
                };
                across(0, ks.x, qs.x);
                across(1, ks.y, qs.y);
                across(2, ks.z, qs.z);
                across(3, ks.w, qs.w);
            }
        }
        __syncthreads();
        // <dS1, S0> while the states change places
        float dot = 0.f;
#pragma unroll 4
        for (int r = warp; r < A.d; r += 8)
#pragma unroll
            for (int j = lane; j < kMaxDim; j += 32) {
                const float ds = j < A.e ? dS1c[static_cast<size_t>(r) * A.e + j] : 0.f;
                dot = fmaf(ds, sm.S[r][j], dot);
                sm.S[r][j] = ds;
            }
        for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
        if (lane == 0) sm.red[warp] = dot;
        __syncthreads();
        if (i < A.d) {
            for (int j = 0; j < A.e; j += 4) {
                const float4 s = make_float4(sm.S[i][j], sm.S[i][j + 1], sm.S[i][j + 2], sm.S[i][j + 3]);
#pragma unroll
                for (int m = 0; m < kRows; ++m) colS[m] = dot4(at4(&sm.u[r0 + m][j]), s, colS[m]);
            }
        }
        // row sums over i (kWarps warps have the same rows), then <dS1, S1>
        float gc = 0.f;
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
            const int t = r0 + m;
            const float ki = i < A.d ? sm.k[t][i] : 0.f, qi = i < A.d ? sm.q[t][i] : 0.f;
            colS[m] *= expf((sm.G[C - 1] - sm.G[t]) + (sm.Gl[C - 1] - sm.Gl[t]));
            col[m] += colS[m];
            gc = fmaf(ki, colS[m], gc);
            float s = fmaf(qi, fq[m], -ki * col[m]);
            for (int z = 16; z; z >>= 1) s += __shfl_xor_sync(0xffffffffu, s, z);
            if (lane == 0) sm.part[warp][t] = s;
            accq[m] += fq[m];
            acck[m] += row[m] + col[m];
        }
        for (int z = 16; z; z >>= 1) gc += __shfl_xor_sync(0xffffffffu, gc, z);
        __syncthreads();
        if (lane == 0) sm.red[warp] = fmaf(expf(sm.G[C - 1]) * (1.f + sm.Gl[C - 1]), sm.red[warp], gc);
        __syncthreads();
        if (tid < C) {
            float s = sm.xr[tid];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += sm.part[tid / kRows * kWarps + w][tid];
            if (tid == C - 1)
                for (int w = 0; w < 8; ++w) s += sm.red[w];
            sm.dG[tid] = s;
        }
        __syncthreads();
        if (tid < n) {
            const size_t at = row_at(A, b, h, A.H, t0 + tid, 1);
            A.dbeta[at] = sm.db[tid];
            if (A.dg) {
                float s = 0.f;
#pragma unroll
                for (int t = C - 1; t >= 0; --t) s += t >= tid ? sm.dG[t] : 0.f;
                A.dg[at] = s;
            }
        }
    }
    if (i < A.d) {
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
            const int t = r0 + m;
            if (t < n) {
                const size_t at = row_at(A, b, hk, A.Hk, t0 + t, A.d) + i;
                put(A.dq, at, accq[m], A.out_bf16);
                put(A.dk, at, acck[m], A.out_bf16);
            }
        }
    }
}

}  // namespace gdr
}  // namespace la2
