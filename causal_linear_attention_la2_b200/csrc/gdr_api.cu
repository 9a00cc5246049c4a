// gdr_api.cu -- the C ABI of the gated delta rule and of the state pool
// (la2_gdr_*, la2_state_copy in include/la2.h): argument checks, workspace
// layout and launches.  The kernels are in gdr_chunk.cuh (bf16, d and e 64 or
// 128), gdr_rec.cuh (everything else) and state_pool.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "gdr_chunk.cuh"
#include "gdr_common.cuh"
#include "gdr_grad_sm100.cuh"
#include "gdr_rec.cuh"
#include "gdr_walk_sm100.cuh"
#include "la2.h"
#include "state_pool.cuh"

namespace la2 {
int* status_word();  // la2_api.cu
}

namespace {

using la2::gdr::Args;

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 4-D map over bf16 rows [B, heads, T, width] (or [B, T, heads, width]): boxes of
// 64 columns x 64 rows of one (b, head), 128-byte swizzle, rows past T zero.
bool row_map(CUtensorMap* m, const void* ptr, int B, int heads, int T, int width, int bthd) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t w = width, t = T, h = heads, b = B, rows = la2::gdr::kC;
    const cuuint64_t dims[4] = {w, bthd ? h : t, bthd ? t : h, b};
    const cuuint64_t strides[3] = {w * 2, (bthd ? h : t) * w * 2, t * h * w * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(bthd ? 1 : rows), static_cast<cuuint32_t>(bthd ? rows : 1), 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;
constexpr int kSMs = 148;

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int cdiv(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

bool set(const void* f, size_t bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) == cudaSuccess;
}

template <int D>
bool set_chunk_attrs() {
    using namespace la2::gdr;
    return set(reinterpret_cast<const void*>(gdr_prep<D>), sizeof(PrepSmem<D>)) &&
           set(reinterpret_cast<const void*>(gdr_chain<D>), sizeof(WalkSmem<D>)) &&
           set(reinterpret_cast<const void*>(gdr_chains<D>), sizeof(WalkSmem<D>)) &&
           set(reinterpret_cast<const void*>(walk::gdr_walk<D, walk::kForward>), sizeof(walk::Smem<D>)) &&
           set(reinterpret_cast<const void*>(walk::gdr_walks<D>), sizeof(walk::Smem<D>)) &&
           set(reinterpret_cast<const void*>(walk::gdr_join<D>), sizeof(walk::JoinSmem<D>)) &&
           set(reinterpret_cast<const void*>(walk::gdr_walk<D, walk::kTransfer>), sizeof(walk::Smem<D>)) &&
           set(reinterpret_cast<const void*>(grad::gdr_grad_tc<D, 64>), sizeof(grad::Smem<D, 64>)) &&
           set(reinterpret_cast<const void*>(grad::gdr_grad_tc<D, 128>), sizeof(grad::Smem<D, 128>));
}

template <int kCols>
bool set_rec_attrs() {
    using namespace la2::gdr;
    return set(reinterpret_cast<const void*>(gdr_grad_rec<float, kCols>), sizeof(GradSmem)) &&
           set(reinterpret_cast<const void*>(gdr_grad_rec<__nv_bfloat16, kCols>), sizeof(GradSmem));
}

template <int kTeam>
bool set_bulk_attrs() {
    using namespace la2::gdr;
    return set(reinterpret_cast<const void*>(gdr_step_bulk<float, kTeam>), bulk_smem_bytes<kTeam>()) &&
           set(reinterpret_cast<const void*>(gdr_step_bulk<__nv_bfloat16, kTeam>), bulk_smem_bytes<kTeam>());
}

// The kernels of la2_gdr_selftest_timeout
bool set_held_attrs() {
    using namespace la2::gdr;
    return set(reinterpret_cast<const void*>(walk::gdr_walk<128, walk::kForward, true>), sizeof(walk::Smem<128>)) &&
           set(reinterpret_cast<const void*>(walk::gdr_walks<128, true>), sizeof(walk::Smem<128>)) &&
           set(reinterpret_cast<const void*>(grad::gdr_grad_tc<128, 128, true>), sizeof(grad::Smem<128, 128>)) &&
           set(reinterpret_cast<const void*>(gdr_step_bulk<__nv_bfloat16, 512, true>), bulk_smem_bytes<512>());
}

bool set_smem_attrs() {
    return set_chunk_attrs<64>() && set_chunk_attrs<128>() &&
           set_rec_attrs<64>() && set_rec_attrs<128>() &&
           set_held_attrs() && set_bulk_attrs<128>() && set_bulk_attrs<256>() && set_bulk_attrs<512>() &&
           set(reinterpret_cast<const void*>(la2::gdr::pool_copy<float4>), 200 << 10) &&
           set(reinterpret_cast<const void*>(la2::gdr::pool_copy<float>), 200 << 10);
}

// Once per device: the shared-memory limits of the kernels that need more than
// 48 KB.  A failed attempt is tried again by the next call.
bool device_setup() {
    static std::mutex m;
    static bool done[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    std::lock_guard<std::mutex> lock(m);
    if (!done[dev]) done[dev] = set_smem_attrs();
    return done[dev];
}

la2_status launched() { return cudaGetLastError() == cudaSuccess ? LA2_OK : LA2_ERR_CUDA; }

// Workspace of a backward on the token-by-token kernels.
struct RecWs {
    size_t S0, dS1, W, X, bytes;
};

RecWs rec_ws(long long BH, int T, int d, int e) {
    const size_t seqs = static_cast<size_t>(BH);
    const size_t chunks = cdiv(T, la2::gdr::kRecChunk);
    const size_t pages = align256(seqs * chunks * d * e * sizeof(float));
    const size_t rows = align256(seqs * T * e * sizeof(float));
    RecWs w;
    w.S0 = 0;
    w.dS1 = w.S0 + pages;
    w.W = w.dS1 + pages;
    w.X = w.W + rows;
    w.bytes = w.X + rows;
    return w;
}

template <typename Tin>
la2_status rec_forward(const Args& A, cudaStream_t stream) {
    const dim3 grid(A.B * A.H, cdiv(A.e, la2::gdr::kRecCols));
    if (A.d <= 64) la2::gdr::gdr_rec_fwd<Tin, 8><<<grid, la2::gdr::kRecThreads, 0, stream>>>(A);
    else la2::gdr::gdr_rec_fwd<Tin, 16><<<grid, la2::gdr::kRecThreads, 0, stream>>>(A);
    return launched();
}

template <typename Tin>
la2_status rec_backward(const Args& A, char* ws, cudaStream_t stream) {
    const RecWs w = rec_ws(static_cast<long long>(A.B) * A.H, A.T, A.d, A.e);
    float* S0 = reinterpret_cast<float*>(ws + w.S0);
    float* dS1 = reinterpret_cast<float*>(ws + w.dS1);
    float* W = reinterpret_cast<float*>(ws + w.W);
    float* X = reinterpret_cast<float*>(ws + w.X);
    const dim3 grid(A.B * A.H, 2 * cdiv(A.e, la2::gdr::kRecCols));
    const unsigned chunks = static_cast<unsigned>(A.B) * A.Hk * cdiv(A.T, la2::gdr::kRecChunk);
    const auto go = [&](auto rows, auto cols) {
        la2::gdr::gdr_rec_walks<Tin, decltype(rows)::value>
            <<<grid, la2::gdr::kRecThreads, 0, stream>>>(A, S0, dS1, W, X);
        if (A.T > 0)
            la2::gdr::gdr_grad_rec<Tin, decltype(cols)::value>
                <<<chunks, la2::gdr::kGradThreads, sizeof(la2::gdr::GradSmem), stream>>>(A, S0, dS1, W, X);
    };
    if (A.d <= 64) go(std::integral_constant<int, 8>(), std::integral_constant<int, 64>());
    else go(std::integral_constant<int, 16>(), std::integral_constant<int, 128>());
    return launched();
}

// The tensor-core kernels' sizes.
bool by_chunks(la2_dtype dtype, int d, int e) {
    return dtype == LA2_DTYPE_BF16 && (d == 64 || d == 128) && (e == 64 || e == 128);
}

// Segments of the forward walk (gdr_walk_sm100.cuh) for `seqs` sequences of
// `chunks` chunks, by the chunks that the busiest SM walks: a segment's own and,
// with segments, those of the two walks that make its entering state; a join takes
// about a chunk's time.  The whole forward, d = e = 128, cut and not: 16 sequences of 1024
// chunks (T = 65,536) 1219 and 3057 us, of 256 chunks 349 and 777 us; 40 of 128 chunks
// 356 and 458 us; 60 of 128 and 80 of 96 are not cut (507 and 421 us).
struct SegPlan {
    int segs, per;
};

SegPlan seg_plan(long long seqs, int chunks) {
    SegPlan best = {1, chunks};
    long long cost = static_cast<long long>(chunks) * ((seqs + kSMs - 1) / kSMs);
    for (int g = 2; g <= 32 && chunks / g >= 8; ++g) {
        const int per = cdiv(chunks, g), segs = cdiv(chunks, per);
        const long long waves = (seqs * segs + kSMs - 1) / kSMs + (seqs * (2 * (segs - 1) - 1) + kSMs - 1) / kSMs;
        const long long c = waves * per + segs + 8;
        if (c < cost) {
            cost = c;
            best = {segs, per};
        }
    }
    return best;
}

struct ChunkLayout {
    size_t prep, S0, dS1, W, X, sums, segs, bytes;
};

ChunkLayout chunk_ws(long long BH, int T, int d, int e, bool bwd) {
    const size_t seqs = static_cast<size_t>(BH), chunks = cdiv(T, la2::gdr::kC);
    ChunkLayout w = {};
    size_t at = align256(seqs * chunks * sizeof(la2::gdr::ChunkWs));
    if (bwd) {
        const size_t pages = align256(seqs * chunks * 2 * d * e * 2);  // two bf16 parts
        const size_t rows = align256(seqs * T * e * sizeof(float));
        w.S0 = at;
        w.dS1 = w.S0 + pages;
        w.W = w.dS1 + pages;
        w.X = w.W + rows;
        w.sums = w.X + rows;
        at = w.sums + static_cast<size_t>(kSMs) * (64 << 10);
    }
    if (!bwd && e == la2::gdr::walk::kE) {
        w.segs = at;
        at += static_cast<size_t>(seg_plan(BH, static_cast<int>(chunks)).segs - 1) * seqs * 3 * d * e * sizeof(float);
    }
    w.bytes = at;
    return w;
}

// One walk along every sequence: e = 128 on tcgen05 (T = 0 has no rows to map).
template <int D, int kMode, bool kHold = false>
la2_status walk_tc(const Args& A, const la2::gdr::ChunkWs* cw, const la2::gdr::walk::Segments& sg, int chunks,
                   cudaStream_t stream) {
    using namespace la2::gdr;
    CUtensorMap mk, mq, mv;
    if (!row_map(&mk, A.k, A.B, A.Hk, A.T, D, A.bthd) || !row_map(&mq, A.q, A.B, A.Hk, A.T, D, A.bthd) ||
        !row_map(&mv, A.v, A.B, A.H, A.T, walk::kE, A.bthd))
        return LA2_ERR_CUDA;
    int* status = la2::status_word();
    if (!status) return LA2_ERR_CUDA;
    const int parts = kMode == walk::kTransfer ? 2 * (sg.segs - 1) - 1 : sg.segs;
    walk::gdr_walk<D, kMode, kHold><<<A.B * A.H * parts, walk::kThreads, sizeof(walk::Smem<D>), stream>>>(
        A, cw, sg, chunks, mk, mq, mv, status);
    return LA2_OK;
}

// Both walks of a backward
template <int D, bool kHold = false>
la2_status walks_tc(const Args& A, const la2::gdr::ChunkWs* cw, const la2::gdr::Saved& sv, int chunks, cudaStream_t stream) {
    using namespace la2::gdr;
    CUtensorMap mk, mq, mv, md;
    if (!row_map(&mk, A.k, A.B, A.Hk, A.T, D, A.bthd) || !row_map(&mq, A.q, A.B, A.Hk, A.T, D, A.bthd) ||
        !row_map(&mv, A.v, A.B, A.H, A.T, walk::kE, A.bthd) || !row_map(&md, A.dout, A.B, A.H, A.T, walk::kE, A.bthd))
        return LA2_ERR_CUDA;
    int* status = la2::status_word();
    if (!status) return LA2_ERR_CUDA;
    walk::gdr_walks<D, kHold><<<2 * A.B * A.H, walk::kThreads, sizeof(walk::Smem<D>), stream>>>(A, cw, sv, chunks, mk, mq, mv,
                                                                                              md, status);
    return LA2_OK;
}

template <int D, int E, bool kHold = false>
la2_status grad_tc(const Args& A, const la2::gdr::ChunkWs* cw, const la2::gdr::Saved& sv, int chunks, cudaStream_t stream) {
    using namespace la2::gdr;
    CUtensorMap mk, mq, md;
    if (!row_map(&mk, A.k, A.B, A.Hk, A.T, D, A.bthd) || !row_map(&mq, A.q, A.B, A.Hk, A.T, D, A.bthd) ||
        !row_map(&md, A.dout, A.B, A.H, A.T, E, A.bthd))
        return LA2_ERR_CUDA;
    int* status = la2::status_word();
    if (!status) return LA2_ERR_CUDA;
    const int units = A.B * A.Hk * chunks;
    grad::gdr_grad_tc<D, E, kHold><<<units < kSMs ? units : kSMs, grad::kThreads, sizeof(grad::Smem<D, E>), stream>>>(
        A, cw, sv, chunks, units * (A.H / A.Hk), mk, mq, md, status);
    return LA2_OK;
}

bool on_tc(const Args& A) { return A.e == la2::gdr::walk::kE && A.T > 0; }

template <int D, bool kHold = false>
la2_status chunk_forward(const Args& A, char* ws, cudaStream_t stream) {
    using namespace la2::gdr;
    const int chunks = cdiv(A.T, kC);
    ChunkWs* cw = reinterpret_cast<ChunkWs*>(ws);
    if (chunks > 0)
        gdr_prep<D><<<static_cast<unsigned>(A.B) * A.H * chunks, kPrepThreads, sizeof(PrepSmem<D>), stream>>>(A, cw, chunks);
    if (on_tc(A)) {
        const long long seqs = static_cast<long long>(A.B) * A.H;
        const SegPlan pl = seg_plan(seqs, chunks);
        const walk::Segments sg = {pl.segs, pl.per, reinterpret_cast<float*>(ws + chunk_ws(seqs, A.T, A.d, A.e, false).segs)};
        la2_status st = LA2_OK;
        if (pl.segs > 1) {
            st = walk_tc<D, walk::kTransfer>(A, cw, sg, chunks, stream);
            if (st != LA2_OK) return st;
            walk::gdr_join<D><<<dim3(A.B * A.H, walk::kE / 32), walk::kJoinThreads, sizeof(walk::JoinSmem<D>), stream>>>(A, sg);
        }
        st = walk_tc<D, walk::kForward, kHold>(A, cw, sg, chunks, stream);
        return st == LA2_OK ? launched() : st;
    }
    gdr_chain<D><<<A.B * A.H * (A.e / kWalkCols), kWalkThreads, sizeof(WalkSmem<D>), stream>>>(A, cw, chunks);
    return launched();
}

template <int D, bool kHoldWalks = false, bool kHoldGrad = false>
la2_status chunk_backward(const Args& A, char* ws, cudaStream_t stream) {
    using namespace la2::gdr;
    const int chunks = cdiv(A.T, kC);
    const ChunkLayout w = chunk_ws(static_cast<long long>(A.B) * A.H, A.T, A.d, A.e, true);
    ChunkWs* cw = reinterpret_cast<ChunkWs*>(ws + w.prep);
    Saved sv;
    sv.S0 = reinterpret_cast<__nv_bfloat16*>(ws + w.S0);
    sv.dS1 = reinterpret_cast<__nv_bfloat16*>(ws + w.dS1);
    sv.W = reinterpret_cast<float*>(ws + w.W);
    sv.X = reinterpret_cast<float*>(ws + w.X);
    sv.sums = reinterpret_cast<float*>(ws + w.sums);
    if (chunks > 0)
        gdr_prep<D><<<static_cast<unsigned>(A.B) * A.H * chunks, kPrepThreads, sizeof(PrepSmem<D>), stream>>>(A, cw, chunks);
    la2_status st = LA2_OK;
    if (on_tc(A)) {
        st = walks_tc<D, kHoldWalks>(A, cw, sv, chunks, stream);
        if (kHoldWalks) return st == LA2_OK ? launched() : st;
        if (st == LA2_OK) st = grad_tc<D, 128, kHoldGrad>(A, cw, sv, chunks, stream);
    } else {
        gdr_chains<D><<<2 * A.B * A.H * (A.e / kWalkCols), kWalkThreads, sizeof(WalkSmem<D>), stream>>>(A, cw, sv, chunks);
        if (chunks > 0) st = grad_tc<D, 64>(A, cw, sv, chunks, stream);
    }
    return st == LA2_OK ? launched() : st;
}

// Sizes and enums of a sequence call; *empty: nothing to do (no batch entry or
// no head: there is neither a row nor a state).
la2_status size_checks(int B, int Hk, int H, int T, int d, int e, la2_dtype dtype, la2_dtype out_dtype,
                       la2_layout layout, bool* empty) {
    if (dtype != LA2_DTYPE_F32 && dtype != LA2_DTYPE_BF16) return LA2_ERR_INVALID_ARG;
    if (out_dtype != LA2_DTYPE_F32 && out_dtype != LA2_DTYPE_BF16) return LA2_ERR_INVALID_ARG;
    if (layout != LA2_LAYOUT_BHTD && layout != LA2_LAYOUT_BTHD) return LA2_ERR_INVALID_ARG;
    if (B < 0 || Hk < 0 || H < 0 || T < 0 || d < 1 || e < 1) return LA2_ERR_INVALID_ARG;
    if (H > 0 && (Hk == 0 || H % Hk != 0)) return LA2_ERR_INVALID_ARG;
    if (d > la2::gdr::kMaxDim || e > la2::gdr::kMaxDim) return LA2_ERR_UNSUPPORTED;
    if (dtype == LA2_DTYPE_F32 && out_dtype == LA2_DTYPE_BF16) return LA2_ERR_UNSUPPORTED;
    // the kernels step a chunk past a sequence's last row, in 32 bits
    if (T > INT_MAX - (la2::gdr::kC - 1)) return LA2_ERR_UNSUPPORTED;
    // one CTA per (sequence, chunk), or four per sequence, at most, in one grid dimension
    if (B > 0 && H > 0 && static_cast<long long>(B) * H > (INT_MAX - 1) / (static_cast<long long>(T) / 32 + 4))
        return LA2_ERR_UNSUPPORTED;
    *empty = B == 0 || H == 0;
    return LA2_OK;
}

}  // namespace

extern "C" {

size_t la2_gdr_workspace_bytes(int B, int Hk, int H, int T, int d, int e, la2_dtype dtype, int is_bwd) {
    bool empty = false;
    if (size_checks(B, Hk, H, T, d, e, dtype, LA2_DTYPE_F32, LA2_LAYOUT_BHTD, &empty) != LA2_OK)
        return static_cast<size_t>(-1);
    if (empty || T == 0) return 0;
    if (by_chunks(dtype, d, e)) return chunk_ws(static_cast<long long>(B) * H, T, d, e, is_bwd != 0).bytes;
    if (!is_bwd) return 0;
    return rec_ws(static_cast<long long>(B) * H, T, d, e).bytes;
}

la2_status la2_gdr_fwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                       void* out, const float* init_state, float* final_state, const int* seq_lens, int B,
                       int Hk, int H, int T, int d, int e, la2_dtype dtype, la2_dtype out_dtype,
                       la2_layout layout, void* workspace, size_t workspace_bytes, la2_stream_t stream) {
    bool empty = false;
    const la2_status st = size_checks(B, Hk, H, T, d, e, dtype, out_dtype, layout, &empty);
    if (st != LA2_OK) return st;
    if (empty || (T == 0 && !final_state)) return LA2_OK;
    if (T > 0 && (!q || !k || !v || !beta || !out)) return LA2_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(g, 4) ||
        !aligned(beta, 4) || !aligned(init_state, 4) || !aligned(final_state, 4) || !aligned(seq_lens, 4))
        return LA2_ERR_INVALID_ARG;
    const size_t need = la2_gdr_workspace_bytes(B, Hk, H, T, d, e, dtype, 0);
    if (need && (!workspace || workspace_bytes < need)) return LA2_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return LA2_ERR_INVALID_ARG;
    if (!device_setup()) return LA2_ERR_CUDA;
    Args A = {};
    A.q = q; A.k = k; A.v = v; A.g = g; A.beta = beta; A.o = out;
    A.init = init_state; A.fin = final_state; A.lens = seq_lens;
    A.B = B; A.Hk = Hk; A.H = H; A.T = T; A.d = d; A.e = e;
    A.bthd = layout == LA2_LAYOUT_BTHD;
    A.out_bf16 = out_dtype == LA2_DTYPE_BF16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (by_chunks(dtype, d, e)) {
        char* ws = static_cast<char*>(workspace);
        return d == 64 ? chunk_forward<64>(A, ws, s) : chunk_forward<128>(A, ws, s);
    }
    return dtype == LA2_DTYPE_BF16 ? rec_forward<__nv_bfloat16>(A, s) : rec_forward<float>(A, s);
}

la2_status la2_gdr_bwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                       const void* dout, const float* init_state, const float* d_final_state, void* dq,
                       void* dk, void* dv, float* dg, float* dbeta, float* d_init_state, const int* seq_lens,
                       int B, int Hk, int H, int T, int d, int e, la2_dtype dtype, la2_dtype out_dtype,
                       la2_layout layout, void* workspace, size_t workspace_bytes, la2_stream_t stream) {
    bool empty = false;
    const la2_status st = size_checks(B, Hk, H, T, d, e, dtype, out_dtype, layout, &empty);
    if (st != LA2_OK) return st;
    if (empty || (T == 0 && !d_init_state)) return LA2_OK;
    if (T > 0 && (!q || !k || !v || !beta || !dout || !dq || !dk || !dv || !dbeta)) return LA2_ERR_INVALID_ARG;
    if (dg && !g) return LA2_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dout, 16) || !aligned(dq, 16) ||
        !aligned(dk, 16) || !aligned(dv, 16) || !aligned(g, 4) || !aligned(beta, 4) || !aligned(dg, 4) ||
        !aligned(dbeta, 4) || !aligned(init_state, 4) || !aligned(d_final_state, 4) ||
        !aligned(d_init_state, 4) || !aligned(seq_lens, 4))
        return LA2_ERR_INVALID_ARG;
    const size_t need = la2_gdr_workspace_bytes(B, Hk, H, T, d, e, dtype, 1);
    if (need && (!workspace || workspace_bytes < need)) return LA2_ERR_WORKSPACE;
    if (need && !aligned(workspace, 256)) return LA2_ERR_INVALID_ARG;
    if (!device_setup()) return LA2_ERR_CUDA;
    Args A = {};
    A.q = q; A.k = k; A.v = v; A.dout = dout; A.g = g; A.beta = beta;
    A.dq = dq; A.dk = dk; A.dv = dv; A.dg = dg; A.dbeta = dbeta;
    A.init = init_state; A.dfinal = d_final_state; A.dinit = d_init_state; A.lens = seq_lens;
    A.B = B; A.Hk = Hk; A.H = H; A.T = T; A.d = d; A.e = e;
    A.bthd = layout == LA2_LAYOUT_BTHD;
    A.out_bf16 = out_dtype == LA2_DTYPE_BF16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    if (by_chunks(dtype, d, e)) return d == 64 ? chunk_backward<64>(A, ws, s) : chunk_backward<128>(A, ws, s);
    return dtype == LA2_DTYPE_BF16 ? rec_backward<__nv_bfloat16>(A, ws, s) : rec_backward<float>(A, ws, s);
}

la2_status la2_gdr_decode(const void* q, const void* k, const void* v, const float* g, const float* beta,
                          float* states, const int* slots, int n_slots, float* out, int B, int Hk, int H,
                          int d, int e, la2_dtype dtype, la2_stream_t stream) {
    bool empty = false;
    const la2_status st =
        size_checks(B, Hk, H, 1, d, e, dtype, LA2_DTYPE_F32, LA2_LAYOUT_BHTD, &empty);
    if (st != LA2_OK) return st;
    if (n_slots < 0) return LA2_ERR_INVALID_ARG;
    if (empty) return LA2_OK;
    if (!q || !k || !v || !beta || !out || (n_slots > 0 && !states)) return LA2_ERR_INVALID_ARG;
    const uintptr_t el = dtype == LA2_DTYPE_BF16 ? 2 : 4;
    if (!aligned(q, el) || !aligned(k, el) || !aligned(v, el) || !aligned(g, 4) || !aligned(beta, 4) ||
        !aligned(states, 4) || !aligned(slots, 4) || !aligned(out, 4))
        return LA2_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = e % 4 == 0 && aligned(states, 16);
    const long long blocks = static_cast<long long>(B) * H * cdiv(e, la2::gdr::kStepUnits * (vec ? 4 : 1));
    if (blocks > INT_MAX) return LA2_ERR_UNSUPPORTED;
    const unsigned grid = static_cast<unsigned>(blocks);
    // From two states per SM on the pipelined kernel; it and the other one, in us: states of 64 x 64: 148 of them
    // 8.2 and 8.2, 296 10.2 and 10.2, 592 12.3 and 14.3, 2560 25 and 41; of 128 x 128: 148 12.3 and 11, 296 16.4 and
    // 16.4, 592 22.5 and 26.6, 2560 63 and 90; of 16 x 16: 296 8.2 and 8.2, 5120 29 and 33.
    const bool bulk = vec && n_slots > 0 && static_cast<long long>(B) * H >= 2 * kSMs;
    int* status = nullptr;
    if (bulk && (!device_setup() || !(status = la2::status_word()))) return LA2_ERR_CUDA;
    const auto go = [&](auto tag) {
        using Tin = decltype(tag);
        const Tin *qq = static_cast<const Tin*>(q), *kk = static_cast<const Tin*>(k), *vv = static_cast<const Tin*>(v);
        const auto pipelined = [&](auto team) {
            constexpr int kTeam = decltype(team)::value;
            la2::gdr::gdr_step_bulk<Tin, kTeam><<<kSMs, la2::gdr::kBulkThreads, la2::gdr::bulk_smem_bytes<kTeam>(), s>>>(
                qq, kk, vv, g, beta, states, slots, n_slots, out, B * H, Hk, H, d, e, la2::gdr::bulk_stages(d, e), status);
        };
        const int team = bulk ? la2::gdr::bulk_team(d, e) : 0;  // (e >= 4)
        if (team == 128) pipelined(std::integral_constant<int, 128>());
        else if (team == 256) pipelined(std::integral_constant<int, 256>());
        else if (team == 512) pipelined(std::integral_constant<int, 512>());
        else if (vec)
            la2::gdr::gdr_step<Tin, 4><<<grid, la2::gdr::kStepThreads, 0, s>>>(qq, kk, vv, g, beta, states, slots,
                                                                             n_slots, out, Hk, H, d, e);
        else
            la2::gdr::gdr_step<Tin, 1><<<grid, la2::gdr::kStepThreads, 0, s>>>(qq, kk, vv, g, beta, states, slots,
                                                                             n_slots, out, Hk, H, d, e);
    };
    if (dtype == LA2_DTYPE_BF16) go(__nv_bfloat16());
    else go(float());
    return launched();
}

la2_status la2_gdr_selftest_timeout(la2_gdr_kernel kernel, void* workspace, size_t workspace_bytes, la2_stream_t stream) {
    if (kernel < LA2_GDR_KERNEL_DECODE || kernel > LA2_GDR_KERNEL_WALKS) return LA2_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < LA2_GDR_SELFTEST_BYTES) return LA2_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return LA2_ERR_INVALID_ARG;
    int* status = nullptr;
    if (!device_setup() || !(status = la2::status_word())) return LA2_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(workspace, 0, LA2_GDR_SELFTEST_BYTES, s) != cudaSuccess) return LA2_ERR_CUDA;
    char* at = static_cast<char*>(workspace);
    const auto take = [&](size_t bytes) {
        char* p = at;
        at += align256(bytes);
        return p;
    };
    using la2::gdr::kMaxDim;
    constexpr int d = kMaxDim, e = kMaxDim;
    if (kernel == LA2_GDR_KERNEL_DECODE) {  // one CTA, six rows one after the other
        constexpr int B = 6;
        const auto *q = reinterpret_cast<__nv_bfloat16*>(take(B * d * 2)), *k = reinterpret_cast<__nv_bfloat16*>(take(B * d * 2)),
                   *v = reinterpret_cast<__nv_bfloat16*>(take(B * e * 2));
        const float* beta = reinterpret_cast<float*>(take(B * sizeof(float)));
        float* states = reinterpret_cast<float*>(take(B * d * e * sizeof(float)));
        float* out = reinterpret_cast<float*>(take(B * e * sizeof(float)));
        la2::gdr::gdr_step_bulk<__nv_bfloat16, 512, true><<<1, la2::gdr::kBulkThreads, la2::gdr::bulk_smem_bytes<512>(), s>>>(
            q, k, v, nullptr, beta, states, nullptr, B, out, B, 1, 1, d, e, la2::gdr::bulk_stages(d, e), status);
        return launched();
    }
    // Two sequences of two value heads and up to four chunks; one ends inside its second chunk, whose padding
    // takes the copies' other way (kRaw).
    static const int lens[2] = {100, 200};
    Args A = {};
    A.B = 2; A.Hk = 1; A.H = 2; A.T = 200; A.d = d; A.e = e;
    const size_t keys = static_cast<size_t>(A.B) * A.Hk * A.T * d * 2, values = static_cast<size_t>(A.B) * A.H * A.T * e * 2,
                 gates = static_cast<size_t>(A.B) * A.H * A.T * sizeof(float);
    A.out_bf16 = 1;
    A.q = take(keys); A.k = take(keys); A.v = take(values); A.dout = take(values);
    A.beta = reinterpret_cast<float*>(take(gates));
    A.o = take(values); A.dq = take(keys); A.dk = take(keys); A.dv = take(values);
    A.dbeta = reinterpret_cast<float*>(take(gates));
    int* n = reinterpret_cast<int*>(take(sizeof(lens)));
    if (cudaMemcpyAsync(n, lens, sizeof(lens), cudaMemcpyHostToDevice, s) != cudaSuccess) return LA2_ERR_CUDA;
    A.lens = n;
    const size_t need = chunk_ws(static_cast<long long>(A.B) * A.H, A.T, d, e, true).bytes;
    char* ws = take(need);
    if (at > static_cast<char*>(workspace) + LA2_GDR_SELFTEST_BYTES) return LA2_ERR_WORKSPACE;
    if (kernel == LA2_GDR_KERNEL_WALK) return chunk_forward<d, true>(A, ws, s);
    return kernel == LA2_GDR_KERNEL_WALKS ? chunk_backward<d, true, false>(A, ws, s) : chunk_backward<d, false, true>(A, ws, s);
}

la2_status la2_state_copy(float* states, const int* src, const int* dst, int n, int n_slots,
                          long long slot_elems, la2_stream_t stream) {
    if (n < 0 || n_slots < 0 || slot_elems < 0) return LA2_ERR_INVALID_ARG;
    if (n == 0 || n_slots == 0 || slot_elems == 0) return LA2_OK;
    if (n > la2::gdr::kPoolMaxPairs) return LA2_ERR_UNSUPPORTED;
    if (!states || !src || !dst || !aligned(states, 4) || !aligned(src, 4) || !aligned(dst, 4))
        return LA2_ERR_INVALID_ARG;
    if (!device_setup()) return LA2_ERR_CUDA;
    const bool vec = slot_elems % 4 == 0 && aligned(states, 16);
    const size_t item = vec ? 16 : 4;
    const long long page = vec ? slot_elems / 4 : slot_elems;
    // slices of at most 32 KB of shared memory, so that several CTAs share an SM
    // and one reads while another writes, down to 32 bytes of a page
    int units = la2::gdr::kPoolThreads;
    while (units > static_cast<int>(32 / item) && static_cast<size_t>(n) * units * item > (32u << 10)) units >>= 1;
    const size_t smem = static_cast<size_t>(n) * (units * item + 2 * sizeof(int)) +
                        (n_slots <= la2::gdr::kPoolTable ? n_slots * sizeof(int) : 0);
    const long long grid = (page + units - 1) / units;
    if (grid > INT_MAX) return LA2_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (vec)
        la2::gdr::pool_copy<float4><<<static_cast<unsigned>(grid), la2::gdr::kPoolThreads, smem, s>>>(
            reinterpret_cast<float4*>(states), src, dst, n, n_slots, page, units);
    else
        la2::gdr::pool_copy<float><<<static_cast<unsigned>(grid), la2::gdr::kPoolThreads, smem, s>>>(
            states, src, dst, n, n_slots, page, units);
    return launched();
}

}  // extern "C"
