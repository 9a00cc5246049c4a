// gdr_common.cuh -- what the kernels of the gated delta rule share: the call's
// arguments, where a row of a tensor lies, element conversions.
//
// The rule, per batch entry b and value head h with a d x e state S (fp32):
//
//   S_t = a_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   a_t = exp(g_t),
//   o_t = S_t^T q_t,
//
// i.e. with the decayed state D_t = a_t S_{t-1}: w_t = v_t - D_t^T k_t (what the
// state does not yet predict), u_t = beta_t w_t, S_t = D_t + k_t u_t^T.  Value
// head h reads key head h / (H / Hk).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>

namespace la2 {
namespace gdr {

struct Args {
    const void *q, *k, *v, *dout;
    const float *g, *beta;       // g may be null (no gate: a_t = 1)
    void *o, *dq, *dk, *dv;
    float *dg, *dbeta;           // dg null when g is
    const float *init, *dfinal;  // null: zero
    float *fin, *dinit;          // null: not wanted
    const int* lens;             // [B] or null: every sequence has T rows
    int B, Hk, H, T, d, e;
    int bthd;                    // rows [B, T, heads, width], else [B, heads, T, width]
    int out_bf16;
};

// Element offset of row t of head h (of nh heads of `width`) in batch entry b.
__device__ __forceinline__ size_t row_at(const Args& a, int b, int h, int nh, int t, int width) {
    const size_t r = a.bthd ? (static_cast<size_t>(b) * a.T + t) * nh + h
                            : (static_cast<size_t>(b) * nh + h) * a.T + t;
    return r * width;
}

// Rows of sequence b: lens[b] brought into 0 .. T.
__device__ __forceinline__ int length_of(const Args& a, int b) {
    if (!a.lens) return a.T;
    return min(max(a.lens[b], 0), a.T);
}

// exp(g) underflows fp32 below -104; a gate of -inf (or far below) is brought
// to where its exponential is 0 all the same, so that differences of
// cumulative gates stay finite.  A comparison, not fmaxf, which would bring a
// NaN to the bound as well: a NaN gate has to be seen in the results.
constexpr float kMinGate = -128.f;

__device__ __forceinline__ float bounded_gate(float g) { return g < kMinGate ? kMinGate : g; }

__device__ __forceinline__ float gate_at(const Args& a, size_t i) { return a.g ? bounded_gate(a.g[i]) : 0.f; }

// 2^x, off by at most 2 units in the last place (results below 2^-126 are zero);
// without a branch, so that it can be computed where it is not used.
__device__ __forceinline__ float exp2_flat(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ void put(void* p, size_t i, float x, int bf16) {
    if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
    else static_cast<float*>(p)[i] = x;
}

}  // namespace gdr
}  // namespace la2
