// Device parts shared by the gated linear recurrence's kernels: pairs of channels, the gate
// function and its chain rule.
//
//   g_t = g_raw_t  (gate "log")   or   -e^{A_log} softplus(g_raw_t + dt_bias)  (gate "softplus")
//   a_t = e^{g_t},   s_t = 1  or  1 - a_t  (complement),   h_t = a_t h_{t-1} + s_t x_t
#pragma once
#include "gdr_block.h"
#include "gdr_common.cuh"

namespace gdr {

enum { GLR_LOG = 0, GLR_SOFTPLUS = 1 };

// two consecutive channels of a row as loaded, and as fp32
template <class T> struct PairOf;
template <> struct PairOf<__nv_bfloat16> {
    using raw = uint32_t;
    static __device__ __forceinline__ float2 widen(raw r) { return unpack_bf16(r); }
    static __device__ __forceinline__ raw narrow(float2 v) { return pack_bf16(v.x, v.y); }
    static __device__ __forceinline__ raw zero() { return 0u; }
};
template <> struct PairOf<float> {
    using raw = float2;
    static __device__ __forceinline__ float2 widen(raw r) { return r; }
    static __device__ __forceinline__ raw narrow(float2 v) { return v; }
    static __device__ __forceinline__ raw zero() { return make_float2(0.f, 0.f); }
};

// a = e^g and, where asked for, s = 1 - e^g.  A slow channel (|g| below 1/4) keeps its state
// for hundreds of tokens, over which a relative error of a that has one sign grows by the
// number of tokens; there both come from the Taylor series of e^g - 1 (seven terms, truncation
// |g|^7 / 7! < 1.3e-8 absolute and 5e-8 relative to g), so a is rounded once and s does not
// cancel.  Elsewhere the memory is a few tokens and the hardware exponential's 2^-22 is enough.
__device__ __forceinline__ void decay(float g, float& a, float& s) {
    const float m = g * (1.f + g * (0.5f + g * (1.f / 6.f + g * (1.f / 24.f + g * (1.f / 120.f + g * (1.f / 720.f))))));
    const float e = __expf(g);
    const bool slow = fabsf(g) < 0.25f;
    a = slow ? 1.f + m : e;
    s = slow ? -m : 1.f - e;
}

// one channel's gate: its parameters and the log gate of a raw value
template <int GATE>
struct GlrGate {
    float nA, bias;  // -e^{A_log}, dt_bias
    __device__ __forceinline__ void load(const float* A_log, const float* dt_bias, int c) {
        if constexpr (GATE == GLR_SOFTPLUS) {
            nA = -expf(A_log[c]);
            bias = dt_bias[c];
        }
    }
    __device__ __forceinline__ float log_gate(float raw) const {
        if constexpr (GATE == GLR_LOG) return raw;
        else return nA * softplus_f(raw + bias);
    }
    // the log gate, and dg/d(raw) = -e^{A_log} sigmoid(z)
    __device__ __forceinline__ float log_gate_slope(float raw, float& slope) const {
        if constexpr (GATE == GLR_LOG) {
            slope = 1.f;
            return raw;
        } else {
            float sp, sg;
            softplus_sigmoid(raw + bias, sp, sg);
            slope = nA * sg;
            return nA * sp;
        }
    }
};

// [begin, end) of sequence n, clamped so that inconsistent cu_seqlens stay inside the tensors
__device__ __forceinline__ void glr_bounds(const int64_t* cu, int64_t seq_len, int64_t T, int n, int64_t& b,
                                           int64_t& e) {
    if (!cu) {
        b = (int64_t)n * seq_len;
        e = b + seq_len;
        return;
    }
    b = cu[n];
    e = cu[n + 1];
    b = b < 0 ? 0 : (b > T ? T : b);
    e = e < b ? b : (e > T ? T : e);
}

// cu_seqlens against its contract: sequences n, n + step, ... checked by the calling thread
__device__ __forceinline__ void glr_check_seqlens(const int64_t* cu, int N, int64_t T, int n, int step, int* status) {
    if (!cu) return;
    bool bad = false;
    if (n == 0) bad = cu[0] != 0 || cu[N] != T;
    for (; n < N; n += step) bad |= cu[n + 1] < cu[n];
    if (bad) atomicOr(status, ST_BAD_SEQLENS);
}

// Calls f.run<TX, TG, GATE, COMP>() for the run-time choice of types, gate
// function and input scale (bf16 / fp32 activations; a bf16 or fp32 gate for bf16 activations).
template <class F>
cudaError_t glr_dispatch(int act_f32, int gate_f32, int gate, int comp, const F& f) {
    using bf = __nv_bfloat16;
#define GLR_PICK(TX, TG)                                                                     \
    do {                                                                                     \
        if (gate == GLR_LOG) return comp ? f.template run<TX, TG, GLR_LOG, true>()            \
                                         : f.template run<TX, TG, GLR_LOG, false>();          \
        return comp ? f.template run<TX, TG, GLR_SOFTPLUS, true>()                            \
                    : f.template run<TX, TG, GLR_SOFTPLUS, false>();                          \
    } while (0)
    if (act_f32) GLR_PICK(float, float);
    if (!gate_f32) GLR_PICK(bf, bf);
    GLR_PICK(bf, float);
#undef GLR_PICK
}

}  // namespace gdr
