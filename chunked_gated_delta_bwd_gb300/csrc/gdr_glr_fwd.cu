// Gated linear recurrence, forward and single-token step: h_t = a_t h_{t-1} + s_t x_t per
// channel, the state kept in fp32.
//
// The simplest form: a thread owns two channels and walks every sequence from its first to its
// last token.
#include "gdr_glr.cuh"
#include "gdr_internal.h"

namespace gdr {

template <class TX, class TG, int GATE, bool COMP>
__global__ void __launch_bounds__(64) k_glr_fwd(const GlrParams p) {
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    if (blockIdx.x == 0) glr_check_seqlens(p.cu_seqlens, p.N, p.T, threadIdx.x, 64, p.status);
    const int c = (blockIdx.x * 64 + threadIdx.x) * 2;
    if (c >= p.C) return;
    GlrGate<GATE> g0, g1;
    g0.load(p.A_log, p.dt_bias, c);
    g1.load(p.A_log, p.dt_bias, c + 1);
    const TX* x = static_cast<const TX*>(p.x) + c;
    const TG* g = static_cast<const TG*>(p.g) + c;
    TX* h = static_cast<TX*>(p.h) + c;
    for (int n = 0; n < p.N; ++n) {
        int64_t b, e;
        glr_bounds(p.cu_seqlens, p.seq_len, p.T, n, b, e);
        float2 st = make_float2(0.f, 0.f);
        if (p.h0) st = *reinterpret_cast<const float2*>(p.h0 + (int64_t)n * p.C + c);
        for (int64_t t = b; t < e; ++t) {
            const float2 xv = PX::widen(*reinterpret_cast<const typename PX::raw*>(x + t * p.ldx));
            const float2 gv = PG::widen(*reinterpret_cast<const typename PG::raw*>(g + t * p.ldg));
            float2 a, s;
            decay(g0.log_gate(gv.x), a.x, s.x);
            decay(g1.log_gate(gv.y), a.y, s.y);
            st.x = fmaf(a.x, st.x, COMP ? s.x * xv.x : xv.x);
            st.y = fmaf(a.y, st.y, COMP ? s.y * xv.y : xv.y);
            *reinterpret_cast<typename PX::raw*>(h + t * p.C) = PX::narrow(st);
        }
        if (p.ht) *reinterpret_cast<float2*>(p.ht + (int64_t)n * p.C + c) = st;
    }
}

namespace {
struct Launch {
    const GlrParams& p;
    cudaStream_t s;
    template <class TX, class TG, int GATE, bool COMP>
    cudaError_t run() const {
        k_glr_fwd<TX, TG, GATE, COMP><<<(p.C / 2 + 63) / 64, 64, 0, s>>>(p);
        return cudaGetLastError();
    }
};
}  // namespace

cudaError_t launch_glr_fwd(const GlrParams& p, cudaStream_t s) {
    return glr_dispatch(p.act_f32, p.gate_f32, p.gate, p.complement, Launch{p, s});
}

// One token for each row: y = h = a h + s x on the row's state, in place.  A row whose slot is
// negative (padding of the batch) or past the pool reads and writes no state; its y is zero.
template <class TX, class TG, int GATE, bool COMP>
__global__ void __launch_bounds__(128) k_glr_step(const GlrStepParams p) {
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    const int c = (blockIdx.x * 128 + threadIdx.x) * 2;
    if (c >= p.C) return;
    for (int64_t n = blockIdx.y; n < p.N; n += gridDim.y) {
        const int64_t slot = p.slots ? p.slots[n] : n;
        float2 st = make_float2(0.f, 0.f);
        if (slot >= 0 && slot < p.pool) {
            float2* home = reinterpret_cast<float2*>(p.state + slot * p.C + c);
            GlrGate<GATE> g0, g1;
            g0.load(p.A_log, p.dt_bias, c);
            g1.load(p.A_log, p.dt_bias, c + 1);
            const float2 xv = PX::widen(*reinterpret_cast<const typename PX::raw*>(static_cast<const TX*>(p.x) + n * p.ldx + c));
            const float2 gv = PG::widen(*reinterpret_cast<const typename PG::raw*>(static_cast<const TG*>(p.g) + n * p.ldg + c));
            st = *home;
            float2 a, s;
            decay(g0.log_gate(gv.x), a.x, s.x);
            decay(g1.log_gate(gv.y), a.y, s.y);
            st.x = fmaf(a.x, st.x, COMP ? s.x * xv.x : xv.x);
            st.y = fmaf(a.y, st.y, COMP ? s.y * xv.y : xv.y);
            *home = st;
        }
        *reinterpret_cast<typename PX::raw*>(static_cast<TX*>(p.y) + n * p.C + c) = PX::narrow(st);
    }
}

namespace {
struct StepLaunch {
    const GlrStepParams& p;
    cudaStream_t s;
    template <class TX, class TG, int GATE, bool COMP>
    cudaError_t run() const {
        const dim3 grid((p.C / 2 + 127) / 128, p.N < 65535 ? p.N : 65535);
        k_glr_step<TX, TG, GATE, COMP><<<grid, 128, 0, s>>>(p);
        return cudaGetLastError();
    }
};
}  // namespace

cudaError_t launch_glr_step(const GlrStepParams& p, cudaStream_t s) {
    return glr_dispatch(p.act_f32, p.gate_f32, p.gate, p.complement, StepLaunch{p, s});
}

}  // namespace gdr
