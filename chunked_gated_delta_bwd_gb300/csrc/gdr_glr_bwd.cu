// Gated linear recurrence, backward.  With l_t the gradient of h_t through every later token
// of its sequence (l = dh + dht at the last one):
//
//   l_t = dh_t + a_{t+1} l_{t+1},   dx_t = s_t l_t,   dh0 = a l at the first token
//   dg_t = l_t a_t (h_{t-1} - [complement] x_t)     (ds/dg = -a)
//   softplus gate, z = g_raw + dt_bias: dg_raw = dg (-e^{A_log} sigmoid z),
//   ddt_bias = sum_t dg_raw,  dA_log = sum_t dg g
//
// The simplest form: a thread owns two channels and walks every sequence backwards, so the
// sums over tokens have a fixed order.
#include "gdr_glr.cuh"
#include "gdr_internal.h"

namespace gdr {

template <class TX, class TG, int GATE, bool COMP>
__global__ void __launch_bounds__(64) k_glr_bwd(const GlrParams p) {
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    if (blockIdx.x == 0) glr_check_seqlens(p.cu_seqlens, p.N, p.T, threadIdx.x, 64, p.status);
    const int c = (blockIdx.x * 64 + threadIdx.x) * 2;
    if (c >= p.C) return;
    GlrGate<GATE> gt[2];
    gt[0].load(p.A_log, p.dt_bias, c);
    gt[1].load(p.A_log, p.dt_bias, c + 1);
    const TX* x = static_cast<const TX*>(p.x) + c;
    const TG* g = static_cast<const TG*>(p.g) + c;
    const TX* h = static_cast<const TX*>(p.h_in) + c;
    const TX* dh = static_cast<const TX*>(p.dh) + c;
    TX* dx = static_cast<TX*>(p.dx) + c;
    TG* dg = static_cast<TG*>(p.dg) + c;
    float sumA[2] = {0.f, 0.f}, sumB[2] = {0.f, 0.f};
    for (int n = 0; n < p.N; ++n) {
        int64_t b, e;
        glr_bounds(p.cu_seqlens, p.seq_len, p.T, n, b, e);
        const int64_t row = (int64_t)n * p.C + c;
        float2 carry = make_float2(0.f, 0.f), h0 = make_float2(0.f, 0.f);  // carry: a_{t+1} l_{t+1}
        if (p.dht) carry = *reinterpret_cast<const float2*>(p.dht + row);
        if (p.h0) h0 = *reinterpret_cast<const float2*>(p.h0 + row);
        for (int64_t t = e - 1; t >= b; --t) {
            const float2 gv = PG::widen(*reinterpret_cast<const typename PG::raw*>(g + t * p.ldg));
            const float2 dv = PX::widen(*reinterpret_cast<const typename PX::raw*>(dh + t * p.C));
            const float2 hv = t > b ? PX::widen(*reinterpret_cast<const typename PX::raw*>(h + (t - 1) * p.C)) : h0;
            float2 xv = make_float2(0.f, 0.f);
            if (COMP) xv = PX::widen(*reinterpret_cast<const typename PX::raw*>(x + t * p.ldx));
            float2 odx, odg;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float slope, a, s;
                const float lg = gt[j].log_gate_slope(j ? gv.y : gv.x, slope);
                decay(lg, a, s);
                float& cr = j ? carry.y : carry.x;
                const float l = (j ? dv.y : dv.x) + cr;
                cr = a * l;
                const float d = cr * ((j ? hv.y : hv.x) - (j ? xv.y : xv.x));
                (j ? odx.y : odx.x) = COMP ? s * l : l;
                if (GATE == GLR_SOFTPLUS) {
                    sumA[j] = fmaf(d, lg, sumA[j]);
                    sumB[j] = fmaf(d, slope, sumB[j]);
                }
                (j ? odg.y : odg.x) = d * slope;
            }
            *reinterpret_cast<typename PX::raw*>(dx + t * p.C) = PX::narrow(odx);
            *reinterpret_cast<typename PG::raw*>(dg + t * p.C) = PG::narrow(odg);
        }
        *reinterpret_cast<float2*>(p.dh0 + row) = carry;
    }
    if (GATE == GLR_SOFTPLUS) {
        *reinterpret_cast<float2*>(p.dA_log + c) = make_float2(sumA[0], sumA[1]);
        *reinterpret_cast<float2*>(p.ddt_bias + c) = make_float2(sumB[0], sumB[1]);
    }
}

namespace {
struct Launch {
    const GlrParams& p;
    cudaStream_t s;
    template <class TX, class TG, int GATE, bool COMP>
    cudaError_t run() const {
        k_glr_bwd<TX, TG, GATE, COMP><<<(p.C / 2 + 63) / 64, 64, 0, s>>>(p);
        return cudaGetLastError();
    }
};
}  // namespace

cudaError_t launch_glr_bwd(const GlrParams& p, cudaStream_t s) {
    return glr_dispatch(p.act_f32, p.gate_f32, p.gate, p.complement, Launch{p, s});
}

}  // namespace gdr
