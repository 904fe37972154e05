// Gated linear recurrence, backward.  With l_t the gradient of h_t through every later token
// of its sequence (l = dh + dht at the last one):
//
//   l_t = dh_t + a_{t+1} l_{t+1},   dx_t = s_t l_t,   dh0 = a l at the first token
//   dg_t = l_t a_t (h_{t-1} - [complement] x_t)     (ds/dg = -a)
//   softplus gate, z = g_raw + dt_bias: dg_raw = dg (-e^{A_log} sigmoid z),
//   ddt_bias = sum_t dg_raw,  dA_log = sum_t dg g
//
// The scan (gdr_glr.cuh) runs against time on y_t = a_t l_t = a_t (dh_t + y_{t+1}), restarted from
// dht at each sequence's last token; what it leaves at the first token is dh0.
#include "gdr_glr.cuh"
#include "gdr_internal.h"

namespace gdr {

// Bytes bound it: g, h, dh (and x with the complement) are read once, dx and dg written once (10
// or 12 bytes a token and channel in bf16).  g and dh are loaded first, for the run that is
// published; h and x only then, so that they arrive while the block waits for the state.
template <class TX, class TG, int GATE, bool COMP>
__global__ void __launch_bounds__(GLR_THREADS, 2) k_glr_bwd(const GlrParams p) {
    constexpr int SUB = glr_sub(sizeof(TX) == 4), CHUNK = SUB * GLR_WARPS;
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    using RX = typename PX::raw;
    using RG = typename PG::raw;
    __shared__ GlrShared sm;
    const int chunks = glr_chunks(p.T, sizeof(TX) == 4);
    const int tiles = (p.C + GLR_TILE - 1) / GLR_TILE;
    const unsigned id = glr_ticket(p, sm, chunks);
    const int k = id / (unsigned)tiles, kc = chunks - 1 - k;  // the chunk's number against and in the order of time
    const int tile = id - k * tiles, w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int c = tile * GLR_TILE + 2 * lane, i0 = w * SUB, ld = p.C / 2;
    const bool live = c < p.C;
    const int64_t t0 = (int64_t)kc * CHUNK, t = t0 + i0;  // the chunk's first token, this warp's
    const int len = (int)min((int64_t)CHUNK, p.T - t0);
    const int nt = (int)min((int64_t)SUB, max((int64_t)0, p.T - t));  // tokens of this warp
    const int64_t ldx = p.ldx / 2, ldg = p.ldg / 2;
    const RG* g = reinterpret_cast<const RG*>(static_cast<const TG*>(p.g) + t * p.ldg + c);
    const RX* dh = reinterpret_cast<const RX*>(static_cast<const TX*>(p.dh) + t * p.C + c);
    const RX* h = reinterpret_cast<const RX*>(static_cast<const TX*>(p.h_in) + (t - 1) * p.C + c);  // the state before
    const RX* x = COMP ? reinterpret_cast<const RX*>(static_cast<const TX*>(p.x) + t * p.ldx + c) : nullptr;
    RX* dx = reinterpret_cast<RX*>(static_cast<TX*>(p.dx) + t * p.C + c);
    RG* dg = reinterpret_cast<RG*>(static_cast<TG*>(p.dg) + t * p.C + c);
    RG gr[SUB];
    RX dr[SUB], hr[SUB], xr[SUB];
    if (nt == SUB && live) {
#pragma unroll
        for (int i = SUB - 1; i >= 0; --i) {
            gr[i] = __ldg(g + i * ldg);
            dr[i] = __ldg(dh + i * ld);
        }
    } else {
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            gr[i] = PG::zero();
            dr[i] = PX::zero();
        }
    }
    GlrGate<GATE> gate;
    if (live) gate.load(p.A_log, p.dt_bias, c);
    if (w == 0) glr_find_sequences(p, sm, t0, len, lane);
    if (w == GLR_WARPS - 1) glr_empty_sequences(p, p.dht, p.dh0, kc, chunks, c, live, tile == 0);
    __syncthreads();
    const uint32_t bits = glr_start_bits(sm, i0, nt);  // of this warp's tokens and the one after
    const bool whole = bits == 0 && nt == SUB;
    float2 sumA = splat(0.f), sumB = splat(0.f);

    // one token's gradients from l a (y) and the state before it
    auto token = [&](float2 tg, typename PG::raw graw, float2 l, float2 s, float2 y, float2 before, float2 xv, RX* to_dx,
                     RG* to_dg) {
        float2 d = __fmul2_rn(y, COMP ? __fadd2_rn(before, make_float2(-xv.x, -xv.y)) : before);
        if (GATE == GLR_SOFTPLUS) {
            sumA = __ffma2_rn(d, tg, sumA);
            d = __fmul2_rn(d, gate.slope(PG::widen(graw)));
            sumB = __fadd2_rn(sumB, d);
        }
        if (live) {
            *to_dx = PX::narrow(COMP ? __fmul2_rn(s, l) : l);
            *to_dg = PG::narrow(d);
        }
    };
    auto state_of = [&](const float* from, int i) {
        return from && live ? *reinterpret_cast<const float2*>(from + (int64_t)glr_seq_at(sm, i) * p.C + c) : splat(0.f);
    };
    // the rolled walk from the state y (or, for the run, from none), with outputs or without
    auto walk = [&](Run r, bool out) {
#pragma unroll 1
        for (int i = nt - 1; i >= 0; --i) {
            const RG graw = live ? g[i * ldg] : PG::zero();
            const float2 tg = gate.log2_gate(PG::widen(graw));
            float2 a, s;
            decay(tg, a, s);
            if (bits >> (i + 1) & 1) {
                r.A = splat(-0.f);
                r.H = state_of(p.dht, i0 + i);
            } else {
                r.A = __fmul2_rn(r.A, a);
            }
            const float2 l = __fadd2_rn(r.H, live ? PX::widen(dh[i * ld]) : splat(0.f));
            r.H = __fmul2_rn(a, l);
            if (out) {
                const bool first = bits >> i & 1;
                const float2 before = first ? state_of(p.h0, i0 + i) : live && t + i > 0 ? PX::widen(h[i * ld]) : splat(0.f);
                token(tg, graw, l, s, r.H, before, COMP && live ? PX::widen(x[i * ldx]) : splat(0.f), dx + i * ld, dg + i * ld);
                if (first && live) *reinterpret_cast<float2*>(p.dh0 + (int64_t)glr_seq_at(sm, i0 + i) * p.C + c) = r.H;
            }
        }
        return r;
    };
    Run r = run_identity();
    float2 tg[SUB];  // the base-2 log gates
    if (whole) {
#pragma unroll
        for (int i = SUB - 1; i >= 0; --i) {
            tg[i] = gate.log2_gate(PG::widen(gr[i]));
            const float2 a = decay(tg[i]);
            r.A = __fmul2_rn(r.A, a);
            r.H = __fmul2_rn(a, __fadd2_rn(r.H, PX::widen(dr[i])));
        }
    } else {
        r = walk(r, false);
    }
    const int pos = GLR_WARPS - 1 - w;
    sm.sub[pos][lane] = run_bits(r);
    if (whole && live) {
#pragma unroll
        for (int i = SUB - 1; i >= 0; --i) {
            hr[i] = t + i > 0 ? __ldg(h + i * ld) : PX::zero();
            xr[i] = COMP ? __ldg(x + i * ldx) : PX::zero();
        }
    }
    __syncthreads();
    float2 y = glr_carry(p, sm, chunks, k, chunks - 1 - (int)((uint64_t)(sm.end1 - 1) / CHUNK),
                         sm.starts[len >> 5] >> (len & 31) & 1, pos, lane, c / 2, live);

    if (whole) {
        dx += (SUB - 1) * ld;
        dg += (SUB - 1) * ld;
#pragma unroll
        for (int i = SUB - 1; i >= 0; --i, dx -= ld, dg -= ld) {
            forget(tg[i]);
            forget(dr[i]);
            forget(gr[i]);
            float2 a, s;
            decay(tg[i], a, s);
            const float2 l = __fadd2_rn(y, PX::widen(dr[i]));
            y = __fmul2_rn(a, l);
            token(tg[i], gr[i], l, s, y, PX::widen(hr[i]), PX::widen(xr[i]), dx, dg);
        }
    } else {
        r.H = y;
        walk(r, true);
    }
    if (GATE == GLR_SOFTPLUS) {  // the chunk's sums, the warps' in a fixed order
        __shared__ float4 sums[GLR_WARPS][32];
        sums[w][lane] = make_float4(kLn2f * sumA.x, kLn2f * sumA.y, sumB.x, sumB.y);
        __syncthreads();
        if (w == 0 && live) {
            float4 v = sums[0][lane];
            for (int q = 1; q < GLR_WARPS; ++q) {
                const float4 u = sums[q][lane];
                v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
            p.sums[(int64_t)kc * ld + c / 2] = v;
        }
    }
}

// dA_log and ddt_bias: the chunks' sums, added in a fixed order.  A block takes 32 pairs of
// channels, each of its 32 warps every 32nd chunk.
__global__ void __launch_bounds__(1024) k_glr_sums(const float4* sums, int chunks, int C, float* dA_log, float* ddt_bias) {
    __shared__ float4 part[32][33];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, c2 = blockIdx.x * 32 + lane;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c2 < C / 2) {
#pragma unroll 4
        for (int k = w; k < chunks; k += 32) {
            const float4 u = sums[(int64_t)k * (C / 2) + c2];
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
    }
    part[w][lane] = v;
    __syncthreads();
    v = part[lane][w];  // the pair w of the block, the warps' sums across the lanes
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        v.x += __shfl_xor_sync(~0u, v.x, o);
        v.y += __shfl_xor_sync(~0u, v.y, o);
        v.z += __shfl_xor_sync(~0u, v.z, o);
        v.w += __shfl_xor_sync(~0u, v.w, o);
    }
    const int c = (blockIdx.x * 32 + w) * 2;
    if (lane == 0 && c < C) {
        *reinterpret_cast<float2*>(dA_log + c) = make_float2(v.x, v.y);
        *reinterpret_cast<float2*>(ddt_bias + c) = make_float2(v.z, v.w);
    }
}

size_t glr_sums_bytes(const GlrParams& p) {
    return p.gate == GLR_SOFTPLUS ? sizeof(float4) * (size_t)(p.C / 2) * glr_chunks(p.T, p.act_f32) : 0;
}

namespace {
struct Launch {
    const GlrParams& p;
    cudaStream_t s;
    template <class TX, class TG, int GATE, bool COMP>
    cudaError_t run() const {
        const int chunks = glr_chunks(p.T, sizeof(TX) == 4);
        k_glr_bwd<TX, TG, GATE, COMP><<<(unsigned)(chunks * ((p.C + GLR_TILE - 1) / GLR_TILE)), GLR_THREADS, 0, s>>>(p);
        if (GATE == GLR_SOFTPLUS)
            k_glr_sums<<<(p.C / 2 + 31) / 32, 1024, 0, s>>>(p.sums, chunks, p.C, p.dA_log, p.ddt_bias);
        return cudaGetLastError();
    }
};
}  // namespace

cudaError_t launch_glr_bwd(const GlrParams& p, cudaStream_t s) {
    return glr_dispatch(p.act_f32, p.gate_f32, p.gate, p.complement, Launch{p, s});
}

}  // namespace gdr
