// Gated linear recurrence, forward and single-token step: h_t = a_t h_{t-1} + s_t x_t per
// channel, the state kept in fp32 (the scan's scheme is in gdr_glr.cuh).
#include "gdr_glr.cuh"
#include "gdr_internal.h"

namespace gdr {

size_t glr_published_bytes(const GlrParams& p) { return glr_runs_bytes(glr_chunks(p.T, p.act_f32), p.C); }

// Bytes bound it: x and g are read once and h is written once (6 bytes a token and channel in
// bf16).  A thread keeps its tokens' x as loaded and their decays in fp32 in registers from the
// one evaluation of the gate to the second walk, after the state in front of the chunk is known.
// A warp among whose tokens a sequence begins or ends walks them in a rolled loop that reads
// them again: unrolled, those branches made three quarters of the code and the instruction
// cache bound the kernel.
template <class TX, class TG, int GATE, bool COMP>
__global__ void __launch_bounds__(GLR_THREADS, sizeof(TX) == 2 ? 3 : 4) k_glr_fwd(const GlrParams p) {
    constexpr int SUB = glr_sub(sizeof(TX) == 4), CHUNK = SUB * GLR_WARPS;
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    using RX = typename PX::raw;
    using RG = typename PG::raw;
    __shared__ GlrShared sm;
    const int chunks = glr_chunks(p.T, sizeof(TX) == 4);
    const int tiles = (p.C + GLR_TILE - 1) / GLR_TILE;
    const unsigned id = glr_ticket(p, sm, chunks);
    const int k = id / (unsigned)tiles;
    const int tile = id - k * tiles, w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int c = tile * GLR_TILE + 2 * lane, i0 = w * SUB, ld = p.C / 2;
    const bool live = c < p.C;
    const int64_t t0 = (int64_t)k * CHUNK, t = t0 + i0;  // the chunk's first token, this warp's
    const int nt = (int)min((int64_t)SUB, max((int64_t)0, p.T - t));  // tokens of this warp
    const RX* x = reinterpret_cast<const RX*>(static_cast<const TX*>(p.x) + t * p.ldx + c);
    const RG* g = reinterpret_cast<const RG*>(static_cast<const TG*>(p.g) + t * p.ldg + c);
    const int64_t ldx = p.ldx / 2, ldg = p.ldg / 2;
    RX* h = reinterpret_cast<RX*>(static_cast<TX*>(p.h) + t * p.C + c);
    RX xr[SUB];
    RG gr[SUB];
    if (nt == SUB && live) {
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            gr[i] = __ldg(g + i * ldg);
            xr[i] = __ldg(x + i * ldx);
        }
    } else {
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            gr[i] = PG::zero();
            xr[i] = PX::zero();
        }
    }
    GlrGate<GATE> gate;
    if (live) gate.load(p.A_log, p.dt_bias, c);
    if (w == 0) glr_find_sequences(p, sm, t0, (int)min((int64_t)CHUNK, p.T - t0), lane);
    if (w == GLR_WARPS - 1) glr_empty_sequences(p, p.h0, p.ht, k, chunks, c, live, tile == 0);
    __syncthreads();
    const uint32_t bits = glr_start_bits(sm, i0, nt);  // of this warp's tokens and the one after
    const bool whole = bits == 0 && nt == SUB;
    float2 a[SUB];

    // the rolled walk from the state y (or, for the run, from none), with outputs or without
    auto walk = [&](Run r, bool out) {
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            const float2 d = decay(gate.log2_gate(live ? PG::widen(g[i * ldg]) : splat(0.f)));
            const float2 xv = live ? PX::widen(x[i * ldx]) : splat(0.f);
            if (bits >> i & 1) {
                r.A = splat(-0.f);
                r.H = p.h0 && live ? *reinterpret_cast<const float2*>(p.h0 + (int64_t)glr_seq_at(sm, i0 + i) * p.C + c)
                                   : splat(0.f);
            } else {
                r.A = __fmul2_rn(r.A, d);
            }
            r.H = glr_update<COMP>(d, r.H, xv);
            if (out && live) {
                h[(int64_t)i * ld] = PX::narrow(r.H);
                if (p.ht && (bits >> (i + 1) & 1))
                    *reinterpret_cast<float2*>(p.ht + (int64_t)glr_seq_at(sm, i0 + i) * p.C + c) = r.H;
            }
        }
        return r;
    };
    Run r = run_identity();
    if (whole) {
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            a[i] = decay(gate.log2_gate(PG::widen(gr[i])));
            r.A = __fmul2_rn(r.A, a[i]);
            r.H = glr_update<COMP>(a[i], r.H, PX::widen(xr[i]));
        }
    } else {
        r = walk(r, false);
    }
    sm.sub[w][lane] = run_bits(r);
    __syncthreads();
    float2 y = glr_carry(p, sm, chunks, k, (int)((uint64_t)sm.begin0 / CHUNK), sm.starts[0] & 1, w, lane, c / 2, live);

    if (whole) {
#pragma unroll
        for (int i = 0; i < SUB; ++i, h += ld) {
            forget(xr[i]);
            y = glr_update<COMP>(a[i], y, PX::widen(xr[i]));
            if (live) *h = PX::narrow(y);
        }
    } else {
        r.H = y;
        walk(r, true);
    }
}

namespace {
struct Launch {
    const GlrParams& p;
    cudaStream_t s;
    template <class TX, class TG, int GATE, bool COMP>
    cudaError_t run() const {
        const int chunks = glr_chunks(p.T, sizeof(TX) == 4);
        k_glr_fwd<TX, TG, GATE, COMP><<<(unsigned)(chunks * ((p.C + GLR_TILE - 1) / GLR_TILE)), GLR_THREADS, 0, s>>>(p);
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
            GlrGate<GATE> gate;
            gate.load(p.A_log, p.dt_bias, c);
            const float2 xv = PX::widen(*reinterpret_cast<const typename PX::raw*>(static_cast<const TX*>(p.x) + n * p.ldx + c));
            const float2 gv = PG::widen(*reinterpret_cast<const typename PG::raw*>(static_cast<const TG*>(p.g) + n * p.ldg + c));
            st = *home;
            st = glr_update<COMP>(decay(gate.log2_gate(gv)), st, xv);
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
