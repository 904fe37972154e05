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
// or 12 bytes a token and channel in bf16).  g and dh, which the published run needs, are copied
// a tile ahead; h and x arrive while a tile waits for the state behind it.  The base-2 log gates
// stay in registers between the two walks, the decays are derived from them again.
template <class TX, class TG, bool COMP>
struct GlrBwdTile {
    static constexpr int SUB = glr_sub(sizeof(TX) == 4, sizeof(TG) == 4);
    TX dh[2][GLR_WARPS][SUB][GLR_TILE];
    TG g[2][GLR_WARPS][SUB][GLR_TILE];
    TX h[GLR_WARPS][SUB][GLR_TILE];  // of the token before
    TX x[COMP ? GLR_WARPS : 1][COMP ? SUB : 1][GLR_TILE];
    float4 sums[GLR_WARPS][32];
    GlrShared sm;
};

template <class TX, class TG, int GATE, bool COMP>
__global__ void __launch_bounds__(GLR_THREADS, 2) k_glr_bwd(const GlrParams p) {
    using Tile = GlrBwdTile<TX, TG, COMP>;
    constexpr int SUB = Tile::SUB, CHUNK = SUB * GLR_WARPS;
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    using RX = typename PX::raw;
    using RG = typename PG::raw;
    extern __shared__ __align__(16) unsigned char smem[];
    Tile& tl = *reinterpret_cast<Tile*>(smem);
    GlrShared& sm = tl.sm;
    const int chunks = glr_chunks(p.T, sizeof(TX) == 4, sizeof(TG) == 4);
    const unsigned tiles = (p.C + GLR_TILE - 1) / GLR_TILE, all = tiles * chunks;
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, i0 = w * SUB, ld = p.C / 2;
    const int pos = GLR_WARPS - 1 - w;  // this warp's place in the order of the scan
    const GlrRuns runs = glr_runs(p.status, chunks, p.C);

    auto copy = [&](unsigned id, int b) {  // this warp's g and dh of a tile
        if (id < all) {
            const int k = id / tiles, c0 = (id - k * tiles) * GLR_TILE;
            const int64_t t = (int64_t)(chunks - 1 - k) * CHUNK + i0;
            const int nt = (int)min((int64_t)SUB, max((int64_t)0, p.T - t));
            const TX* dh = static_cast<const TX*>(p.dh);
            const TG* g = static_cast<const TG*>(p.g);
            glr_copy_rows<SUB>(&tl.g[b][w][0][0], g + t * p.ldg + c0, p.ldg, 0, nt, p.C - c0, p.wide, lane, g);
            glr_copy_rows<SUB>(&tl.dh[b][w][0][0], dh + t * p.C + c0, p.C, 0, nt, p.C - c0, p.wide, lane, dh);
        }
        copies_commit();
    };
    auto look = [&](unsigned id, int b) {  // the sequences of a tile's tokens; one warp
        if (id >= all) return;
        const int k = id / tiles, c = (id - k * tiles) * GLR_TILE + 2 * lane, kc = chunks - 1 - k;
        glr_find_sequences(p, sm.info[b], (int64_t)kc * CHUNK, (int)min((int64_t)CHUNK, p.T - (int64_t)kc * CHUNK), lane);
        glr_empty_sequences(p, p.dht, p.dh0, kc, chunks, c, c < p.C, id == k * tiles);
    };
    unsigned summed = all;  // the tile whose warps' sums lie in tl.sums
    auto add_sums = [&]() {  // ... its sums, in a fixed order; one warp
        const int k = summed / tiles, c = (summed - k * tiles) * GLR_TILE + 2 * lane;
        if (summed >= all || c >= p.C) return;
        float4 v = tl.sums[0][lane];
        for (int q = 1; q < GLR_WARPS; ++q) {
            const float4 u = tl.sums[q][lane];
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
        p.sums[(int64_t)k * ld + c / 2] = v;
    };

    if (threadIdx.x == 0) sm.ticket = chunks == 1 ? blockIdx.x : glr_next(p, chunks, 0);
    __syncthreads();
    unsigned id = sm.ticket;
    copy(id, 0);
    if (w == GLR_WARPS - 1) look(id, 0);
    __syncthreads();
    if (threadIdx.x == 0) sm.ticket = glr_next(p, chunks, id);
    __syncthreads();
    for (int b = 0; id < all; b ^= 1) {
        const unsigned next = sm.ticket;
        const int k = id / tiles, kc = chunks - 1 - k, tile = id - k * tiles, c0 = tile * GLR_TILE, c = c0 + 2 * lane;
        const bool live = c < p.C;
        const int64_t t0 = (int64_t)kc * CHUNK, t = t0 + i0;  // the chunk's first token, this warp's
        const int len = (int)min((int64_t)CHUNK, p.T - t0);
        const int nt = (int)min((int64_t)SUB, max((int64_t)0, p.T - t));
        {
            const TX* h = static_cast<const TX*>(p.h_in);
            glr_copy_rows<SUB>(&tl.h[w][0][0], h + (t - 1) * p.C + c0, p.C, t == 0, nt, p.C - c0, p.wide, lane, h);
            if (COMP) {
                const TX* x = static_cast<const TX*>(p.x);
                glr_copy_rows<SUB>(&tl.x[w][0][0], x + t * p.ldx + c0, p.ldx, 0, nt, p.C - c0, p.wide, lane, x);
            }
            copies_commit();
        }
        copy(next, b ^ 1);
        const GlrInfo& info = sm.info[b];
        const uint32_t bits = glr_start_bits(info, i0, nt);  // of this warp's tokens and the one after
        const bool whole = bits == 0 && nt == SUB;
        const GlrPlace at(k, chunks - 1 - (int)((uint64_t)(info.end1 - 1) / CHUNK), info.starts[len >> 5] >> (len & 31) & 1);
        GlrGate<GATE> gate;
        gate.load(p.A_log, p.dt_bias, live ? c : 0);
        RX* dx = reinterpret_cast<RX*>(static_cast<TX*>(p.dx) + t * p.C + c);
        RG* dg = reinterpret_cast<RG*>(static_cast<TG*>(p.dg) + t * p.C + c);
        auto gv = [&](int i) { return PG::widen(*reinterpret_cast<const RG*>(&tl.g[b][w][i][2 * lane])); };
        auto dv = [&](int i) { return PX::widen(*reinterpret_cast<const RX*>(&tl.dh[b][w][i][2 * lane])); };
        auto state_of = [&](const float* from, int i) {
            return from && live ? *reinterpret_cast<const float2*>(from + (int64_t)glr_seq_at(info, i) * p.C + c) : splat(0.f);
        };
        float2 sumA = splat(0.f), sumB = splat(0.f);
        // a token's gradients from l and y = a l; h before it from the tile or, at a start, given
        auto token = [&](int i, float2 tg, float2 s, float2 l, float2 y, float2 before) {
            if (COMP) before = __ffma2_rn(PX::widen(*reinterpret_cast<const RX*>(&tl.x[w][i][2 * lane])), splat(-1.f), before);
            float2 d = __fmul2_rn(y, before);
            if (GATE == GLR_SOFTPLUS) {
                sumA = __ffma2_rn(d, tg, sumA);
                d = __fmul2_rn(d, gate.slope(gv(i)));
                sumB = __fadd2_rn(sumB, d);
            }
            if (live) {
                dx[(int64_t)i * ld] = PX::narrow(COMP ? __fmul2_rn(s, l) : l);
                dg[(int64_t)i * ld] = PG::narrow(d);
            }
        };
        auto hv = [&](int i) { return PX::widen(*reinterpret_cast<const RX*>(&tl.h[w][i][2 * lane])); };
        // the rolled walk from the state r.H, with outputs or (for the run) without
        auto walk = [&](Run r, bool out) {
#pragma unroll 1
            for (int i = nt - 1; i >= 0; --i) {
                const float2 tg = gate.log2_gate(gv(i));
                float2 a, s;
                decay(tg, a, s);
                if (bits >> (i + 1) & 1) {
                    r.A = splat(-0.f);
                    r.H = state_of(p.dht, i0 + i);
                } else {
                    r.A = __fmul2_rn(r.A, a);
                }
                const float2 l = __fadd2_rn(r.H, dv(i));
                r.H = __fmul2_rn(a, l);
                if (out) {
                    const bool first = bits >> i & 1;
                    token(i, tg, s, l, r.H, first ? state_of(p.h0, i0 + i) : hv(i));
                    if (first && live) *reinterpret_cast<float2*>(p.dh0 + (int64_t)glr_seq_at(info, i0 + i) * p.C + c) = r.H;
                }
            }
            return r;
        };
        copies_wait<2>();
        Run r = run_identity();
        float2 tg[SUB];
        if (whole) {
#pragma unroll
            for (int i = SUB - 1; i >= 0; --i) {
                tg[i] = gate.log2_gate(gv(i));
                const float2 a = decay(tg[i]);
                r.A = __fmul2_rn(r.A, a);
                r.H = __fmul2_rn(a, __fadd2_rn(r.H, dv(i)));
            }
        } else {
            r = walk(r, false);
        }
        sm.sub[pos][lane] = run_bits(r);
        __syncthreads();
        const bool restarts = info.starts[0] | info.starts[1] | info.starts[2] | info.starts[3] | info.starts[4];
        Run before = glr_before_warp(sm, pos, lane, restarts), own;
        if (chunks > 1) own = glr_exchange(p, sm, at, runs, w, lane, c / 2, live);
        if (w == GLR_WARPS - 1) {
            if (lane == 0) sm.ticket = glr_next(p, chunks, next);
            look(next, b ^ 1);
            if (GATE == GLR_SOFTPLUS) add_sums();
        }
        __syncthreads();
        float2 y = glr_after(before, glr_state_before(sm, at, lane));
        if (w == 0 && chunks > 1) glr_publish_groups(p, sm, at, runs, own, lane, c / 2, live);
        copies_wait<1>();
        if (whole) {
#pragma unroll
            for (int i = SUB - 1; i >= 0; --i) {
                forget(tg[i]);
                float2 a, s;
                decay(tg[i], a, s);
                const float2 l = __fadd2_rn(y, dv(i));
                y = __fmul2_rn(a, l);
                token(i, tg[i], s, l, y, hv(i));
            }
        } else {
            walk(Run{splat(1.f), y}, true);
        }
        if (GATE == GLR_SOFTPLUS) tl.sums[w][lane] = make_float4(kLn2f * sumA.x, kLn2f * sumA.y, sumB.x, sumB.y);
        __syncwarp();  // the warp's rows are free for the next copies
        summed = id;
        id = next;
    }
    copies_wait<0>();
    if (GATE == GLR_SOFTPLUS) {
        __syncthreads();
        if (w == 0) add_sums();
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
    return p.gate == GLR_SOFTPLUS ? sizeof(float4) * (size_t)(p.C / 2) * glr_chunks(p.T, p.act_f32, p.gate_f32) : 0;
}

namespace {
struct Launch {
    const GlrParams& p;
    cudaStream_t s;
    template <class TX, class TG, int GATE, bool COMP>
    cudaError_t run() const {
        static std::atomic<uint64_t> ready{0};
        cudaError_t e = glr_launch(k_glr_bwd<TX, TG, GATE, COMP>, ready, sizeof(GlrBwdTile<TX, TG, COMP>), 2, p, s);
        if (e != cudaSuccess || GATE != GLR_SOFTPLUS) return e;
        k_glr_sums<<<(p.C / 2 + 31) / 32, 1024, 0, s>>>(p.sums, glr_chunks(p.T, p.act_f32, p.gate_f32), p.C, p.dA_log,
                                                        p.ddt_bias);
        return cudaGetLastError();
    }
};
}  // namespace

cudaError_t launch_glr_bwd(const GlrParams& p, cudaStream_t s) {
    return glr_dispatch(p.act_f32, p.gate_f32, p.gate, p.complement, Launch{p, s});
}

}  // namespace gdr
