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
// or 12 bytes a token and channel in bf16).  The first walk leaves the base-2 log gates in fp32
// where g was; the second derives the decays, and the softplus gate's slope, from them.  g and dh
// are copied two tiles ahead, h and x, which only the second walk needs, one.
constexpr int BWD_WARPS = 8, BWD_SUB = GLR_CHUNK / BWD_WARPS;
template <class TX, bool COMP, bool SUMS>
struct GlrBwdTile {
    float2 t[3][BWD_WARPS][BWD_SUB][32];    // g as copied (a row in the first bytes of its 256), then the log gates
    TX dh[3][BWD_WARPS][BWD_SUB][GLR_TILE];
    TX h[BWD_WARPS][BWD_SUB][GLR_TILE];     // of the token before
    TX x[COMP ? BWD_WARPS : 1][COMP ? BWD_SUB : 1][GLR_TILE];
    float4 sums[SUMS ? 3 : 1][BWD_WARPS][32];  // of each warp's tokens, for the softplus gate's parameters
    GlrRing<BWD_WARPS, 1> ring;
};

template <class TX, class TG, int GATE, bool COMP>
__global__ void __launch_bounds__(32 * (BWD_WARPS + 4), 2) k_glr_bwd(const GlrParams p) {
    using Tile = GlrBwdTile<TX, COMP, GATE == GLR_SOFTPLUS>;
    constexpr int SUB = BWD_SUB;
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    using RX = typename PX::raw;
    using RG = typename PG::raw;
    extern __shared__ __align__(16) unsigned char smem[];
    Tile& tl = *reinterpret_cast<Tile*>(smem);
    using Ring = decltype(Tile::ring);
    Ring& ring = tl.ring;
    const int chunks = glr_chunks(p);
    const unsigned tiles = (p.C + GLR_TILE - 1) / GLR_TILE, all = tiles * chunks;
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, i0 = w * SUB, ld = p.C / 2;
    glr_ring_init(ring);
    if (w >= BWD_WARPS) {
        const GlrRuns runs = glr_runs(p.status, chunks, p.C);
        // tile j's sums are added before place j + 4 is signalled, and written again only after that
        auto add_sums = [&](int4 tick, int j) {
            const int c = tick.y + 2 * lane;
            if (GATE != GLR_SOFTPLUS || c >= p.C) return;
            float4 v = tl.sums[j % 3][0][lane];
#pragma unroll
            for (int q = 1; q < BWD_WARPS; ++q) {
                const float4 u = tl.sums[j % 3][q][lane];
                v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
            p.sums[(int64_t)tick.x * ld + c / 2] = v;
        };
        int4 tick = glr_look<true>(p, ring, chunks, w - BWD_WARPS, lane);
        for (int j = w - BWD_WARPS; tick.x >= 0; j += 4) {
            glr_exchange<true>(p, ring, runs, chunks, j, tick, lane);
            glr_wait<50>(p, ring, GLR_FREE, j);
            add_sums(tick, j);
            tick = glr_look<true>(p, ring, chunks, j + 4, lane);
        }
        return;
    }
    const int pos = BWD_WARPS - 1 - w;  // this warp's place in the order of the scan

    constexpr int XP = GLR_TILE * sizeof(TX);
    const GlrRows<SUB, 256, TG> g_rows(p.g, p.ldg, i0, lane);
    const GlrRows<SUB, XP, TX> dh_rows(p.dh, p.C, i0, lane), h_rows(p.h_in, p.C, i0 - 1, lane), x_rows(p.x, p.ldx, i0, lane);
    const bool wide = p.wide;
    auto copy = [&](int j) {  // this warp's g and dh of tile j
        glr_wait<0>(p, ring, GLR_TICK, j);
        const int4 tick = ring.tick[j & 7];
        if (tick.x >= 0) {
            const int kc = chunks - 1 - tick.x;
            const int64_t left = p.T - ((int64_t)kc * GLR_CHUNK + i0);
            g_rows.copy(&tl.t[j % 3][w][0][0], kc, tick.y, tick.z, wide, 0, left, p.C - tick.y, lane);
            dh_rows.copy(&tl.dh[j % 3][w][0][0], kc, tick.y, tick.z, wide, 0, left, p.C - tick.y, lane);
        }
        copies_commit();
    };
    auto copy_h = [&](int4 tick) {  // its h, of the token before each, and x
        if (tick.x >= 0) {
            const int kc = chunks - 1 - tick.x;
            const int64_t left = p.T - ((int64_t)kc * GLR_CHUNK + i0);
            h_rows.copy(&tl.h[w][0][0], kc, tick.y, tick.z, wide, kc == 0 && w == 0, left, p.C - tick.y, lane);
            if (COMP) x_rows.copy(&tl.x[w][0][0], kc, tick.y, tick.z, wide, 0, left, p.C - tick.y, lane);
        }
        copies_commit();
    };
    const bool takes = w == 0 && lane == 0;  // the tickets
    for (int j = 0; j < 3; ++j) {
        if (w == 0) {
            if (takes) glr_set_tick<true>(p, ring, chunks, j, glr_ticket(p, chunks, j), tiles, all);
            glr_signal(ring, GLR_TICK, j);
        }
        if (j < 2) copy(j);
        if (j == 0) copies_commit();  // (an h of no tile, so that every tile waits for the same number of groups)
    }
    int4 before = make_int4(-1, 0, 0, 0);  // tile j - 1
    for (int j = 0;; ++j) {
        glr_wait<0>(p, ring, GLR_PLACE, j);
        const int4 tick = ring.tick[j & 7];
        unsigned id = 0;
        if (tick.x >= 0) {
            if (takes) id = glr_ticket(p, chunks, j + 3);
            const GlrInfo& info = ring.info[j & 7];
            const int c = tick.y + 2 * lane;
            const bool live = c < p.C;
            GlrGate<GATE> gate;
            gate.set(ring.gate[j & 3][lane]);
            copies_wait<2>();
            const TX* ds = &tl.dh[j % 3][w][0][2 * lane];
            float2* ts = &tl.t[j % 3][w][0][lane];
            const TG* gs = reinterpret_cast<const TG*>(&tl.t[j % 3][w][0][0]) + 2 * lane;
            constexpr int GP = 256 / sizeof(TG);
            Run r = run_identity();
            if (!info.any) {
#pragma unroll 1
                for (int i = SUB - 4; i >= 0; i -= 4) {
                    RG graw[4];
                    float2 dv[4];
#pragma unroll
                    for (int q = 3; q >= 0; --q) {
                        graw[q] = *reinterpret_cast<const RG*>(gs + (i + q) * GP);
                        dv[q] = PX::widen(*reinterpret_cast<const RX*>(ds + (i + q) * GLR_TILE));
                    }
                    __syncwarp();  // every lane has its g of these rows
#pragma unroll
                    for (int q = 3; q >= 0; --q) {
                        const float2 t = gate.log2_gate(PG::widen(graw[q]));
                        const float2 a = decay(t);
                        ts[(i + q) * 32] = t;
                        r.A = __fmul2_rn(r.A, a);
                        r.H = __fmul2_rn(a, __fadd2_rn(r.H, dv[q]));
                    }
                }
            } else {
                const int nt = (int)min((int64_t)SUB, max((int64_t)0, p.T - ((int64_t)(chunks - 1 - tick.x) * GLR_CHUNK + i0)));
                const uint32_t bits = glr_start_bits(info, i0, nt);
#pragma unroll 1
                for (int i = nt - 1; i >= 0; --i) {
                    const RG graw = *reinterpret_cast<const RG*>(gs + i * GP);
                    __syncwarp();
                    const float2 t = gate.log2_gate(PG::widen(graw));
                    const float2 a = decay(t);
                    ts[i * 32] = t;
                    if (bits >> (i + 1) & 1) {
                        r.A = splat(-0.f);
                        r.H = p.dht && live ? *reinterpret_cast<const float2*>(p.dht + (int64_t)glr_seq_at(info, i0 + i) * p.C + c)
                                            : splat(0.f);
                    } else {
                        r.A = __fmul2_rn(r.A, a);
                    }
                    r.H = __fmul2_rn(a, __fadd2_rn(r.H, PX::widen(*reinterpret_cast<const RX*>(ds + i * GLR_TILE))));
                }
            }
            ring.sub[j & 1][pos][lane] = run_bits(r);
            glr_runs_there<Ring>(j);
        }
        if (before.x >= 0) {
            const int kc = chunks - 1 - before.x, c = before.y + 2 * lane;
            const bool live = c < p.C;
            const int64_t t0 = (int64_t)kc * GLR_CHUNK + i0;
            GlrGate<GATE> gate;
            gate.set(ring.gate[(j - 1) & 3][lane]);
            copies_wait<1>();
            glr_wait<0>(p, ring, GLR_STATE, j - 1);
            const GlrInfo& info = ring.info[(j - 1) & 7];
            const int nt = info.any ? (int)min((int64_t)SUB, max((int64_t)0, p.T - t0)) : SUB;
            const TX* ds = &tl.dh[(j - 1) % 3][w][0][2 * lane];
            const TX* hs = &tl.h[w][0][2 * lane];
            const TX* xs = &tl.x[COMP ? w : 0][0][2 * lane];
            const float2* ts = &tl.t[(j - 1) % 3][w][0][lane];
            RX* dx = reinterpret_cast<RX*>(static_cast<TX*>(p.dx) + (t0 + nt - 1) * p.C + c);
            RG* dg = reinterpret_cast<RG*>(static_cast<TG*>(p.dg) + (t0 + nt - 1) * p.C + c);
            float2 sumA = splat(0.f), sumB = splat(0.f);
            float2 y = *reinterpret_cast<const float2*>(&ring.sub[(j - 1) & 1][pos][lane]);
            auto token = [&](int i, float2 prev) {
                const float2 t = ts[i * 32];
                float2 a, s;
                decay(t, a, s);
                const float2 l = __fadd2_rn(y, PX::widen(*reinterpret_cast<const RX*>(ds + i * GLR_TILE)));
                y = __fmul2_rn(a, l);
                if (COMP) prev = __ffma2_rn(PX::widen(*reinterpret_cast<const RX*>(xs + i * GLR_TILE)), splat(-1.f), prev);
                float2 d = __fmul2_rn(y, prev);
                if (GATE == GLR_SOFTPLUS) {
                    sumA = __ffma2_rn(d, t, sumA);
                    d = __fmul2_rn(d, gate.slope(t));
                    sumB = __fadd2_rn(sumB, d);
                }
                if (live) {
                    *dx = PX::narrow(COMP ? __fmul2_rn(s, l) : l);
                    *dg = PG::narrow(d);
                }
                dx -= ld;
                dg -= ld;
            };
            if (!info.any) {
#pragma unroll 1
                for (int i = SUB - 4; i >= 0; i -= 4) {
#pragma unroll
                    for (int q = 3; q >= 0; --q) token(i + q, PX::widen(*reinterpret_cast<const RX*>(hs + (i + q) * GLR_TILE)));
                }
            } else {
                const uint32_t bits = glr_start_bits(info, i0, nt);
#pragma unroll 1
                for (int i = nt - 1; i >= 0; --i) {
                    const int64_t row = (int64_t)glr_seq_at(info, i0 + i) * p.C + c;
                    const bool first = bits >> i & 1;
                    if (bits >> (i + 1) & 1) y = p.dht && live ? *reinterpret_cast<const float2*>(p.dht + row) : splat(0.f);
                    float2 prev = PX::widen(*reinterpret_cast<const RX*>(hs + i * GLR_TILE));
                    if (first) prev = p.h0 && live ? *reinterpret_cast<const float2*>(p.h0 + row) : splat(0.f);
                    token(i, prev);
                    if (first && live) *reinterpret_cast<float2*>(p.dh0 + row) = y;
                }
            }
            if (GATE == GLR_SOFTPLUS)
                tl.sums[(j - 1) % 3][w][lane] = make_float4(kLn2f * sumA.x, kLn2f * sumA.y, sumB.x, sumB.y);
            glr_signal(ring, GLR_FREE, j - 1);
        }
        if (w == 0) {
            if (takes) glr_set_tick<true>(p, ring, chunks, j + 3, tick.x < 0 ? all : id, tiles, all);
            glr_signal(ring, GLR_TICK, j + 3);
        }
        if (tick.x < 0) break;
        copy_h(tick);
        copy(j + 2);
        before = tick;
    }
    copies_wait<0>();
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
    return p.gate == GLR_SOFTPLUS ? sizeof(float4) * (size_t)(p.C / 2) * glr_chunks(p) : 0;
}

namespace {
struct Launch {
    const GlrParams& p;
    cudaStream_t s;
    template <class TX, class TG, int GATE, bool COMP>
    cudaError_t run() const {
        static std::atomic<uint64_t> ready{0};
        cudaError_t e = glr_launch(k_glr_bwd<TX, TG, GATE, COMP>, ready, 32 * (BWD_WARPS + 4), sizeof(GlrBwdTile<TX, COMP, GATE == GLR_SOFTPLUS>), 2,
                                   p, s);
        if (e != cudaSuccess || GATE != GLR_SOFTPLUS) return e;
        k_glr_sums<<<(p.C / 2 + 31) / 32, 1024, 0, s>>>(p.sums, glr_chunks(p), p.C, p.dA_log,
                                                        p.ddt_bias);
        return cudaGetLastError();
    }
};
}  // namespace

cudaError_t launch_glr_bwd(const GlrParams& p, cudaStream_t s) {
    return glr_dispatch(p.act_f32, p.gate_f32, p.gate, p.complement, Launch{p, s});
}

}  // namespace gdr
