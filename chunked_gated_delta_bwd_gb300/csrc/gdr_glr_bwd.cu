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

// Bytes bound it with a given log gate (g, h, dh, and x with the complement, are read once, dx and
// dg written once: 10 or 12 bytes a token and channel in bf16, 20 in float32: 8192 x 2048 71 us, 71%
// of the measured copy rate, one block an SM by the tiles' shared memory).  With the softplus gate no pipe is
// saturated (32768 x 2048 with the complement: 229 us, 53%; FMA 59%, issue slots 62%, DRAM 45% of its peak):
// see the forward.
// The first walk leaves the base-2 log gates in fp32 where g was; the second derives the decays, and
// the softplus gate's slope, from them.  g and dh are copied ahead, h and x, which only the second
// walk needs, when their one buffer is free.
// Warps without a sequence's beginning or end among their tokens walk in the short loops also where
// the chunk has one (512 sequences of 32768 tokens, 2048 channels, softplus: 285 us, 5% more when all of
// the chunk's warps walked token by token).
// tokens of an unrolled step: the instruction cache holds more of the walks the shorter it is (against 2,
// 4: 3% slower for 32768 x 2048 with the softplus gate, 1: 5%)
constexpr int BWD_WARPS = 8, BWD_SUB = GLR_CHUNK / BWD_WARPS, AT_ONCE = 2;
template <class TX, bool COMP, bool SUMS>
struct GlrBwdTile {
    float2 t[3][BWD_WARPS][BWD_SUB][32];    // g as copied (glr_raw_offset), then the log gates
    TX dh[3][BWD_WARPS][BWD_SUB][GLR_TILE];
    TX h[BWD_WARPS][BWD_SUB][GLR_TILE];     // of the token before
    TX x[COMP ? BWD_WARPS : 1][COMP ? BWD_SUB : 1][GLR_TILE];
    float4 sums[SUMS ? 3 : 1][BWD_WARPS][32];  // of each warp's tokens, for the softplus gate's parameters
    GlrRing<BWD_WARPS, 1> ring;
};

template <class TX, class TG, int GATE, bool COMP>
__global__ void __launch_bounds__(32 * (BWD_WARPS + GLR_X + 1), glr_per_sm(sizeof(GlrBwdTile<TX, COMP, GATE == GLR_SOFTPLUS>)))
    k_glr_bwd(const GlrParams p, const __grid_constant__ GlrMaps maps) {
    using Tile = GlrBwdTile<TX, COMP, GATE == GLR_SOFTPLUS>;
    constexpr int SUB = BWD_SUB;
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    using RX = typename PX::raw;
    using RG = typename PG::raw;
    constexpr int RAW = glr_raw_offset<TG>(true);
    extern __shared__ __align__(128) unsigned char smem[];
    Tile& tl = *reinterpret_cast<Tile*>(smem);
    using Ring = decltype(Tile::ring);
    Ring& ring = tl.ring;
    const int chunks = glr_chunks(p);
    const unsigned tiles = (p.C + GLR_TILE - 1) / GLR_TILE, all = tiles * chunks;
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, i0 = w * SUB, ld = p.C / 2;
    const bool wide = p.wide;
    glr_ring_init(ring, wide);
    if (w == BWD_WARPS + GLR_X) {  // tickets and copies: g and dh of tile j, then h and x of tile j - 2
        constexpr int XP = GLR_TILE * sizeof(TX);
        unsigned id = lane == 0 ? glr_ticket(p, chunks, 0) : 0;
        int k1 = -1, c1 = 0, k2 = -1, c2 = 0;  // tiles j - 1, j - 2
        int copied = 0, late = 0;
        for (int j = 0, over = 0; over < GLR_X; ++j) {
            id = __shfl_sync(~0u, id, 0);
            const int k = id < all ? (int)(id / tiles) : -1, c0 = (int)(id - id / tiles * tiles) * GLR_TILE;
            if (lane == 0) ring.tick[j & 7] = make_int4(k, c0, 0, 0);
            glr_signal(ring, GLR_TICK, j);
            if (j >= 3 && (k >= 0 || k2 >= 0) && !glr_wait_long<20>(p, ring, GLR_FREE, j - 3)) break;
            if (glr_stalled(p, ring, j)) break;
            if (k >= 0) {
                const int64_t t0 = (int64_t)(chunks - 1 - k) * GLR_CHUNK;
                const int rows = (int)min((int64_t)GLR_CHUNK, p.T - t0), cols = min(GLR_TILE, p.C - c0);
                const uint32_t bar = glr_announce(ring, GLR_FULL, j, wide, GLR_CHUNK * GLR_TILE * (sizeof(TX) + sizeof(TG)), lane);
                glr_copy_rows<GLR_TILE * sizeof(TG), 2048>(reinterpret_cast<char*>(&tl.t[j % 3]) + RAW, &maps.g,
                                                           static_cast<const TG*>(p.g), p.ldg, t0, 0, rows, c0, cols, wide, bar, lane);
                glr_copy_rows<XP, 8 * XP>(&tl.dh[j % 3], &maps.dh, static_cast<const TX*>(p.dh), p.C, t0, 0, rows, c0, cols, wide, bar, lane);
                glr_report(bar, wide);
                copied = j + 1;
                if (wide && lane == 0) {  // h and x have one buffer: on their way to L2 until it is free
                    tc::tma_prefetch_2d(&maps.h, c0, (int)t0 - 1);
                    if (COMP) tc::tma_prefetch_2d(&maps.x, c0, (int)t0);
                }
            } else {
                if (over++ == 0) glr_report(glr_announce(ring, GLR_FULL, j, wide, 0, lane), wide);
            }
            if (k2 >= 0) {
                const int64_t t0 = (int64_t)(chunks - 1 - k2) * GLR_CHUNK;
                const int rows = (int)min((int64_t)GLR_CHUNK, p.T - t0), cols = min(GLR_TILE, p.C - c2);
                const uint32_t bar = glr_announce(ring, GLR_LATE, j - 2, wide, GLR_CHUNK * XP * (COMP ? 2 : 1), lane);
                glr_copy_rows<XP, 8 * XP>(&tl.h, &maps.h, static_cast<const TX*>(p.h_in), p.C, t0 - 1, t0 == 0, rows, c2, cols, wide, bar, lane);
                if (COMP)
                    glr_copy_rows<XP, 8 * XP>(&tl.x, &maps.x, static_cast<const TX*>(p.x), p.ldx, t0, 0, rows, c2, cols, wide, bar, lane);
                glr_report(bar, wide);
                late = j - 1;
            }
            k2 = k1; c2 = c1; k1 = k; c1 = c0;
            // (taken as late as that, so that tiles with near tickets are worked on at the same time)
            id = lane == 0 && id < all ? glr_ticket(p, chunks, j + 1) : id;
        }
        glr_landed(p, ring, copied - 3, copied);
        for (int j = max(late - 2, 0); j < late; ++j) tc::mbar_wait(glr_bar(ring, GLR_LATE, j), glr_phase(GLR_LATE, j), GLR_SPIN_COMPUTE);
        return;
    }
    if (w >= BWD_WARPS) {
        const GlrRuns runs = glr_runs(p.status, chunks, p.C);
        // tile j's sums are added before tile j + 3 is looked at, and written again only after that
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
        for (int j = w - BWD_WARPS; tick.x >= 0; j += GLR_X) {
            if (!glr_exchange<true>(p, ring, runs, chunks, j, tick, lane) || !glr_wait_long<50>(p, ring, GLR_FREE, j)) break;
            add_sums(tick, j);
            tick = glr_look<true>(p, ring, chunks, j + GLR_X, lane);
        }
        glr_leave(ring);
        return;
    }
    const int pos = BWD_WARPS - 1 - w;  // this warp's place in the order of the scan

    int4 before = make_int4(-1, 0, 0, 0);  // tile j - 1
    for (int j = 0;; ++j) {
        glr_wait(p, ring, GLR_FULL, j);
        const int4 tick = ring.tick[j & 7];
        if (tick.x >= 0) {
            const GlrInfo& info = ring.info[j & 7];
            const int c = tick.y + 2 * lane;
            const bool live = c < p.C;
            GlrGate<GATE> gate;
            gate.set(ring.gate[j & 3][lane]);
            const TX* ds = &tl.dh[j % 3][w][0][2 * lane];
            float2* ts = &tl.t[j % 3][w][0][lane];
            const TG* gs = reinterpret_cast<const TG*>(reinterpret_cast<char*>(&tl.t[j % 3][w]) + RAW) + 2 * lane;
            constexpr int GP = GLR_TILE;
            Run r = run_identity();
            const int nt =
                info.any ? (int)min((int64_t)SUB, max((int64_t)0, p.T - ((int64_t)(chunks - 1 - tick.x) * GLR_CHUNK + i0))) : SUB;
            const uint32_t bits = info.any ? glr_start_bits(info, i0, nt) : 0;
            if (bits == 0 && nt == SUB) {
                float2 sum = splat(0.f);
#pragma unroll 1
                for (int i = SUB - AT_ONCE; i >= 0; i -= AT_ONCE) {
                    RG graw[AT_ONCE];
                    float2 dv[AT_ONCE];
#pragma unroll
                    for (int q = AT_ONCE - 1; q >= 0; --q) {
                        graw[q] = *reinterpret_cast<const RG*>(gs + (i + q) * GP);
                        dv[q] = PX::widen(*reinterpret_cast<const RX*>(ds + (i + q) * GLR_TILE));
                    }
                    __syncwarp();  // every lane has its g of these rows
#pragma unroll
                    for (int q = AT_ONCE - 1; q >= 0; --q) {
                        const float2 t = gate.log2_gate(PG::widen(graw[q]));
                        const float2 a = decay(t);
                        ts[(i + q) * 32] = t;
                        sum = __fadd2_rn(sum, t);
                        r.H = __fmul2_rn(a, __fadd2_rn(r.H, dv[q]));
                    }
                }
                r.A = run_decay<GATE>(sum);
            } else {
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
            glr_arrive(ring, GLR_RUNS, j);
        }
        if (before.x >= 0) {
            const int kc = chunks - 1 - before.x, c = before.y + 2 * lane;
            const bool live = c < p.C;
            const int64_t t0 = (int64_t)kc * GLR_CHUNK + i0;
            GlrGate<GATE> gate;
            gate.set(ring.gate[(j - 1) & 3][lane]);
            glr_wait(p, ring, GLR_LATE, j - 1);
            glr_wait(p, ring, GLR_STATE, j - 1);
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
            const uint32_t bits = info.any ? glr_start_bits(info, i0, nt) : 0;
            if (bits == 0 && nt == SUB) {
#pragma unroll 1
                for (int i = SUB - AT_ONCE; i >= 0; i -= AT_ONCE) {
#pragma unroll
                    for (int q = AT_ONCE - 1; q >= 0; --q) token(i + q, PX::widen(*reinterpret_cast<const RX*>(hs + (i + q) * GLR_TILE)));
                }
            } else {
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
            tc::fence_async_smem();  // (the next copy into these rows comes after the reads and writes above)
            glr_signal(ring, GLR_FREE, j - 1);
        }
        if (tick.x < 0) break;
        before = tick;
    }
}

// dA_log and ddt_bias: the chunks' sums, added in a fixed order.  A block takes 32 pairs of
// channels, each of its 32 warps every 32nd chunk.
__global__ void __launch_bounds__(1024) k_glr_sums(const float4* sums, int chunks, int C, float* dA_log, float* ddt_bias) {
    __shared__ float4 part[32][33];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, c2 = blockIdx.x * 32 + lane;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    cudaGridDependencySynchronize();  // (launched ahead of the end of the kernel before it)
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
        GlrMaps maps;
        if (p.wide && !(encode_plain_map(&maps.g, p.g, p.gate_f32, p.T, p.C, p.ldg, p.gate_f32 ? 64 : 8) &&
                        encode_plain_map(&maps.dh, p.dh, p.act_f32, p.T, p.C, p.C, 64) &&
                        encode_plain_map(&maps.h, p.h_in, p.act_f32, p.T, p.C, p.C, 64) &&
                        (!COMP || encode_plain_map(&maps.x, p.x, p.act_f32, p.T, p.C, p.ldx, 64))))
            return cudaErrorInvalidValue;
        using Tile = GlrBwdTile<TX, COMP, GATE == GLR_SOFTPLUS>;
        static_assert(sizeof(TX) == 4 || glr_per_sm(sizeof(Tile)) == 2, "bf16 tiles: two blocks an SM");
        cudaError_t e = glr_launch<Tile>(k_glr_bwd<TX, TG, GATE, COMP>, ready, p, maps, s);
        if (e != cudaSuccess || GATE != GLR_SOFTPLUS) return e;
        return launch_after((p.C / 2 + 31) / 32, 1024, s, k_glr_sums, (const float4*)p.sums, glr_chunks(p), (int)p.C, p.dA_log,
                            p.ddt_bias);
    }
};
}  // namespace

cudaError_t launch_glr_bwd(const GlrParams& p, cudaStream_t s) {
    return glr_dispatch(p.act_f32, p.gate_f32, p.gate, p.complement, Launch{p, s});
}

}  // namespace gdr
