// Gated linear recurrence, forward and single-token step: h_t = a_t h_{t-1} + s_t x_t per
// channel, the state kept in fp32 (the scan's scheme is in gdr_glr.cuh).
#include "gdr_glr.cuh"
#include "gdr_internal.h"

namespace gdr {

size_t glr_published_bytes(const GlrParams& p) { return glr_runs_bytes(glr_chunks(p), p.C); }

// Bytes bound it with a given log gate (x and g are read once, h is written once: 6 bytes a token
// and channel in bf16; 32768 x 2048 with a float32 gate, 8 bytes: 109 us, 74% of the measured copy
// rate).  With the softplus gate no pipe is saturated (30011 x 4096 with the complement, some 50
// instructions a token and channel, all warps' counted: 241 us, 46%; issue slots 66%, FMA 49%, ALU 46%, DRAM
// 39% of its peak): a tile waits for its rows, for issue slots between twelve warps a block, and for the
// states' way from block to block.  The gate is
// evaluated once: the first walk leaves the decays (glr_update) in fp32 where g was, for the second one,
// after the state in front of the chunk is known.  Both walk in rolled loops (unrolled over restarts too, the
// code did not fit the instruction cache, which then bound the kernel); a warp in whose tokens a
// sequence begins or ends folds its run again, token by token, from the decays it has just left
// (32768 tokens in 512 sequences, 2048 channels, softplus: 177 us, a tenth more with the gates evaluated
// token by token in every warp of such a chunk; 132 for one sequence).
// (tokens of an unrolled step: 30011 x 4096 took 234 us with 8, 237 with 4)
constexpr int FWD_WARPS = 8, FWD_SUB = GLR_CHUNK / FWD_WARPS, AT_ONCE = 8;
template <class TX>
struct GlrFwdTile {
    static constexpr int LATE = 2, SLOTS = LATE + 2;
    float2 a[SLOTS][FWD_WARPS][FWD_SUB][32];    // g as copied (glr_raw_offset), then what is kept of the decays
    TX x[SLOTS][FWD_WARPS][FWD_SUB][GLR_TILE];
    GlrRing<FWD_WARPS, LATE> ring;
};

template <class TX, class TG, int GATE, bool COMP>
__global__ void __launch_bounds__(32 * (FWD_WARPS + GLR_X + 1), glr_per_sm(sizeof(GlrFwdTile<TX>))) k_glr_fwd(const GlrParams p, const __grid_constant__ GlrMaps maps) {
    constexpr int SUB = FWD_SUB;
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    using RX = typename PX::raw;
    using RG = typename PG::raw;
    constexpr int RAW = glr_raw_offset<TG>(false);
    extern __shared__ __align__(128) unsigned char smem[];
    using Tile = GlrFwdTile<TX>;
    using Ring = decltype(Tile::ring);
    constexpr int LATE = Tile::LATE, SLOTS = Tile::SLOTS;
    Tile& tl = *reinterpret_cast<Tile*>(smem);
    Ring& ring = tl.ring;
    const int chunks = glr_chunks(p);
    const unsigned tiles = (p.C + GLR_TILE - 1) / GLR_TILE, all = tiles * chunks;
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, i0 = w * SUB, ld = p.C / 2;
    const bool wide = p.wide;
    glr_ring_init(ring, wide);
    if (w == FWD_WARPS + GLR_X) {  // tickets and copies
        unsigned id = lane == 0 ? glr_ticket(p, chunks, 0) : 0;
        int copied = 0, over = 0;
        for (int j = 0; over < GLR_X; ++j) {
            id = __shfl_sync(~0u, id, 0);
            const int k = id < all ? (int)(id / tiles) : -1, c0 = (int)(id - id / tiles * tiles) * GLR_TILE;
            if (lane == 0) ring.tick[j & 7] = make_int4(k, c0, 0, 0);
            glr_signal(ring, GLR_TICK, j);
            if ((k >= 0 || over == 0) && j >= SLOTS && !glr_wait_long<20>(p, ring, GLR_FREE, j - SLOTS)) break;
            if (glr_stalled(p, ring, j)) break;
            if (k >= 0) {
                const int64_t t0 = (int64_t)k * GLR_CHUNK;
                const int rows = (int)min((int64_t)GLR_CHUNK, p.T - t0), cols = min(GLR_TILE, p.C - c0);
                const uint32_t bar = glr_announce(ring, GLR_FULL, j, wide, GLR_CHUNK * GLR_TILE * (sizeof(TX) + sizeof(TG)), lane);
                glr_copy_rows<GLR_TILE * sizeof(TG), 2048>(reinterpret_cast<char*>(&tl.a[j % SLOTS]) + RAW, &maps.g,
                                                           static_cast<const TG*>(p.g), p.ldg, t0, 0, rows, c0, cols, wide, bar, lane);
                glr_copy_rows<GLR_TILE * sizeof(TX), 8 * GLR_TILE * sizeof(TX)>(
                    &tl.x[j % SLOTS], &maps.x, static_cast<const TX*>(p.x), p.ldx, t0, 0, rows, c0, cols, wide, bar, lane);
                glr_report(bar, wide);
                copied = j + 1;
            } else {
                if (over++ == 0) glr_report(glr_announce(ring, GLR_FULL, j, wide, 0, lane), wide);
            }
            // (taken as late as that, so that tiles with near tickets are worked on at the same time)
            id = lane == 0 && id < all ? glr_ticket(p, chunks, j + 1) : id;
        }
        glr_landed(p, ring, copied - SLOTS + (over > 0), copied);  // (the end's mark has the next tile's barrier)
        return;
    }
    if (w >= FWD_WARPS) {
        const GlrRuns runs = glr_runs(p.status, chunks, p.C);
        int4 tick = glr_look<false>(p, ring, chunks, w - FWD_WARPS, lane);
        for (int j = w - FWD_WARPS; tick.x >= 0; j += GLR_X) {
            if (!glr_exchange<false>(p, ring, runs, chunks, j, tick, lane)) break;
            tick = glr_look<false>(p, ring, chunks, j + GLR_X, lane);
        }
        glr_leave(ring);
        return;
    }
    int4 before[LATE];  // tiles j - LATE .. j - 1
#pragma unroll
    for (int i = 0; i < LATE; ++i) before[i] = make_int4(-1, 0, 0, 0);
    int4 tick = make_int4(0, 0, 0, 0);
    for (int j = 0;; ++j) {
        const bool more = tick.x >= 0;  // (past the last tile only second walks are left)
        if (more) {
            glr_wait(p, ring, GLR_FULL, j);
            tick = ring.tick[j & 7];
        }
        if (tick.x >= 0) {
            const GlrInfo& info = ring.info[j & 7];
            const int c = tick.y + 2 * lane;
            const bool live = c < p.C;
            GlrGate<GATE> gate;
            gate.set(ring.gate[j & 3][lane]);
            const TX* xs = &tl.x[j % SLOTS][w][0][2 * lane];
            float2* as = &tl.a[j % SLOTS][w][0][lane];
            const TG* gs = reinterpret_cast<const TG*>(reinterpret_cast<char*>(&tl.a[j % SLOTS][w]) + RAW) + 2 * lane;
            constexpr int GP = GLR_TILE;
            Run r = run_identity();
            float2 sum = splat(0.f);
            const int nt = info.any ? (int)min((int64_t)SUB, max((int64_t)0, p.T - ((int64_t)tick.x * GLR_CHUNK + i0))) : SUB;
            const uint32_t bits = info.any ? glr_start_bits(info, i0, nt) : 0;
#pragma unroll 1
            for (int i = 0; i < SUB; i += AT_ONCE) {
                RG graw[AT_ONCE];
                float2 xv[AT_ONCE];
#pragma unroll
                for (int q = 0; q < AT_ONCE; ++q) {
                    graw[q] = *reinterpret_cast<const RG*>(gs + (i + q) * GP);
                    xv[q] = PX::widen(*reinterpret_cast<const RX*>(xs + (i + q) * GLR_TILE));
                }
                __syncwarp();  // every lane has its g of these rows
#pragma unroll
                for (int q = 0; q < AT_ONCE; ++q) {
                    const float2 t = gate.log2_gate(PG::widen(graw[q]));
                    as[(i + q) * 32] = glr_update_by_gate<GATE, COMP>(t, r.H, xv[q]);
                    sum = __fadd2_rn(sum, t);
                }
            }
            r.A = run_decay<GATE>(sum);
            if (bits != 0 || nt < SUB) {  // again with the restarts
                r = run_identity();
#pragma unroll 1
                for (int i = 0; i < nt; ++i) {
                    const float2 v = as[i * 32];
                    if (bits >> i & 1) {
                        r.A = splat(-0.f);
                        r.H = p.h0 && live ? *reinterpret_cast<const float2*>(p.h0 + (int64_t)glr_seq_at(info, i0 + i) * p.C + c)
                                           : splat(0.f);
                    } else {
                        r.A = __fmul2_rn(r.A, decay_of_kept<COMP>(v));
                    }
                    r.H = glr_update<COMP>(v, r.H, PX::widen(*reinterpret_cast<const RX*>(xs + i * GLR_TILE)));
                }
            }
            ring.sub[j % (LATE + 1)][w][lane] = run_bits(r);
            glr_arrive(ring, GLR_RUNS, j);
        }
        if (before[0].x >= 0) {
            glr_wait(p, ring, GLR_STATE, j - LATE);
            const GlrInfo& info = ring.info[(j - LATE) & 7];
            const int c = before[0].y + 2 * lane;
            const bool live = c < p.C;
            const int64_t t = (int64_t)before[0].x * GLR_CHUNK + i0;
            RX* h = reinterpret_cast<RX*>(static_cast<TX*>(p.h) + t * p.C + c);
            const TX* xs = &tl.x[(j - LATE) % SLOTS][w][0][2 * lane];
            const float2* as = &tl.a[(j - LATE) % SLOTS][w][0][lane];
            float2 y = *reinterpret_cast<const float2*>(&ring.sub[(j - LATE) % (LATE + 1)][w][lane]);
            const int nt = info.any ? (int)min((int64_t)SUB, max((int64_t)0, p.T - t)) : SUB;
            const uint32_t bits = info.any ? glr_start_bits(info, i0, nt) : 0;
            if (bits == 0 && nt == SUB) {
#pragma unroll 1
                for (int i = 0; i < SUB; i += 4) {
#pragma unroll
                    for (int q = 0; q < 4; ++q, h += ld) {
                        y = glr_update<COMP>(as[(i + q) * 32], y, PX::widen(*reinterpret_cast<const RX*>(xs + (i + q) * GLR_TILE)));
                        if (live) *h = PX::narrow(y);
                    }
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < nt; ++i, h += ld) {
                    if (bits >> i & 1)
                        y = p.h0 && live ? *reinterpret_cast<const float2*>(p.h0 + (int64_t)glr_seq_at(info, i0 + i) * p.C + c)
                                         : splat(0.f);
                    y = glr_update<COMP>(as[i * 32], y, PX::widen(*reinterpret_cast<const RX*>(xs + i * GLR_TILE)));
                    if (live) {
                        *h = PX::narrow(y);
                        if (p.ht && (bits >> (i + 1) & 1))
                            *reinterpret_cast<float2*>(p.ht + (int64_t)glr_seq_at(info, i0 + i) * p.C + c) = y;
                    }
                }
            }
            tc::fence_async_smem();  // (the next copy into these rows comes after the reads and writes above)
            glr_signal(ring, GLR_FREE, j - LATE);
        }
#pragma unroll
        for (int i = 0; i + 1 < LATE; ++i) before[i] = before[i + 1];
        before[LATE - 1] = tick;
        bool left = tick.x >= 0;
#pragma unroll
        for (int i = 0; i < LATE; ++i) left |= before[i].x >= 0;
        if (!left) break;
    }
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
                        encode_plain_map(&maps.x, p.x, p.act_f32, p.T, p.C, p.ldx, 64)))
            return cudaErrorInvalidValue;
        static_assert(sizeof(TX) == 4 || glr_per_sm(sizeof(GlrFwdTile<TX>)) == 2, "bf16 tiles: two blocks an SM");
        return glr_launch<GlrFwdTile<TX>>(k_glr_fwd<TX, TG, GATE, COMP>, ready, p, maps, s);
    }
};
}  // namespace

cudaError_t launch_glr_fwd(const GlrParams& p, cudaStream_t s) {
    return glr_dispatch(p.act_f32, p.gate_f32, p.gate, p.complement, Launch{p, s});
}

// One token for each row: y = h = a h + s x on the row's state, in place.  A row whose slot is
// negative (padding of the batch) or past the pool reads and writes no state; its y is zero.
//
// Bytes bound it, and at the sizes of a decoding batch the two memory latencies of a slot and its
// state: a thread takes V channels, four (8 bytes of bf16, 16 of the state) where rows are whole
// numbers of aligned pieces, else two, and asks for everything else while the slot is on its way.
// 509 x 4096 with slots and the softplus gate, from cold caches: 7.4 us (a sixth more with two channels and the slot first).
template <class R, int P>
struct __align__(sizeof(R) * P) Pairs {
    R v[P];
};
template <class TX, class TG, int GATE, bool COMP, int V>
__global__ void __launch_bounds__(128) k_glr_step(const GlrStepParams p) {
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    constexpr int P = V / 2;
    using XS = Pairs<typename PX::raw, P>;
    using GS = Pairs<typename PG::raw, P>;
    using States = Pairs<float2, P>;
    const int c = (blockIdx.x * 128 + threadIdx.x) * V;
    if (c >= p.C) return;
    for (int64_t n = blockIdx.y; n < p.N; n += gridDim.y) {
        const int64_t slot = p.slots ? p.slots[n] : n;
        const XS x = *reinterpret_cast<const XS*>(static_cast<const TX*>(p.x) + n * p.ldx + c);
        const GS g = *reinterpret_cast<const GS*>(static_cast<const TG*>(p.g) + n * p.ldg + c);
        float2 t[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            GlrGate<GATE> gate;
            gate.load(p.A_log, p.dt_bias, c + 2 * i);
            t[i] = gate.log2_gate(PG::widen(g.v[i]));
        }
        XS y;
        if (slot >= 0 && slot < p.pool) {
            States* home = reinterpret_cast<States*>(p.state + slot * p.C + c);
            States st = *home;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float2 a, s, xv = PX::widen(x.v[i]);
                decay(t[i], a, s);
                st.v[i] = __ffma2_rn(a, st.v[i], COMP ? __fmul2_rn(s, xv) : xv);
                y.v[i] = PX::narrow(st.v[i]);
            }
            *home = st;
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) y.v[i] = PX::zero();
        }
        *reinterpret_cast<XS*>(static_cast<TX*>(p.y) + n * p.C + c) = y;
    }
}

namespace {
struct StepLaunch {
    const GlrStepParams& p;
    cudaStream_t s;
    template <class TX, class TG, int GATE, bool COMP>
    cudaError_t run() const {
        const unsigned rows = p.N < 65535 ? p.N : 65535;
        const bool wide = p.C % 4 == 0 && p.ldx % 4 == 0 && p.ldg % 4 == 0 &&
                          ((reinterpret_cast<uintptr_t>(p.x) % (4 * sizeof(TX))) | (reinterpret_cast<uintptr_t>(p.g) % (4 * sizeof(TG)))) == 0;
        if (wide) k_glr_step<TX, TG, GATE, COMP, 4><<<dim3((p.C / 4 + 127) / 128, rows), 128, 0, s>>>(p);
        else k_glr_step<TX, TG, GATE, COMP, 2><<<dim3((p.C / 2 + 127) / 128, rows), 128, 0, s>>>(p);
        return cudaGetLastError();
    }
};
}  // namespace

cudaError_t launch_glr_step(const GlrStepParams& p, cudaStream_t s) {
    return glr_dispatch(p.act_f32, p.gate_f32, p.gate, p.complement, StepLaunch{p, s});
}

}  // namespace gdr
