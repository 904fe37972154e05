// Gated linear recurrence, forward and single-token step: h_t = a_t h_{t-1} + s_t x_t per
// channel, the state kept in fp32 (the scan's scheme is in gdr_glr.cuh).
#include "gdr_glr.cuh"
#include "gdr_internal.h"

namespace gdr {

size_t glr_published_bytes(const GlrParams& p) { return glr_runs_bytes(glr_chunks(p.T, p.act_f32, p.gate_f32), p.C); }

// Bytes bound it: x and g are read once and h is written once (6 bytes a token and channel in
// bf16).  A thread keeps its tokens' decays in fp32 in registers from the one evaluation of the
// gate to the second walk, after the state in front of the chunk is known.  A warp among whose
// tokens a sequence begins or ends walks them in a rolled loop: unrolled, those branches made
// three quarters of the code and the instruction cache bound the kernel.
template <class TX, class TG>
struct GlrFwdTile {
    static constexpr int SUB = glr_sub(sizeof(TX) == 4, sizeof(TG) == 4);
    TX x[2][GLR_WARPS][SUB][GLR_TILE];
    TG g[2][GLR_WARPS][SUB][GLR_TILE];
    GlrShared sm;
};

template <class TX, class TG, int GATE, bool COMP>
__global__ void __launch_bounds__(GLR_THREADS, 3) k_glr_fwd(const GlrParams p) {
    constexpr int SUB = GlrFwdTile<TX, TG>::SUB, CHUNK = SUB * GLR_WARPS;
    using PX = PairOf<TX>;
    using PG = PairOf<TG>;
    using RX = typename PX::raw;
    using RG = typename PG::raw;
    extern __shared__ __align__(16) unsigned char smem[];
    GlrFwdTile<TX, TG>& tl = *reinterpret_cast<GlrFwdTile<TX, TG>*>(smem);
    GlrShared& sm = tl.sm;
    const int chunks = glr_chunks(p.T, sizeof(TX) == 4, sizeof(TG) == 4);
    const unsigned tiles = (p.C + GLR_TILE - 1) / GLR_TILE, all = tiles * chunks;
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, i0 = w * SUB, ld = p.C / 2;
    const GlrRuns runs = glr_runs(p.status, chunks, p.C);

    auto copy = [&](unsigned id, int b) {  // this warp's tokens of a tile
        if (id < all) {
            const int k = id / tiles, c0 = (id - k * tiles) * GLR_TILE;
            const int64_t t = (int64_t)k * CHUNK + i0;
            const int nt = (int)min((int64_t)SUB, max((int64_t)0, p.T - t));
            const TX* x = static_cast<const TX*>(p.x);
            const TG* g = static_cast<const TG*>(p.g);
            glr_copy_rows<SUB>(&tl.g[b][w][0][0], g + t * p.ldg + c0, p.ldg, 0, nt, p.C - c0, p.wide, lane, g);
            glr_copy_rows<SUB>(&tl.x[b][w][0][0], x + t * p.ldx + c0, p.ldx, 0, nt, p.C - c0, p.wide, lane, x);
        }
        copies_commit();
    };
    auto look = [&](unsigned id, int b) {  // the sequences of a tile's tokens; one warp
        if (id >= all) return;
        const int k = id / tiles, c = (id - k * tiles) * GLR_TILE + 2 * lane;
        glr_find_sequences(p, sm.info[b], (int64_t)k * CHUNK, (int)min((int64_t)CHUNK, p.T - (int64_t)k * CHUNK), lane);
        glr_empty_sequences(p, p.h0, p.ht, k, chunks, c, c < p.C, id == k * tiles);
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
        copy(next, b ^ 1);
        const int k = id / tiles, tile = id - k * tiles, c = tile * GLR_TILE + 2 * lane;
        const bool live = c < p.C;
        const int64_t t = (int64_t)k * CHUNK + i0;  // this warp's first token
        const int nt = (int)min((int64_t)SUB, max((int64_t)0, p.T - t));
        const GlrInfo& info = sm.info[b];
        const uint32_t bits = glr_start_bits(info, i0, nt);  // of this warp's tokens and the one after
        const bool whole = bits == 0 && nt == SUB;
        const GlrPlace at(k, (int)((uint64_t)info.begin0 / CHUNK), info.starts[0] & 1);
        GlrGate<GATE> gate;
        gate.load(p.A_log, p.dt_bias, live ? c : 0);
        RX* h = reinterpret_cast<RX*>(static_cast<TX*>(p.h) + t * p.C + c);
        auto xv = [&](int i) { return PX::widen(*reinterpret_cast<const RX*>(&tl.x[b][w][i][2 * lane])); };
        auto tv = [&](int i) { return gate.log2_gate(PG::widen(*reinterpret_cast<const RG*>(&tl.g[b][w][i][2 * lane]))); };
        // the rolled walk from the state r.H, with outputs or (for the run) without
        auto walk = [&](Run r, bool out) {
#pragma unroll 1
            for (int i = 0; i < nt; ++i) {
                const float2 d = decay(tv(i));
                if (bits >> i & 1) {
                    r.A = splat(-0.f);
                    r.H = p.h0 && live ? *reinterpret_cast<const float2*>(p.h0 + (int64_t)glr_seq_at(info, i0 + i) * p.C + c)
                                       : splat(0.f);
                } else {
                    r.A = __fmul2_rn(r.A, d);
                }
                r.H = glr_update<COMP>(d, r.H, xv(i));
                if (out && live) {
                    h[(int64_t)i * ld] = PX::narrow(r.H);
                    if (p.ht && (bits >> (i + 1) & 1))
                        *reinterpret_cast<float2*>(p.ht + (int64_t)glr_seq_at(info, i0 + i) * p.C + c) = r.H;
                }
            }
            return r;
        };
        copies_wait<1>();
        Run r = run_identity();
        float2 a[SUB];
        if (whole) {
#pragma unroll
            for (int i = 0; i < SUB; ++i) {
                a[i] = decay(tv(i));
                r.A = __fmul2_rn(r.A, a[i]);
                r.H = glr_update<COMP>(a[i], r.H, xv(i));
            }
        } else {
            r = walk(r, false);
        }
        sm.sub[w][lane] = run_bits(r);
        __syncthreads();
        const bool restarts = info.starts[0] | info.starts[1] | info.starts[2] | info.starts[3];
        Run before = glr_before_warp(sm, w, lane, restarts), own;
        if (chunks > 1) own = glr_exchange(p, sm, at, runs, w, lane, c / 2, live);
        if (w == GLR_WARPS - 1) {
            if (lane == 0) sm.ticket = glr_next(p, chunks, next);
            look(next, b ^ 1);
        }
        __syncthreads();
        float2 y = glr_after(before, glr_state_before(sm, at, lane));
        if (w == 0 && chunks > 1) glr_publish_groups(p, sm, at, runs, own, lane, c / 2, live);
        if (whole) {
#pragma unroll
            for (int i = 0; i < SUB; ++i, h += ld) {
                y = glr_update<COMP>(a[i], y, xv(i));
                if (live) *h = PX::narrow(y);
            }
        } else {
            walk(Run{splat(1.f), y}, true);
        }
        __syncwarp();  // the warp's rows are free for the copies of the tile after next
        id = next;
    }
    copies_wait<0>();
}

namespace {
struct Launch {
    const GlrParams& p;
    cudaStream_t s;
    template <class TX, class TG, int GATE, bool COMP>
    cudaError_t run() const {
        static std::atomic<uint64_t> ready{0};
        return glr_launch(k_glr_fwd<TX, TG, GATE, COMP>, ready, sizeof(GlrFwdTile<TX, TG>), 3, p, s);
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
