// Linear attention with a decay for each head, forward and backward, in chunks of 128 tokens.
//
//   S_t = gamma S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   gamma = e^g
//
// One operator gives every output.  With operands (X, Y, Z), per chunk of L tokens and incoming state C:
//
//   out = (X Y^T o D) Z + diag(r) X C,    C' = gamma^L C + sum_t w_t y_t z_t^T
//
// forward in time  D_ij = gamma^{i-j} (i >= j), r_i = gamma^{i+1}, w_t = gamma^{L-1-t}:
//   o: (q, k, v);  dq: (dO, v, k), on the transposed state
// back in time     D_ij = gamma^{j-i} (j >= i), r_i = gamma^{L-1-i}, w_t = gamma^{t+1}:
//   dv: (k, q, dO), with dh0 as its last state;  dk: (v, dO, q), on the transposed state
//
// so that the backward is three such walks in one launch, which meet in the second-level cache: dv's and
// dk's walk the same chunks at the same time.
//
// Bytes bound it: a chunk and head of 128 moves 128 KB (2.9 us of a multiprocessor's share of the
// measured copy rate) for five products of 128^3 (1.3 us of tensor cores).  So one block a multiprocessor
// walks a range of chunks (gdr_dla_plan.cuh) with the loads of the next chunk in flight, the state in fp32
// registers, and four roles that overlap:
//   loader   Y, Z, X tiles of the chunks to come, by TMA, through a ring of tiles
//   issuer   the products: P = X Y^T, X C, P Z (P from tensor memory), Y'^T Z
//   group A  P times the decays, rounded to bf16 (tensor memory); out, staged in X's tile for a TMA store
//   group B  Y' = w Y as two bf16 tiles (the first in Y's place): their products with Z make the state's
//            terms good to 2^-16, so that the states that leave (ht, dh0) are fp32 results; the state's
//            sum, and its bf16 copy for X C
// P and the state's copy are rounded to bf16: each adds 2^-9 at most to a term of an output that is
// rounded to bf16 itself.
//
// A chain that crosses from one range into the next: k_dla_tail first sums, for each range, the terms of
// its last chain's tokens (it reads only Y and Z, from the range's end backwards, and stops where the decay
// has underflowed), k_dla_join carries them along the chain, and the walk starts from there.
#include "gdr_dla.h"
#include "gdr_dla_plan.cuh"
#include "gdr_internal.h"
#include "gdr_tc.cuh"
#include "gdr_tma.h"

namespace gdr {
namespace {

using namespace dla;

template <int D>
struct Cfg {
    static constexpr int TILE = CHUNK * D * 2, RING = D == 128 ? 5 : 8;
    static constexpr int oLo = RING * TILE, oS = oLo + TILE, oTab = oS + D * D * 2;
    // (the product Y'^T Z has 128 rows; with 64 channels the upper ones read what lies behind the tile)
    static constexpr int oEnd = (oTab + 1024 > oLo + 2 * CHUNK * 128 ? oTab + 1024 : oLo + 2 * CHUNK * 128);
    static constexpr int oBar = oEnd, BARS = 2 * RING + 10;
    static constexpr int SMEM = oBar + 8 * BARS + 128 + 1024;
};
template <int D>
struct TailCfg {
    static constexpr int TILE = CHUNK * D * 2, RING = D == 128 ? 5 : 8;
    static constexpr int oLo = RING * TILE, oEnd = oLo + 2 * TILE + (D == 128 ? 0 : CHUNK * 128);
    static constexpr int oBar = oEnd, BARS = 2 * RING + 5;
    static constexpr int SMEM = oBar + 8 * BARS + 128 + 1024;
};

struct Walk {
    CUtensorMap X, Y, Z, out;
    int gx, gy, gz;                 // value heads that share a head of the tensor
    int back, turned;               // walked back in time; on transposed states
    float p_scale, o_scale, w_scale;  // of P, of X C, of the state's terms
    const float* init;              // [N][H][D][D] or nullptr
    const float* joined;            // incoming states of ranges that begin inside a chain
    float* last;                    // final states or nullptr
    __nv_bfloat16* o;
    float* o32;                     // fp32 outputs for each value head instead
};
template <int WALKS>
struct Walks {
    Walk w[WALKS];
};

struct Grid {
    int N, H, D, ranges, snap;
    int64_t T, seq_len;
    const int64_t* cu;
    const float* g;
    int* status;
};
__device__ __forceinline__ Line line_of(const Grid& p, int back) { return Line{p.N, p.H, p.T, p.seq_len, p.cu, back}; }

// Waits are bounded: one that runs out records it, and turns every later wait and issue of the block into nothing.
struct Waiter {
    volatile int* gone;
    int* status;
    __device__ __forceinline__ bool ok() const { return *gone == 0; }
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) const {
        if (ok() && !tc::mbar_wait(bar, parity, 1 << 22)) {
            *gone = 1;
            atomicOr(status, ST_MMA_TIMEOUT);
        }
    }
};

// Row `row` of a tile times w, as two bf16 rows: the first over the row, the rest into `lo`.  w = 0 takes
// whatever the row holds as zero.
template <int D>
__device__ __forceinline__ void split_row(unsigned char* tile, unsigned char* lo, int row, float w) {
#pragma unroll 4
    for (int j = 0; j < D / 8; ++j) {
        const uint32_t at = tc::sw_chunk(row, j, CHUNK);
        uint4 hi4 = make_uint4(0, 0, 0, 0), lo4 = hi4;
        if (w != 0.f) {
            const uint4 u = *reinterpret_cast<const uint4*>(tile + at);
            const uint32_t in[4] = {u.x, u.y, u.z, u.w};
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __fmul2_rn(make_float2(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xffff0000u)), make_float2(w, w));
                h[i] = pack_bf16(f.x, f.y);
                l[i] = pack_bf16(f.x - __uint_as_float(h[i] << 16), f.y - __uint_as_float(h[i] & 0xffff0000u));
            }
            hi4 = make_uint4(h[0], h[1], h[2], h[3]);
            lo4 = make_uint4(l[0], l[1], l[2], l[3]);
        }
        *reinterpret_cast<uint4*>(tile + at) = hi4;
        *reinterpret_cast<uint4*>(lo + at) = lo4;
    }
}
// row `row` of a tile made zero (a row of another sequence, whose values must not reach a product)
template <int D>
__device__ __forceinline__ void clear_row(unsigned char* tile, int row) {
#pragma unroll
    for (int j = 0; j < D / 8; ++j) *reinterpret_cast<uint4*>(tile + tc::sw_chunk(row, j, CHUNK)) = make_uint4(0, 0, 0, 0);
}

// the state's terms of a chunk: Y'^T Z from both halves of Y'
template <int D>
__device__ __forceinline__ void issue_terms(uint32_t to, uint32_t hi, uint32_t lo, uint32_t z) {
    constexpr uint32_t id = tc::idesc(128, D, 1, 1);
#pragma unroll
    for (int k = 0; k < CHUNK; k += 16) tc::mma(to, tc::mdesc(hi, CHUNK, 0, k), tc::mdesc(z, CHUNK, 0, k), id, k > 0);
#pragma unroll
    for (int k = 0; k < CHUNK; k += 16) tc::mma(to, tc::mdesc(lo, CHUNK, 0, k), tc::mdesc(z, CHUNK, 0, k), id, 1);
}

template <int D, int WALKS>
__global__ void __launch_bounds__(384, 1) k_dla(const __grid_constant__ Walks<WALKS> walks, const Grid p) {
    using K = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Plan plan_s;
    __shared__ int scratch[12];
    __shared__ int gone_s;
    __shared__ uint32_t tslot;
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int range = blockIdx.x / WALKS;
    const Walk& w = walks.w[WALKS == 1 ? 0 : blockIdx.x % WALKS];
    const Line line = line_of(p, w.back);

    const uint32_t bar0 = sb + K::oBar;
    auto full = [&](int slot) { return bar0 + 8 * slot; };
    auto empty = [&](int slot) { return bar0 + 8 * (K::RING + slot); };
    const uint32_t more_bars = bar0 + 16 * K::RING;
    const uint32_t p_full = more_bars, p_ready = more_bars + 8, o_full = more_bars + 16, o_free = more_bars + 24,
                   s_ready = more_bars + 32, s_free = more_bars + 40, y_ready = more_bars + 48, d_full = more_bars + 56,
                   staged = more_bars + 64, ended = more_bars + 72;
    if (tid == 0) {
        for (int i = 0; i < 2 * K::RING; ++i) tc::mbar_init(bar0 + 8 * i, 1);
        tc::mbar_init(p_full, 1);
        tc::mbar_init(p_ready, 128);
        tc::mbar_init(o_full, 1);
        tc::mbar_init(o_free, 128);
        tc::mbar_init(s_ready, 128);
        tc::mbar_init(s_free, 1);
        tc::mbar_init(y_ready, 128);
        tc::mbar_init(d_full, 1);
        tc::mbar_init(staged, 128);
        tc::mbar_init(ended, 1);
        gone_s = 0;
    }
    if (warp == 0) tc::alloc(smem_u32(&tslot), 512);
    make_plan<384>(line, range, p.ranges, p.snap, &plan_s, scratch);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tslot;
    const Waiter wait{&gone_s, p.status};
    const Plan plan = plan_s;
    if (plan.total < 0 && tid == 0) atomicOr(p.status, ST_BAD_SEQLENS);

    // load l of the block: Y, Z, X of its chunk l / 3
    auto slot_of = [&](int l) { return l % K::RING; };
    auto parity_of = [&](int l) { return (uint32_t)((l / K::RING) & 1); };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
        if (warp == 0 && lane == 0) {
            // ---------------- loader ----------------
            tc::prefetch_map(&w.Y);
            tc::prefetch_map(&w.Z);
            tc::prefetch_map(&w.X);
            int l = 0;
            Place at = plan.at;
            for (int f = plan.f0; more(plan, at, f, p.snap); ++f, line.next(at)) {
                const int t0 = line.token(at);
#pragma unroll
                for (int j = 0; j < 3; ++j, ++l) {
                    const int s = slot_of(l);
                    if (l >= K::RING) wait(empty(s), parity_of(l) ^ 1);
                    if (!wait.ok()) break;
                    const CUtensorMap* m = j == 0 ? &w.Y : j == 1 ? &w.Z : &w.X;
                    const int h = at.head / (j == 0 ? w.gy : j == 1 ? w.gz : w.gx);
                    tc::mbar_expect_tx(full(s), K::TILE);
                    tc::tma_load_4d(sb + s * K::TILE, m, 0, h, t0, 0, full(s));
                }
                if (!wait.ok()) break;
            }
            // (where the block gave up: its copies have to land before it ends)
            if (!wait.ok())
                for (int i = l > K::RING ? l - K::RING : 0; i < l; ++i) tc::mbar_wait(full(slot_of(i)), parity_of(i));
        } else if (warp == 1 && lane == 0) {
            // ---------------- issuer ----------------
            const uint32_t tP = tmem, tO1 = tmem + 128, tO2 = tmem + 256, tD = tmem + 384;
            constexpr uint32_t idP = tc::idesc(128, 128, 0, 0), idO = tc::idesc(128, D, 0, 1);
            Place at = plan.at;
            int it = 0;
            for (int f = plan.f0; more(plan, at, f, p.snap); ++f, line.next(at), ++it) {
                const int ly = 3 * it, lz = ly + 1, lx = ly + 2;
                const uint32_t Y = sb + slot_of(ly) * K::TILE, Z = sb + slot_of(lz) * K::TILE, X = sb + slot_of(lx) * K::TILE;
                const uint32_t ph = it & 1;
                wait(full(slot_of(ly)), parity_of(ly));
                wait(full(slot_of(lx)), parity_of(lx));
                if (it) wait(o_full, ph ^ 1);  // (P Z of the chunk before has read P)
                if (!wait.ok()) break;
                tc::fence_after();
#pragma unroll
                for (int k = 0; k < D; k += 16) tc::mma(tP, tc::kdesc(X, CHUNK, 0, k), tc::kdesc(Y, CHUNK, 0, k), idP, k > 0);
                tc::commit(p_full);
                wait(s_ready, ph);
                if (it) wait(o_free, ph ^ 1);
                if (!wait.ok()) break;
                tc::fence_after();
#pragma unroll
                for (int k = 0; k < D; k += 16) tc::mma(tO2, tc::kdesc(X, CHUNK, 0, k), tc::mdesc(sb + K::oS, D, 0, k), idO, k > 0);
                tc::commit(s_free);
                wait(full(slot_of(lz)), parity_of(lz));
                const bool part = line.rows(at) < CHUNK;
                if (part) wait(y_ready, ph);  // (group B clears rows of Z)
                wait(p_ready, ph);
                if (!wait.ok()) break;
                tc::fence_after();
#pragma unroll
                for (int k = 0; k < CHUNK; k += 16) tc::mma_ts(tO1, tP + k / 2, tc::mdesc(Z, CHUNK, 0, k), idO, k > 0);
                tc::commit(o_full);
                if (!part) wait(y_ready, ph);
                if (!wait.ok()) break;
                tc::fence_after();
                issue_terms<D>(tD, Y, sb + K::oLo, Z);
                tc::commit(d_full);
                tc::commit(empty(slot_of(ly)));
                tc::commit(empty(slot_of(lz)));
            }
            if (!wait.ok()) {  // (the products in flight have to end before the tensor memory is given back)
                tc::commit(ended);
                tc::mbar_wait(ended, 0);
            }
        } else if (warp == 2 && lane == 0) {
            // ---------------- stores ----------------
            Place at = plan.at;
            int it = 0;
            for (int f = plan.f0; more(plan, at, f, p.snap); ++f, line.next(at), ++it) {
                const int s = slot_of(3 * it + 2);
                wait(staged, it & 1);
                if (!wait.ok()) break;
                if (!w.o32 && line.rows(at) == CHUNK) {
                    tc::tma_store_4d(&w.out, 0, at.head, line.token(at), 0, sb + s * K::TILE);
                    tc::bulk_commit();
                    tc::bulk_wait_read();
                }
                tc::mbar_arrive(empty(s));
            }
            tc::bulk_wait_all();
        }
    } else if (warp < 8) {
        // ---------------- group A: P, outputs ----------------
        const int q4 = warp & 3, i = 32 * q4 + lane;  // row of the chunk
        const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16);
        float* tab = reinterpret_cast<float*>(smem + K::oTab);  // tab[i - j + 127] = D_ij
        Place at = plan.at;
        int it = 0, head = -1;
        float r_full = 0.f, g = 0.f;
        for (int f = plan.f0; more(plan, at, f, p.snap); ++f, line.next(at), ++it) {
            const uint32_t ph = it & 1;
            if (at.head != head) {
                head = at.head;
                g = log_decay(p.g, head);
                r_full = w.o_scale * power(g, w.back ? CHUNK - 1 - i : i + 1);
                tc::named_sync(1, 128);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int n = w.back ? 127 - (i + 128 * u) : i + 128 * u - 127;
                    tab[i + 128 * u] = n >= 0 ? w.p_scale * power(g, n) : 0.f;
                }
                tc::named_sync(1, 128);
            }
            const int rows = line.rows(at);
            wait(p_full, ph);
            tc::fence_after();
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t out[16];
                if (w.back ? s < q4 : s > q4) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[j] = 0;
                } else {
                    float v[32];
                    tc::ld32(lanes + 32 * s, v);
                    const float* d = tab + i - 32 * s + 127;
                    // (what the mask leaves out is set to zero, not multiplied by it: it may not be finite)
                    const int from = w.back ? i - 32 * s : 0, to = (w.back ? rows - 1 : i) - 32 * s;
                    if (s == q4 || (w.back && rows < CHUNK)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = j >= from && j <= to ? v[j] * d[-j] : 0.f;
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] *= d[-j];
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
                }
                tc::st16u_nowait(lanes + 16 * s, out);
            }
            tc::st_wait();
            tc::fence_before();
            tc::mbar_arrive(p_ready);

            float r = r_full;
            if (w.back && rows < CHUNK) r = i < rows ? w.o_scale * power(g, rows - 1 - i) : 0.f;
            const int slot = slot_of(3 * it + 2);
            unsigned char* stage = smem + slot * K::TILE;
            const int64_t row = (int64_t)line.token(at) + i;
            wait(o_full, ph);
            tc::fence_after();
#pragma unroll
            for (int s = 0; s < D / 32; ++s) {
                float a[32], b[32];
                tc::ld32(lanes + 128 + 32 * s, a);
                tc::ld32(lanes + 256 + 32 * s, b);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 u = __ffma2_rn(make_float2(r, r), F2(b, j), F2(a, j));
                    a[j] = u.x;
                    a[j + 1] = u.y;
                }
                if (w.o32) {
                    if (i < rows && wait.ok()) {
                        float4* to = reinterpret_cast<float4*>(w.o32 + (row * p.H + head) * D + 32 * s);
#pragma unroll
                        for (int j = 0; j < 8; ++j) to[j] = make_float4(a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 u = make_uint4(pack_bf16(a[8 * j], a[8 * j + 1]), pack_bf16(a[8 * j + 2], a[8 * j + 3]),
                                                   pack_bf16(a[8 * j + 4], a[8 * j + 5]), pack_bf16(a[8 * j + 6], a[8 * j + 7]));
                        if (rows == CHUNK) *reinterpret_cast<uint4*>(stage + tc::sw_chunk(i, 4 * s + j, CHUNK)) = u;
                        else if (i < rows && wait.ok()) *reinterpret_cast<uint4*>(w.o + (row * p.H + head) * D + 32 * s + 8 * j) = u;
                    }
                }
            }
            tc::fence_before();
            tc::mbar_arrive(o_free);
            tc::fence_async_smem();
            tc::mbar_arrive(staged);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 248;\n");
        // ---------------- group B: Y', the state ----------------
        const int q4 = warp & 3, i = 32 * q4 + lane;  // token of Y; row of the state
        const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16) + 384;
        const bool mine = i < D;  // (warps without rows of the state)
        float S[D];
        Place at = plan.at;
        int it = 0;
        float g = 0.f, w_full = 0.f;
        float2 c_full = make_float2(0.f, 0.f);
        auto incoming = [&]() {
            const float* from = nullptr;
            if (at.pos != 0) from = w.joined + (int64_t)(range - 1) * D * D;
            else if (w.init) from = w.init + ((int64_t)at.seq * p.H + at.head) * D * D;
            if (from && mine) {
                if (w.turned) {
#pragma unroll
                    for (int c = 0; c < D; ++c) S[c] = from[c * D + i];
                } else {
#pragma unroll
                    for (int c = 0; c < D; c += 4) {
                        const float4 u = *reinterpret_cast<const float4*>(from + i * D + c);
                        S[c] = u.x, S[c + 1] = u.y, S[c + 2] = u.z, S[c + 3] = u.w;
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < D; ++c) S[c] = 0.f;
            }
            g = log_decay(p.g, at.head);
            w_full = w.w_scale * power(g, w.back ? i + 1 : CHUNK - 1 - i);
            c_full = carry(g, CHUNK);
        };
        auto copy_state = [&]() {
            if (mine) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    *reinterpret_cast<uint4*>(smem + K::oS + tc::sw_chunk(i, j, D)) =
                        make_uint4(pack_bf16(S[8 * j], S[8 * j + 1]), pack_bf16(S[8 * j + 2], S[8 * j + 3]),
                                   pack_bf16(S[8 * j + 4], S[8 * j + 5]), pack_bf16(S[8 * j + 6], S[8 * j + 7]));
            }
            tc::fence_async_smem();
            tc::mbar_arrive(s_ready);
        };
        int f = plan.f0;
        if (more(plan, at, f, p.snap)) {
            incoming();
            copy_state();
        }
        while (more(plan, at, f, p.snap)) {
            const uint32_t ph = it & 1;
            const int ly = 3 * it, lz = ly + 1;
            const int rows = line.rows(at);
            float wt = w_full;
            float2 c = c_full;
            if (rows < CHUNK) {
                wt = i < rows ? w.w_scale * power(g, w.back ? i + 1 : rows - 1 - i) : 0.f;
                c = carry(g, rows);
                wait(full(slot_of(lz)), parity_of(lz));
                if (i >= rows && wait.ok()) clear_row<D>(smem + slot_of(lz) * K::TILE, i);
            }
            wait(full(slot_of(ly)), parity_of(ly));
            wait(p_full, ph);  // (X Y^T has read Y)
            if (wait.ok()) split_row<D>(smem + slot_of(ly) * K::TILE, smem + K::oLo, i, wt);
            tc::fence_async_smem();
            tc::mbar_arrive(y_ready);
            wait(d_full, ph);
            tc::fence_after();
            if (32 * q4 < D) {
#pragma unroll
                for (int s = 0; s < D / 32; ++s) {
                    float v[32];
                    tc::ld32(lanes + 32 * s, v);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 old = F2(S, 32 * s + j);
                        const float2 t = __ffma2_rn(make_float2(c.x, c.x), old, F2(v, j));
                        ACC2(S, 32 * s + j, __ffma2_rn(make_float2(c.y, c.y), old, t));
                    }
                }
            }
            tc::fence_before();
            const bool ends = at.pos + 1 == at.count;
            if (ends && w.last && mine && wait.ok()) {
                float* to = w.last + (((int64_t)at.seq * p.H + at.head) * D + i) * D;
#pragma unroll
                for (int j = 0; j < D; j += 4) *reinterpret_cast<float4*>(to + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
            }
            ++f, ++it;
            line.next(at);
            if (!more(plan, at, f, p.snap)) break;
            if (ends) incoming();
            wait(s_free, ph);  // (X C has read the copy)
            copy_state();
        }
    }
    // empty sequences pass their states through
    if (w.last && plan.total >= 0 && p.cu) {
        const int64_t size = (int64_t)p.H * D * D;
        for (int n = range; n < p.N; n += p.ranges) {
            if (p.cu[n] != p.cu[n + 1]) continue;
            for (int64_t e = tid; e < size; e += 384) w.last[n * size + e] = w.init ? w.init[n * size + e] : 0.f;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::dealloc(tmem, 512);
}

struct TailWalk {
    CUtensorMap Y, Z;
    int gy, gz, back;
    float w_scale;
    float* sums;        // [ranges][D][D]
    const float* init;  // [N][H][D][D] or nullptr
};
template <int WALKS>
struct TailWalks {
    TailWalk w[WALKS];
};

// The part of range `range` that its last chain has, where that chain goes on: the first chunk's place.
struct Tail {
    Place first, last;
    int chunks;  // 0: none
};
__device__ __forceinline__ Tail tail_of(const Line& line, const Plan& plan) {
    Tail t;
    t.chunks = 0;
    t.first = plan.at;
    if (plan.total <= 0 || plan.f0 >= plan.f1) return t;
    // chain by chain to the one that holds the range's last chunk
    Place at = plan.at;
    int f = plan.f0;
    while (f + (at.count - at.pos) < plan.f1) {
        f += at.count - at.pos;
        at.pos = at.count - 1;
        line.next(at);
    }
    t.first = at;
    t.last = at;
    t.last.pos = at.pos + (plan.f1 - 1 - f);
    if (t.last.pos + 1 < at.count) t.chunks = plan.f1 - f;
    return t;
}

// For each range the sum of its last chain's terms, as the next range's state takes them.
template <int D, int WALKS>
__global__ void __launch_bounds__(256, 1) k_dla_tail(const __grid_constant__ TailWalks<WALKS> walks, const Grid p) {
    using K = TailCfg<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Plan plan_s;
    __shared__ int scratch[8];
    __shared__ int gone_s;
    __shared__ uint32_t tslot;
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int range = blockIdx.x / WALKS;
    const TailWalk& w = walks.w[WALKS == 1 ? 0 : blockIdx.x % WALKS];
    const Line line = line_of(p, w.back);
    const uint32_t bar0 = sb + K::oBar;
    auto full = [&](int slot) { return bar0 + 8 * slot; };
    auto empty = [&](int slot) { return bar0 + 8 * (K::RING + slot); };
    const uint32_t y_ready = bar0 + 16 * K::RING, d_full = y_ready + 16 /* two each */, ended = d_full + 16;
    if (tid == 0) {
        for (int i = 0; i < 2 * K::RING; ++i) tc::mbar_init(bar0 + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(y_ready + 8 * i, 128);
            tc::mbar_init(d_full + 8 * i, 1);
        }
        tc::mbar_init(ended, 1);
        gone_s = 0;
    }
    if (warp == 0) tc::alloc(smem_u32(&tslot), 256);
    make_plan<256>(line, range, p.ranges, 0, &plan_s, scratch);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tslot;
    const Waiter wait{&gone_s, p.status};
    const Tail tail = tail_of(line, plan_s);
    const float g = tail.chunks ? log_decay(p.g, tail.first.head) : 0.f;
    const int end = tail.chunks ? line.before(tail.first, tail.last.pos + 1) : 0;  // tokens of the chain before the next range
    // chunk `it` of the walk: from the last one backwards, as long as any decay is left
    auto chunk = [&](int it, Place& at) {
        at = tail.last;
        at.pos -= it;
        return it < tail.chunks && power(g, end - line.before(at, at.pos + 1)) != 0.f;
    };
    auto slot_of = [&](int l) { return l % K::RING; };
    auto parity_of = [&](int l) { return (uint32_t)((l / K::RING) & 1); };
    Place at;
    if (warp == 0 && lane == 0) {
        int l = 0;
        for (int it = 0; chunk(it, at); ++it) {
            const int t0 = line.token(at);
#pragma unroll
            for (int j = 0; j < 2; ++j, ++l) {
                const int s = slot_of(l);
                if (l >= K::RING) wait(empty(s), parity_of(l) ^ 1);
                if (!wait.ok()) break;
                tc::mbar_expect_tx(full(s), K::TILE);
                tc::tma_load_4d(sb + s * K::TILE, j ? &w.Z : &w.Y, 0, at.head / (j ? w.gz : w.gy), t0, 0, full(s));
            }
            if (!wait.ok()) break;
        }
        if (!wait.ok())
            for (int i = l > K::RING ? l - K::RING : 0; i < l; ++i) tc::mbar_wait(full(slot_of(i)), parity_of(i));
    } else if (warp == 1 && lane == 0) {
        for (int it = 0; chunk(it, at); ++it) {
            const int b = it & 1;
            const uint32_t ph = (it >> 1) & 1;
            wait(full(slot_of(2 * it + 1)), parity_of(2 * it + 1));
            wait(y_ready + 8 * b, ph);
            if (!wait.ok()) break;
            tc::fence_after();
            issue_terms<D>(tmem + 128 * b, sb + slot_of(2 * it) * K::TILE, sb + K::oLo + b * K::TILE, sb + slot_of(2 * it + 1) * K::TILE);
            tc::commit(d_full + 8 * b);
            tc::commit(empty(slot_of(2 * it)));
            tc::commit(empty(slot_of(2 * it + 1)));
        }
        if (!wait.ok()) {
            tc::commit(ended);
            tc::mbar_wait(ended, 0);
        }
    } else if (warp >= 4) {
        const int q4 = warp & 3, i = 32 * q4 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16);
        float S[D];
#pragma unroll
        for (int c = 0; c < D; ++c) S[c] = 0.f;
        auto bring = [&](int it) {
            Place c;
            if (!chunk(it, c)) return false;
            const int rows = line.rows(c), l = 2 * it;
            // tokens of the walk from token i on to the next range's first
            const int away = end - line.before(c, c.pos) - (w.back ? rows - 1 - i : i);
            const float wt = i < rows ? w.w_scale * power(g, w.back ? away : away - 1) : 0.f;
            wait(full(slot_of(l)), parity_of(l));
            if (wait.ok()) split_row<D>(smem + slot_of(l) * K::TILE, smem + K::oLo + (it & 1) * K::TILE, i, wt);
            if (rows < CHUNK) {
                wait(full(slot_of(l + 1)), parity_of(l + 1));
                if (i >= rows && wait.ok()) clear_row<D>(smem + slot_of(l + 1) * K::TILE, i);
            }
            tc::fence_async_smem();
            tc::mbar_arrive(y_ready + 8 * (it & 1));
            return true;
        };
        bool on = bring(0);
        for (int it = 0; on; ++it) {
            on = bring(it + 1);
            wait(d_full + 8 * (it & 1), (it >> 1) & 1);
            tc::fence_after();
            if (32 * q4 < D) {
#pragma unroll
                for (int s = 0; s < D / 32; ++s) {
                    float v[32];
                    tc::ld32(lanes + 128 * (it & 1) + 32 * s, v);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) ACC2(S, 32 * s + j, __fadd2_rn(F2(S, 32 * s + j), F2(v, j)));
                }
            }
            tc::fence_before();
        }
        if (tail.chunks && i < D && wait.ok()) {
            float* to = w.sums + ((int64_t)range * D + i) * D;
#pragma unroll
            for (int j = 0; j < D; j += 4) *reinterpret_cast<float4*>(to + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::dealloc(tmem, 256);
}

// The states at the beginnings of ranges that begin inside a chain, in the place of the sums of the ranges
// before them: along each such chain, from its initial state.  One block an eighth of a state.
template <int D, int WALKS>
__global__ void __launch_bounds__(256) k_dla_join(const __grid_constant__ TailWalks<WALKS> walks, const Grid p) {
    constexpr int SLICES = D * D / 2048;  // of 256 threads' two float4
    __shared__ Plan plan_s;
    __shared__ int scratch[8];
    const int slice = blockIdx.x % SLICES, which = blockIdx.x / SLICES % WALKS, range = blockIdx.x / SLICES / WALKS + 1;
    const TailWalk& w = walks.w[which];
    const Line line = line_of(p, w.back);
    make_plan<256>(line, range, p.ranges, 0, &plan_s, scratch);
    const Plan plan = plan_s;
    if (plan.total <= 0 || plan.f0 >= plan.f1 || plan.at.pos == 0) return;
    const Place at = plan.at;
    const int begin = plan.f0 - at.pos;  // the chain's first chunk
    if (begin < range_begin(plan.total, range - 1, plan.ranges)) return;  // (the chain's first crossing does them all)
    const float g = log_decay(p.g, at.head);
    const int e = slice * 2048 + threadIdx.x * 4;
    float4 s[2] = {};
    if (w.init) {
        const float* from = w.init + ((int64_t)at.seq * p.H + at.head) * D * D + e;
#pragma unroll
        for (int u = 0; u < 2; ++u) s[u] = *reinterpret_cast<const float4*>(from + 1024 * u);
    }
    int done = 0;
    for (int r = range; r < plan.ranges; ++r) {
        const int f = range_begin(plan.total, r, plan.ranges);
        if (f >= begin + at.count) break;
        const int upto = line.before(at, f - begin);
        const float2 c = carry(g, upto - done);
        done = upto;
        float* sum = w.sums + (int64_t)(r - 1) * D * D + e;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float4* to = reinterpret_cast<float4*>(sum + 1024 * u);
            const float4 t = *to;
            s[u] = make_float4(fmaf(c.y, s[u].x, fmaf(c.x, s[u].x, t.x)), fmaf(c.y, s[u].y, fmaf(c.x, s[u].y, t.y)),
                               fmaf(c.y, s[u].z, fmaf(c.x, s[u].z, t.z)), fmaf(c.y, s[u].w, fmaf(c.x, s[u].w, t.w)));
            *to = s[u];
        }
    }
}

// the gradients of shared heads: sums over the value heads of a group
__global__ void __launch_bounds__(256) k_dla_groups(const float* a, __nv_bfloat16* out, int64_t pairs, int group, int D) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= pairs) return;
    const int64_t row = i * 2 / D;  // (token, k head)
    const float* from = a + row * group * D + (i * 2 - row * D);
    float2 s = make_float2(0.f, 0.f);
    for (int j = 0; j < group; ++j) {
        const float2 u = *reinterpret_cast<const float2*>(from + (int64_t)j * D);
        s = make_float2(s.x + u.x, s.y + u.y);
    }
    reinterpret_cast<uint32_t*>(out)[i] = pack_bf16(s.x, s.y);
}

// How a call's chunks are shared out: the number of ranges (of each walk), and whether they end with whole chains.
struct Shares {
    int ranges, snap;
};
Shares shares_of(const DlaParams& p, int walks) {
    const int64_t chains = (int64_t)p.N * p.H;
    const int64_t longest = p.cu_seqlens ? (p.T + CHUNK - 1) / CHUNK : (p.seq_len + CHUNK - 1) / CHUNK;
    const int64_t most = p.cu_seqlens ? (p.T / CHUNK + p.N) * p.H : longest * chains;
    const int sms = num_sms();
    int64_t fit = sms / walks > 0 ? sms / walks : 1;
    if (longest <= 4) return {(int)(chains < fit ? chains : fit), 1};
    const int64_t ranges = (most + 3) / 4;  // of at least four chunks
    return {(int)(ranges < fit ? ranges : fit), 0};
}

template <int D, int WALKS, int TAILS>
cudaError_t go(const DlaParams& p, const Shares& sh, const Walks<WALKS>& walks, const TailWalks<TAILS>& tails, cudaStream_t s) {
    const Grid grid{p.N, p.H, D, sh.ranges, sh.snap, p.T, p.seq_len, p.cu_seqlens, p.g, p.status};
    cudaError_t e = cudaMemsetAsync(p.status, 0, 256, s);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(k_dla<D, WALKS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    // (the groups' shares of the registers, 88 + 168 + 248 a thread of 128, have to be there at the launch)
    static const int regs = [] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, k_dla<D, WALKS>) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs != 168) return cudaErrorInvalidConfiguration;
    if (!sh.snap && sh.ranges > 1) {
        e = cudaFuncSetAttribute(k_dla_tail<D, TAILS>, cudaFuncAttributeMaxDynamicSharedMemorySize, TailCfg<D>::SMEM);
        if (e != cudaSuccess) return e;
        k_dla_tail<D, TAILS><<<(sh.ranges - 1) * TAILS, 256, TailCfg<D>::SMEM, s>>>(tails, grid);
        k_dla_join<D, TAILS><<<(sh.ranges - 1) * TAILS * (D * D / 2048), 256, 0, s>>>(tails, grid);
    }
    k_dla<D, WALKS><<<sh.ranges * WALKS, 384, Cfg<D>::SMEM, s>>>(walks, grid);
    return cudaGetLastError();
}

struct Tensor {
    const void* at;
    int heads;
    int64_t ld;
};
bool encode(CUtensorMap* m, const Tensor& t, const DlaParams& p) {
    return encode_heads_map(m, t.at, p.T, t.heads, p.D, t.ld, CHUNK);
}
bool make_walk(Walk* w, const DlaParams& p, const Tensor& x, const Tensor& y, const Tensor& z, void* out, int out_heads) {
    w->gx = p.H / x.heads, w->gy = p.H / y.heads, w->gz = p.H / z.heads;
    w->o = static_cast<__nv_bfloat16*>(out);
    return encode(&w->X, x, p) && encode(&w->Y, y, p) && encode(&w->Z, z, p) &&
           encode(&w->out, Tensor{out, out_heads, (int64_t)out_heads * p.D}, p);
}

template <int D>
cudaError_t forward(const DlaParams& p, cudaStream_t s) {
    const Shares sh = shares_of(p, 1);
    const Tensor q{p.q, p.Hk, p.ldq}, k{p.k, p.Hk, p.ldk}, v{p.v, p.H, p.ldv};
    Walks<1> w;
    memset(&w, 0, sizeof(w));
    TailWalks<1> t;
    memset(&t, 0, sizeof(t));
    Walk& o = w.w[0];
    if (!make_walk(&o, p, q, k, v, p.o, p.H)) return cudaErrorInvalidValue;
    o.p_scale = o.o_scale = p.scale, o.w_scale = 1.f;
    o.init = p.h0, o.joined = p.states, o.last = p.ht;
    t.w[0] = TailWalk{o.Y, o.Z, o.gy, o.gz, 0, 1.f, p.states, p.h0};
    return go<D, 1, 1>(p, sh, w, t, s);
}

template <int D>
cudaError_t backward(const DlaParams& p, cudaStream_t s) {
    const Shares sh = shares_of(p, 3);
    const Tensor q{p.q, p.Hk, p.ldq}, k{p.k, p.Hk, p.ldk}, v{p.v, p.H, p.ldv}, dO{p.dO, p.H, (int64_t)p.H * D};
    Walks<3> w;
    memset(&w, 0, sizeof(w));
    TailWalks<2> t;
    memset(&t, 0, sizeof(t));
    Walk &dq = w.w[0], &dk = w.w[1], &dv = w.w[2];
    if (!make_walk(&dq, p, dO, v, k, p.dq, p.Hk) || !make_walk(&dk, p, v, dO, q, p.dk, p.Hk) || !make_walk(&dv, p, k, q, dO, p.dv, p.H))
        return cudaErrorInvalidValue;
    float* back = p.states + (size_t)sh.ranges * D * D;
    dq.turned = 1, dq.p_scale = dq.o_scale = p.scale, dq.w_scale = 1.f;
    dq.init = p.h0, dq.joined = p.states, dq.o32 = p.dq_heads;
    dk.turned = 1, dk.back = 1, dk.p_scale = dk.w_scale = p.scale, dk.o_scale = 1.f;
    dk.init = p.dht, dk.joined = back, dk.o32 = p.dk_heads;
    dv.back = 1, dv.p_scale = dv.w_scale = p.scale, dv.o_scale = 1.f;
    dv.init = p.dht, dv.joined = back, dv.last = p.dh0;
    t.w[0] = TailWalk{dq.Z, dq.Y, dq.gz, dq.gy, 0, 1.f, p.states, p.h0};
    t.w[1] = TailWalk{dv.Y, dv.Z, dv.gy, dv.gz, 1, p.scale, back, p.dht};
    cudaError_t e = go<D, 3, 2>(p, sh, w, t, s);
    if (e != cudaSuccess || !p.dq_heads) return e;
    const int64_t pairs = p.T * p.Hk * D / 2;
    const unsigned grid = (unsigned)((pairs + 255) / 256);
    k_dla_groups<<<grid, 256, 0, s>>>(p.dq_heads, p.dq, pairs, p.H / p.Hk, D);
    k_dla_groups<<<grid, 256, 0, s>>>(p.dk_heads, p.dk, pairs, p.H / p.Hk, D);
    return cudaGetLastError();
}

}  // namespace

size_t dla_states_bytes(const DlaParams& p, bool backward) {
    const Shares sh = shares_of(p, backward ? 3 : 1);
    return sh.snap || sh.ranges < 2 ? 0 : (backward ? 2 : 1) * sizeof(float) * (size_t)sh.ranges * p.D * p.D;
}
int dla_kernels(const DlaParams& p, bool backward) {
    const Shares sh = shares_of(p, backward ? 3 : 1);
    return (sh.snap || sh.ranges < 2 ? 1 : 3) + (backward && p.H != p.Hk ? 2 : 0);
}

cudaError_t launch_dla_fwd(const DlaParams& p, cudaStream_t s) { return p.D == 64 ? forward<64>(p, s) : forward<128>(p, s); }
cudaError_t launch_dla_bwd(const DlaParams& p, cudaStream_t s) { return p.D == 64 ? backward<64>(p, s) : backward<128>(p, s); }

}  // namespace gdr
