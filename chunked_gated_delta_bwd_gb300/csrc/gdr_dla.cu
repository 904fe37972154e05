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
// Bytes bound it: a chunk and head of 128 channels moves 128 KB (2.9 us of a multiprocessor's share of the measured copy
// rate) for five products of 128^3 and one more for the states' accuracy (1.6 us of tensor cores).  So one block a
// multiprocessor walks chunks (gdr_dla_plan.cuh: a range, or whole chains from a queue), the state in fp32 registers, in
// roles that overlap:
//   loader    Y, X, Z tiles of the chunks to come, by TMA, through a ring of tiles; what the others have to know of a chunk
//   issuer 1  P = X Y^T, and P Z (P from tensor memory)
//   issuer 3  the state's terms Y'^T Z, and X C
//   stores    the outputs, by TMA
//   group A   (eight warps) P times the decays, rounded to bf16 (tensor memory); out, staged in X's tile
//   group B   (eight warps) Y' = w Y as two bf16 tiles, whose products with Z make the state's terms good to 2^-17; the
//             state's sum in fp32, and its bf16 copy for X C
// P and the state's copy are rounded to bf16: each adds up to 2^-8 of a term of an output that is rounded to bf16 itself
// (o and the gradients are off by 2.3e-3 in the 2-norm; their own rounding alone is 1.7e-3).  The tokens' terms of the
// states keep 2^-17: the first part leaves 2^-8 of a value's power of two at most, whose half step is 2^-17 (ht, dh0: 2.5e-6; a
// plain fp32 form 3e-7.  A third part does not fit: the seven tiles of 128 channels fill shared memory.  Y itself as an exact part
// for long memories, and a third one in Y's place for the chunks near a chain's end, took 6.4e-7, and 12 to 20% more time, most of
// it in calls that hardly ran them).  With one half of Y' in the walks whose states do not leave, dq and dk were off by
// 2.7e-3, for 2 us in 355.
//
// Measured (32768 tokens, 16 heads of 128): forward 155 us, its walk 98 (5.5 TB/s); backward 355, its three walks 265.  A
// chunk takes 6000 cycles where 5400 are its bytes' time (forward) and 2560 its products': what is left is the turn of P,
// decays, P Z and output, which wait for one another in group A, beside split, product and sum in group B.  With 64
// channels it is this turn alone: 4500 cycles a chunk of half the bytes.  Tried: Y' of 64 channels as one operand of 128
// columns (98 -> 103 us at 2 x 4095 backward, 16 heads); two tiles of Y; tiles asked into the second-level cache two chunks
// ahead; more columns a tensor memory load; two loaders: all as fast or slower.
//
// A chain that crosses from one range into the next: k_dla_tail first sums, for each range, the terms of
// its last chain's tokens (it reads only Y and Z, from the range's end backwards, and stops where the decay
// has underflowed, so that a NaN from there on does not reach the next range; 41 us forward, 77 for the
// backward's two sums), k_dla_join carries them along the chain (8 to 12 us),
// and the walk starts from there.
#include "gdr_dla.h"
#include "gdr_dla_plan.cuh"
#include "gdr_internal.h"
#include "gdr_tc.cuh"
#include "gdr_tma.h"

namespace gdr {
namespace {

using namespace dla;

// Tiles in shared memory: X, Y and Z of the chunks to come (a slot of X is free when its output has been
// stored from it, of Y when P is there and Y' has been made from it, of Z when its products are done), both halves of Y',
// the state's copy.
template <int D>
struct Cfg {
    static constexpr int TILE = CHUNK * D * 2;
    static constexpr int NX = D == 128 ? 2 : 3, NY = D == 128 ? 1 : 2, NZ = NY, SLOTS = NX + NY + NZ;
    static constexpr int oHi = SLOTS * TILE, oLo = oHi + TILE, oS = oLo + TILE, oTab = oS + D * D * 2;
    // (the product Y'^T Z has 128 rows; with 64 channels the upper ones read what lies behind the tile)
    static constexpr int oEnd = (oTab + 512 > oLo + 2 * CHUNK * 128 ? oTab + 512 : oLo + 2 * CHUNK * 128);
    // (an fp32 output is twice X's tile: with 64 channels there is room for it, with 128 one half goes out after the other)
    static constexpr int oWide = (oEnd + 1023) / 1024 * 1024;
    static constexpr int oBar = D == 64 ? oWide + 2 * TILE : oEnd, BARS = 2 * SLOTS + 13 + 2 * NX;
    static constexpr int SMEM = oBar + 8 * BARS + 1024;
    static constexpr int THREADS = 640;  // a warpgroup of single threads' roles, two each for groups A and B
    static constexpr int REGS = 96, REGS_1 = 80, REGS_B = 104;  // at the launch (and group A), of the single threads, of group B
};
static_assert(Cfg<128>::REGS_1 + 2 * Cfg<128>::REGS_B <= 3 * Cfg<128>::REGS, "the groups' registers come out of the launch's");
template <int D>
struct TailCfg {
    static constexpr int TILE = CHUNK * D * 2, RING = D == 128 ? 5 : 8;
    static constexpr int oLo = RING * TILE, oEnd = oLo + 2 * TILE + (D == 128 ? 0 : CHUNK * 128);
    static constexpr int oBar = oEnd, BARS = 2 * RING + 5;
    static constexpr int SMEM = oBar + 8 * BARS + 1024;
    static constexpr int THREADS = 384;
};

struct Walk {
    CUtensorMap X, Y, Z, out;       // (out: bf16, or fp32 where value heads share a head of it)
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
    int N, H, D, ranges, mode;
    int pieces;  // blocks that share the sum of a range's last chain
    int64_t T, seq_len;
    const int64_t* cu;
    const float* g;
    int* status;
    int* taken;  // for each walk the chains that its blocks have taken from the queue beyond their first
};
__device__ __forceinline__ Line line_of(const Grid& p, int back, const Plan* plan) {
    return Line{p.N, p.H, p.T, p.seq_len, p.cu, back, plan};
}

// Waits are bounded: one that runs out records it, and ends every role of the block at its next wait.
struct Waiter {
    volatile int* gone;
    int* status;
    __device__ __forceinline__ bool ok() const { return *gone == 0; }
    // by one thread
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        if (tc::mbar_try(bar, parity)) return true;
#pragma unroll 1
        for (int i = 0; i < 1 << 22; ++i) {
            if (!ok()) return false;
            if (tc::mbar_try(bar, parity)) return true;
        }
        give_up();
        return false;
    }
    // by a whole warp, which goes on converged
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {
        if (__all_sync(~0u, tc::mbar_try(bar, parity))) return true;
#pragma unroll 1
        for (int i = 0; i < 1 << 22; ++i) {
            if (__any_sync(~0u, !ok())) return false;
            if (__all_sync(~0u, tc::mbar_try(bar, parity))) return true;
        }
        give_up();
        return false;
    }
    __device__ __forceinline__ void give_up() const {
        *gone = 1;
        atomicOr(status, ST_MMA_TIMEOUT);
    }
};

// Chunks j0 to j0 + N of 16 bytes of row `row` of a tile times w, rounded to bf16 (`hi`) and what that leaves (`lo`).
// (Not unrolled: what eight warps of two groups run in turn has to stay in the instruction caches.)
template <int N>
__device__ __forceinline__ void split_row(const unsigned char* tile, unsigned char* hi, unsigned char* lo, int row, int j0, float w) {
#pragma unroll 1
    for (int j2 = j0; j2 < j0 + N; j2 += 2) {
        uint4 u[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) u[j] = *reinterpret_cast<const uint4*>(tile + tc::sw_chunk(row, j2 + j, CHUNK));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t in[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __fmul2_rn(make_float2(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xffff0000u)), make_float2(w, w));
                h[i] = pack_bf16(f.x, f.y);
                const float2 r = __ffma2_rn(make_float2(__uint_as_float(h[i] << 16), __uint_as_float(h[i] & 0xffff0000u)), make_float2(-1.f, -1.f), f);
                l[i] = pack_bf16(r.x, r.y);
            }
            const uint32_t at = tc::sw_chunk(row, j2 + j, CHUNK);
            *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    }
}
// the same chunks of a row made zero (a row of another sequence, whose values must not reach a product)
template <int N>
__device__ __forceinline__ void clear_row(unsigned char* tile, int row, int j0) {
#pragma unroll
    for (int j = 0; j < N; ++j) *reinterpret_cast<uint4*>(tile + tc::sw_chunk(row, j0 + j, CHUNK)) = make_uint4(0, 0, 0, 0);
}
// What the loader tells the other roles of a chunk (the walk along the line costs registers that they need for sums).
struct Chunk {
    int t0;     // first token
    int rows;   // tokens, and the bits below
    int head;
    int chain;  // seq * H + head
    // the chain ends with it; it is the block's last; the next one is another chain's first (a range may end inside a chain)
    static constexpr int ENDS = 256, LAST = 512, TURNS = 1024;
    __device__ __forceinline__ int tokens() const { return rows & 255; }
    __device__ __forceinline__ bool ends() const { return rows & ENDS; }
    __device__ __forceinline__ bool last() const { return rows & LAST; }
    __device__ __forceinline__ bool turns() const { return rows & TURNS; }
};
__device__ __forceinline__ Chunk chunk_at(const int4* chunks, int it) {
    const int4 c = chunks[it & 7];
    return Chunk{c.x, c.y, c.z, c.w};
}

// one arrival for a warp, after all of its threads' work
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

// the state's terms of a chunk, transposed: Z^T Y', from both halves of Y'
template <int D>
__device__ __forceinline__ void issue_terms(uint32_t on, uint32_t to, uint32_t hi, uint32_t lo, uint32_t z) {
    constexpr uint32_t id = tc::idesc(128, D, 1, 1);
#pragma unroll 1
    for (int k = 0; k < CHUNK; k += 16) tc::mma_if(on, to, tc::mdesc(z, CHUNK, 0, k), tc::mdesc(hi, CHUNK, 0, k), id, k > 0);
#pragma unroll 1
    for (int k = 0; k < CHUNK; k += 16) tc::mma_if(on, to, tc::mdesc(z, CHUNK, 0, k), tc::mdesc(lo, CHUNK, 0, k), id, 1);
}

template <int D, int WALKS>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1) k_dla(const __grid_constant__ Walks<WALKS> walks, const Grid p) {
    using K = Cfg<D>;
    constexpr int HALF = D / 2;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Plan plan_s;
    __shared__ int scratch[K::THREADS / 32];
    __shared__ int gone_s;
    __shared__ uint32_t tslot;
    __shared__ int4 chunks[8];
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int range = blockIdx.x / WALKS;
    const Walk& w = walks.w[WALKS == 1 ? 0 : blockIdx.x % WALKS];
    const bool back = WALKS > 1 && w.back, wide = WALKS > 1 && w.o32;  // (the forward is one walk, forward in time, into bf16)
    const Line line = line_of(p, back, &plan_s);

    // slot of chunk `it`'s tile, and how often that slot has been used before
    const uint32_t bar0 = sb + K::oBar;
    auto full = [&](int slot) { return bar0 + 8 * slot; };
    auto empty = [&](int slot) { return bar0 + 8 * (K::SLOTS + slot); };
    auto slot_x = [&](int it) { return it % K::NX; };
    auto slot_y = [&](int it) { return K::NX + it % K::NY; };
    auto slot_z = [&](int it) { return K::NX + K::NY + it % K::NZ; };
    auto turn = [&](int it, int n) { return (uint32_t)(it / n & 1); };
    const uint32_t more_bars = bar0 + 16 * K::SLOTS;
    const uint32_t p_full = more_bars, p_ready = more_bars + 8, o_full = more_bars + 16, o_free = more_bars + 24,
                   s_ready = more_bars + 32, s_free = more_bars + 40, y_ready = more_bars + 48, d_full = more_bars + 56,
                   half_out = more_bars + 64, ended = more_bars + 72, ended_3 = more_bars + 80 + 16 * K::NX,
                   tab_free = ended_3 + 8, tab_ready = ended_3 + 16;
    // (group A may be chunks ahead of the stores: a barrier for each of X's slots, and each half of a wide output)
    auto staged = [&](int it, int half) { return more_bars + 80 + 16 * slot_x(it) + 8 * half; };
    if (tid == 64) {  // (beside the warp that makes the plan)
        // (Y's slots are given back by P's product and by group B's eight warps, Z's by the products of both issuers)
        for (int i = 0; i < K::SLOTS; ++i) {
            tc::mbar_set(full(i), 1);
            tc::mbar_set(empty(i), i < K::NX ? 1 : i < K::NX + K::NY ? 9 : 2);
        }
        tc::mbar_set(p_full, 1);
        tc::mbar_set(p_ready, 8);
        tc::mbar_set(o_full, 2);  // P Z and X C
        tc::mbar_set(o_free, 8);
        tc::mbar_set(s_ready, 8);
        tc::mbar_set(s_free, 1);
        tc::mbar_set(y_ready, 8);
        tc::mbar_set(d_full, 1);
        for (int i = 0; i < 2 * K::NX; ++i) tc::mbar_set(staged(0, 0) + 8 * i, wide && D == 128 ? 4 : 8);
        tc::mbar_set(half_out, 1);
        tc::mbar_set(ended, 1);
        tc::mbar_set(ended_3, 1);
        tc::mbar_set(tab_free, 8);
        tc::mbar_set(tab_ready, 8);
        tc::mbar_set_fence();
        gone_s = 0;
    }
    if (warp == 1) tc::alloc(smem_u32(&tslot), 512);
    make_plan<K::THREADS>(line, range, p.ranges, p.mode, &plan_s, scratch);
    // (blocks without a range begin with the first chains of the queue, a chain each)
    const int first_chain = range - plan_s.ranges;
    const bool queued = plan_s.f0 == plan_s.f1 && first_chain >= 0 && first_chain < plan_s.chains;
    if (tid == 0 && queued) plan_s.at = line.chain(first_chain);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tslot;
    const Waiter wait{&gone_s, p.status};
    if (plan_s.total < 0 && tid == 0) atomicOr(p.status, ST_BAD_SEQLENS);
    const bool any = queued || more(plan_s, plan_s.at, plan_s.f, p.mode);


    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(K::REGS_1));
        if (warp == 0 && lane == 0 && any) {
            // ---------------- loader ----------------
            tc::prefetch_map(&w.X);
            tc::prefetch_map(&w.Y);
            tc::prefetch_map(&w.Z);
            int it = 0;
            bool on[3] = {};  // copies issued into Y's, X's, Z's slots in the last turn that was begun
            const Plan& plan = plan_s;
            Place at = plan.at;
            bool go_on = true;
            bool in_line = plan.f0 < plan.f1;
            int f = plan.f, taken = -1;
            auto take = [&]() { return p.ranges - plan.ranges + atomicAdd(p.taken + (WALKS == 1 ? 0 : blockIdx.x % WALKS), 1); };
#pragma unroll 1
            for (; go_on; ++it) {
                const int t0 = line.token(at), h0 = at.head;
                int4 c = make_int4(t0, line.rows(at), h0, at.seq * p.H + h0);
                if (at.pos == 0 && w.init && it)  // (the chain's state will be asked for soon)
                    tc::prefetch_l2(w.init + (int64_t)c.w * D * D, D * D * sizeof(float));
                if (at.pos + 1 == at.count) c.y |= Chunk::ENDS;
                if (in_line) {
                    line.next(at, f);
                    go_on = more(plan, at, f, p.mode);
                } else {
                    go_on = ++at.pos < at.count;
                }
                if (plan.chains) {  // (the next chain is asked for a chunk ahead)
                    if (taken < 0 && (!go_on || (in_line ? f + 2 >= plan.f1 : at.pos + 1 == at.count))) taken = take();
                    if (!go_on && taken < plan.chains) {
                        at = line.chain(taken);
                        taken = -1;
                        in_line = false;
                        go_on = true;
                    }
                }
                c.y |= !go_on ? Chunk::LAST : at.pos == 0 ? Chunk::TURNS : 0;
                chunks[it & 7] = c;
                on[0] = on[1] = on[2] = false;
#pragma unroll 1
                for (int j = 0; j < 3; ++j) {
                    const int n = j == 0 ? K::NY : j == 1 ? K::NX : K::NZ, s = j == 0 ? slot_y(it) : j == 1 ? slot_x(it) : slot_z(it);
                    if (it >= n && !wait(empty(s), turn(it, n) ^ 1)) break;
                    const CUtensorMap* m = j == 0 ? &w.Y : j == 1 ? &w.X : &w.Z;
                    const int h = h0 / (j == 0 ? w.gy : j == 1 ? w.gx : w.gz);
                    tc::mbar_expect_tx(full(s), K::TILE);
                    tc::tma_load_4d(sb + s * K::TILE, m, 0, h, t0, 0, full(s));
                    on[j] = true;
                }
                if (!wait.ok()) break;
            }
            if (!wait.ok()) {  // (the block gave up: its copies have to land before it ends)
                auto landed = [&](int last, int n, int which) {
#pragma unroll 1
                    for (int i = last - n + 1 > 0 ? last - n + 1 : 0; i <= last; ++i)
                        tc::mbar_wait(full(which == 0 ? slot_y(i) : which == 1 ? slot_x(i) : slot_z(i)), turn(i, n));
                };
                landed(on[0] ? it : it - 1, K::NY, 0);
                landed(on[1] ? it : it - 1, K::NX, 1);
                landed(on[2] ? it : it - 1, K::NZ, 2);
            }
        } else if ((warp == 1 || warp == 3) && any) {
            // ---------------- issuers (whole warps, converged; lane 0 issues) ----------------
            // A warp that waits, commits or fences issues no product (60 to 120 cycles each, against 64 for a product
            // of 16 of the inner dimension, and products do not queue up): two share them, P's chain and the state's.
            const uint32_t on = lane == 0;
            const uint32_t tP = tmem, tO1 = tmem + 128, tO2 = tmem + 256, tD = tmem + 384;
            constexpr uint32_t idP = tc::idesc(128, 128, 0, 0), idO = tc::idesc(128, D, 0, 1), idS = tc::idesc(128, D, 0, 0);
#pragma unroll 1
            for (int it = 0;; ++it) {
                const int sx = slot_x(it), sy = slot_y(it), sz = slot_z(it);
                const uint32_t X = sb + sx * K::TILE, Y = sb + sy * K::TILE, Z = sb + sz * K::TILE;
                const uint32_t ph = it & 1;
                if (warp == 1) {
                    if (!wait.warp(full(sy), turn(it, K::NY)) || !wait.warp(full(sx), turn(it, K::NX))) break;
                    if (it && !wait.warp(o_full, ph ^ 1)) break;  // (P Z of the chunk before has read P)
                    tc::fence_after();
#pragma unroll 1
                    for (int k = 0; k < D; k += 16) tc::mma_if(on, tP, tc::kdesc(X, CHUNK, 0, k), tc::kdesc(Y, CHUNK, 0, k), idP, k > 0);
                    tc::commit_if(on, p_full);
                    tc::commit_if(on, empty(sy));
                    if (!wait.warp(full(sz), turn(it, K::NZ))) break;
                    if ((it && !wait.warp(o_free, ph ^ 1)) || !wait.warp(p_ready, ph)) break;
                    tc::fence_after();
                    // (bf16 P: the 32 columns of slice s lie in the first 16 of the 32 that held them in fp32)
#pragma unroll 1
                    for (int k = 0; k < CHUNK; k += 16) tc::mma_ts_if(on, tO1, tP + (k & ~31) + (k & 31) / 2, tc::mdesc(Z, CHUNK, 0, k), idO, k > 0);
                } else {
                    if (!wait.warp(full(sz), turn(it, K::NZ)) || !wait.warp(y_ready, ph)) break;
                    tc::fence_after();
                    issue_terms<D>(on, tD, sb + K::oHi, sb + K::oLo, Z);
                    tc::commit_if(on, d_full);
                    tc::commit_if(on, empty(sz));
                    if (!wait.warp(full(sx), turn(it, K::NX)) || !wait.warp(s_ready, ph) || (it && !wait.warp(o_free, ph ^ 1))) break;
                    tc::fence_after();
#pragma unroll 1
                    for (int k = 0; k < D; k += 16) tc::mma_if(on, tO2, tc::kdesc(X, CHUNK, 0, k), tc::kdesc(sb + K::oS, D, 0, k), idS, k > 0);
                    tc::commit_if(on, s_free);
                }
                tc::commit_if(on, o_full);
                if (warp == 1) tc::commit_if(on, empty(sz));
                if (__any_sync(~0u, chunk_at(chunks, it).last())) break;
            }
            if (!wait.ok()) {  // (the products in flight have to end before the tensor memory is given back)
                tc::commit_if(on, warp == 1 ? ended : ended_3);
                tc::mbar_wait(warp == 1 ? ended : ended_3, 0);
            }
        } else if (warp == 2 && lane == 0 && any) {
            // ---------------- stores ----------------
#pragma unroll 1
            for (int it = 0;; ++it) {
                const uint32_t X = sb + slot_x(it) * K::TILE;
                if (wide) {
                    if (!wait(staged(it, 0), turn(it, K::NX))) break;
                    const Chunk now = chunk_at(chunks, it);
                    const bool whole = now.tokens() == CHUNK;
                    auto put = [&](int half, uint32_t from) {
                        if (whole) tc::tma_store_4d(&w.out, 0, now.head, now.t0, half * (D / 64), from);
                    };
                    auto out = [&]() {
                        tc::bulk_commit();
                        tc::bulk_wait_read();
                        tc::mbar_arrive(half_out);
                    };
                    if (D == 64) {
                        tc::mbar_arrive(empty(slot_x(it)));
                        put(0, sb + K::oWide);
                        put(1, sb + K::oWide + K::TILE);
                        out();
                    } else {
                        put(0, X);
                        out();
                        if (!wait(staged(it, 1), turn(it, K::NX))) break;
                        put(1, X);
                        tc::bulk_commit();
                        tc::bulk_wait_read();
                        tc::mbar_arrive(empty(slot_x(it)));
                    }
                    if (now.last()) break;
                    continue;
                }
                if (!wait(staged(it, 0), turn(it, K::NX))) break;
                const Chunk now = chunk_at(chunks, it);
                if (now.tokens() == CHUNK) {
                    tc::tma_store_4d(&w.out, 0, now.head, now.t0, 0, X);
                    tc::bulk_commit();
                    tc::bulk_wait_read();
                }
                tc::mbar_arrive(empty(slot_x(it)));
                if (now.last()) break;
            }
        }
    } else if (warp < 12) {
        // ---------------- group A: P, outputs ----------------
        // two warps for each 32 rows: of P's slices of 32 columns one takes 0 and 2, the other 1 and 3; of an output's
        // columns each takes half
        const int q4 = warp & 3, half = (warp - 4) >> 2, i = 32 * q4 + lane;  // row of the chunk
        const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16);
        // decays: on the diagonal slice D_ij from a table (tab[lane - j + 31], j the column in the slice); elsewhere a
        // factor of the column (cols[j]) times one of the row, neither above 1: forward gamma^{31-j} and
        // gamma^{i - 32 s - 31}, back gamma^j and gamma^{32 s - i}
        float* tab = reinterpret_cast<float*>(smem + K::oTab);
        float* cols = tab + 64;
        int head = -1;
        uint32_t tables = 0;  // heads whose tables have been made
        float r_full = 0.f, g = 0.f, rf0 = 0.f, rf1 = 0.f;
#pragma unroll 1
        for (int it = 0; any; ++it) {
            const uint32_t ph = it & 1;
            if (!wait.warp(full(slot_x(it)), turn(it, K::NX))) break;
            const Chunk now = chunk_at(chunks, it);
            if (now.head != head) {
                head = now.head;
                g = log_decay(p.g, head);
                r_full = w.o_scale * power(g, back ? CHUNK - 1 - i : i + 1);
                const int n0 = back ? 32 * half - i : i - 32 * half - 31, n1 = back ? n0 + 64 : n0 - 64;
                rf0 = n0 >= 0 ? power(g, n0) : 0.f;
                rf1 = n1 >= 0 ? power(g, n1) : 0.f;
                // (barriers with bounded waits, as all: a warp that gives up arrives at none)
                warp_arrive(tab_free);
                if (!wait.warp(tab_free, tables & 1)) break;
                if (warp == 4 || warp == 5) {  // 64 entries
                    const int e = 32 * (warp & 1) + lane, n = back ? 31 - e : e - 31;
                    tab[e] = n >= 0 ? w.p_scale * power(g, n) : 0.f;
                } else if (warp == 6) {
                    cols[lane] = w.p_scale * power(g, back ? lane : 31 - lane);
                }
                warp_arrive(tab_ready);
                if (!wait.warp(tab_ready, tables++ & 1)) break;
            }
            const int rows = now.tokens();
            if (!wait.warp(p_full, ph)) break;
            tc::fence_after();
#pragma unroll 1
            for (int s = half; s < 4; s += 2) {
                const float rf = s < 2 ? rf0 : rf1;
                uint32_t out[16];
                if (back ? s < q4 : s > q4) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[j] = 0;
                } else {
                    float v[32];
                    tc::ld32(lanes + 32 * s, v);
                    if (s == q4) {
                        const float* d = tab + lane + 31;
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] *= d[-j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 c = *reinterpret_cast<const float4*>(cols + j);
                            ACC2(v, j, __fmul2_rn(__fmul2_rn(F2(v, j), make_float2(c.x, c.y)), make_float2(rf, rf)));
                            ACC2(v, j + 2, __fmul2_rn(__fmul2_rn(F2(v, j + 2), make_float2(c.z, c.w)), make_float2(rf, rf)));
                        }
                    }
                    if (rows < CHUNK) {
                        // (columns of the next sequence are set to zero, not multiplied by it: they may not be finite)
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 32 * s + j < rows ? v[j] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
                }
                tc::st16u_nowait(lanes + 32 * s, out);
            }
            if (rows < CHUNK) {  // (the rows of Z that belong to the next sequence: each group clears them for its product)
                if (!wait.warp(full(slot_z(it)), turn(it, K::NZ))) break;
                if (i >= rows) clear_row<HALF / 8>(smem + slot_z(it) * K::TILE, i, half * (HALF / 8));
                tc::fence_async_smem();
            }
            tc::st_wait();
            tc::fence_before();
            warp_arrive(p_ready);

            float r = r_full;
            if (back && rows < CHUNK) r = i < rows ? w.o_scale * power(g, rows - 1 - i) : 0.f;
            unsigned char* stage = smem + (wide && D == 64 ? K::oWide + half * K::TILE : slot_x(it) * K::TILE);
            const int64_t row = (int64_t)now.t0 + i;
            if (!wait.warp(o_full, ph)) break;
            // (a wide output's first half has left X's tile; the last chunk's output has left its own)
            if (wide && (D == 64 ? it && !wait.warp(half_out, ph ^ 1) : half == 1 && !wait.warp(half_out, ph))) break;
            tc::fence_after();
#pragma unroll 1
            for (int c = 0; c < HALF; c += 16) {
                const int n = half * HALF + c;
                uint32_t a[16], b[16];
                tc::ld16_nowait(lanes + 128 + n, a);
                tc::ld16_nowait(lanes + 256 + n, b);
                tc::ld_wait(a, b);
                float o[16];
#pragma unroll
                for (int j = 0; j < 16; j += 2)
                    ACC2(o, j, __ffma2_rn(make_float2(r, r), make_float2(__uint_as_float(b[j]), __uint_as_float(b[j + 1])),
                                          make_float2(__uint_as_float(a[j]), __uint_as_float(a[j + 1]))));
                if (wide) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 v = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                        if (rows == CHUNK) *reinterpret_cast<float4*>(stage + tc::sw_chunk(i, c / 4 + j, CHUNK)) = v;
                        else if (i < rows) *reinterpret_cast<float4*>(w.o32 + (row * p.H + head) * D + n + 4 * j) = v;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 v = make_uint4(pack_bf16(o[8 * j], o[8 * j + 1]), pack_bf16(o[8 * j + 2], o[8 * j + 3]),
                                                   pack_bf16(o[8 * j + 4], o[8 * j + 5]), pack_bf16(o[8 * j + 6], o[8 * j + 7]));
                        if (rows == CHUNK) *reinterpret_cast<uint4*>(stage + tc::sw_chunk(i, n / 8 + j, CHUNK)) = v;
                        else if (i < rows) *reinterpret_cast<uint4*>(w.o + (row * p.H + head) * D + n + 8 * j) = v;
                    }
                }
            }
            tc::fence_before();
            warp_arrive(o_free);
            tc::fence_async_smem();
            warp_arrive(staged(it, wide && D == 128 ? half : 0));
            if (now.last()) break;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(K::REGS_B));
        // ---------------- group B: Y', the state ----------------
        // two warps for each 32 tokens of Y and 32 columns of the state (Z's channels, so that what one instruction
        // moves of a state in memory is contiguous), each with half of Y's channels
        const int q4 = warp & 3, half = (warp - 12) >> 2, i = 32 * q4 + lane, col = half * HALF;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16) + 384 + col;
        const bool mine = 32 * q4 < D;  // (warps without columns of the state)
        float S[HALF];  // rows `col` and on of column i
        float g = 0.f, w_full = 0.f;
        float2 c_full = make_float2(0.f, 0.f);
        auto incoming = [&](int chain, int head, bool inside) {
            const float* from = nullptr;
            if (inside) from = w.joined + (int64_t)(range - 1) * p.pieces * D * D;
            else if (w.init) from = w.init + (int64_t)chain * D * D;
            if (from && mine) {
                if (WALKS > 1 && w.turned) {
#pragma unroll
                    for (int c = 0; c < HALF; c += 4) {
                        const float4 u = *reinterpret_cast<const float4*>(from + i * D + col + c);
                        S[c] = u.x, S[c + 1] = u.y, S[c + 2] = u.z, S[c + 3] = u.w;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < HALF; ++c) S[c] = from[(col + c) * D + i];
                }
            } else {
#pragma unroll
                for (int c = 0; c < HALF; ++c) S[c] = 0.f;
            }
            g = log_decay(p.g, head);
            w_full = w.w_scale * power(g, back ? i + 1 : CHUNK - 1 - i);
            c_full = carry(g, CHUNK);
        };
        auto copy_state = [&]() {
            if (mine) {
#pragma unroll
                for (int j = 0; j < HALF / 8; ++j)
                    *reinterpret_cast<uint4*>(smem + K::oS + tc::sw_chunk(i, col / 8 + j, D)) =
                        make_uint4(pack_bf16(S[8 * j], S[8 * j + 1]), pack_bf16(S[8 * j + 2], S[8 * j + 3]),
                                   pack_bf16(S[8 * j + 4], S[8 * j + 5]), pack_bf16(S[8 * j + 6], S[8 * j + 7]));
            }
            tc::fence_async_smem();
            warp_arrive(s_ready);
        };
        cudaGridDependencySynchronize();  // (the states that k_dla_join carries)
        if (any) incoming(plan_s.at.seq * p.H + plan_s.at.head, plan_s.at.head, plan_s.at.pos != 0);
#pragma unroll 1
        for (int it = 0; any; ++it) {
            const uint32_t ph = it & 1;
            if (!wait.warp(full(slot_y(it)), turn(it, K::NY))) break;
            const Chunk now = chunk_at(chunks, it);
            const int rows = now.tokens();
            float wt = w_full;
            float2 c = c_full;
            const unsigned char* tile = smem + slot_y(it) * K::TILE;
            if (rows < CHUNK) {
                wt = w.w_scale * power(g, back ? i + 1 : rows - 1 - i);
                c = carry(g, rows);
                if (!wait.warp(full(slot_z(it)), turn(it, K::NZ))) break;
            }
            // (Y' of the chunk before has been read: this group has waited for its terms)
            if (i >= rows) {
                clear_row<HALF / 8>(smem + K::oHi, i, col / 8);
                clear_row<HALF / 8>(smem + K::oLo, i, col / 8);
                clear_row<HALF / 8>(smem + slot_z(it) * K::TILE, i, col / 8);
            } else {
                split_row<HALF / 8>(tile, smem + K::oHi, smem + K::oLo, i, col / 8, wt);
            }
            tc::fence_async_smem();
            warp_arrive(y_ready);
            if (lane == 0) tc::mbar_arrive(empty(slot_y(it)));
            if (it && !wait.warp(s_free, ph ^ 1)) break;  // (X C of the chunk before has read the copy)
            copy_state();
            if (!wait.warp(d_full, ph)) break;
            tc::fence_after();
            if (mine) {
#pragma unroll
                for (int s = 0; s < HALF; s += 16) {
                    uint32_t v[16];
                    tc::ld16_nowait(lanes + s, v);
                    tc::ld_wait(v);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float2 old = F2(S, s + j);
                        const float2 t = __ffma2_rn(make_float2(c.x, c.x), old, make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])));
                        ACC2(S, s + j, __ffma2_rn(make_float2(c.y, c.y), old, t));
                    }
                }
            }
            tc::fence_before();
            if (now.ends() && w.last && mine) {
                float* to = w.last + ((int64_t)now.chain * D + col) * D + i;
#pragma unroll
                for (int j = 0; j < HALF; ++j) to[j * D] = S[j];
            }
            if (now.last()) break;
            if (now.turns()) {
                if (!wait.warp(full(slot_y(it + 1)), turn(it + 1, K::NY))) break;
                const Chunk next = chunk_at(chunks, it + 1);
                incoming(next.chain, next.head, false);
            }
        }
    }
    // empty sequences pass their states through, chain by chain shared by all blocks
    if (w.last && plan_s.total >= 0 && p.cu) {
        const int chains = p.N * p.H;
#pragma unroll 1
        for (int c = range; c < chains; c += p.ranges) {
            if (p.cu[c / p.H] != p.cu[c / p.H + 1]) continue;
            const float4* from = reinterpret_cast<const float4*>(w.init + (int64_t)c * D * D);
            float4* to = reinterpret_cast<float4*>(w.last + (int64_t)c * D * D);
#pragma unroll 4
            for (int e = tid; e < D * D / 4; e += K::THREADS) to[e] = w.init ? from[e] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) tc::dealloc(tmem, 512);
}

struct TailWalk {
    CUtensorMap Y, Z;
    int gy, gz, back;
    float w_scale;
    float* sums;        // [ranges][pieces][D][D]
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
    int f = plan.f;
#pragma unroll 1
    while (f + (at.count - at.pos) + 1 < plan.f1) {
        f += at.count - 1 - at.pos;
        at.pos = at.count - 1;
        line.next(at, f);
    }
    t.first = at;
    t.last = at;
    t.last.pos = at.pos + (plan.f1 - 1 - f);
    if (f < plan.f1 && t.last.pos + 1 < at.count) t.chunks = plan.f1 - f;
    return t;
}

// the chunks of the last chain's part, counted from its end, that piece `piece` sums
__device__ __forceinline__ int piece_begin(int chunks, int piece, int pieces) { return chunks * piece / pieces; }

// For each range the sum of its last chain's terms, as the next range's state takes them.  `pieces` blocks share
// one: with more chains than ranges the parts' lengths differ, and short blocks even that out.
template <int D, int WALKS>
__global__ void __launch_bounds__(TailCfg<D>::THREADS, 1) k_dla_tail(const __grid_constant__ TailWalks<WALKS> walks, const Grid p) {
    using K = TailCfg<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Plan plan_s;
    __shared__ int scratch[K::THREADS / 32];
    __shared__ int gone_s;
    __shared__ uint32_t tslot;
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int piece = blockIdx.x % p.pieces, range = blockIdx.x / p.pieces / WALKS;
    const TailWalk& w = walks.w[WALKS == 1 ? 0 : blockIdx.x / p.pieces % WALKS];
    const Line line = line_of(p, w.back, &plan_s);
    make_plan<K::THREADS>(line, range, p.ranges, RANGES, &plan_s, scratch);
    const Tail tail = tail_of(line, plan_s);
    const int begin = piece_begin(tail.chunks, piece, p.pieces), stop = piece_begin(tail.chunks, piece + 1, p.pieces);
    if (begin == stop) return;
    const uint32_t bar0 = sb + K::oBar;
    auto full = [&](int slot) { return bar0 + 8 * slot; };
    auto empty = [&](int slot) { return bar0 + 8 * (K::RING + slot); };
    const uint32_t y_ready = bar0 + 16 * K::RING, d_full = y_ready + 16 /* two each */, ended = d_full + 16;
    if (tid == 0) {
        for (int i = 0; i < 2 * K::RING; ++i) tc::mbar_set(bar0 + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_set(y_ready + 8 * i, 8);
            tc::mbar_set(d_full + 8 * i, 1);
        }
        tc::mbar_set(ended, 1);
        tc::mbar_set_fence();
        gone_s = 0;
    }
    if (warp == 1) tc::alloc(smem_u32(&tslot), 256);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tslot;
    const Waiter wait{&gone_s, p.status};
    const float g = log_decay(p.g, tail.first.head);
    const int end = line.before(tail.first, tail.last.pos + 1);  // tokens of the chain before the next range
    // chunk `it` of the walk: from the piece's last one backwards, as long as any decay is left
    auto chunk = [&](int it, Place& at) {
        at = tail.last;
        at.pos -= begin + it;
        return begin + it < stop && power(g, end - line.before(at, at.pos + 1)) != 0.f;
    };
    auto slot_of = [&](int l) { return l % K::RING; };
    auto parity_of = [&](int l) { return (uint32_t)((l / K::RING) & 1); };
    Place at;
    if (warp == 0 && lane == 0) {
        int l = 0;
#pragma unroll 1
        for (int it = 0; chunk(it, at); ++it) {
            const int t0 = line.token(at);
#pragma unroll
            for (int j = 0; j < 2; ++j, ++l) {
                const int s = slot_of(l);
                if (l >= K::RING && !wait(empty(s), parity_of(l) ^ 1)) break;
                tc::mbar_expect_tx(full(s), K::TILE);
                tc::tma_load_4d(sb + s * K::TILE, j ? &w.Z : &w.Y, 0, at.head / (j ? w.gz : w.gy), t0, 0, full(s));
            }
            if (!wait.ok()) break;
        }
        if (!wait.ok())
#pragma unroll 1
            for (int i = l > K::RING ? l - K::RING : 0; i < l; ++i) tc::mbar_wait(full(slot_of(i)), parity_of(i));
    } else if (warp == 1) {
        const uint32_t on = lane == 0;
#pragma unroll 1
        for (int it = 0; __any_sync(~0u, chunk(it, at)); ++it) {
            const int b = it & 1;
            const uint32_t ph = (it >> 1) & 1;
            const uint32_t y = sb + slot_of(2 * it) * K::TILE, z = sb + slot_of(2 * it + 1) * K::TILE;
            if (!wait.warp(full(slot_of(2 * it + 1)), parity_of(2 * it + 1)) || !wait.warp(y_ready + 8 * b, ph)) break;
            tc::fence_after();
            issue_terms<D>(on, tmem + 128 * b, y, sb + K::oLo + b * K::TILE, z);
            tc::commit_if(on, d_full + 8 * b);
            tc::commit_if(on, empty(slot_of(2 * it)));
            tc::commit_if(on, empty(slot_of(2 * it + 1)));
        }
        if (!wait.ok()) {
            tc::commit_if(on, ended);
            tc::mbar_wait(ended, 0);
        }
    } else if (warp >= 4) {
        constexpr int HALF = D / 2;
        const int q4 = warp & 3, half = (warp - 4) >> 2, i = 32 * q4 + lane, col = half * HALF;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16) + col;
        const bool mine = 32 * q4 < D;
        float S[HALF];
#pragma unroll
        for (int c = 0; c < HALF; ++c) S[c] = 0.f;
        auto bring = [&](int it) {
            Place c;
            if (!chunk(it, c)) return false;
            const int rows = line.rows(c), l = 2 * it;
            // tokens of the walk from token i on to the next range's first
            const int away = end - line.before(c, c.pos) - (w.back ? rows - 1 - i : i);
            const float wt = w.w_scale * power(g, w.back ? away : away - 1);
            unsigned char *tile = smem + slot_of(l) * K::TILE, *lo = smem + K::oLo + (it & 1) * K::TILE;
            if (!wait.warp(full(slot_of(l)), parity_of(l))) return false;
            if (rows < CHUNK && !wait.warp(full(slot_of(l + 1)), parity_of(l + 1))) return false;
            if (i < rows) {
                split_row<HALF / 8>(tile, tile, lo, i, col / 8, wt);
            } else {
                clear_row<HALF / 8>(tile, i, col / 8);
                clear_row<HALF / 8>(lo, i, col / 8);
                clear_row<HALF / 8>(smem + slot_of(l + 1) * K::TILE, i, col / 8);
            }
            tc::fence_async_smem();
            warp_arrive(y_ready + 8 * (it & 1));
            return true;
        };
        bool on = bring(0);
#pragma unroll 1
        for (int it = 0; on; ++it) {
            on = bring(it + 1);
            if (!wait.warp(d_full + 8 * (it & 1), (it >> 1) & 1)) break;
            tc::fence_after();
            if (mine) {
#pragma unroll
                for (int s = 0; s < HALF; s += 32) {
                    uint32_t v0[16], v1[16];
                    tc::ld16_nowait(lanes + 128 * (it & 1) + s, v0);
                    tc::ld16_nowait(lanes + 128 * (it & 1) + s + 16, v1);
                    tc::ld_wait(v0, v1);
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const uint32_t* v = (j < 16 ? v0 : v1) + j % 16;
                        ACC2(S, s + j, __fadd2_rn(F2(S, s + j), make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]))));
                    }
                }
            }
            tc::fence_before();
        }
        if (mine && wait.ok()) {
            float* to = w.sums + (((int64_t)range * p.pieces + piece) * D + col) * D + i;
#pragma unroll
            for (int j = 0; j < HALF; ++j) to[j * D] = S[j];
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) tc::dealloc(tmem, 256);
}

// The states at the beginnings of ranges that begin inside a chain, in the place of the first piece of the sum of
// the range before: along each such chain, from its initial state.  A few blocks a state (most blocks have
// nothing to do and have to end soon), the sums of four ranges asked for together.
constexpr int JOIN_THREADS = 256;
template <int D>
__host__ __device__ constexpr int join_slices() { return D == 128 ? 8 : 2; }
template <int D, int WALKS>
__global__ void __launch_bounds__(JOIN_THREADS) k_dla_join(const __grid_constant__ TailWalks<WALKS> walks, const Grid p) {
    constexpr int SLICES = join_slices<D>(), AHEAD = 4, QUADS = D * D / SLICES / (4 * JOIN_THREADS);  // float4 of a thread
    __shared__ Plan plan_s;
    __shared__ int scratch[JOIN_THREADS / 32];
    const int slice = blockIdx.x % SLICES, which = blockIdx.x / SLICES % WALKS, range = blockIdx.x / SLICES / WALKS + 1;
    const TailWalk& w = walks.w[which];
    const Line line = line_of(p, w.back, &plan_s);
    make_plan<JOIN_THREADS>(line, range, p.ranges, RANGES, &plan_s, scratch);
    const Plan& plan = plan_s;
    cudaGridDependencySynchronize();  // (the sums of k_dla_tail)
    if (plan.total <= 0 || plan.f0 >= plan.f1 || plan.at.pos == 0) return;
    const Place at = plan.at;
    const int first = plan.f0 - at.pos, stop = first + at.count;  // the places of the chain's chunks
    if (range_begin(plan.total, range - 1, plan.ranges) > first) return;  // (the chain's first crossing does them all)
    const float g = log_decay(p.g, at.head);
    const int e = slice * (D * D / SLICES) + threadIdx.x * 4;
    float4 s[QUADS] = {};
    if (w.init) {
        const float* from = w.init + ((int64_t)at.seq * p.H + at.head) * D * D + e;
#pragma unroll
        for (int q = 0; q < QUADS; ++q) s[q] = *reinterpret_cast<const float4*>(from + q * 4 * JOIN_THREADS);
    }
    int done = 0;
#pragma unroll 1
    for (int r0 = range; r0 < plan.ranges && range_begin(plan.total, r0, plan.ranges) < stop; r0 += AHEAD) {
        float4 t[AHEAD][QUADS] = {};
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int r = r0 + u, f = range_begin(plan.total, r, plan.ranges);
            if (r >= plan.ranges || f >= stop) continue;
            const int chunks = f - max(first, range_begin(plan.total, r - 1, plan.ranges));
            const float* from = w.sums + (int64_t)(r - 1) * p.pieces * D * D + e;
#pragma unroll 1
            for (int k = 0; k < p.pieces; ++k) {
                if (piece_begin(chunks, k, p.pieces) == piece_begin(chunks, k + 1, p.pieces)) continue;
#pragma unroll
                for (int q = 0; q < QUADS; ++q) {
                    const float4 v = *reinterpret_cast<const float4*>(from + (int64_t)k * D * D + q * 4 * JOIN_THREADS);
                    t[u][q] = make_float4(t[u][q].x + v.x, t[u][q].y + v.y, t[u][q].z + v.z, t[u][q].w + v.w);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int r = r0 + u, f = range_begin(plan.total, r, plan.ranges);
            if (r >= plan.ranges || f >= stop) break;
            const int upto = line.before(at, f - first);
            const float2 c = carry(g, upto - done);
            done = upto;
            float* to = w.sums + (int64_t)(r - 1) * p.pieces * D * D + e;
#pragma unroll
            for (int q = 0; q < QUADS; ++q) {
                s[q] = make_float4(fmaf(c.y, s[q].x, fmaf(c.x, s[q].x, t[u][q].x)), fmaf(c.y, s[q].y, fmaf(c.x, s[q].y, t[u][q].y)),
                                   fmaf(c.y, s[q].z, fmaf(c.x, s[q].z, t[u][q].z)), fmaf(c.y, s[q].w, fmaf(c.x, s[q].w, t[u][q].w)));
                *reinterpret_cast<float4*>(to + q * 4 * JOIN_THREADS) = s[q];
            }
        }
    }
}

// The gradients of shared heads: sums over the value heads of a group, in fp32; dq and dk (blockIdx.y), four channels a thread.
// (Nothing where the sequences' borders are inconsistent: the walks have written no gradients to add up.)
__global__ void __launch_bounds__(256) k_dla_groups(const float* dq_heads, const float* dk_heads, __nv_bfloat16* dq, __nv_bfloat16* dk, int64_t quads,
                                                    int group, int D, const int* status) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= quads || (*status & ST_BAD_SEQLENS)) return;
    const int per = D / 4;
    const int64_t row = i / per;  // (token, k head)
    const float* from = (blockIdx.y ? dk_heads : dq_heads) + (row * group * per + (i - row * per)) * 4;
    float4 s = *reinterpret_cast<const float4*>(from);
    for (int j = 1; j < group; ++j) {
        const float4 u = *reinterpret_cast<const float4*>(from + (int64_t)j * D);
        s = make_float4(s.x + u.x, s.y + u.y, s.z + u.z, s.w + u.w);
    }
    reinterpret_cast<uint2*>(blockIdx.y ? dk : dq)[i] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
}

// How a call's chunks are shared out: the number of ranges (of each walk), what they are, and the blocks that share the
// sum of a range's last chain.
struct Shares {
    int ranges;
    Mode mode;
    int pieces;
};
Shares shares_of(const DlaParams& p, int walks) {
    const int64_t chains = (int64_t)p.N * p.H;
    const int64_t longest = p.cu_seqlens ? (p.T + CHUNK - 1) / CHUNK : (p.seq_len + CHUNK - 1) / CHUNK;
    const int64_t most = p.cu_seqlens ? (p.T / CHUNK + p.N) * p.H : longest * chains;
    const int sms = num_sms();
    int64_t fit = sms / walks > 0 ? sms / walks : 1;
    // Chains of four chunks are walked whole (10 sequences of 512, 16 heads: ranges 50 us, whole chains 35).
    const int all_chains = (int)(chains < fit ? chains : fit);
    if (longest <= 4) return {all_chains, p.cu_seqlens ? SNAP : WHOLE, 1};
    // Ranges of at least four chunks: against two, 900 tokens of 8 heads 33 us (29), 16384 of one head 87 (93), the backward
    // of 4096 of 4 heads 43 (52).
    const int64_t ranges = (most + 3) / 4;
    Shares sh{(int)(ranges < fit ? ranges : fit), RANGES, 1};
    if (!p.cu_seqlens) {
        const int64_t places = longest + 1;
        if (short_enough((chains + sh.ranges - 1) / sh.ranges * places, chains * places / sh.ranges)) return {all_chains, WHOLE, 1};
    }
    // The sums of the ranges' last chains: with more chains than ranges they are of all lengths, and two blocks each even
    // that out (30011 tokens in 8 sequences, 32 heads: 263 us with one, 240 with two, 246 with four); else as many as end
    // soonest, at 1.5 us a chunk and 2.5 us for each more sum that the join adds (T = 32768, 16 heads: three for the
    // backward's two sums of 49 ranges each, two rounds of a third, 75 us where one took 105; one forward, where two would
    // take 13 us more.  4096 tokens of 4 heads, chains of 32 chunks: two, 44 us, against one 48 and four 49).
    if (chains > fit) {
        sh.pieces = 2;
    } else {
        const int blocks = (sh.ranges - 1) * (walks == 1 ? 1 : 2);
        const double chunks = (double)most / sh.ranges;
        double best = 1e30;
        for (int n = 1; n <= 4; ++n) {
            const double us = 1.5 * chunks * ((blocks * n + sms - 1) / sms) / n + 2.5 * n;
            if (us < best) best = us, sh.pieces = n;
        }
    }
    return sh;
}

// Launches a kernel whose blocks may be in place before the kernel ahead of it has ended: it waits for that one itself
// (cudaGridDependencySynchronize) before it reads what that has written.
template <class... P, class... A>
cudaError_t launch_after(unsigned grid, unsigned threads, size_t smem, cudaStream_t s, void (*kernel)(P...), const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int WALKS, int TAILS>
cudaError_t go(const DlaParams& p, const Shares& sh, const Walks<WALKS>& walks, const TailWalks<TAILS>& tails, cudaStream_t s) {
    const Grid grid{p.N, p.H, D, sh.ranges, sh.mode, sh.pieces, p.T, p.seq_len, p.cu_seqlens, p.g, p.status, p.status + 1};
    cudaError_t e = cudaMemsetAsync(p.status, 0, 256, s);
    if (e != cudaSuccess) return e;
    static bool allowed[64], allowed_tail[64];
    e = allow_smem((const void*)k_dla<D, WALKS>, Cfg<D>::SMEM, allowed);
    if (e != cudaSuccess) return e;
    // (the groups' shares of the registers have to be there at the launch)
    static const int regs = [] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, k_dla<D, WALKS>) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs != Cfg<D>::REGS) return cudaErrorInvalidConfiguration;
    if (sh.mode == RANGES && sh.ranges > 1) {
        e = allow_smem((const void*)k_dla_tail<D, TAILS>, TailCfg<D>::SMEM, allowed_tail);
        if (e != cudaSuccess) return e;
        k_dla_tail<D, TAILS><<<(sh.ranges - 1) * TAILS * sh.pieces, TailCfg<D>::THREADS, TailCfg<D>::SMEM, s>>>(tails, grid);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = launch_after((sh.ranges - 1) * TAILS * join_slices<D>(), JOIN_THREADS, 0, s, k_dla_join<D, TAILS>, tails, grid);
        if (e == cudaSuccess) e = launch_after(sh.ranges * WALKS, Cfg<D>::THREADS, Cfg<D>::SMEM, s, k_dla<D, WALKS>, walks, grid);
        return e;
    }
    k_dla<D, WALKS><<<sh.ranges * WALKS, Cfg<D>::THREADS, Cfg<D>::SMEM, s>>>(walks, grid);
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
bool make_walk(Walk* w, const DlaParams& p, const Tensor& x, const Tensor& y, const Tensor& z, void* out, int out_heads, float* out32) {
    w->gx = p.H / x.heads, w->gy = p.H / y.heads, w->gz = p.H / z.heads;
    w->o = static_cast<__nv_bfloat16*>(out);
    w->o32 = out32;
    if (!encode(&w->X, x, p) || !encode(&w->Y, y, p) || !encode(&w->Z, z, p)) return false;
    return out32 ? encode_heads_f32_map(&w->out, out32, p.T, p.H, p.D, CHUNK) : encode(&w->out, Tensor{out, out_heads, (int64_t)out_heads * p.D}, p);
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
    if (!make_walk(&o, p, q, k, v, p.o, p.H, nullptr)) return cudaErrorInvalidValue;
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
    if (!make_walk(&dq, p, dO, v, k, p.dq, p.Hk, p.dq_heads) || !make_walk(&dk, p, v, dO, q, p.dk, p.Hk, p.dk_heads) ||
        !make_walk(&dv, p, k, q, dO, p.dv, p.H, nullptr))
        return cudaErrorInvalidValue;
    float* back = p.states + (size_t)sh.ranges * sh.pieces * D * D;
    dq.turned = 1, dq.p_scale = dq.o_scale = p.scale, dq.w_scale = 1.f;
    dq.init = p.h0, dq.joined = p.states;
    dk.turned = 1, dk.back = 1, dk.p_scale = dk.w_scale = p.scale, dk.o_scale = 1.f;
    dk.init = p.dht, dk.joined = back;
    dv.back = 1, dv.p_scale = dv.w_scale = p.scale, dv.o_scale = 1.f;
    dv.init = p.dht, dv.joined = back, dv.last = p.dh0;
    t.w[0] = TailWalk{dq.Z, dq.Y, dq.gz, dq.gy, 0, 1.f, p.states, p.h0};
    t.w[1] = TailWalk{dv.Y, dv.Z, dv.gy, dv.gz, 1, p.scale, back, p.dht};
    cudaError_t e = go<D, 3, 2>(p, sh, w, t, s);
    if (e != cudaSuccess || !p.dq_heads) return e;
    const int64_t quads = p.T * p.Hk * D / 4;
    k_dla_groups<<<dim3((unsigned)((quads + 255) / 256), 2), 256, 0, s>>>(p.dq_heads, p.dk_heads, p.dq, p.dk, quads, p.H / p.Hk, D, p.status);
    return cudaGetLastError();
}

}  // namespace

size_t dla_states_bytes(const DlaParams& p, bool backward) {
    const Shares sh = shares_of(p, backward ? 3 : 1);
    return sh.mode != RANGES || sh.ranges < 2 ? 0 : (backward ? 2 : 1) * sizeof(float) * (size_t)sh.ranges * sh.pieces * p.D * p.D;
}
int dla_kernels(const DlaParams& p, bool backward) {
    const Shares sh = shares_of(p, backward ? 3 : 1);
    return (sh.mode != RANGES || sh.ranges < 2 ? 1 : 3) + (backward && p.H != p.Hk ? 1 : 0);
}

cudaError_t launch_dla_fwd(const DlaParams& p, cudaStream_t s) { return p.D == 64 ? forward<64>(p, s) : forward<128>(p, s); }
cudaError_t launch_dla_bwd(const DlaParams& p, cudaStream_t s) { return p.D == 64 ? backward<64>(p, s) : backward<128>(p, s); }

}  // namespace gdr
