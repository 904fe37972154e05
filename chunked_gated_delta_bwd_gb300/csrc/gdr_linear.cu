// The product of e4m3 operands with a scale for each block of 128 of the inner dimension:
//
//   y[m, n] = bias[n] + sum_b xs[m, b] ws[n / 128, b] sum_{k in b} x[m, k] w[n, k]
//
// The scales are any fp32 numbers, so the tensor cores cannot apply them: each block's product (four
// steps of 32 of the inner dimension) goes into tensor memory by itself, and groups of threads add it, times its scale,
// to sums in fp32 registers while the next blocks' products run into other columns of the tensor memory.
//
// What bounds it with many rows is no part alone.  32768 x 2048 x 6144 takes 305 us, 2.7 PFLOP/s (340 in a long loop, under the
// power cap), with the tensor cores at 59% of their cycles (512 for 128 x 256 sums of a block of 128).  Copies of the kernel that
// leave out the sums take 288, the tiles' loads (4.8 GB from the second-level cache, 16 TB/s) 283, both 256: what is left then
// is products and the hand-over of two accumulators between the warps that issue and those that add.
//
// Two forms, the same loop:
//   rows of x as the product's rows  (many rows of x): a thread holds one row, its scale is one number; blocks
//       walk the tiles, and the output leaves through shared memory by TMA.
//   rows of w as the product's rows  (up to 64 rows of x, decoding): the weights' bytes bound it; the tile is 128 outputs by
//       all rows of x, and a thread holds one output, its scales come from shared memory.
// Where there are fewer tiles than multiprocessors the inner dimension is split over the blocks of a cluster (up
// to 8), which add up their parts through one another's shared memory in a fixed order.
#include "gdr_common.cuh"
#include "gdr_e4m3.h"
#include "gdr_internal.h"
#include "gdr_tc.cuh"
#include "gdr_tma.h"

namespace gdr {
namespace {

constexpr int KB = 128;  // inner block

// X_ROWS: rows of x as the product's rows; BN: its columns
template <bool X_ROWS, int BN>
struct Lin {
    static constexpr int GROUPS = BN >= 128 ? 2 : 1, COLS = BN / GROUPS, THREADS = 128 + 128 * GROUPS;
    static constexpr int A = 128 * KB, B = BN * KB, STAGE = A + B;
    static constexpr int STAGES = BN == 256 ? 3 : BN == 128 ? 6 : BN == 64 ? 8 : BN == 32 ? 5 : 6;
    static constexpr int oStore = STAGES * STAGE;  // (rows of x: 128 x 64 bf16 tiles, COLS / 64 for each group)
    static constexpr int oScale = oStore + (X_ROWS ? BN / 64 * 16384 : 0);
    static constexpr int oBar = oScale + (X_ROWS ? 0 : 2 * 8 * BN * 4);
    // accumulators in tensor memory (with two, what a block's product takes from its issue to its sums is not hidden
    // where products are short: 1024 x 4096 x 2048 took 15.8 us)
    static constexpr int BUFS = BN == 256 ? 2 : 4;
    static constexpr int BARS = 2 * STAGES + 2 * BUFS + 6;
    static constexpr int SMEM = oBar + 8 * BARS + 8 + 1024;
    static constexpr int TMEM = BUFS * BN;
    static constexpr bool MOVE_REGS = BN == 256;  // 64 x 128 + 216 x 256 registers out of the launch's 168 x 384
};

struct Maps {
    CUtensorMap a, b, y;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ float4 ld_peer(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %4, %5;\nld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}\n"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

template <bool X_ROWS, int BN>
__global__ void __launch_bounds__(Lin<X_ROWS, BN>::THREADS, BN <= 32 ? 2 : 1)
    k_linear(const __grid_constant__ Maps maps, const LinearParams p, int tiles_b, int tiles, int split) {
    using L = Lin<X_ROWS, BN>;
    constexpr int COLS = L::COLS;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t tslot;
    __shared__ int gone_s;
    __shared__ volatile int asked_s;  // tiles that the loader has asked for, once it asks for no more
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nkb = (p.K + KB - 1) / KB;
    const int rank = split > 1 ? (int)cluster_rank() : 0;
    const int kb0 = (int)((int64_t)nkb * rank / split), kb1 = (int)((int64_t)nkb * (rank + 1) / split);

    const uint32_t bar0 = sb + L::oBar;
    auto full = [&](int s) { return bar0 + 8 * s; };
    auto empty = [&](int s) { return bar0 + 8 * (L::STAGES + s); };
    const uint32_t t_full = bar0 + 16 * L::STAGES, t_empty = t_full + 8 * L::BUFS, sc_full = t_empty + 8 * L::BUFS, sc_empty = sc_full + 16,
                   ended = sc_empty + 16;
    if (tid == 0) {
        for (int i = 0; i < 2 * L::STAGES; ++i) tc::mbar_set(bar0 + 8 * i, 1);
        for (int i = 0; i < L::BUFS; ++i) {
            tc::mbar_set(t_full + 8 * i, 1);
            tc::mbar_set(t_empty + 8 * i, 4 * L::GROUPS);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_set(sc_full + 8 * i, 32);
            tc::mbar_set(sc_empty + 8 * i, 4 * L::GROUPS);
        }
        for (int i = 0; i < 2; ++i) tc::mbar_set(ended + 8 * i, 1);
        tc::mbar_set_fence();
        gone_s = 0;
        asked_s = -1;
    }
    if (warp == 1) tc::alloc(smem_u32(&tslot), L::TMEM);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tslot;
    // Waits are bounded: one that runs out turns every later wait and issue of the block into nothing, and its outputs into NaN.
    volatile int* gone = &gone_s;
    auto ok = [&]() { return *gone == 0; };
    auto wait = [&](uint32_t bar, uint32_t parity) {  // by one thread
        if (tc::mbar_try(bar, parity)) return true;
#pragma unroll 1
        for (int i = 0; i < 1 << 22; ++i) {
            if (!ok()) return false;
            if (tc::mbar_try(bar, parity)) return true;
        }
        *gone = 1;
        return false;
    };
    auto wait_warp = [&](uint32_t bar, uint32_t parity) {  // by a whole warp, which goes on converged
        if (__all_sync(~0u, tc::mbar_try(bar, parity))) return true;
#pragma unroll 1
        for (int i = 0; i < 1 << 22; ++i) {
            if (__any_sync(~0u, !ok())) return false;
            if (__all_sync(~0u, tc::mbar_try(bar, parity))) return true;
        }
        *gone = 1;
        return false;
    };
    auto landed = [&](int asked) {  // (of a block that gave up: all copies that it asked for)
#pragma unroll 1
        for (int i = asked > L::STAGES ? asked - L::STAGES : 0; i < asked; ++i) tc::mbar_wait(full(i % L::STAGES), i / L::STAGES & 1);
    };
    const int first = blockIdx.x / split, step = gridDim.x / split;

    // (the registers of group sums: 128, and the 64 that come in; all warps of a group of four take part)
    if (warp < 4) {
        if (L::MOVE_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
        if (warp == 0) {
            if (lane == 0) {
                // ---------------- loader ----------------
                tc::prefetch_map(&maps.a);
                tc::prefetch_map(&maps.b);
                int l = 0;
#pragma unroll 1
                for (int t = first; t < tiles && ok(); t += step) {
                    const int a0 = t / tiles_b * 128, b0 = t % tiles_b * BN;
#pragma unroll 1
                    for (int kb = kb0; kb < kb1; ++kb, ++l) {
                        const int s = l % L::STAGES;
                        if (l >= L::STAGES && !wait(empty(s), (l / L::STAGES & 1) ^ 1)) break;
                        tc::mbar_expect_tx(full(s), L::STAGE);
                        tc::tma_load_2d(sb + s * L::STAGE, &maps.a, kb * KB, a0, full(s));
                        tc::tma_load_2d(sb + s * L::STAGE + L::A, &maps.b, kb * KB, b0, full(s));
                    }
                }
                asked_s = l;
                if (!ok()) landed(l);
            }
        } else if (warp == 1 || warp == 3) {
            // ---------------- issuers (whole warps, converged; lane 0 issues) ----------------
            // A warp that waits, commits or fences issues no product (60 to 120 cycles each, 400 a block of 128, against 512
            // for its products of 128 x 256, and products do not queue up): two take the blocks in turn.
            constexpr uint32_t id = tc::idesc_e4m3(128, BN);
            const uint32_t on = lane == 0;
            const int mine = warp == 3;
            int l = 0;
            bool fine = true;
#pragma unroll 1
            for (int t = first; t < tiles && fine; t += step) {
#pragma unroll 1
                for (int kb = kb0; kb < kb1; ++kb, ++l) {
                    if ((l & 1) != mine) continue;
                    const int s = l % L::STAGES, b = l % L::BUFS;
                    fine = (l < L::BUFS || wait_warp(t_empty + 8 * b, (l / L::BUFS & 1) ^ 1)) && wait_warp(full(s), l / L::STAGES & 1);
                    if (!fine) break;
                    tc::fence_after();
                    const uint64_t da = tc::desc(sb + s * L::STAGE, 16, 1024), db = tc::desc(sb + s * L::STAGE + L::A, 16, 1024);
#pragma unroll
                    for (int k = 0; k < KB / 32; ++k) tc::mma_e4m3_if(on, tmem + b * BN, da + 2 * k, db + 2 * k, id, k > 0);
                    tc::commit_if(on, empty(s));
                    tc::commit_if(on, t_full + 8 * b);
                }
            }
            if (!fine) {
                tc::commit_if(on, ended + 8 * mine);
                tc::mbar_wait(ended + 8 * mine, 0);
            }
        } else if (warp == 2 && !X_ROWS) {
            // ---------------- scales of the columns, eight blocks at a time ----------------
            int u = 0;
#pragma unroll 1
            for (int t = first; t < tiles; t += step) {
                const int nb = t / tiles_b;
                const int64_t m0 = (int64_t)(t % tiles_b) * BN;
#pragma unroll 1
                for (int kb = kb0; kb < kb1; kb += 8, ++u) {
                    if (u >= 2) wait_warp(sc_empty + 8 * (u & 1), (u >> 1 & 1) ^ 1);
                    float* sc = reinterpret_cast<float*>(smem + L::oScale) + (u & 1) * 8 * BN;
                    for (int j = lane; j < BN; j += 32) {
                        float v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const bool on = m0 + j < p.M && kb + i < kb1;
                            v[i] = on ? p.xs[(m0 + j) * p.x_blocks + (p.x_blocks > 1 ? kb + i : 0)] * p.ws[(int64_t)nb * nkb + kb + i] : 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) sc[i * BN + j] = v[i];
                    }
                    tc::mbar_arrive(sc_full + 8 * (u & 1));
                }
            }
        }
    } else {
        if (L::MOVE_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n");
        // ---------------- sums ----------------
        const int q4 = warp & 3, group = (warp - 4) >> 2, i = 32 * q4 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * q4) << 16) + group * COLS;
        int l = 0, u = 0;
        bool there = false;  // the next block's product has been seen to be done
        // The two factors of a block's scale, asked for two blocks ahead (a tile's first ones before the last tile's outputs
        // are written) and multiplied when they are wanted: a product of look-ups that are still on their way stops
        // the thread (400 of 700 cycles a block).
        const float *xs = nullptr, *ws = nullptr;
        float2 next = make_float2(0.f, 0.f), then = next;
        auto scales_at = [&](int kb) {
            return xs && kb < kb1 ? make_float2(__ldg(xs + (p.x_blocks > 1 ? kb : 0)), __ldg(ws + kb)) : make_float2(0.f, 0.f);
        };
        auto begin = [&](int t) {
            if (!X_ROWS || t >= tiles) return;
            const int64_t row = (int64_t)(t / tiles_b) * 128 + i;
            xs = row < p.M ? p.xs + row * p.x_blocks : nullptr;
            ws = p.ws + (int64_t)min((t % tiles_b * BN + group * COLS) / 128, (p.N - 1) / 128) * nkb;
            next = scales_at(kb0), then = scales_at(kb0 + 1);
        };
        begin(first);
#pragma unroll 1
        for (int t = first; t < tiles; t += step) {
            const int a0 = t / tiles_b * 128, b0 = t % tiles_b * BN;
            float acc[COLS];
#pragma unroll
            for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
#pragma unroll 1
            for (int kb = kb0; kb < kb1; ++kb, ++l) {
                const int b = l % L::BUFS;
                const float s = next.x * next.y;
                next = then;
                if (X_ROWS) then = scales_at(kb + 2);
                const float* sc = reinterpret_cast<const float*>(smem + L::oScale) + (u & 1) * 8 * BN + ((kb - kb0) & 7) * BN;
                if (!X_ROWS && ((kb - kb0) & 7) == 0) wait_warp(sc_full + 8 * (u & 1), u >> 1 & 1);
                if (!there) wait_warp(t_full + 8 * b, l / L::BUFS & 1);
                tc::fence_after();
                // (64 columns asked for at once, and the buffer given back before the last ones are added: what bounds the
                // loop is how soon the next product may have it)
                constexpr int PART = COLS < 64 ? COLS : 64;
#pragma unroll
                for (int c = 0; c < COLS; c += PART) {
                    uint32_t v[PART / 16][16];
#pragma unroll
                    for (int h = 0; h < PART / 16; ++h) tc::ld16_nowait(lanes + b * BN + c + 16 * h, v[h]);
#pragma unroll
                    for (int h = 0; h < PART / 16; ++h) tc::ld_wait(v[h]);
                    if (c + PART == COLS) {
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(t_empty + 8 * b);
                        // (looked at now, decided on when the last columns have been added: 5% of narrow tiles' time; with 256
                        // columns it costs 8%)
                        if (BN < 256) there = tc::mbar_test(t_full + 8 * ((l + 1) % L::BUFS), (l + 1) / L::BUFS & 1);
                    }
#pragma unroll
                    for (int j = 0; j < PART; j += 4) {
                        float4 f = make_float4(s, s, s, s);
                        if (!X_ROWS) f = *reinterpret_cast<const float4*>(sc + c + j);
                        const uint32_t* w = v[j / 16] + j % 16;
                        ACC2(acc, c + j, __ffma2_rn(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), make_float2(f.x, f.y), F2(acc, c + j)));
                        ACC2(acc, c + j + 2, __ffma2_rn(make_float2(__uint_as_float(w[2]), __uint_as_float(w[3])), make_float2(f.z, f.w), F2(acc, c + j + 2)));
                    }
                }
                if (BN < 256) there = __all_sync(~0u, there);
                if (!X_ROWS && (((kb - kb0) & 7) == 7 || kb + 1 == kb1)) {
                    __syncwarp();  // (all lanes have read the scales before they are given back)
                    if (lane == 0) tc::mbar_arrive(sc_empty + 8 * (u & 1));
                    ++u;
                }
            }
            begin(t + step);
            if (!ok()) {
#pragma unroll
                for (int j = 0; j < COLS; ++j) acc[j] = __int_as_float(0x7fffffff);
                if (BN < 256 && (!X_ROWS || split > 1)) {  // (what follows takes the memory that copies may still be on their way to)
#pragma unroll 1
                    for (int n = 0; asked_s < 0 && n < 1 << 22; ++n) {}
                    landed(asked_s);
                }
            }
            if (X_ROWS && split == 1) {
                // out through 128 x 64 tiles in shared memory, which the copies have left by the next time (what lies
                // outside y is cut off by the copy)
                unsigned char* stage = smem + L::oStore + group * (COLS / 64) * 16384;
                const int n0 = b0 + group * COLS;
                if (i == 0) tc::bulk_wait_read();
                tc::named_sync(1 + group, 128);
#pragma unroll
                for (int j = 0; j < COLS / 8; ++j) {
                    float* a = acc + 8 * j;
                    if (p.bias) {
#pragma unroll
                        for (int h = 0; h < 8; h += 4) {
                            if (n0 + 8 * j + h >= p.N) continue;
                            const float4 f = __ldg(reinterpret_cast<const float4*>(p.bias + n0 + 8 * j + h));
                            a[h] += f.x, a[h + 1] += f.y, a[h + 2] += f.z, a[h + 3] += f.w;
                        }
                    }
                    *reinterpret_cast<uint4*>(stage + tc::sw_chunk(i, j, 128)) =
                        make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7]));
                }
                tc::fence_async_smem();
                tc::named_sync(1 + group, 128);
                if (i == 0) {
#pragma unroll
                    for (int c = 0; c < COLS; c += 64)
                        if (n0 + c < p.N) tc::tma_store_2d(&maps.y, n0 + c, a0, smem_u32(stage) + c / 64 * 16384);
                    tc::bulk_commit();
                }
            } else {
                // the part of this block, for the cluster (the tiles' memory is free: this is the block's only tile)
                float* part = reinterpret_cast<float*>(smem);
                if (X_ROWS) {
#pragma unroll
                    for (int j = 0; j < COLS; j += 4)
                        *reinterpret_cast<float4*>(part + ((group * COLS + j) / 4 * 128 + i) * 4) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
                } else {
#pragma unroll
                    for (int j = 0; j < COLS; ++j) part[j * 128 + i] = acc[j];
                }
            }
        }
        if (X_ROWS && split == 1 && i == 0) tc::bulk_wait_read();
    }
    __syncwarp();
    if (!X_ROWS || split > 1) {
        if (split > 1) cluster_sync();
        else __syncthreads();
        const int a0 = first / tiles_b * 128, b0 = first % tiles_b * BN;
        auto total = [&](int word) {  // (all parts asked for before any is added)
            float4 v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < split) v[r] = split > 1 ? ld_peer(sb + 4 * word, r) : *reinterpret_cast<const float4*>(smem + 4 * word);
            float4 s = v[0];
#pragma unroll
            for (int r = 1; r < 8; ++r)
                if (r < split) s = make_float4(s.x + v[r].x, s.y + v[r].y, s.z + v[r].z, s.w + v[r].w);
            return s;
        };
        auto put = [&](int64_t m, int n, const float4& s) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.bias) f = __ldg(reinterpret_cast<const float4*>(p.bias + n));
            *reinterpret_cast<uint2*>(p.y + m * p.N + n) = make_uint2(pack_bf16(s.x + f.x, s.y + f.y), pack_bf16(s.z + f.z, s.w + f.w));
        };
        // the ranks share out the tile's quadruples of outputs
        constexpr int QUADS = 128 * BN / 4;
#pragma unroll 1
        for (int e = rank * L::THREADS + tid; e < QUADS; e += split * L::THREADS) {
            if (X_ROWS) {  // quadruple e: columns 4 (e / 128), row e % 128
                const int n = b0 + e / 128 * 4;
                const int64_t m = (int64_t)a0 + e % 128;
                if (m < p.M && n < p.N) put(m, n, total(4 * e));
            } else {       // column (row of x) e / 32, outputs 4 (e % 32)
                const int64_t m = (int64_t)b0 + e / 32;
                const int n = a0 + e % 32 * 4;
                if (m < p.M && n < p.N) put(m, n, total(4 * e));
            }
        }
        if (split > 1) cluster_sync();
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) tc::dealloc(tmem, L::TMEM);
}

// Clusters of `split` blocks of a kernel that the device holds at once (asked once a device).
template <bool X_ROWS, int BN>
int clusters_at_once(int split) {
    using L = Lin<X_ROWS, BN>;
    static int known[64][4];
    int dev = 0, which = split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (known[dev][which]) return known[dev][which];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split);
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = L::SMEM;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k_linear<X_ROWS, BN>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    return known[dev][which] = n > 0 ? n : 1;
}

// Blocks that share a tile's inner dimension: as many as leave all tiles in place at once (a second round would cost what
// the split gains: 128 x 2048 x 6144 in 48 clusters of four 17 us, of two 10), at most 8, two blocks of 128 each at least.
template <bool X_ROWS, int BN>
int split_of(int64_t tiles, int K) {
    const int nkb = (K + KB - 1) / KB;
    int s = 1;
    while (s < 8 && 4 * s <= nkb && tiles <= clusters_at_once<X_ROWS, BN>(2 * s)) s *= 2;
    return s;
}

template <bool X_ROWS, int BN>
cudaError_t go(const LinearParams& p, cudaStream_t s) {
    using L = Lin<X_ROWS, BN>;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    const int a_rows = X_ROWS ? (int)p.M : p.N, b_rows = X_ROWS ? p.N : (int)p.M;
    if (!encode_bytes_map(&maps.a, X_ROWS ? p.x : p.w, a_rows, p.K, 128) || !encode_bytes_map(&maps.b, X_ROWS ? p.w : p.x, b_rows, p.K, BN))
        return cudaErrorInvalidValue;
    const int tiles_b = (b_rows + BN - 1) / BN;
    const int64_t tiles = (int64_t)((a_rows + 127) / 128) * tiles_b;
    if (tiles > (1 << 30) / 8) return cudaErrorInvalidValue;
    static bool allowed[64];
    cudaError_t e = allow_smem((const void*)k_linear<X_ROWS, BN>, L::SMEM, allowed);
    if (e != cudaSuccess) return e;
    const int split = BN == 256 ? 1 : split_of<X_ROWS, BN>(tiles, p.K);
    if (X_ROWS && split == 1 && !encode_rows_map(&maps.y, p.y, p.M, p.N, 128)) return cudaErrorInvalidValue;
    if (L::MOVE_REGS) {  // (the groups' shares of the registers have to be there at the launch)
        static const int regs = [] {
            cudaFuncAttributes at;
            return cudaFuncGetAttributes(&at, k_linear<X_ROWS, BN>) == cudaSuccess ? at.numRegs : 0;
        }();
        if (regs != 168) return cudaErrorInvalidConfiguration;
    }
    cudaLaunchConfig_t cfg = {};
    // (one tile a cluster; blocks that store by TMA walk the tiles)
    cfg.gridDim = dim3((unsigned)(X_ROWS && split == 1 ? (tiles < num_sms() ? tiles : num_sms()) : tiles * split));
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = L::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_linear<X_ROWS, BN>, maps, p, tiles_b, (int)tiles, split);
}

}  // namespace

cudaError_t launch_linear(const LinearParams& p, cudaStream_t s) {
    // Weights as rows against rows of x as rows, K = 2048, N = 6144, in a graph: 5 rows 5.9 and 9.2 us, 32 6.5 and 9.2,
    // 64 7.8 and 8.6.  Of the narrow ones the narrowest (16 rows in 16 columns 5.8 us, in 64 6.7).
    if (p.M <= 16) return go<false, 16>(p, s);
    if (p.M <= 32) return go<false, 32>(p, s);
    if (p.M <= 64) return go<false, 64>(p, s);
    // Tiles of 128 x 128 where all of them are in place at once, else of 128 x 256, K = N = 2048: 1024 rows 8.9 and 11.0 us, 1280
    // 13.7 and 11.1, 8192 37.8 and 32.3.
    if ((p.M + 127) / 128 * ((p.N + 127) / 128) > num_sms()) return go<true, 256>(p, s);
    return go<true, 128>(p, s);
}

}  // namespace gdr
