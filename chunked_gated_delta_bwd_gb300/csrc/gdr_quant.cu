// Quantisation to 8 bits (e4m3) with a scale for each 128 channels of a row, or for each tile of 128 x 128:
//
//   scale = max |x| / 448 (1 where all are zero),  y = e4m3(x / scale)
//
// Bytes bound it: every value is read once and held in registers between the maximum and its code.
// Rows: eight threads hold 128 channels, 16 each, of two rows, with their loads in flight together
// (instructions bound it next: 16 threads with eight each took 45 us for 8191 x 6144 in bf16, this 27, 5.6 TB/s).  Tiles: a
// block of 512 threads holds a tile, 32 values each; the transposed copy is turned round in shared memory (6144 x 2048 in
// fp32, both copies: 17 us, 4.4 TB/s; 768 blocks at two a multiprocessor are 2.5 rounds).
#include "gdr_e4m3.h"
#include "gdr_internal.h"
#include "gdr_rows.cuh"

namespace gdr {
namespace {

constexpr int ROWS_AT_ONCE = 2;  // rows a group of eight threads holds at once

__device__ __forceinline__ float most_of(const Eight& e) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(e.v[i]));
    return m;
}
__device__ __forceinline__ float most_of(const RawOf<float>& r) { return most_of(r.widen()); }
__device__ __forceinline__ float most_of(const RawOf<__nv_bfloat16>& r) {  // (in pairs)
    const uint32_t w[4] = {r.u.x & 0x7fff7fffu, r.u.y & 0x7fff7fffu, r.u.z & 0x7fff7fffu, r.u.w & 0x7fff7fffu};
    __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(w);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(w + i));
    const float2 f = __bfloat1622float2(m);
    return fmaxf(fmaxf(f.x, f.y), 0.f);
}
// The codes of y / scale, the quotient rounded to fp32 as the division rounds it: from inv, the reciprocal rounded to
// nearest, by one correction of y inv with its exact remainder (P. Markstein, IBM J. Res. Dev. 34, 1990).  A quotient that
// lies on a tie between two codes is exact in fp32, and the correction returns it exactly; bf16 values have many (x / max is
// a ratio of 8-bit numbers), so that trying products to either side and dividing where they disagree, as the norm does
// for its fp32 values, divides in many of the warps (8191 x 6144: 41 us, this 27).  Where the remainder could leave the
// normal numbers the division itself is taken.
__device__ __forceinline__ void quotient_codes(const Eight& y, float scale, uint32_t (&h)[4]) {
    if (scale > 0x1p-80f && scale < 0x1p100f) {
        const float inv = -__frcp_rn(scale);  // (all negative, so that a remainder of zero leaves a zero its sign)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 v = two(y, q), first = __fmul2_rn(v, make_float2(inv, inv));
            const float2 rest = __ffma2_rn(first, make_float2(scale, scale), v), f = __ffma2_rn(rest, make_float2(inv, inv), first);
            h[q] = e4m3x2(f.x, f.y) ^ 0x8080u;
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = e4m3x2(y.v[2 * q] / scale, y.v[2 * q + 1] / scale);
    }
}
// eight codes of a row whose `n` channels from here on exist
__device__ __forceinline__ void put_codes(uint8_t* y, const uint32_t (&h)[4], int n, bool wide) {
    if (wide) {
        *reinterpret_cast<uint2*>(y) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (2 * q < n) *reinterpret_cast<uint16_t*>(y + 2 * q) = (uint16_t)h[q];
    }
}

// Eight threads hold a block of 128 channels, two pieces of eight each (64 channels apart).  A warp takes 4 of them: 1 << cw
// blocks side by side, of 4 >> cw rows.
template <class T, bool wide>
__global__ void __launch_bounds__(256) k_quant_rows(const QuantParams p, int nb, int across, int cw) {
    const int lane = threadIdx.x % 8, group = threadIdx.x / 8;
    const int down = blockIdx.x / across, block = (blockIdx.x - down * across) << cw | (group & ((1 << cw) - 1)), c = block * 128 + 8 * lane;
    const int below = 32 >> cw;  // rows of a block at once
    const int64_t row0 = (int64_t)down * (below * ROWS_AT_ONCE) + (group >> cw);
    const int64_t ahead = below * p.ldx;
    const T* x = static_cast<const T*>(p.x) + row0 * p.ldx + c;
    RawOf<T> raw[ROWS_AT_ONCE][2];
#pragma unroll
    for (int i = 0; i < ROWS_AT_ONCE; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = p.C - c - 64 * h;
            raw[i][h] = RawOf<T>{};
            if (row0 + i * below < p.R && n > 0) raw[i][h] = ld8(x + i * ahead + 64 * h, n, wide);
        }
#pragma unroll
    for (int i = 0; i < ROWS_AT_ONCE; ++i) {
        const int64_t row = row0 + i * below;
        float m = fmaxf(most_of(raw[i][0]), most_of(raw[i][1]));
#pragma unroll
        for (int o = 4; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if (row >= p.R || block >= nb) continue;
        const float scale = scale_of(m);
        if (lane == 0) p.scale[row * nb + block] = scale;
        uint8_t* y = p.y + row * p.C + c;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = p.C - c - 64 * h;
            if (n <= 0) continue;
            uint32_t code[4];
            quotient_codes(raw[i][h].widen(), scale, code);
            put_codes(y + 64 * h, code, n, wide);
        }
    }
}

// A tile: 16 threads hold a row's 128 channels, each eight channels of four rows.
template <class T>
__global__ void __launch_bounds__(512, 2) k_quant_tiles(const QuantParams p, int nb, int nr, int wide, int wide_t) {
    __shared__ float red[16];
    __shared__ uint32_t turned[128][32];  // [channel][four rows]: word w of a channel at w ^ (channel / 8)
    const int lane = threadIdx.x % 16, r4 = threadIdx.x / 16;
    const int64_t tr = blockIdx.x / nb;
    const int tc = (int)(blockIdx.x - tr * nb), c = tc * 128 + 8 * lane;
    const int n = p.C - c;
    RawOf<T> raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = tr * 128 + 4 * r4 + i;
        raw[i] = RawOf<T>{};
        if (row < p.R && n > 0) raw[i] = ld8(static_cast<const T*>(p.x) + row * p.ldx + c, n, wide);
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, most_of(raw[i]));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, red[i]);
    const float scale = scale_of(m);
    if (threadIdx.x == 0) {
        p.scale[tr * nb + tc] = scale;
        if (p.yt) p.scale_t[tc * (int64_t)nr + tr] = scale;
    }
    uint32_t code[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = tr * 128 + 4 * r4 + i;
        uint32_t h[4];
        quotient_codes(raw[i].widen(), scale, h);
        code[i][0] = h[0] | h[1] << 16;
        code[i][1] = h[2] | h[3] << 16;
        if (row < p.R && n > 0) put_codes(p.y + row * p.C + c, h, n, wide);
    }
    if (!p.yt) return;
    // four rows' codes of a channel in one word
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int q = j / 4, b = j % 4;
        const uint32_t lo = __byte_perm(code[0][q], code[1][q], b | (4 + b) << 4), hi = __byte_perm(code[2][q], code[3][q], b | (4 + b) << 4);
        turned[8 * lane + j][r4 ^ lane] = __byte_perm(lo, hi, 0x5410);
    }
    __syncthreads();
    // rows of the transposed copy: eight threads write 128 bytes
    for (int j = threadIdx.x / 8; j < 128; j += 64) {
        const int64_t ch = (int64_t)tc * 128 + j;
        if (ch >= p.C) break;
        const int b = threadIdx.x % 8;
        const int64_t row = tr * 128 + 16 * b;
        uint8_t* to = p.yt + ch * p.R + row;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = turned[j][(4 * b + i) ^ (j / 8)];
        if (wide_t && row + 16 <= p.R) {
            *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (row + i < p.R) to[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
        }
    }
}

template <class T>
cudaError_t go(const QuantParams& p, cudaStream_t s) {
    const int nb = (p.C + 127) / 128;
    const int wide = (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 && p.ldx % 8 == 0 && p.C % 8 == 0;
    if (!p.tiles) {
        const int cw = nb > 2 ? 2 : nb - 1, across = (nb + (1 << cw) - 1) >> cw, rows = (32 >> cw) * ROWS_AT_ONCE;
        const unsigned grid = (unsigned)((p.R + rows - 1) / rows * across);
        if (wide) k_quant_rows<T, true><<<grid, 256, 0, s>>>(p, nb, across, cw);
        else k_quant_rows<T, false><<<grid, 256, 0, s>>>(p, nb, across, cw);
    } else {
        const int64_t nr = (p.R + 127) / 128;
        k_quant_tiles<T><<<(unsigned)(nr * nb), 512, 0, s>>>(p, nb, (int)nr, wide, p.R % 16 == 0);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant(const QuantParams& p, cudaStream_t s) {
    return p.x_f32 ? go<float>(p, s) : go<__nv_bfloat16>(p, s);
}

}  // namespace gdr
