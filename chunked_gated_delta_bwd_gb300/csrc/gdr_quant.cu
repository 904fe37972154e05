// Quantisation to 8 bits (e4m3) with a scale for each 128 channels of a row, or for each tile of 128 x 128:
//
//   scale = max |x| / 448 (1 where all are zero),  y = e4m3(x / scale)
//
// Bytes bound it: every value is read once and held in registers between the maximum and its code.
// Rows: eight threads hold 128 channels, 16 each, of two rows, with their loads in flight together
// (instructions bound it next: 16 threads with eight each took 45 us for 8191 x 6144 in bf16).  Tiles: a block of 256 threads holds a tile, 64 values each; the transposed
// copy is turned round in shared memory.
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
template <class T>
__global__ void __launch_bounds__(256) k_quant_rows(const QuantParams p, int nb, int across, int cw, int wide) {
    const int lane = threadIdx.x % 8, group = threadIdx.x / 8;
    const int down = blockIdx.x / across, block = (blockIdx.x - down * across) << cw | (group & ((1 << cw) - 1)), c = block * 128 + 8 * lane;
    const int64_t row0 = (int64_t)down * ((32 >> cw) * ROWS_AT_ONCE) + (group >> cw);
    RawOf<T> raw[ROWS_AT_ONCE][2];
#pragma unroll
    for (int i = 0; i < ROWS_AT_ONCE; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = row0 + i * (32 >> cw);
            const int n = p.C - c - 64 * h;
            raw[i][h] = RawOf<T>{};
            if (row < p.R && n > 0) raw[i][h] = ld8(static_cast<const T*>(p.x) + row * p.ldx + c + 64 * h, n, wide);
        }
#pragma unroll
    for (int i = 0; i < ROWS_AT_ONCE; ++i) {
        const int64_t row = row0 + i * (32 >> cw);
        float m = fmaxf(most_of(raw[i][0]), most_of(raw[i][1]));
#pragma unroll
        for (int o = 4; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if (row >= p.R || block >= nb) continue;
        const float scale = scale_of(m);
        if (lane == 0) p.scale[row * nb + block] = scale;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = p.C - c - 64 * h;
            if (n <= 0) continue;
            uint32_t code[4];
            codes_of(raw[i][h].widen(), scale, code);
            put_codes(p.y + row * p.C + c + 64 * h, code, n, wide);
        }
    }
}

template <class T>
__global__ void __launch_bounds__(256) k_quant_tiles(const QuantParams p, int nb, int nr, int wide, int wide_t) {
    __shared__ float red[8];
    __shared__ uint32_t turned[128][33];  // [channel][row / 4]
    const int lane = threadIdx.x % 16, r0 = threadIdx.x / 16;
    const int64_t tr = blockIdx.x / nb;
    const int tc = (int)(blockIdx.x - tr * nb), c = tc * 128 + 8 * lane;
    const int n = p.C - c;
    // (rows 8 r0 + i: a thread's eight rows are eight consecutive bytes of a turned row)
    RawOf<T> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = tr * 128 + 8 * r0 + i;
        raw[i] = RawOf<T>{};
        if (row < p.R && n > 0) raw[i] = ld8(static_cast<const T*>(p.x) + row * p.ldx + c, n, wide);
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, most_of(raw[i].widen()));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
    const float scale = scale_of(m);
    if (threadIdx.x == 0) {
        p.scale[tr * nb + tc] = scale;
        if (p.yt) p.scale_t[tc * (int64_t)nr + tr] = scale;
    }
    uint32_t code[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = tr * 128 + 8 * r0 + i;
        uint32_t h[4];
        codes_of(raw[i].widen(), scale, h);
        code[i][0] = h[0] | h[1] << 16;
        code[i][1] = h[2] | h[3] << 16;
        if (row < p.R && n > 0) put_codes(p.y + row * p.C + c, h, n, wide);
    }
    if (!p.yt) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t u = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) u |= (code[4 * q + i][j / 4] >> (8 * (j % 4)) & 255u) << (8 * i);
            turned[8 * lane + j][2 * r0 + q] = u;
        }
    }
    __syncthreads();
    // rows of the transposed copy: eight threads write 128 bytes
    for (int j = threadIdx.x / 8; j < 128; j += 32) {
        const int64_t ch = (int64_t)tc * 128 + j;
        if (ch >= p.C) break;
        const int b = threadIdx.x % 8;
        const int64_t row = tr * 128 + 16 * b;
        uint8_t* to = p.yt + ch * p.R + row;
        const uint32_t* w = &turned[j][4 * b];
        if (wide_t && row + 16 <= p.R) {
            *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int i = 0; i < 16 && row + i < p.R; ++i) to[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
        }
    }
}

template <class T>
cudaError_t go(const QuantParams& p, cudaStream_t s) {
    const int nb = (p.C + 127) / 128;
    const int wide = (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 && p.ldx % 8 == 0 && p.C % 8 == 0;
    if (!p.tiles) {
        const int cw = nb > 2 ? 2 : nb - 1, across = (nb + (1 << cw) - 1) >> cw, rows = (32 >> cw) * ROWS_AT_ONCE;
        k_quant_rows<T><<<(unsigned)((p.R + rows - 1) / rows * across), 256, 0, s>>>(p, nb, across, cw, wide);
    } else {
        const int64_t nr = (p.R + 127) / 128;
        k_quant_tiles<T><<<(unsigned)(nr * nb), 256, 0, s>>>(p, nb, (int)nr, wide, p.R % 16 == 0);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant(const QuantParams& p, cudaStream_t s) {
    return p.x_f32 ? go<float>(p, s) : go<__nv_bfloat16>(p, s);
}

}  // namespace gdr
