// RMS norm with the residual's addition, forward (bf16, or e4m3 with scales) and backward.
//
//   s = round(x + r),  rstd = 1 / sqrt(mean s^2 + eps),  y = s rstd w
//
// The norm is taken of the sum as it is stored (rounded to the residual stream's type), so that
// the backward, which sees only the stored sum, differentiates what the forward computed.
// 8-bit output: scale = max |y| / 448 over the row or over each 128 channels (1 where all of
// them are zero), y8 = e4m3(y / scale).
//
// backward, n = s rstd, u = w dy:  dx = rstd (u - n mean(u n)) + dres,  dweight = sum_rows dy n
//
// Bytes bound both.  A group of threads holds a row in registers, eight channels (16 bytes of
// bf16) a thread at a time, from its loads to its stores, so that every tensor passes once; the
// next row's loads are in flight meanwhile (without that the 8-bit forward of 32768 x 2048 took
// 175 us; now 85, 83% of the measured copy rate; the backward of 8191 x 2048 with a
// float32 stream takes 44 us, 79%).  The group is the smallest with one piece a thread: a row of up to
// 256 channels needs no barrier but the warp's shuffles.
#include <cuda_fp8.h>

#include "gdr_block.h"
#include "gdr_common.cuh"
#include "gdr_internal.h"

namespace gdr {

namespace {

// eight consecutive channels, and as loaded
struct Eight {
    float v[8];
};
__device__ __forceinline__ float2 two(const Eight& e, int q) { return make_float2(e.v[2 * q], e.v[2 * q + 1]); }
__device__ __forceinline__ void set_two(Eight& e, int q, float2 f) {
    e.v[2 * q] = f.x;
    e.v[2 * q + 1] = f.y;
}
// two bf16, by a shift and a mask (the conversion function takes three instructions)
__device__ __forceinline__ float2 widen_pair(uint32_t r) { return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u)); }
template <class T> struct RawOf;
template <> struct RawOf<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ Eight widen() const {
        Eight e;
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = widen_pair(w[i]);
            e.v[2 * i] = f.x;
            e.v[2 * i + 1] = f.y;
        }
        return e;
    }
};
template <> struct RawOf<float> {
    float4 a, b;
    __device__ __forceinline__ Eight widen() const { return Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
// `n` channels of a row from p on; `wide`: rows are whole numbers of aligned pieces, else pairs
__device__ __forceinline__ RawOf<__nv_bfloat16> ld8(const __nv_bfloat16* p, int n, bool wide) {
    if (wide) return {__ldcs(reinterpret_cast<const uint4*>(p))};
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
    return {make_uint4(__ldcs(q), n > 2 ? __ldcs(q + 1) : 0u, n > 4 ? __ldcs(q + 2) : 0u, n > 6 ? __ldcs(q + 3) : 0u)};
}
__device__ __forceinline__ RawOf<float> ld8(const float* p, int n, bool wide) {
    if (wide) return {__ldcs(reinterpret_cast<const float4*>(p)), __ldcs(reinterpret_cast<const float4*>(p) + 1)};
    const float2* q = reinterpret_cast<const float2*>(p);
    const float2 none = make_float2(0.f, 0.f), f0 = __ldcs(q), f1 = n > 2 ? __ldcs(q + 1) : none, f2 = n > 4 ? __ldcs(q + 2) : none,
                 f3 = n > 6 ? __ldcs(q + 3) : none;
    return {make_float4(f0.x, f0.y, f1.x, f1.y), make_float4(f2.x, f2.y, f3.x, f3.y)};
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const Eight& e) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(e.v[0], e.v[1]), pack_bf16(e.v[2], e.v[3]), pack_bf16(e.v[4], e.v[5]),
                                              pack_bf16(e.v[6], e.v[7]));
}
__device__ __forceinline__ void st8(float* p, const Eight& e) {
    reinterpret_cast<float4*>(p)[0] = make_float4(e.v[0], e.v[1], e.v[2], e.v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(e.v[4], e.v[5], e.v[6], e.v[7]);
}
// pairs
template <class T> __device__ __forceinline__ float2 ld2(const T* p);
template <> __device__ __forceinline__ float2 ld2(const __nv_bfloat16* p) { return unpack_bf16(__ldcs(reinterpret_cast<const uint32_t*>(p))); }
template <> __device__ __forceinline__ float2 ld2(const float* p) { return __ldcs(reinterpret_cast<const float2*>(p)); }
__device__ __forceinline__ void st2(__nv_bfloat16* p, float2 v) { *reinterpret_cast<uint32_t*>(p) = pack_bf16(v.x, v.y); }
__device__ __forceinline__ void st2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
template <class T>
__device__ __forceinline__ void st8n(T* p, const Eight& e, int n, bool wide) {
    if (wide) {
        st8(p, e);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        if (i < n) st2(p + i, make_float2(e.v[i], e.v[i + 1]));
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// The scale of values up to m: m / 448, 1 where all are zero.  Where m / 448 rounds to zero it is the
// smallest float32, so that zeros stay zero.
__device__ __forceinline__ float scale_of(float m) { return m > 0.f ? fmaxf(m / 448.f, 1.4e-45f) : 1.f; }
// The codes of y / scale.  A product with 1 / scale (two steps of the last place off at most) is within
// 3 2^-23 of the quotient, so that products to either side by 2^-21 have the quotient's code unless a tie
// lies between them: then (some 10^-5 of the values), or where 1 / scale is far from the normal numbers,
// the division itself decides.  (Dividing every value of 32768 x 2048 takes 98 us, this 85, the product
// alone, which takes the other code next to a tie and is infinite for scales below 2^-128, 81.)
__device__ __forceinline__ void codes_of(const Eight& y, float scale, uint32_t (&h)[4]) {
    const float inv = __fdividef(1.f, scale), under = inv * (1.f - 0x1p-21f), over = inv * (1.f + 0x1p-21f);
    uint32_t differ = scale > 0x1p-120f && scale < 0x1p120f ? 0 : 1;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 a = __fmul2_rn(two(y, q), make_float2(under, under)), b = __fmul2_rn(two(y, q), make_float2(over, over));
        h[q] = e4m3x2(a.x, a.y);
        differ |= h[q] ^ e4m3x2(b.x, b.y);
    }
    if (differ) {
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = e4m3x2(y.v[2 * q] / scale, y.v[2 * q + 1] / scale);
    }
}

// A row of C channels is walked in pieces of 8 by G threads: thread t has pieces t, t + G, ...
// Sum (or maximum) over the G threads of a row; `red`: a word for each warp of the block (G > 32).
template <int G, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red) {
#pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o; o >>= 1) {
        const float u = __shfl_xor_sync(~0u, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    if (G > 32) {
        __syncthreads();  // (red may still be read from the last time)
        if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
        __syncthreads();
        const float* mine = red + threadIdx.x / G * (G / 32);
        v = mine[0];
#pragma unroll
        for (int i = 1; i < G / 32; ++i) v = MAX ? fmaxf(v, mine[i]) : v + mine[i];
    }
    return v;
}

}  // namespace

// G threads a row, P pieces a thread (G * P * 8 >= C); blocks of `threads` hold threads / G rows and
// walk the rows with the grid's stride.  TR: the residual stream's type.
template <int G, int P, class TR, bool RES, int QUANT>
__global__ void __launch_bounds__(G > 128 ? G : 128, P == 1 ? 1280 / (G > 128 ? G : 128) : 1) k_rmsnorm_fwd(const NormParams p, int wide) {
    constexpr int THREADS = G > 128 ? G : 128, ROWS = THREADS / G;
    __shared__ float red[THREADS / 32];
    const int t = threadIdx.x % G, C = p.C;
    const float invC = 1.f / (float)C;
    Eight w[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
            const int c = (t + i * G) * 8 + q;
            const float2 f = c < C ? *reinterpret_cast<const float2*>(p.weight + c) : make_float2(0.f, 0.f);
            w[i].v[q] = f.x;
            w[i].v[q + 1] = f.y;
        }
    RawOf<__nv_bfloat16> xr[P];
    RawOf<TR> rr[P];
    auto load = [&](int64_t row) {
        if (row < p.R) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = (t + i * G) * 8;
                if (c < C) {
                    xr[i] = ld8(p.x + row * p.ldx + c, C - c, wide);
                    if (RES) rr[i] = ld8(static_cast<const TR*>(p.residual) + row * C + c, C - c, wide);
                }
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * ROWS;
    load((int64_t)blockIdx.x * ROWS + threadIdx.x / G);
    for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < p.R; row0 += step) {
        const int64_t row = row0 + threadIdx.x / G;
        const bool live = row < p.R;
        Eight s[P];
        float2 ss = make_float2(0.f, 0.f);
        if (live) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = (t + i * G) * 8;
                if (c < C) {
                    s[i] = xr[i].widen();
                    if (RES) {
                        const Eight r = rr[i].widen();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float2 v = __fadd2_rn(two(s[i], q), two(r, q));
                            set_two(s[i], q, sizeof(TR) == 4 ? v : widen_pair(pack_bf16(v.x, v.y)));
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) ss = __ffma2_rn(two(s[i], q), two(s[i], q), ss);
                }
            }
        }
        load(row + step);
        if (RES && live) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = (t + i * G) * 8;
                if (c < C) st8n(static_cast<TR*>(p.res_out) + row * C + c, s[i], C - c, wide);
            }
        }
        const float rstd = rsqrtf(fmaf(row_reduce<G, false>(ss.x + ss.y, red), invC, p.eps));
        if (live && t == 0) p.rstd[row] = rstd;
        float most[QUANT == 2 ? P : 1];
        most[0] = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (t + i * G) * 8;
            float m = 0.f;
            if (live && c < C) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 y = __fmul2_rn(__fmul2_rn(two(s[i], q), make_float2(rstd, rstd)), two(w[i], q));
                    set_two(s[i], q, y);
                    if (QUANT) m = fmaxf(m, fmaxf(fabsf(y.x), fabsf(y.y)));
                }
            }
            if (QUANT == 1) most[0] = fmaxf(most[0], m);
            if (QUANT == 2) {  // 128 channels are 16 threads' pieces (fewer threads hold a row of at most 64)
#pragma unroll
                for (int o = (G < 16 ? G : 16) / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
                most[QUANT == 2 ? i : 0] = m;
            }
        }
        if (QUANT == 1) most[0] = row_reduce<G, true>(most[0], red);
        if (!live) continue;  // (with several rows a block no barrier follows)
        const int nb = QUANT == 2 ? (C + 127) / 128 : 1;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (t + i * G) * 8;
            if (c >= C) continue;
            if (QUANT == 0) {
                st8n(static_cast<__nv_bfloat16*>(p.y) + row * C + c, s[i], C - c, wide);
            } else {
                const float scale = scale_of(most[QUANT == 2 ? i : 0]);
                if (QUANT == 2 ? c % 128 == 0 : c == 0) p.scale[row * nb + (QUANT == 2 ? c / 128 : 0)] = scale;
                uint32_t h[4];
                codes_of(s[i], scale, h);
                unsigned char* y = static_cast<unsigned char*>(p.y) + row * C + c;
                if (wide) {
                    *reinterpret_cast<uint2*>(y) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (2 * q < C - c) *reinterpret_cast<uint16_t*>(y + 2 * q) = (uint16_t)h[q];
                }
            }
        }
    }
}

// Rows too long for registers: a block walks a row three times, from memory and then from the caches.
template <class TR>
__global__ void __launch_bounds__(512) k_rmsnorm_fwd_long(const NormParams p) {
    __shared__ float red[16];
    const int C = p.C;
    for (int64_t row = blockIdx.x; row < p.R; row += gridDim.x) {
        auto sum_at = [&](int c) {
            float2 v = unpack_bf16(__ldg(reinterpret_cast<const uint32_t*>(p.x + row * p.ldx + c)));
            if (p.residual) {
                const float2 r = ld2(static_cast<const TR*>(p.residual) + row * C + c);
                v = make_float2(v.x + r.x, v.y + r.y);
                if (sizeof(TR) == 2) v = unpack_bf16(pack_bf16(v.x, v.y));
            }
            return v;
        };
        auto stored = [&](int c) {  // the sum once it is written (residual_out may be the residual's buffer)
            return p.residual ? ld2(static_cast<const TR*>(static_cast<const void*>(p.res_out)) + row * C + c) : sum_at(c);
        };
        float ss = 0.f;
        for (int c = threadIdx.x * 2; c < C; c += 1024) {
            const float2 v = sum_at(c);
            ss = fmaf(v.x, v.x, fmaf(v.y, v.y, ss));
            if (p.residual) st2(static_cast<TR*>(p.res_out) + row * C + c, v);
        }
        const float rstd = rsqrtf(row_reduce<512, false>(ss, red) / C + p.eps);
        if (threadIdx.x == 0) p.rstd[row] = rstd;
        auto y_at = [&](int c) {
            const float2 v = stored(c), w = *reinterpret_cast<const float2*>(p.weight + c);
            return make_float2(v.x * rstd * w.x, v.y * rstd * w.y);
        };
        float most = 0.f;
        if (p.quant == 1) {
            for (int c = threadIdx.x * 2; c < C; c += 1024) {
                const float2 y = y_at(c);
                most = fmaxf(most, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
            most = row_reduce<512, true>(most, red);
        }
        const int nb = p.quant == 2 ? (C + 127) / 128 : 1;
        // (64 threads hold 128 channels; whole warps go round, so that each block of channels is whole)
        for (int c0 = 0; c0 < C; c0 += 1024) {
            const int c = c0 + threadIdx.x * 2;
            const float2 y = c < C ? y_at(c) : make_float2(0.f, 0.f);
            if (p.quant == 0) {
                if (c < C) st2(static_cast<__nv_bfloat16*>(p.y) + row * C + c, y);
                continue;
            }
            float m = most;
            if (p.quant == 2) {
                m = fmaxf(fabsf(y.x), fabsf(y.y));
#pragma unroll
                for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
                __syncthreads();
                if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = m;
                __syncthreads();
                m = fmaxf(red[threadIdx.x / 64 * 2], red[threadIdx.x / 64 * 2 + 1]);
            }
            const float scale = scale_of(m);
            if (c < C) {
                if (p.quant == 2 ? threadIdx.x % 64 == 0 : c == 0) p.scale[row * nb + (p.quant == 2 ? c / 128 : 0)] = scale;
                *reinterpret_cast<uint16_t*>(static_cast<unsigned char*>(p.y) + row * C + c) = (uint16_t)e4m3x2(y.x / scale, y.y / scale);
            }
        }
    }
}

// dx of a row held in registers, and dweight's sum over the rows of this group of threads, which
// walks the rows with the grid's stride: one partial row of sums for each block.
template <int G, int P, class TR, bool DRES>
__global__ void __launch_bounds__(G > 128 ? G : 128, P == 1 ? (768 + G - 1) / (G > 128 ? G : 128) : 1) k_rmsnorm_bwd(const NormParams p, int wide) {
    constexpr int THREADS = G > 128 ? G : 128, ROWS = THREADS / G;
    __shared__ float red[THREADS / 32];
    const int t = threadIdx.x % G, C = p.C;
    const float invC = 1.f / (float)C;
    Eight w[P], dw[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int c = (t + i * G) * 8 + q;
            w[i].v[q] = c < C ? p.weight[c] : 0.f;
            dw[i].v[q] = 0.f;
        }
    RawOf<TR> sr[P], dr[P];
    RawOf<__nv_bfloat16> yr[P];
    float next_rstd = 0.f;
    auto load = [&](int64_t row) {
        if (row < p.R) {
            next_rstd = p.rstd_in[row];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = (t + i * G) * 8;
                if (c < C) {
                    sr[i] = ld8(static_cast<const TR*>(p.s) + row * C + c, C - c, wide);
                    yr[i] = ld8(p.dy + row * C + c, C - c, wide);
                    if (DRES) dr[i] = ld8(static_cast<const TR*>(p.dres) + row * C + c, C - c, wide);
                }
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * ROWS;
    load((int64_t)blockIdx.x * ROWS + threadIdx.x / G);
    for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < p.R; row0 += step) {
        const int64_t row = row0 + threadIdx.x / G;
        const bool live = row < p.R;
        Eight s[P], dy[P], dres[DRES ? P : 1];
        float m = 0.f;
        const float rstd = next_rstd;
        if (live) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = (t + i * G) * 8;
                if (c < C) {
                    s[i] = sr[i].widen();
                    dy[i] = yr[i].widen();
                    if (DRES) dres[DRES ? i : 0] = dr[i].widen();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        s[i].v[q] *= rstd;  // n
                        dw[i].v[q] = fmaf(dy[i].v[q], s[i].v[q], dw[i].v[q]);
                        dy[i].v[q] *= w[i].v[q];  // u
                        m = fmaf(dy[i].v[q], s[i].v[q], m);
                    }
                }
            }
        }
        load(row + step);
        m = row_reduce<G, false>(m, red) * invC;
        if (!live) continue;  // (with several rows a block no barrier follows)
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (t + i * G) * 8;
            if (c < C) {
                Eight d;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    d.v[q] = rstd * fmaf(-m, s[i].v[q], dy[i].v[q]);
                    if (DRES) d.v[q] += dres[DRES ? i : 0].v[q];
                }
                st8n(static_cast<TR*>(p.dx) + row * C + c, d, C - c, wide);
            }
        }
    }
    if (ROWS > 1) {  // the groups' sums of a block, in a fixed order
        __shared__ Eight sums[ROWS > 1 ? THREADS : 1];
        sums[ROWS > 1 ? threadIdx.x : 0] = dw[0];
        __syncthreads();
        if (threadIdx.x >= G) return;
#pragma unroll
        for (int r = 1; r < ROWS; ++r)
#pragma unroll
            for (int q = 0; q < 8; ++q) dw[0].v[q] += sums[ROWS > 1 ? r * G + t : 0].v[q];
    }
    float* part = p.partial + (int64_t)blockIdx.x * C;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (t + i * G) * 8;
#pragma unroll
        for (int q = 0; q < 8; q += 2)
            if (c + q < C) *reinterpret_cast<float2*>(part + c + q) = make_float2(dw[i].v[q], dw[i].v[q + 1]);
    }
}

// Rows too long for registers: a block walks a row twice; the sums of its rows lie in its partial row.
template <class TR>
__global__ void __launch_bounds__(512) k_rmsnorm_bwd_long(const NormParams p) {
    __shared__ float red[16];
    const int C = p.C;
    float* part = p.partial + (int64_t)blockIdx.x * C;
    for (int c = threadIdx.x * 2; c < C; c += 1024) *reinterpret_cast<float2*>(part + c) = make_float2(0.f, 0.f);
    for (int64_t row = blockIdx.x; row < p.R; row += gridDim.x) {
        const float rstd = p.rstd_in[row];
        const int64_t at = row * C;
        float m = 0.f;
        for (int c = threadIdx.x * 2; c < C; c += 1024) {
            const float2 s = ld2(static_cast<const TR*>(p.s) + at + c), dy = ld2(p.dy + at + c);
            const float2 n = make_float2(s.x * rstd, s.y * rstd);
            m = fmaf(dy.x * p.weight[c], n.x, fmaf(dy.y * p.weight[c + 1], n.y, m));
            float2 d = *reinterpret_cast<float2*>(part + c);
            d = make_float2(fmaf(dy.x, n.x, d.x), fmaf(dy.y, n.y, d.y));
            *reinterpret_cast<float2*>(part + c) = d;
        }
        m = row_reduce<512, false>(m, red) / C;
        for (int c = threadIdx.x * 2; c < C; c += 1024) {
            const float2 s = ld2(static_cast<const TR*>(p.s) + at + c), dy = ld2(p.dy + at + c);
            float2 d = make_float2(rstd * fmaf(-m, s.x * rstd, dy.x * p.weight[c]), rstd * fmaf(-m, s.y * rstd, dy.y * p.weight[c + 1]));
            if (p.dres) {
                const float2 r = ld2(static_cast<const TR*>(p.dres) + at + c);
                d = make_float2(d.x + r.x, d.y + r.y);
            }
            st2(static_cast<TR*>(p.dx) + at + c, d);
        }
    }
}

// dweight: the partial rows added in a fixed order.  A block takes 32 channels, each of its 32 warps
// every 32nd row.  (The workspace's status word: there is nothing to report.)
__global__ void __launch_bounds__(1024) k_rmsnorm_dw(const float* partial, int rows, int C, float* dw, int* status) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    cudaGridDependencySynchronize();  // (launched ahead of the end of the kernel before it)
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
    if (c < C) {
#pragma unroll 8
        for (int i = w; i < rows; i += 32) v += partial[(int64_t)i * C + c];
    }
    part[w][lane] = v;
    __syncthreads();
    v = part[lane][w];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if (lane == 0 && blockIdx.x * 32 + w < C) dw[blockIdx.x * 32 + w] = v;
}

namespace {

// The threads that hold a row: the fewest with one piece of 8 channels each, up to 512 threads with
// four.  Longer rows go by the long kernels.
struct Split {
    int group, pieces;  // group 0: long
};
Split split_of(int C) {
    const int pieces = (C + 7) / 8;
    for (int g = 8; g <= 512; g *= 2)
        if (pieces <= g) return {g, 1};
    return pieces <= 1024 ? Split{512, 2} : pieces <= 1536 ? Split{512, 3} : pieces <= 2048 ? Split{512, 4} : Split{0, 0};
}

int grid_of(int64_t rows, int group, int per_sm) {
    const int in_block = group >= 128 ? 1 : 128 / group;
    const int64_t blocks = (rows + in_block - 1) / in_block, most = (int64_t)per_sm * num_sms();
    return (int)(blocks < most ? (blocks > 0 ? blocks : 1) : most);
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <class TR, bool RES, int QUANT>
cudaError_t fwd(const NormParams& p, cudaStream_t s) {
    const Split sp = split_of(p.C);
    const int wide = p.C % 8 == 0 && p.ldx % 8 == 0 && aligned(p.x);
    if (sp.group == 0) {
        k_rmsnorm_fwd_long<TR><<<grid_of(p.R, 512, 4), 512, 0, s>>>(p);
        return cudaGetLastError();
    }
    const int threads = sp.group > 128 ? sp.group : 128, grid = grid_of(p.R, sp.group, sp.pieces == 1 ? 1280 / threads : 1);
    switch (sp.group * 8 + sp.pieces) {
#define ROWS_OF(G, P)                                                               \
    case G * 8 + P:                                                                 \
        k_rmsnorm_fwd<G, P, TR, RES, QUANT><<<grid, threads, 0, s>>>(p, wide);      \
        break
        ROWS_OF(8, 1); ROWS_OF(16, 1); ROWS_OF(32, 1); ROWS_OF(64, 1); ROWS_OF(128, 1); ROWS_OF(256, 1); ROWS_OF(512, 1);
        ROWS_OF(512, 2); ROWS_OF(512, 3); ROWS_OF(512, 4);
#undef ROWS_OF
    }
    return cudaGetLastError();
}
template <class TR, bool RES>
cudaError_t fwd_q(const NormParams& p, cudaStream_t s) {
    return p.quant == 0 ? fwd<TR, RES, 0>(p, s) : p.quant == 1 ? fwd<TR, RES, 1>(p, s) : fwd<TR, RES, 2>(p, s);
}

template <class TR, bool DRES>
cudaError_t bwd(const NormParams& p, cudaStream_t s) {
    const Split sp = split_of(p.C);
    const int wide = p.C % 8 == 0, grid = rmsnorm_bwd_blocks(p.R, p.C);
    if (sp.group == 0) {
        k_rmsnorm_bwd_long<TR><<<grid, 512, 0, s>>>(p);
    } else {
        const int threads = sp.group > 128 ? sp.group : 128;
        switch (sp.group * 8 + sp.pieces) {
#define ROWS_OF(G, P)                                                               \
    case G * 8 + P:                                                                 \
        k_rmsnorm_bwd<G, P, TR, DRES><<<grid, threads, 0, s>>>(p, wide);            \
        break
            ROWS_OF(8, 1); ROWS_OF(16, 1); ROWS_OF(32, 1); ROWS_OF(64, 1); ROWS_OF(128, 1); ROWS_OF(256, 1); ROWS_OF(512, 1);
            ROWS_OF(512, 2); ROWS_OF(512, 3); ROWS_OF(512, 4);
#undef ROWS_OF
        }
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after((p.C + 31) / 32, 1024, s, k_rmsnorm_dw, (const float*)p.partial, grid, (int)p.C, p.dweight, p.status);
}

}  // namespace

// Blocks of the backward: what is resident without spilling registers (768 threads), so that each
// walks many rows and the partial rows stay few.
int rmsnorm_bwd_blocks(int64_t R, int C) {
    const Split sp = split_of(C);
    if (sp.group == 0) return grid_of(R, 512, 1);
    return grid_of(R, sp.group, sp.group == 512 ? (sp.pieces == 1 ? 2 : 1) : 768 / (sp.group > 128 ? sp.group : 128));
}
size_t rmsnorm_partial_bytes(int64_t R, int C) { return sizeof(float) * (size_t)rmsnorm_bwd_blocks(R, C) * C; }

cudaError_t launch_rmsnorm_fwd(const NormParams& p, cudaStream_t s) {
    if (!p.residual) return fwd_q<__nv_bfloat16, false>(p, s);
    return p.res_f32 ? fwd_q<float, true>(p, s) : fwd_q<__nv_bfloat16, true>(p, s);
}

cudaError_t launch_rmsnorm_bwd(const NormParams& p, cudaStream_t s) {
    if (p.res_f32) return p.dres ? bwd<float, true>(p, s) : bwd<float, false>(p, s);
    return p.dres ? bwd<__nv_bfloat16, true>(p, s) : bwd<__nv_bfloat16, false>(p, s);
}

}  // namespace gdr
