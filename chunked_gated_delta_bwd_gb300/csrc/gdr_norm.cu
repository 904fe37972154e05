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
// The simplest form: one block per row (forward, dx), one thread per channel (dweight).
#include <cuda_fp8.h>

#include "gdr_block.h"
#include "gdr_common.cuh"

namespace gdr {

namespace {

constexpr int NT = 128;

__device__ __forceinline__ float ld(const void* p, int f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void st(void* p, int f32, int64_t i, float v) {
    if (f32) static_cast<float*>(p)[i] = v;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// over the block's threads; every thread gets the result
__device__ float block_reduce(float v, bool max_of) {
    __shared__ float part[NT / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float w = __shfl_xor_sync(~0u, v, o);
        v = max_of ? fmaxf(v, w) : v + w;
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = part[0];
    for (int i = 1; i < NT / 32; ++i) v = max_of ? fmaxf(v, part[i]) : v + part[i];
    return v;
}

// element i of the stored sum
__device__ __forceinline__ float sum_at(const NormParams& p, int64_t row, int i) {
    const float x = __bfloat162float(p.x[row * p.ldx + i]);
    if (!p.residual) return x;
    const float s = x + ld(p.residual, p.res_f32, row * p.C + i);
    return p.res_f32 ? s : __bfloat162float(__float2bfloat16_rn(s));
}

__global__ void __launch_bounds__(NT) k_rmsnorm_fwd(const NormParams p) {
    const int64_t row = blockIdx.x;
    float ss = 0.f;
    for (int i = threadIdx.x; i < p.C; i += NT) {
        const float s = sum_at(p, row, i);
        ss = fmaf(s, s, ss);
        if (p.res_out) st(p.res_out, p.res_f32, row * p.C + i, s);
    }
    const float rstd = rsqrtf(block_reduce(ss, false) / p.C + p.eps);
    if (threadIdx.x == 0) p.rstd[row] = rstd;
    if (p.quant == 0) {
        for (int i = threadIdx.x; i < p.C; i += NT)
            st(p.y, 0, row * p.C + i, sum_at(p, row, i) * rstd * p.weight[i]);
        return;
    }
    const int block = p.quant == 1 ? p.C : 128, nb = (p.C + block - 1) / block;
    for (int b = 0; b < nb; ++b) {
        const int end = min(p.C, (b + 1) * block);
        float most = 0.f;
        for (int i = b * block + threadIdx.x; i < end; i += NT)
            most = fmaxf(most, fabsf(sum_at(p, row, i) * rstd * p.weight[i]));
        most = block_reduce(most, true);
        const float scale = most > 0.f ? most / 448.f : 1.f;
        if (threadIdx.x == 0) p.scale[row * nb + b] = scale;
        for (int i = b * block + threadIdx.x; i < end; i += NT) {
            const float y = sum_at(p, row, i) * rstd * p.weight[i];
            static_cast<__nv_fp8_storage_t*>(p.y)[row * p.C + i] = __nv_cvt_float_to_fp8(y / scale, __NV_SATFINITE, __NV_E4M3);
        }
    }
}

__global__ void __launch_bounds__(NT) k_rmsnorm_dx(const NormParams p) {
    const int64_t row = blockIdx.x;
    const float rstd = p.rstd_in[row];
    float m = 0.f;
    for (int i = threadIdx.x; i < p.C; i += NT)
        m = fmaf(ld(p.s, p.res_f32, row * p.C + i) * rstd, __bfloat162float(p.dy[row * p.C + i]) * p.weight[i], m);
    m = block_reduce(m, false) / p.C;
    for (int i = threadIdx.x; i < p.C; i += NT) {
        const int64_t at = row * p.C + i;
        const float n = ld(p.s, p.res_f32, at) * rstd;
        float d = rstd * (__bfloat162float(p.dy[at]) * p.weight[i] - n * m);
        if (p.dres) d += ld(p.dres, p.res_f32, at);
        st(p.dx, p.res_f32, at, d);
    }
}

__global__ void __launch_bounds__(NT) k_rmsnorm_dw(const NormParams p) {
    const int i = blockIdx.x * NT + threadIdx.x;
    if (i >= p.C) return;
    float d = 0.f;
    for (int64_t row = 0; row < p.R; ++row)
        d = fmaf(__bfloat162float(p.dy[row * p.C + i]), ld(p.s, p.res_f32, row * p.C + i) * p.rstd_in[row], d);
    p.dweight[i] = d;
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(const NormParams& p, cudaStream_t s) {
    if (p.R == 0) return cudaSuccess;
    k_rmsnorm_fwd<<<(unsigned)p.R, NT, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_rmsnorm_bwd(const NormParams& p, cudaStream_t s) {
    if (p.R) k_rmsnorm_dx<<<(unsigned)p.R, NT, 0, s>>>(p);
    k_rmsnorm_dw<<<(p.C + NT - 1) / NT, NT, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gdr
