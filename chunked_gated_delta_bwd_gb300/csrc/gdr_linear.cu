// The product of e4m3 operands with a scale for each block of 128 of the inner dimension.
#include <cuda_fp8.h>

#include "gdr_common.cuh"
#include "gdr_e4m3.h"

namespace gdr {
namespace {

__device__ __forceinline__ float wide8(uint8_t c) {
    __nv_fp8_e4m3 v;
    v.__x = c;
    return float(v);
}

// 64 x 64 outputs a block, 4 x 4 a thread, 16 of the inner dimension at a time
__global__ void __launch_bounds__(256) k_linear(const LinearParams p) {
    __shared__ float a[16][68], b[16][68];
    const int64_t m0 = (int64_t)blockIdx.x * 64;
    const int n0 = blockIdx.y * 64, tx = threadIdx.x % 16, ty = threadIdx.x / 16, nb = (p.K + 127) / 128;
    float acc[4][4] = {};
    for (int kb = 0; kb < nb; ++kb) {
        float part[4][4] = {};
        for (int k0 = kb * 128; k0 < p.K && k0 < kb * 128 + 128; k0 += 16) {
            __syncthreads();
            for (int i = threadIdx.x; i < 1024; i += 256) {
                const int r = i / 16, k = i % 16;
                a[k][r] = m0 + r < p.M ? wide8(p.x[(m0 + r) * p.K + k0 + k]) : 0.f;
                b[k][r] = n0 + r < p.N ? wide8(p.w[(int64_t)(n0 + r) * p.K + k0 + k]) : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 16; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[i][j] = fmaf(a[k][ty * 4 + i], b[k][tx * 4 + j], part[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + ty * 4 + i;
            const float s = m < p.M ? p.xs[m * p.x_blocks + (p.x_blocks > 1 ? kb : 0)] : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                if (n < p.N) acc[i][j] = fmaf(part[i][j], s * p.ws[(int64_t)(n / 128) * nb + kb], acc[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty * 4 + i;
            const int n = n0 + tx * 4 + j;
            if (m < p.M && n < p.N) p.y[m * p.N + n] = __float2bfloat16(acc[i][j] + (p.bias ? p.bias[n] : 0.f));
        }
}

}  // namespace

cudaError_t launch_linear(const LinearParams& p, cudaStream_t s) {
    k_linear<<<dim3((unsigned)((p.M + 63) / 64), (p.N + 63) / 64), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gdr
