// Launch parameters of the 8-bit products: the quantisation and the product.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdr {

struct QuantParams {
    int64_t R, ldx;
    int C, x_f32, tiles;
    const void* x;           // [R][C], rows of stride ldx
    uint8_t *y, *yt;         // [R][C], [C][R] or nullptr
    float *scale, *scale_t;
};
cudaError_t launch_quant(const QuantParams& p, cudaStream_t s);

struct LinearParams {
    int64_t M;
    int K, N, x_blocks;            // x_blocks: scales of a row of x (1 or one for each 128 of K)
    const uint8_t *x, *w;          // e4m3 [M][K], [N][K]
    const float *xs, *ws, *bias;   // [M][x_blocks], [ceil(N / 128)][ceil(K / 128)], [N] or nullptr
    __nv_bfloat16* y;              // [M][N]
};
cudaError_t launch_linear(const LinearParams& p, cudaStream_t s);

}  // namespace gdr
