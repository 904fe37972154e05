// Launch parameters of the operators around the delta rule in a recurrent block: the gated
// linear recurrence, the RMS norm with residual and the causal conv1d's forward.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdr {

// Launches a kernel that adds up what the kernel before it wrote, with its blocks already in place
// when that ends (it begins with cudaGridDependencySynchronize): 3 us of 51 in the norm's backward.
template <class... P, class... A>
cudaError_t launch_after(unsigned grid, unsigned threads, cudaStream_t s, void (*kernel)(P...), A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// gated linear recurrence (glr_fwd / glr_bwd)
struct GlrParams {
    int N, C;                   // sequences, channels (even)
    int64_t T;                  // tokens
    int64_t seq_len;            // dense layout: tokens per sequence (T / N)
    double inv_len;             // 1 / seq_len
    const int64_t* cu_seqlens;  // device [N+1] or nullptr (dense)
    int64_t ldx, ldg;           // row strides of x and g in elements
    int gate, complement;       // gate function (gdr.h), x scaled by 1 - a
    int act_f32, gate_f32;      // element types: float32 instead of bf16
    int test_stall;             // test hook: block index + 1 held at its second tile (0: none)
    int wide;                   // every row of every tensor read is a whole number of aligned 16-byte pieces
    int* status;                // workspace: status word, ticket counter, published runs
    float4* sums;               // workspace: per-chunk sums of the softplus gate's parameters
    const void *x, *g;          // [T][C]
    const float *A_log, *dt_bias;  // [C] (softplus gate)
    const float *h0, *dht;      // [N][C] or nullptr
    const void *h_in, *dh;      // backward: the forward's h, dL/dh [T][C]
    void *h, *dx, *dg;          // [T][C]
    float *ht, *dh0;            // [N][C]; ht may be nullptr
    float *dA_log, *ddt_bias;   // [C] (softplus gate)
};
// workspace: the status word and a ticket counter, then what the kernels publish (zero before a
// launch), then the backward's per-chunk sums
size_t glr_published_bytes(const GlrParams& p);
size_t glr_sums_bytes(const GlrParams& p);
cudaError_t launch_glr_fwd(const GlrParams& p, cudaStream_t s);
cudaError_t launch_glr_bwd(const GlrParams& p, cudaStream_t s);

// one token of the recurrence for each of N rows (glr_step)
struct GlrStepParams {
    int N, C, pool;
    int gate, complement, act_f32, gate_f32;
    int64_t ldx, ldg;
    const void *x, *g;             // [N][C]
    const float *A_log, *dt_bias;  // [C]
    const int64_t* slots;          // [N] or nullptr (row n has state n)
    float* state;                  // [pool][C], updated in place
    void* y;                       // [N][C]
};
cudaError_t launch_glr_step(const GlrStepParams& p, cudaStream_t s);

// RMS norm with the residual's addition (gdr_rmsnorm_fwd / gdr_rmsnorm_bwd)
struct NormParams {
    int64_t R;                   // rows
    int C;                       // channels (even)
    int64_t ldx;                 // row stride of x in elements
    int res_f32;                 // residual stream in float32 instead of bf16
    int quant;                   // output: 0 bf16, 1 e4m3 with a scale per row, 2 per 128 channels
    float eps;
    const __nv_bfloat16* x;      // [R][C]
    const void* residual;        // [R][C] or nullptr
    const float* weight;         // [C]
    void *y, *res_out;           // [R][C]; res_out nullptr without a residual
    float *scale, *rstd;         // [R][blocks], [R]
    // backward
    const void *s, *dres;        // the stored sum, its gradient or nullptr [R][C]
    const __nv_bfloat16* dy;     // [R][C]
    const float* rstd_in;        // [R]
    void* dx;                    // [R][C], of the residual stream's type
    float* dweight;              // [C]
    int* status;                 // workspace: status word
    float* partial;              // workspace: sums of dweight, a row for each group of threads
};
int rmsnorm_bwd_blocks(int64_t R, int C);
size_t rmsnorm_partial_bytes(int64_t R, int C);
cudaError_t launch_rmsnorm_fwd(const NormParams& p, cudaStream_t s);
cudaError_t launch_rmsnorm_bwd(const NormParams& p, cudaStream_t s);

// causal depthwise conv1d forward (gdr_conv1d_fwd) and its single-token form (gdr_conv1d_step)
struct ConvFwdParams {
    int N;                       // sequences; rows of the step
    int64_t T, seq_len;
    int C, K, silu;
    int64_t ldx;
    const int64_t* cu_seqlens;
    const __nv_bfloat16* x;      // [T][C]
    const float *w, *bias;       // [C][K], [C] or nullptr
    const __nv_bfloat16* state;  // [N][K-1][C] or nullptr (zero)
    __nv_bfloat16* state_out;    // [N][K-1][C] or nullptr
    __nv_bfloat16* y;            // [T][C]
    const int64_t* slots;        // step: [N] or nullptr
    int pool;                    // step: states in the pool
};
cudaError_t launch_conv1d_fwd(const ConvFwdParams& p, cudaStream_t s);
cudaError_t launch_conv1d_step(const ConvFwdParams& p, cudaStream_t s);

}  // namespace gdr
