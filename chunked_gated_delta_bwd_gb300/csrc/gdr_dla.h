// Launch parameters of linear attention with a decay for each head.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdr {

struct DlaParams {
    int N, H, Hk, D;
    int64_t T, seq_len;            // tokens; dense layout: tokens per sequence
    const int64_t* cu_seqlens;     // device [N+1] or nullptr (dense)
    float scale;
    int64_t ldq, ldk, ldv;         // token strides in elements
    const __nv_bfloat16 *q, *k, *v, *dO;
    const float *g, *h0, *dht;     // [H], [N][H][D][D] or nullptr
    __nv_bfloat16 *o, *dq, *dk, *dv;
    float *ht, *dh0;
    int* status;                   // workspace: status word
    float* states;                 // workspace: states between the ranges of a split call
    float *dq_heads, *dk_heads;    // workspace: [T][H][D] per value head, where heads share q and k
};
size_t dla_states_bytes(const DlaParams& p, bool backward);
cudaError_t launch_dla_fwd(const DlaParams& p, cudaStream_t s);
cudaError_t launch_dla_bwd(const DlaParams& p, cudaStream_t s);
int dla_kernels(const DlaParams& p, bool backward);  // kernels that a launch enqueues

struct DlaStepParams {
    int rows, H, Hk, D, pool;
    float scale;
    int64_t ldq, ldk, ldv;
    const __nv_bfloat16 *q, *k, *v;
    const float* g;
    const int64_t* slots;  // [rows] or nullptr (row n has state n)
    float* state;          // [pool][H][D][D], updated in place
    __nv_bfloat16* o;
};
cudaError_t launch_dla_step(const DlaStepParams& p, cudaStream_t s);
int dla_step_kernels(const DlaStepParams& p);  // kernels that a launch enqueues

}  // namespace gdr
