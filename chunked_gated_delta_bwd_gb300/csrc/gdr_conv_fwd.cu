// Causal depthwise conv1d (optionally followed by SiLU), forward and single-token step; the
// backward is in gdr_conv.cu.  Per channel c, K taps:
//
//   z_t = bias_c + sum_k w_{c,k} x_{t-K+1+k},   y = SiLU(z) (or y = z)
//
// Before a sequence's first token x continues into the given state (its last K - 1 inputs,
// oldest first) or is zero; the state after the sequence is the last K - 1 inputs of both.
//
// The simplest form: a thread computes two channels of one token.
#include "gdr_block.h"
#include "gdr_common.cuh"

namespace gdr {

namespace {

constexpr int NT = 128;

__device__ __forceinline__ int64_t seq_begin(const ConvFwdParams& p, int n) {
    return p.cu_seqlens ? p.cu_seqlens[n] : (int64_t)n * p.seq_len;
}
__device__ __forceinline__ float silu_f(float z) { return z * sigmoid_f(z); }

}  // namespace

template <int K>
__global__ void __launch_bounds__(NT) k_conv1d_fwd(const ConvFwdParams p) {
    const int c = (blockIdx.x * NT + threadIdx.x) * 2;
    if (c >= p.C) return;
    for (int64_t t = blockIdx.y; t < p.T; t += gridDim.y) {
        int lo = 0, hi = p.N - 1;  // the sequence holding t: largest n that begins at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_begin(p, mid) <= t) lo = mid;
            else hi = mid - 1;
        }
        const int64_t begin = seq_begin(p, lo);
        float2 z = p.bias ? make_float2(p.bias[c], p.bias[c + 1]) : make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t at = t - (K - 1) + k;
            uint32_t v = 0;
            if (at >= begin && at >= 0) v = *reinterpret_cast<const uint32_t*>(p.x + at * p.ldx + c);
            else if (p.state && at - begin >= -(K - 1) && at < begin)
                v = *reinterpret_cast<const uint32_t*>(p.state + ((int64_t)lo * (K - 1) + (K - 1) + (at - begin)) * p.C + c);
            const float2 x = unpack_bf16(v);
            z.x = fmaf(p.w[c * K + k], x.x, z.x);
            z.y = fmaf(p.w[(c + 1) * K + k], x.y, z.y);
        }
        if (p.silu) z = make_float2(silu_f(z.x), silu_f(z.y));
        *reinterpret_cast<uint32_t*>(p.y + t * p.C + c) = pack_bf16(z.x, z.y);
    }
}

// the states after the sequences: row j of sequence n is the input K - 1 - j tokens before its end
__global__ void __launch_bounds__(NT) k_conv1d_state(const ConvFwdParams p) {
    const int c = (blockIdx.x * NT + threadIdx.x) * 2;
    if (c >= p.C) return;
    const int K1 = p.K - 1;
    for (int n = blockIdx.y; n < p.N; n += gridDim.y) {
        const int64_t b = min(max(seq_begin(p, n), (int64_t)0), p.T);
        const int64_t e = min(max(seq_begin(p, n + 1), b), p.T);
        for (int j = 0; j < K1; ++j) {
            const int64_t at = e - K1 + j;
            uint32_t v = 0;
            if (at >= b) v = *reinterpret_cast<const uint32_t*>(p.x + at * p.ldx + c);
            else if (p.state) v = *reinterpret_cast<const uint32_t*>(p.state + ((int64_t)n * K1 + j + (e - b)) * p.C + c);
            *reinterpret_cast<uint32_t*>(p.state_out + ((int64_t)n * K1 + j) * p.C + c) = v;
        }
    }
}

// One token for each row on the row's state, in place.  A row whose slot is negative (padding
// of the batch) or past the pool reads and writes no state; its y is zero.
template <int K>
__global__ void __launch_bounds__(NT) k_conv1d_step(const ConvFwdParams p) {
    const int c = (blockIdx.x * NT + threadIdx.x) * 2;
    if (c >= p.C) return;
    for (int64_t n = blockIdx.y; n < p.N; n += gridDim.y) {
        const int64_t slot = p.slots ? p.slots[n] : n;
        uint32_t out = 0;
        if (slot >= 0 && slot < p.pool) {
            uint32_t x[K];
            __nv_bfloat16* home = p.state_out + slot * (K - 1) * p.C + c;
#pragma unroll
            for (int k = 0; k < K - 1; ++k) x[k] = *reinterpret_cast<const uint32_t*>(home + (int64_t)k * p.C);
            x[K - 1] = *reinterpret_cast<const uint32_t*>(p.x + n * p.ldx + c);
            float2 z = p.bias ? make_float2(p.bias[c], p.bias[c + 1]) : make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float2 v = unpack_bf16(x[k]);
                z.x = fmaf(p.w[c * K + k], v.x, z.x);
                z.y = fmaf(p.w[(c + 1) * K + k], v.y, z.y);
            }
#pragma unroll
            for (int k = 0; k < K - 1; ++k) *reinterpret_cast<uint32_t*>(home + (int64_t)k * p.C) = x[k + 1];
            if (p.silu) z = make_float2(silu_f(z.x), silu_f(z.y));
            out = pack_bf16(z.x, z.y);
        }
        *reinterpret_cast<uint32_t*>(p.y + n * p.C + c) = out;
    }
}

namespace {

template <int K>
cudaError_t fwd_k(const ConvFwdParams& p, cudaStream_t s) {
    const unsigned gx = (p.C / 2 + NT - 1) / NT;
    if (p.T) k_conv1d_fwd<K><<<dim3(gx, (unsigned)(p.T < 65535 ? p.T : 65535)), NT, 0, s>>>(p);
    if (p.state_out && K > 1) k_conv1d_state<<<dim3(gx, p.N < 65535 ? p.N : 65535), NT, 0, s>>>(p);
    return cudaGetLastError();
}
template <int K>
cudaError_t step_k(const ConvFwdParams& p, cudaStream_t s) {
    k_conv1d_step<K><<<dim3((p.C / 2 + NT - 1) / NT, p.N < 65535 ? p.N : 65535), NT, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_conv1d_fwd(const ConvFwdParams& p, cudaStream_t s) {
    switch (p.K) {
        case 1: return fwd_k<1>(p, s);
        case 2: return fwd_k<2>(p, s);
        case 3: return fwd_k<3>(p, s);
        case 4: return fwd_k<4>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_conv1d_step(const ConvFwdParams& p, cudaStream_t s) {
    switch (p.K) {
        case 1: return step_k<1>(p, s);
        case 2: return step_k<2>(p, s);
        case 3: return step_k<3>(p, s);
        case 4: return step_k<4>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gdr
