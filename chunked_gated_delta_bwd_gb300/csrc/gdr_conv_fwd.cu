// Causal depthwise conv1d (optionally followed by SiLU), forward and single-token step; the
// backward is in gdr_conv.cu.  Per channel c, K taps:
//
//   z_t = bias_c + sum_k w_{c,k} x_{t-K+1+k},   y = SiLU(z) (or y = z)
//
// Before a sequence's first token x continues into the given state (its last K - 1 inputs,
// oldest first) or is zero; the state after the sequence is the last K - 1 inputs of both.
//
// Bytes bound the forward (x once in, y once out).  A thread owns four channels (8 bytes of bf16 a
// token, or two where rows are not whole numbers of aligned 8-byte pieces) and walks a tile of
// tokens with the last K - 1 inputs in registers, eight tokens' loads issued together.  The
// sigmoid is 1 / (1 + 2^{-z / ln 2}) on the hardware exponential and reciprocal (2^-22 relative;
// y is rounded to bf16).
#include "gdr_block.h"
#include "gdr_common.cuh"
#include "gdr_internal.h"

namespace gdr {

namespace {

constexpr int NT = 128;
constexpr int AHEAD = 8;  // tokens whose loads are issued together

__device__ __forceinline__ int64_t seq_begin(const ConvFwdParams& p, int n) {
    return p.cu_seqlens ? p.cu_seqlens[n] : (int64_t)n * p.seq_len;
}
__device__ __forceinline__ float silu_f(float z) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(-1.4426950408889634f * z));
    return __fdividef(z, 1.f + e);
}

// V channels of a token as loaded
template <int V> struct Raw;
template <> struct Raw<2> { uint32_t u[1]; };
template <> struct __align__(8) Raw<4> { uint32_t u[2]; };
template <int V>
__device__ __forceinline__ Raw<V> ld_raw(const __nv_bfloat16* p) {
    Raw<V> r;
    if (V == 2) {
        r.u[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        r.u[0] = v.x;
        r.u[V / 2 - 1] = v.y;
    }
    return r;
}
// the same of memory that the kernel writes
template <int V>
__device__ __forceinline__ Raw<V> ld_state(const __nv_bfloat16* p) {
    return *reinterpret_cast<const Raw<V>*>(p);
}
template <int V>
__device__ __forceinline__ void st_raw(__nv_bfloat16* p, const Raw<V>& r) {
    if (V == 2) *reinterpret_cast<uint32_t*>(p) = r.u[0];
    else *reinterpret_cast<uint2*>(p) = make_uint2(r.u[0], r.u[V / 2 - 1]);
}
template <int V>
__device__ __forceinline__ Raw<V> no_raw() {
    Raw<V> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.u[i] = 0;
    return r;
}

// one thread's channels: weights, bias and the last K - 1 inputs
template <int K, int V, bool SILU>
struct Lane {
    float2 w[K][V / 2], bias[V / 2], win[K > 1 ? K - 1 : 1][V / 2];
    __device__ __forceinline__ void load(const ConvFwdParams& p, int c) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            bias[i] = p.bias ? *reinterpret_cast<const float2*>(p.bias + c + 2 * i) : make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][i] = make_float2(p.w[(c + 2 * i) * K + k], p.w[(c + 2 * i + 1) * K + k]);
        }
    }
    __device__ __forceinline__ void push(const float2 (&x)[V / 2]) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
#pragma unroll
            for (int k = 0; k + 2 < K; ++k) win[k][i] = win[k + 1][i];
            if (K > 1) win[K > 1 ? K - 2 : 0][i] = x[i];
        }
    }
    __device__ __forceinline__ void push(const Raw<V>& r) {
        float2 x[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) x[i] = unpack_bf16(r.u[i]);
        push(x);
    }
    __device__ __forceinline__ Raw<V> token(const Raw<V>& r) {
        float2 x[V / 2];
        Raw<V> y;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            x[i] = unpack_bf16(r.u[i]);
            float2 z = __ffma2_rn(w[K - 1][i], x[i], bias[i]);
#pragma unroll
            for (int k = 0; k < K - 1; ++k) z = __ffma2_rn(w[k][i], win[k][i], z);
            if (SILU) z = make_float2(silu_f(z.x), silu_f(z.y));
            y.u[i] = pack_bf16(z.x, z.y);
        }
        push(x);
        return y;
    }
};

}  // namespace

// Items: `tiles` tiles of `len` tokens (a multiple of AHEAD) for each group of V channels, then, if
// states are wanted, the sequences' last K - 1 inputs for each group.
template <int K, int V, bool SILU>
__global__ void __launch_bounds__(NT, 6) k_conv1d_fwd(const ConvFwdParams p, int len, int64_t tiles, int64_t items) {
    const int groups = (p.C + V - 1) / V;
    const int64_t item = (int64_t)blockIdx.x * NT + threadIdx.x;
    if (item >= items) return;
    const int64_t tile = item / groups;
    const int c = (int)(item - tile * groups) * V;
    const __nv_bfloat16* x = p.x + c;
    if (tile >= tiles) {  // the state after sequence n: row j is the input K - 1 - j tokens before its end
        const int n = (int)(tile - tiles);
        const int64_t b = min(max(seq_begin(p, n), (int64_t)0), p.T), e = min(max(seq_begin(p, n + 1), b), p.T);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int64_t at = e - (K - 1) + j;
            Raw<V> v = no_raw<V>();
            if (at >= b) v = ld_raw<V>(x + at * p.ldx);
            else if (p.state) v = ld_raw<V>(p.state + ((int64_t)n * (K - 1) + j + (e - b)) * p.C + c);
            st_raw<V>(p.state_out + ((int64_t)n * (K - 1) + j) * p.C + c, v);
        }
        return;
    }
    const int64_t t0 = tile * len, t1 = min(t0 + len, p.T);
    int lo = 0;  // the sequence holding t0: largest n that begins at or before t0
    if (p.cu_seqlens) {
        int hi = p.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cu_seqlens[mid] <= t0) lo = mid;
            else hi = mid - 1;
        }
    } else if (p.N > 1) {
        lo = (int)(t0 / p.seq_len);
    }
    Lane<K, V, SILU> L;
    L.load(p, c);
    __nv_bfloat16* y = p.y + t0 * p.C + c;
    int64_t begin = seq_begin(p, lo), end = seq_begin(p, lo + 1);
    if (t1 - t0 == len && t0 - (K - 1) >= begin && t0 >= K - 1 && t1 <= end) {  // inside one sequence
        const __nv_bfloat16* at = x + (t0 - (K - 1)) * p.ldx;
#pragma unroll
        for (int k = 0; k < K - 1; ++k, at += p.ldx) L.push(ld_raw<V>(at));
#pragma unroll 1
        for (int i = 0; i < len; i += AHEAD) {
            Raw<V> r[AHEAD];
#pragma unroll
            for (int q = 0; q < AHEAD; ++q, at += p.ldx) r[q] = ld_raw<V>(at);
#pragma unroll
            for (int q = 0; q < AHEAD; ++q, y += p.C) st_raw<V>(y, L.token(r[q]));
        }
        return;
    }
    // token by token; `fresh`: the window is to be set up for token t of sequence lo
    bool fresh = true;
#pragma unroll 1
    for (int64_t t = t0; t < t1; ++t, y += p.C) {
        while (t >= end && lo < p.N - 1) {  // (past empty sequences)
            ++lo;
            begin = end;
            end = seq_begin(p, lo + 1);
            fresh = true;
        }
        if (fresh) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k) {
                const int64_t at = t - (K - 1) + k, local = at - begin;
                Raw<V> v = no_raw<V>();
                if (local >= 0 && at >= 0) v = ld_raw<V>(x + at * p.ldx);
                else if (p.state && local >= -(K - 1) && local < 0)
                    v = ld_raw<V>(p.state + ((int64_t)lo * (K - 1) + (K - 1) + local) * p.C + c);
                L.push(v);
            }
            fresh = false;
        }
        st_raw<V>(y, L.token(ld_raw<V>(x + t * p.ldx)));
    }
}

// One token for each row on the row's state, in place.  A row whose slot is negative (padding
// of the batch) or past the pool reads and writes no state; its y is zero.  A thread takes V
// channels as the forward's and asks for its input and weights while the slot is on its way:
// 257 x 6144 with slots, K = 4, from cold caches: 9.9 us (11.4 with two channels and the slot first).
template <int K, int V>
__global__ void __launch_bounds__(NT) k_conv1d_step(const ConvFwdParams p) {
    const int c = (blockIdx.x * NT + threadIdx.x) * V;
    if (c >= p.C) return;
    for (int64_t n = blockIdx.y; n < p.N; n += gridDim.y) {
        const int64_t slot = p.slots ? p.slots[n] : n;
        Raw<V> x[K], out = no_raw<V>();
        x[K - 1] = ld_raw<V>(p.x + n * p.ldx + c);
        float w[V * K];
#pragma unroll
        for (int i = 0; i < V * K / 2; ++i) {
            const float2 v = *reinterpret_cast<const float2*>(p.w + c * K + 2 * i);
            w[2 * i] = v.x;
            w[2 * i + 1] = v.y;
        }
        float2 z[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            z[i] = p.bias ? *reinterpret_cast<const float2*>(p.bias + c + 2 * i) : make_float2(0.f, 0.f);
        if (slot >= 0 && slot < p.pool) {
            __nv_bfloat16* home = p.state_out + slot * (K - 1) * p.C + c;
#pragma unroll
            for (int k = 0; k < K - 1; ++k) x[k] = ld_state<V>(home + (int64_t)k * p.C);
#pragma unroll
            for (int k = 0; k < K - 1; ++k) st_raw<V>(home + (int64_t)k * p.C, x[k + 1]);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float2 v = unpack_bf16(x[k].u[i]);
                    z[i].x = fmaf(w[2 * i * K + k], v.x, z[i].x);
                    z[i].y = fmaf(w[(2 * i + 1) * K + k], v.y, z[i].y);
                }
                if (p.silu) z[i] = make_float2(silu_f(z[i].x), silu_f(z[i].y));
                out.u[i] = pack_bf16(z[i].x, z[i].y);
            }
        }
        st_raw<V>(p.y + n * p.C + c, out);
    }
}

namespace {

template <int K, int V>
cudaError_t fwd_kv(const ConvFwdParams& p, cudaStream_t s) {
    const int groups = (p.C + V - 1) / V;
    // tiles of up to 64 tokens (the K - 1 inputs before a tile are read again), shorter as long as
    // there are not four rounds of resident blocks: 65536 tokens of 512 channels in 64 sequences took
    // 65 us with one round of 64 tokens, 48 us so
    int len = 64;
    while (len > AHEAD && (p.T + len - 1) / len * groups < (int64_t)num_sms() * NT * 6 * 4) len /= 2;
    const int64_t tiles = (p.T + len - 1) / len, items = (tiles + (p.state_out && K > 1 ? p.N : 0)) * groups;
    if (items == 0) return cudaSuccess;
    const unsigned grid = (unsigned)((items + NT - 1) / NT);
    if (p.silu) k_conv1d_fwd<K, V, true><<<grid, NT, 0, s>>>(p, len, tiles, items);
    else k_conv1d_fwd<K, V, false><<<grid, NT, 0, s>>>(p, len, tiles, items);
    return cudaGetLastError();
}
bool four_wide(const ConvFwdParams& p) {
    return p.C % 4 == 0 && p.ldx % 4 == 0 && (reinterpret_cast<uintptr_t>(p.x) & 7) == 0;
}
template <int K>
cudaError_t fwd_k(const ConvFwdParams& p, cudaStream_t s) {
    return four_wide(p) ? fwd_kv<K, 4>(p, s) : fwd_kv<K, 2>(p, s);
}
template <int K>
cudaError_t step_k(const ConvFwdParams& p, cudaStream_t s) {
    const unsigned rows = p.N < 65535 ? p.N : 65535;
    if (four_wide(p)) k_conv1d_step<K, 4><<<dim3((p.C / 4 + NT - 1) / NT, rows), NT, 0, s>>>(p);
    else k_conv1d_step<K, 2><<<dim3((p.C / 2 + NT - 1) / NT, rows), NT, 0, s>>>(p);
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
