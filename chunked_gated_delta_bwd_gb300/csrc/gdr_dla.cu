// Linear attention with a decay for each head, forward and backward: the recurrence token by token.
//
// All outputs are one operator with three operands (X, Y, Z), walked forward or backward in time:
//   C' = e^g C + y z^T  (forward: before the output;  backward: after it, the decay last),  out = x C
// o: (q, k, v);  dq: (dO, v, k) forward;  dv: (k, q, dO), dk: (v, dO, q) backward.
#include "gdr_common.cuh"
#include "gdr_dla.h"
#include "gdr_internal.h"

namespace gdr {
namespace {

struct Role {
    const __nv_bfloat16 *x, *y, *z;
    int64_t ldx, ldy, ldz;
    int gx, gy, gz;       // value heads that share a head of it
    int back, turned;     // walked backward; the states' key channels are the columns
    float y_scale, o_scale;
    const float* init;
    float* final_state;
    __nv_bfloat16* out;
    float* out32;
};

// e^g S + t as c2 S + (c1 S + t): a decay near 1 by its distance from 1, so that its rounding does not add
// up over thousands of tokens
__device__ __forceinline__ float2 decay_of(float g) {
    return g > -0.5f && g < 0.5f ? make_float2(expm1f(g), 1.f) : make_float2(expf(g < -1e4f ? -1e4f : g), 0.f);
}

// one block a (sequence, head); thread = column of the state
template <int D>
__global__ void __launch_bounds__(D) k_dla(const DlaParams p, const Role r) {
    __shared__ float xs[D], ys[D];
    const int n = blockIdx.x / p.H, h = blockIdx.x % p.H, e = threadIdx.x;
    int64_t b = n * p.seq_len, end = b + p.seq_len;
    if (p.cu_seqlens) {
        b = p.cu_seqlens[n];
        end = p.cu_seqlens[n + 1];
        if (b < 0 || end < b || end > p.T || p.cu_seqlens[0] != 0 || p.cu_seqlens[p.N] != p.T) {
            if (e == 0) atomicOr(p.status, ST_BAD_SEQLENS);
            return;
        }
    }
    float S[D];
    const int64_t base = (int64_t)blockIdx.x * D * D;
    for (int d = 0; d < D; ++d) S[d] = r.init ? r.init[base + (r.turned ? e * D + d : d * D + e)] : 0.f;
    const float2 a = decay_of(p.g[h]);
    for (int64_t i = 0; i < end - b; ++i) {
        const int64_t t = r.back ? end - 1 - i : b + i;
        __syncthreads();
        xs[e] = bf2f(r.x[t * r.ldx + h / r.gx * D + e]);
        ys[e] = bf2f(r.y[t * r.ldy + h / r.gy * D + e]) * r.y_scale;
        const float z = bf2f(r.z[t * r.ldz + h / r.gz * D + e]);
        __syncthreads();
        float o = 0.f;
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const float t = ys[d] * z, u = r.back ? S[d] + t : fmaf(a.y, S[d], fmaf(a.x, S[d], t));
            o = fmaf(xs[d], u, o);
            S[d] = r.back ? fmaf(a.y, u, a.x * u) : u;
        }
        o *= r.o_scale;
        if (r.out32) r.out32[(t * p.H + h) * D + e] = o;
        else r.out[(t * p.H + h) * D + e] = __float2bfloat16(o);
    }
    if (r.final_state)
        for (int d = 0; d < D; ++d) r.final_state[base + d * D + e] = S[d];
}

// the gradients of shared heads: sums over the value heads of a group
__global__ void __launch_bounds__(256) k_dla_groups(const float* a, __nv_bfloat16* out, int64_t pairs, int heads, int k_heads, int D) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= pairs) return;
    const int64_t row = i * 2 / D;  // (token, k head)
    const int group = heads / k_heads, d = (int)(i * 2 - row * D);
    const float* from = a + row * group * D + d;
    float2 s = make_float2(0.f, 0.f);
    for (int j = 0; j < group; ++j) {
        const float2 u = *reinterpret_cast<const float2*>(from + (int64_t)j * D);
        s = make_float2(s.x + u.x, s.y + u.y);
    }
    reinterpret_cast<uint32_t*>(out)[i] = pack_bf16(s.x, s.y);
}

cudaError_t walk(const DlaParams& p, const Role& r, cudaStream_t s) {
    if (p.D == 64) k_dla<64><<<p.N * p.H, 64, 0, s>>>(p, r);
    else k_dla<128><<<p.N * p.H, 128, 0, s>>>(p, r);
    return cudaGetLastError();
}

}  // namespace

size_t dla_states_bytes(const DlaParams&, bool) { return 0; }
int dla_kernels(const DlaParams& p, bool backward) { return backward ? (p.dq_heads ? 5 : 3) : 1; }

cudaError_t launch_dla_fwd(const DlaParams& p, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(p.status, 0, 256, s);
    if (e != cudaSuccess) return e;
    const int G = p.H / p.Hk;
    return walk(p, Role{p.q, p.k, p.v, p.ldq, p.ldk, p.ldv, G, G, 1, 0, 0, 1.f, p.scale, p.h0, p.ht, p.o, nullptr}, s);
}

cudaError_t launch_dla_bwd(const DlaParams& p, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(p.status, 0, 256, s);
    const int G = p.H / p.Hk;
    const int64_t ldo = (int64_t)p.H * p.D;
    if (e == cudaSuccess) e = walk(p, Role{p.dO, p.v, p.k, ldo, p.ldv, p.ldk, 1, 1, G, 0, 1, 1.f, p.scale, p.h0, nullptr, p.dq, p.dq_heads}, s);
    if (e == cudaSuccess) e = walk(p, Role{p.v, p.dO, p.q, p.ldv, ldo, p.ldq, 1, 1, G, 1, 1, p.scale, 1.f, p.dht, nullptr, p.dk, p.dk_heads}, s);
    if (e == cudaSuccess) e = walk(p, Role{p.k, p.q, p.dO, p.ldk, p.ldq, ldo, G, G, 1, 1, 0, p.scale, 1.f, p.dht, p.dh0, p.dv, nullptr}, s);
    if (e != cudaSuccess || !p.dq_heads) return e;
    const int64_t pairs = p.T * p.Hk * p.D / 2;
    const unsigned grid = (unsigned)((pairs + 255) / 256);
    k_dla_groups<<<grid, 256, 0, s>>>(p.dq_heads, p.dq, pairs, p.H, p.Hk, p.D);
    k_dla_groups<<<grid, 256, 0, s>>>(p.dk_heads, p.dk, pairs, p.H, p.Hk, p.D);
    return cudaGetLastError();
}

}  // namespace gdr
