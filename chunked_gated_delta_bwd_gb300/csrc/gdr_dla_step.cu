// One token of linear attention with a decay for each head, on a pool of fp32 states:
//
//   S <- e^g S + k v^T,   o = scale S^T q
//
// The states' bytes bound it: each is read and written once, 64 KB each way for a head of 128.  A block of
// 256 threads takes W value columns of one (row, head): a thread holds four columns of every PAR-th key row in
// registers between the loads, all in flight at once, and the stores.  The sum over the key rows is taken in a
// fixed order (a thread's rows, the lanes of a warp, the warps).  Few states of 128 channels take narrow blocks (a
// quarter of the columns), so that their bytes come through more multiprocessors.
//
// 257 rows of 16 heads of 128, some of them padding: 77.9 us, 6.5 TB/s.  One row of 16 heads: 1.9 us in a graph.
#include "gdr_common.cuh"
#include "gdr_dla.h"
#include "gdr_internal.h"

namespace gdr {
namespace {

template <int D, int W>
__global__ void __launch_bounds__(256) k_dla_step(const DlaStepParams p) {
    constexpr int C4 = W / 4, PAR = 256 / C4, PER = D / PAR, SL = D / W;
    __shared__ float2 qk[D];
    __shared__ float4 part[8][C4];
    const int tid = threadIdx.x, slice = blockIdx.x % SL, h = blockIdx.x / SL;
    const int64_t n = blockIdx.y;
    const int64_t slot = p.slots ? p.slots[n] : n;
    const int c = tid % C4, r = tid / C4, col = slice * W + 4 * c;
    __nv_bfloat16* o = p.o + (n * p.H + h) * D + slice * W;
    if (slot < 0 || slot >= p.pool) {
        if (tid < C4) *reinterpret_cast<uint2*>(o + 4 * tid) = make_uint2(0, 0);
        return;
    }
    float4* home = reinterpret_cast<float4*>(p.state + ((slot * p.H + h) * D + r) * D + col);
    float4 s[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = home[i * PAR * (D / 4)];
    const int hk = h / (p.H / p.Hk);
    if (tid < D) qk[tid] = make_float2(bf2f(p.q[n * p.ldq + hk * D + tid]), bf2f(p.k[n * p.ldk + hk * D + tid]));
    const uint2 vr = *reinterpret_cast<const uint2*>(p.v + n * p.ldv + h * D + col);
    const float2 v0 = unpack_bf16(vr.x), v1 = unpack_bf16(vr.y);
    const float a = expf(p.g[h]);
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const float2 w = qk[r + i * PAR];
        s[i] = make_float4(fmaf(a, s[i].x, w.y * v0.x), fmaf(a, s[i].y, w.y * v0.y), fmaf(a, s[i].z, w.y * v1.x),
                           fmaf(a, s[i].w, w.y * v1.y));
        home[i * PAR * (D / 4)] = s[i];
        acc = make_float4(fmaf(w.x, s[i].x, acc.x), fmaf(w.x, s[i].y, acc.y), fmaf(w.x, s[i].z, acc.z), fmaf(w.x, s[i].w, acc.w));
    }
#pragma unroll
    for (int m = C4; m < 32; m *= 2) {
        acc.x += __shfl_xor_sync(~0u, acc.x, m);
        acc.y += __shfl_xor_sync(~0u, acc.y, m);
        acc.z += __shfl_xor_sync(~0u, acc.z, m);
        acc.w += __shfl_xor_sync(~0u, acc.w, m);
    }
    if (tid % 32 < C4) part[tid / 32][c] = acc;
    __syncthreads();
    if (tid < C4) {
        float4 t = part[0][tid];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            const float4 u = part[i][tid];
            t = make_float4(t.x + u.x, t.y + u.y, t.z + u.z, t.w + u.w);
        }
        *reinterpret_cast<uint2*>(o + 4 * tid) = make_uint2(pack_bf16(p.scale * t.x, p.scale * t.y), pack_bf16(p.scale * t.z, p.scale * t.w));
    }
}

constexpr int MOST = 65535;  // rows of a launch: a grid's y

template <int D, int W>
cudaError_t go(const DlaStepParams& p, cudaStream_t s) {
    DlaStepParams part = p;
    for (int n = 0; n < p.rows; n += MOST) {
        part.rows = p.rows - n < MOST ? p.rows - n : MOST;
        part.q = p.q + n * p.ldq;
        part.k = p.k + n * p.ldk;
        part.v = p.v + n * p.ldv;
        part.o = p.o + (int64_t)n * p.H * D;
        if (p.slots) part.slots = p.slots + n;
        else part.state = p.state + (int64_t)n * p.H * D * D, part.pool = p.pool - n;
        k_dla_step<D, W><<<dim3(p.H * (D / W), part.rows), 256, 0, s>>>(part);
    }
    return cudaGetLastError();
}

}  // namespace

int dla_step_kernels(const DlaStepParams& p) { return (p.rows + MOST - 1) / MOST; }

cudaError_t launch_dla_step(const DlaStepParams& p, cudaStream_t s) {
    if (p.D == 64) return go<64, 64>(p, s);
    // one row of so many heads of 128 in blocks of 32 columns and whole ones, in a graph: 16 1.9 and 2.8 us, 64 2.6 and 3.0,
    // 80 3.0 and 3.1, 8 rows of 16 3.1 and 3.0; heads of 64 take 2.0 to 2.2 us either way
    return 2 * (int64_t)p.rows * p.H < num_sms() ? go<128, 32>(p, s) : go<128, 128>(p, s);
}

}  // namespace gdr
