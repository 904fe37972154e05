// C ABI of the operators around the delta rule in a recurrent block (declared in
// include/gdr.h): argument checks and launches.
#include <limits.h>
#include <atomic>
#include <string.h>

#include "gdr_block.h"
#include "gdr_common.cuh"
#include "gdr_host.h"

namespace gdr {

// a pointer to rows read two elements at a time: aligned to a pair
#define NEED_ROWS(ptr, f32)                                                                       \
    do {                                                                                          \
        if (!(ptr)) return fail(GDR_ERR_INVALID, "required pointer %s is NULL", #ptr);            \
        if (!aligned_to(ptr, (f32) ? 8 : 4))                                                      \
            return fail(GDR_ERR_INVALID, "pointer %s is not aligned to two elements", #ptr);      \
    } while (0)

// a row stride in elements: 0 means contiguous rows; resolves it
static gdr_status row_stride(int64_t given, int64_t channels, int64_t* out) {
    if (given == 0) given = channels;
    if (given < channels || given % 2 != 0)
        return fail(GDR_ERR_INVALID, "a row stride must be even and at least the number of channels%s");
    if (given > ((int64_t)1 << 38)) return fail(GDR_ERR_INVALID, "row stride too large%s");
    *out = given;
    return GDR_OK;
}

// whether two buffers (or NULL) share memory
static bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
    const uintptr_t u = reinterpret_cast<uintptr_t>(a), v = reinterpret_cast<uintptr_t>(b);
    return a && b && u < v + b_bytes && v < u + a_bytes;
}

static gdr_status check_channels(int32_t channels) {
    if (channels < 1) return fail(GDR_ERR_INVALID, "channels must be >= 1%s");
    if (channels % 2 != 0) return fail(GDR_ERR_INVALID, "channels must be even%s");
    // (the kernels count channels, and the conv1d's weights of them, in 32 bits)
    if (channels > GDR_MAX_CHANNELS) return fail(GDR_ERR_INVALID, "channels must be at most 2^28%s");
    return GDR_OK;
}

static gdr_status check_glr_choices(int32_t gate, int32_t act_type, int32_t gate_type) {
    if (gate != GLR_GATE_LOG && gate != GLR_GATE_SOFTPLUS) return fail(GDR_ERR_INVALID, "unknown gate function%s");
    if ((act_type != GDR_TYPE_BF16 && act_type != GDR_TYPE_F32) || (gate_type != GDR_TYPE_BF16 && gate_type != GDR_TYPE_F32))
        return fail(GDR_ERR_UNSUPPORTED, "element types are bf16 and float32%s");
    if (act_type == GDR_TYPE_F32 && gate_type == GDR_TYPE_BF16)
        return fail(GDR_ERR_UNSUPPORTED, "float32 activations need a float32 gate%s");
    return GDR_OK;
}

static gdr_status check_tokens(int32_t num_seqs, int64_t total_tokens, const int64_t* cu_seqlens, int64_t channels) {
    if (num_seqs < 1 || total_tokens < 0) return fail(GDR_ERR_INVALID, "num_seqs must be >= 1, total_tokens >= 0%s");
    if (!cu_seqlens && total_tokens % num_seqs != 0)
        return fail(GDR_ERR_INVALID, "dense layout needs total_tokens divisible by num_seqs%s");
    const int64_t most = (int64_t)1 << 40;  // elements (the product of the sizes may leave 64 bits)
    if (total_tokens > ((int64_t)1 << 36) || total_tokens > most / channels || num_seqs > most / channels)
        return fail(GDR_ERR_INVALID, "problem too large%s");
    return GDR_OK;
}

static gdr_status check_glr(const glr_shape* sh, GlrParams* p) {
    if (!sh) return fail(GDR_ERR_INVALID, "shape is NULL%s");
    gdr_status st = check_channels(sh->channels);
    if (st == GDR_OK) st = check_tokens(sh->num_seqs, sh->total_tokens, sh->cu_seqlens, sh->channels);
    if (st == GDR_OK) st = check_glr_choices(sh->gate, sh->act_type, sh->gate_type);
    int64_t ldx = 0, ldg = 0;
    if (st == GDR_OK) st = row_stride(sh->x_stride, sh->channels, &ldx);
    if (st == GDR_OK) st = row_stride(sh->g_stride, sh->channels, &ldg);
    if (st != GDR_OK) return st;
    memset(p, 0, sizeof(*p));
    p->N = sh->num_seqs;
    p->C = sh->channels;
    p->T = sh->total_tokens;
    p->seq_len = sh->cu_seqlens ? 0 : sh->total_tokens / sh->num_seqs;
    p->inv_len = p->seq_len > 0 ? 1.0 / (double)p->seq_len : 0.0;
    p->cu_seqlens = sh->cu_seqlens;
    p->ldx = ldx;
    p->ldg = ldg;
    p->gate = sh->gate;
    p->complement = sh->complement != 0;
    p->act_f32 = sh->act_type == GDR_TYPE_F32;
    p->gate_f32 = sh->gate_type == GDR_TYPE_F32;
    return GDR_OK;
}

static std::atomic<int> g_glr_stall{0};  // glr_test_stall_next_call: block index + 1, or 0

static size_t glr_workspace(const GlrParams& p) { return 256 + glr_published_bytes(p) + glr_sums_bytes(p); }

// whether rows of C elements at this stride are whole numbers of aligned 16-byte pieces
static int rows_wide(const GlrParams& p, const void* at, int64_t ld, int f32) {
    const int piece = f32 ? 4 : 8;
    return aligned16(at) && ld % piece == 0 && p.C % piece == 0 && p.T < ((int64_t)1 << 31);
}

// Clears the workspace (a launch of one chunk writes its status word itself); every
// sequence empty: the states pass through.
static gdr_status glr_front(GlrParams& p, void* ws, float* to, const float* from, cudaStream_t s, bool* done) {
    const size_t published = glr_published_bytes(p);
    cudaError_t e = cudaSuccess;
    if (published || p.T == 0) e = cudaMemsetAsync(ws, 0, 256 + published, s);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(workspace)");
    p.status = static_cast<int*>(ws);
    p.sums = reinterpret_cast<float4*>(static_cast<unsigned char*>(ws) + 256 + published);
    *done = p.T == 0;
    if (p.T || !to) return GDR_OK;
    const size_t bytes = sizeof(float) * (size_t)p.N * p.C;
    e = from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s);
    return e == cudaSuccess ? GDR_OK : cuda_fail(e, "states of empty sequences");
}

}  // namespace gdr

using namespace gdr;

extern "C" {

size_t glr_workspace_bytes(const glr_shape* shape) {
    GlrParams p;
    if (check_glr(shape, &p) != GDR_OK) return 0;
    return glr_workspace(p);
}

gdr_status glr_fwd(const glr_shape* shape, const void* x, const void* g, const float* A_log, const float* dt_bias,
                   const float* h0, void* h, float* ht, void* workspace, size_t workspace_bytes, void* stream) {
    GlrParams p;
    if (gdr_status st = check_glr(shape, &p)) return st;
    if (p.T) {
        NEED_ROWS(x, p.act_f32); NEED_ROWS(g, p.gate_f32); NEED(h);
        if (p.gate == GLR_GATE_SOFTPLUS) { NEED(A_log); NEED(dt_bias); }
    }
    OPT(h0); OPT(ht); NEED(workspace);
    if (workspace_bytes < glr_workspace(p)) return fail(GDR_ERR_WORKSPACE, "workspace smaller than glr_workspace_bytes%s");
    // (h0 is read again when another block may have written ht)
    const size_t states = sizeof(float) * (size_t)p.N * p.C;
    if (p.T && overlap(h0, states, ht, states)) return fail(GDR_ERR_INVALID, "ht must not share memory with h0%s");
    cudaStream_t s = (cudaStream_t)stream;
    bool done = false;
    if (gdr_status st = glr_front(p, workspace, ht, h0, s, &done)) return st;
    if (done) return ok();
    p.x = x; p.g = g; p.A_log = A_log; p.dt_bias = dt_bias; p.h0 = h0; p.h = h; p.ht = ht;
    p.wide = rows_wide(p, x, p.ldx, p.act_f32) && rows_wide(p, g, p.ldg, p.gate_f32);
    p.test_stall = g_glr_stall.exchange(0);
    cudaError_t e = timed(GDR_KERNEL_GLR, s, [&] { return launch_glr_fwd(p, s); });
    return e == cudaSuccess ? ok() : cuda_fail(e, "gated linear recurrence launch");
}

gdr_status glr_bwd(const glr_shape* shape, const void* x, const void* g, const float* A_log, const float* dt_bias,
                   const void* h, const float* h0, const void* dh, const float* dht, void* workspace,
                   size_t workspace_bytes, void* dx, void* dg, float* dh0, float* dA_log, float* ddt_bias,
                   void* stream) {
    GlrParams p;
    if (gdr_status st = check_glr(shape, &p)) return st;
    const bool soft = p.gate == GLR_GATE_SOFTPLUS;
    if (p.T) {
        if (p.complement) NEED_ROWS(x, p.act_f32);
        NEED_ROWS(g, p.gate_f32); NEED(h); NEED(dh); NEED(dx); NEED(dg);
        if (soft) { NEED(A_log); NEED(dt_bias); }
    }
    NEED(dh0); OPT(h0); OPT(dht); NEED(workspace);
    if (soft) { NEED(dA_log); NEED(ddt_bias); }
    if (workspace_bytes < glr_workspace(p)) return fail(GDR_ERR_WORKSPACE, "workspace smaller than glr_workspace_bytes%s");
    // (the states are read again when another block may have written dh0, and h of the token before a tile
    // when another block may have written that token's gradients)
    const size_t states = sizeof(float) * (size_t)p.N * p.C, tokens = (size_t)p.T * p.C;
    if (p.T && (overlap(dht, states, dh0, states) || overlap(h0, states, dh0, states)))
        return fail(GDR_ERR_INVALID, "dh0 must not share memory with dht or h0%s");
    if (overlap(h, tokens * (p.act_f32 ? 4 : 2), dx, tokens * (p.act_f32 ? 4 : 2)) ||
        overlap(h, tokens * (p.act_f32 ? 4 : 2), dg, tokens * (p.gate_f32 ? 4 : 2)))
        return fail(GDR_ERR_INVALID, "dx and dg must not share memory with h%s");
    cudaStream_t s = (cudaStream_t)stream;
    bool done = false;
    if (gdr_status st = glr_front(p, workspace, dh0, dht, s, &done)) return st;
    if (done) {
        if (!soft) return ok();
        cudaError_t e = cudaMemsetAsync(dA_log, 0, sizeof(float) * p.C, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(ddt_bias, 0, sizeof(float) * p.C, s);
        return e == cudaSuccess ? ok() : cuda_fail(e, "cudaMemsetAsync(dA_log/ddt_bias)");
    }
    p.x = x; p.g = g; p.A_log = A_log; p.dt_bias = dt_bias; p.h_in = h; p.h0 = h0; p.dh = dh; p.dht = dht;
    p.dx = dx; p.dg = dg; p.dh0 = dh0; p.dA_log = dA_log; p.ddt_bias = ddt_bias;
    p.wide = (!p.complement || rows_wide(p, x, p.ldx, p.act_f32)) && rows_wide(p, g, p.ldg, p.gate_f32) &&
             rows_wide(p, h, p.C, p.act_f32);
    p.test_stall = g_glr_stall.exchange(0);
    cudaError_t e = timed(GDR_KERNEL_GLR, s, [&] { return launch_glr_bwd(p, s); }, soft ? 2 : 1);
    return e == cudaSuccess ? ok() : cuda_fail(e, "gated linear recurrence backward launch");
}

void glr_test_stall_next_call(int block) { g_glr_stall.store(block >= 0 ? block + 1 : 0); }

gdr_status glr_step(int32_t rows, int32_t channels, int32_t pool, int32_t gate, int32_t complement, int32_t act_type,
                    int32_t gate_type, const void* x, int64_t x_stride, const void* g, int64_t g_stride,
                    const float* A_log, const float* dt_bias, const int64_t* slots, float* state, void* y,
                    void* stream) {
    GlrStepParams p;
    if (gdr_status st = check_channels(channels)) return st;
    if (gdr_status st = check_glr_choices(gate, act_type, gate_type)) return st;
    if (rows < 0 || pool < 0) return fail(GDR_ERR_INVALID, "rows and pool must be >= 0%s");
    if (!slots && pool < rows) return fail(GDR_ERR_INVALID, "the pool holds fewer states than there are rows%s");
    if (gdr_status st = row_stride(x_stride, channels, &p.ldx)) return st;
    if (gdr_status st = row_stride(g_stride, channels, &p.ldg)) return st;
    if (rows == 0) return ok();
    NEED_ROWS(x, act_type == GDR_TYPE_F32); NEED_ROWS(g, gate_type == GDR_TYPE_F32); NEED(y);
    if (pool) NEED(state);
    if (gate == GLR_GATE_SOFTPLUS) { NEED(A_log); NEED(dt_bias); }
    if (slots && !aligned_to(slots, 8)) return fail(GDR_ERR_INVALID, "pointer %s is not 8-byte aligned", "slots");
    p.N = rows; p.C = channels; p.pool = pool;
    p.gate = gate; p.complement = complement != 0;
    p.act_f32 = act_type == GDR_TYPE_F32; p.gate_f32 = gate_type == GDR_TYPE_F32;
    p.x = x; p.g = g; p.A_log = A_log; p.dt_bias = dt_bias; p.slots = slots; p.state = state; p.y = y;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = timed(GDR_KERNEL_GLR, s, [&] { return launch_glr_step(p, s); });
    return e == cudaSuccess ? ok() : cuda_fail(e, "gated linear recurrence step launch");
}

static gdr_status check_norm(int64_t rows, int32_t channels, int32_t res_type) {
    if (rows < 0 || rows > INT_MAX) return fail(GDR_ERR_INVALID, "rows must be 0 to 2^31 - 1%s");
    if (gdr_status st = check_channels(channels)) return st;
    if (res_type != GDR_TYPE_BF16 && res_type != GDR_TYPE_F32)
        return fail(GDR_ERR_UNSUPPORTED, "the residual's type is bf16 or float32%s");
    return GDR_OK;
}

gdr_status gdr_rmsnorm_fwd(int64_t rows, int32_t channels, const void* x, int64_t x_stride, const void* residual,
                           int32_t res_type, const float* weight, float eps, int32_t quant, void* y, float* scale,
                           void* residual_out, float* rstd, void* stream) {
    NormParams p;
    memset(&p, 0, sizeof(p));
    if (gdr_status st = check_norm(rows, channels, res_type)) return st;
    if (quant != GDR_QUANT_NONE && quant != GDR_QUANT_ROW && quant != GDR_QUANT_BLOCK)
        return fail(GDR_ERR_INVALID, "unknown output form%s");
    if (!(eps >= 0.f)) return fail(GDR_ERR_INVALID, "eps must be >= 0%s");
    if (gdr_status st = row_stride(x_stride, channels, &p.ldx)) return st;
    if (rows == 0) return ok();
    NEED_ROWS(x, 0); NEED(weight); NEED(y); NEED(rstd); OPT(residual);
    if (residual) NEED(residual_out);
    if (quant != GDR_QUANT_NONE) NEED(scale);
    p.R = rows; p.C = channels; p.res_f32 = residual && res_type == GDR_TYPE_F32; p.quant = quant; p.eps = eps;
    p.x = (const __nv_bfloat16*)x; p.residual = residual; p.weight = weight; p.y = y; p.scale = scale;
    p.res_out = residual ? residual_out : nullptr; p.rstd = rstd;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = timed(GDR_KERNEL_NORM, s, [&] { return launch_rmsnorm_fwd(p, s); });
    return e == cudaSuccess ? ok() : cuda_fail(e, "rms norm launch");
}

size_t gdr_rmsnorm_workspace_bytes(int64_t rows, int32_t channels) {
    if (check_norm(rows, channels, GDR_TYPE_BF16) != GDR_OK) return 0;
    return 256 + rmsnorm_partial_bytes(rows, channels);
}

gdr_status gdr_rmsnorm_bwd(int64_t rows, int32_t channels, const void* dy, const void* s_in, int32_t res_type,
                           const float* weight, const float* rstd, const void* dres, void* workspace,
                           size_t workspace_bytes, void* dx, float* dweight, void* stream) {
    NormParams p;
    memset(&p, 0, sizeof(p));
    if (gdr_status st = check_norm(rows, channels, res_type)) return st;
    if (rows) {
        NEED(dy); NEED(s_in); NEED(weight); NEED(rstd); NEED(dx);
    }
    NEED(dweight); OPT(dres); NEED(workspace);
    if (workspace_bytes < gdr_rmsnorm_workspace_bytes(rows, channels))
        return fail(GDR_ERR_WORKSPACE, "workspace smaller than gdr_rmsnorm_workspace_bytes%s");
    cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) {  // (the weight may be NULL, as everything of the rows)
        cudaError_t e = cudaMemsetAsync(dweight, 0, sizeof(float) * channels, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(workspace, 0, 256, s);
        return e == cudaSuccess ? ok() : cuda_fail(e, "cudaMemsetAsync(dweight/workspace)");
    }
    p.R = rows; p.C = channels; p.ldx = channels; p.res_f32 = res_type == GDR_TYPE_F32;
    p.dy = (const __nv_bfloat16*)dy; p.s = s_in; p.weight = weight; p.rstd_in = rstd; p.dres = dres; p.dx = dx;
    p.dweight = dweight;
    p.status = static_cast<int*>(workspace);
    p.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + 256);
    cudaError_t e = timed(GDR_KERNEL_NORM, s, [&] { return launch_rmsnorm_bwd(p, s); }, 2);
    return e == cudaSuccess ? ok() : cuda_fail(e, "rms norm backward launch");
}

gdr_status gdr_conv1d_fwd(int32_t num_seqs, int64_t total_tokens, int32_t channels, int32_t width,
                          const int64_t* cu_seqlens, const void* x, int64_t x_stride, const float* weight,
                          const float* bias, const void* state, int32_t silu, void* y, void* state_out,
                          void* stream) {
    ConvFwdParams p;
    memset(&p, 0, sizeof(p));
    if (gdr_status st = check_channels(channels)) return st;
    if (width < 1 || width > 4) return fail(GDR_ERR_UNSUPPORTED, "width must be 1 to 4%s");
    if (gdr_status st = check_tokens(num_seqs, total_tokens, cu_seqlens, channels)) return st;
    if (gdr_status st = row_stride(x_stride, channels, &p.ldx)) return st;
    if (total_tokens) { NEED_ROWS(x, 0); NEED(y); }
    NEED(weight); OPT(bias); OPT(state); OPT(state_out);
    const size_t states = 2 * (size_t)num_seqs * (width - 1) * channels;
    if (overlap(state, states, state_out, states)) return fail(GDR_ERR_INVALID, "state_out must not share memory with the initial state%s");
    p.N = num_seqs; p.T = total_tokens; p.seq_len = cu_seqlens ? 0 : total_tokens / num_seqs;
    p.C = channels; p.K = width; p.silu = silu != 0; p.cu_seqlens = cu_seqlens;
    p.x = (const __nv_bfloat16*)x; p.w = weight; p.bias = bias; p.state = (const __nv_bfloat16*)state;
    p.state_out = (__nv_bfloat16*)state_out; p.y = (__nv_bfloat16*)y;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = timed(GDR_KERNEL_CONV, s, [&] { return launch_conv1d_fwd(p, s); });
    return e == cudaSuccess ? ok() : cuda_fail(e, "conv1d launch");
}

gdr_status gdr_conv1d_step(int32_t rows, int32_t channels, int32_t width, int32_t pool, const void* x,
                           int64_t x_stride, void* state, const float* weight, const float* bias,
                           const int64_t* slots, int32_t silu, void* y, void* stream) {
    ConvFwdParams p;
    memset(&p, 0, sizeof(p));
    if (gdr_status st = check_channels(channels)) return st;
    if (width < 1 || width > 4) return fail(GDR_ERR_UNSUPPORTED, "width must be 1 to 4%s");
    if (rows < 0 || pool < 0) return fail(GDR_ERR_INVALID, "rows and pool must be >= 0%s");
    if (!slots && pool < rows) return fail(GDR_ERR_INVALID, "the pool holds fewer states than there are rows%s");
    if (gdr_status st = row_stride(x_stride, channels, &p.ldx)) return st;
    if (rows == 0) return ok();
    NEED_ROWS(x, 0); NEED(weight); NEED(y); OPT(bias);
    if (pool && width > 1) NEED(state);
    if (slots && !aligned_to(slots, 8)) return fail(GDR_ERR_INVALID, "pointer %s is not 8-byte aligned", "slots");
    p.N = rows; p.C = channels; p.K = width; p.pool = pool; p.silu = silu != 0; p.slots = slots;
    p.x = (const __nv_bfloat16*)x; p.w = weight; p.bias = bias; p.state_out = (__nv_bfloat16*)state;
    p.y = (__nv_bfloat16*)y;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = timed(GDR_KERNEL_CONV, s, [&] { return launch_conv1d_step(p, s); });
    return e == cudaSuccess ? ok() : cuda_fail(e, "conv1d step launch");
}

}  // extern "C"
