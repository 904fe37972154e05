// C ABI of linear attention with a decay for each head (declared in include/gdr.h): argument checks
// and launches.
#include <math.h>
#include <string.h>

#include "gdr_dla.h"
#include "gdr_host.h"

namespace gdr {

static gdr_status check_heads(int32_t heads, int32_t* k_heads, int32_t dim) {
    if (heads < 1 || heads > (1 << 16)) return fail(GDR_ERR_INVALID, "num_heads must be 1 to 65536%s");
    if (*k_heads == 0) *k_heads = heads;
    if (*k_heads < 1 || heads % *k_heads != 0) return fail(GDR_ERR_INVALID, "num_heads must be a multiple of num_k_heads%s");
    if (dim != 64 && dim != 128) return fail(GDR_ERR_UNSUPPORTED, "head_dim must be 64 or 128%s");
    return GDR_OK;
}

// a token stride in elements: 0 means contiguous tokens; resolves it
static gdr_status token_stride(int64_t given, int64_t least, int64_t* out) {
    if (given == 0) given = least;
    if (given < least || given % 8 != 0) return fail(GDR_ERR_INVALID, "a token stride must be a multiple of 8 and at least heads x head_dim%s");
    if (given > ((int64_t)1 << 32)) return fail(GDR_ERR_INVALID, "token stride too large%s");
    *out = given;
    return GDR_OK;
}

static gdr_status check_dla(const dla_shape* sh, DlaParams* p) {
    if (!sh) return fail(GDR_ERR_INVALID, "shape is NULL%s");
    memset(p, 0, sizeof(*p));
    int32_t hk = sh->num_k_heads;
    if (gdr_status st = check_heads(sh->num_heads, &hk, sh->head_dim)) return st;
    if (sh->num_seqs < 1 || sh->total_tokens < 0) return fail(GDR_ERR_INVALID, "num_seqs must be >= 1, total_tokens >= 0%s");
    if (!sh->cu_seqlens && sh->total_tokens % sh->num_seqs != 0)
        return fail(GDR_ERR_INVALID, "dense layout needs total_tokens divisible by num_seqs%s");
    if (sh->cu_seqlens && !aligned_to(sh->cu_seqlens, 8)) return fail(GDR_ERR_INVALID, "pointer %s is not 8-byte aligned", "cu_seqlens");
    if (sh->total_tokens > (1 << 30) || (int64_t)sh->num_seqs * sh->num_heads > (1 << 24) ||
        sh->total_tokens * sh->num_heads > ((int64_t)1 << 36))
        return fail(GDR_ERR_INVALID, "problem too large%s");
    if (!isfinite(sh->scale)) return fail(GDR_ERR_INVALID, "scale must be finite%s");
    p->N = sh->num_seqs; p->H = sh->num_heads; p->Hk = hk; p->D = sh->head_dim;
    p->T = sh->total_tokens;
    p->seq_len = sh->cu_seqlens ? 0 : p->T / p->N;
    p->cu_seqlens = sh->cu_seqlens;
    p->scale = sh->scale;
    const int64_t qk = (int64_t)hk * p->D, vo = (int64_t)p->H * p->D;
    if (gdr_status st = token_stride(sh->q_stride, qk, &p->ldq)) return st;
    if (gdr_status st = token_stride(sh->k_stride, qk, &p->ldk)) return st;
    return token_stride(sh->v_stride, vo, &p->ldv);
}

// workspace: status word, states, then the gradients of each value head where heads share q and k
static size_t heads_bytes(const DlaParams& p) { return p.H == p.Hk ? 0 : sizeof(float) * (size_t)p.T * p.H * p.D; }
static size_t dla_workspace(const DlaParams& p, bool backward) {
    const size_t forward = 256 + dla_states_bytes(p, false);
    if (!backward) return forward;
    const size_t both = 256 + dla_states_bytes(p, true) + 2 * heads_bytes(p);
    return both > forward ? both : forward;
}

static size_t extent(int64_t tokens, int64_t ld, int64_t width) { return tokens ? 2 * (size_t)((tokens - 1) * ld + width) : 0; }

// no tokens: the states pass through
static gdr_status pass_states(const DlaParams& p, float* to, const float* from, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(p.status, 0, 256, s);
    const size_t bytes = sizeof(float) * (size_t)p.N * p.H * p.D * p.D;
    if (e == cudaSuccess && to) e = from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s);
    return e == cudaSuccess ? ok() : cuda_fail(e, "states of empty sequences");
}

}  // namespace gdr

using namespace gdr;

extern "C" {

size_t dla_workspace_bytes(const dla_shape* shape, int32_t backward) {
    DlaParams p;
    if (check_dla(shape, &p) != GDR_OK) return 0;
    return dla_workspace(p, backward != 0);
}

gdr_status dla_fwd(const dla_shape* shape, const void* q, const void* k, const void* v, const float* log_decay,
                   const float* h0, void* o, float* ht, void* workspace, size_t workspace_bytes, void* stream) {
    DlaParams p;
    if (gdr_status st = check_dla(shape, &p)) return st;
    if (p.T) { NEED(q); NEED(k); NEED(v); NEED(o); NEED(log_decay); }
    OPT(h0); OPT(ht); NEED(workspace);
    const size_t ws = dla_workspace(p, false);
    if (workspace_bytes < ws) return fail(GDR_ERR_WORKSPACE, "workspace smaller than dla_workspace_bytes%s");
    const int64_t qk = (int64_t)p.Hk * p.D, vo = (int64_t)p.H * p.D;
    const size_t states = sizeof(float) * (size_t)p.N * vo * p.D;
    const Span in[] = {{q, extent(p.T, p.ldq, qk), "q"}, {k, extent(p.T, p.ldk, qk), "k"}, {v, extent(p.T, p.ldv, vo), "v"},
                       {log_decay, sizeof(float) * p.H, "log_decay"}, {h0, states, "h0"},
                       {p.cu_seqlens, 8 * ((size_t)p.N + 1), "cu_seqlens"}};
    const Span out[] = {{o, extent(p.T, vo, vo), "o"}, {ht, states, "ht"}, {workspace, ws, "workspace"}};
    if (gdr_status st = apart(out, 3, in, 6)) return st;
    cudaStream_t s = (cudaStream_t)stream;
    p.status = static_cast<int*>(workspace);
    p.states = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + 256);
    if (p.T == 0) return pass_states(p, ht, h0, s);
    p.q = (const __nv_bfloat16*)q; p.k = (const __nv_bfloat16*)k; p.v = (const __nv_bfloat16*)v;
    p.g = log_decay; p.h0 = h0; p.o = (__nv_bfloat16*)o; p.ht = ht;
    cudaError_t e = timed(GDR_KERNEL_DLA, s, [&] { return launch_dla_fwd(p, s); }, dla_kernels(p, false));
    return e == cudaSuccess ? ok() : cuda_fail(e, "linear attention launch");
}

gdr_status dla_bwd(const dla_shape* shape, const void* q, const void* k, const void* v, const float* log_decay,
                   const float* h0, const void* dO, const float* dht, void* workspace, size_t workspace_bytes,
                   void* dq, void* dk, void* dv, float* dh0, void* stream) {
    DlaParams p;
    if (gdr_status st = check_dla(shape, &p)) return st;
    if (p.T) { NEED(q); NEED(k); NEED(v); NEED(dO); NEED(dq); NEED(dk); NEED(dv); NEED(log_decay); }
    OPT(h0); OPT(dht); NEED(dh0); NEED(workspace);
    const size_t ws = dla_workspace(p, true);
    if (workspace_bytes < ws) return fail(GDR_ERR_WORKSPACE, "workspace smaller than dla_workspace_bytes%s");
    const int64_t qk = (int64_t)p.Hk * p.D, vo = (int64_t)p.H * p.D;
    const size_t states = sizeof(float) * (size_t)p.N * vo * p.D;
    const Span in[] = {{q, extent(p.T, p.ldq, qk), "q"}, {k, extent(p.T, p.ldk, qk), "k"}, {v, extent(p.T, p.ldv, vo), "v"},
                       {dO, extent(p.T, vo, vo), "dO"}, {log_decay, sizeof(float) * p.H, "log_decay"}, {h0, states, "h0"},
                       {dht, states, "dht"}, {p.cu_seqlens, 8 * ((size_t)p.N + 1), "cu_seqlens"}};
    const Span out[] = {{dq, extent(p.T, qk, qk), "dq"}, {dk, extent(p.T, qk, qk), "dk"}, {dv, extent(p.T, vo, vo), "dv"},
                        {dh0, states, "dh0"}, {workspace, ws, "workspace"}};
    if (gdr_status st = apart(out, 5, in, 8)) return st;
    cudaStream_t s = (cudaStream_t)stream;
    p.status = static_cast<int*>(workspace);
    if (p.T == 0) return pass_states(p, dh0, dht, s);
    unsigned char* at = static_cast<unsigned char*>(workspace) + 256;
    p.states = reinterpret_cast<float*>(at);
    at += dla_states_bytes(p, true);
    if (heads_bytes(p)) {
        p.dq_heads = reinterpret_cast<float*>(at);
        p.dk_heads = reinterpret_cast<float*>(at + heads_bytes(p));
    }
    p.q = (const __nv_bfloat16*)q; p.k = (const __nv_bfloat16*)k; p.v = (const __nv_bfloat16*)v;
    p.dO = (const __nv_bfloat16*)dO; p.g = log_decay; p.h0 = h0; p.dht = dht;
    p.dq = (__nv_bfloat16*)dq; p.dk = (__nv_bfloat16*)dk; p.dv = (__nv_bfloat16*)dv; p.dh0 = dh0;
    cudaError_t e = timed(GDR_KERNEL_DLA, s, [&] { return launch_dla_bwd(p, s); }, dla_kernels(p, true));
    return e == cudaSuccess ? ok() : cuda_fail(e, "linear attention backward launch");
}

gdr_status dla_step(int32_t rows, int32_t num_heads, int32_t num_k_heads, int32_t head_dim, int32_t pool, float scale,
                    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                    const float* log_decay, const int64_t* slots, float* state, void* o, void* stream) {
    DlaStepParams p;
    memset(&p, 0, sizeof(p));
    if (gdr_status st = check_heads(num_heads, &num_k_heads, head_dim)) return st;
    if (rows < 0 || pool < 0) return fail(GDR_ERR_INVALID, "rows and pool must be >= 0%s");
    if ((int64_t)rows * num_heads > (1 << 28)) return fail(GDR_ERR_INVALID, "problem too large%s");
    if (!slots && pool < rows) return fail(GDR_ERR_INVALID, "the pool holds fewer states than there are rows%s");
    if (!isfinite(scale)) return fail(GDR_ERR_INVALID, "scale must be finite%s");
    const int64_t qk = (int64_t)num_k_heads * head_dim, vo = (int64_t)num_heads * head_dim;
    if (gdr_status st = token_stride(q_stride, qk, &p.ldq)) return st;
    if (gdr_status st = token_stride(k_stride, qk, &p.ldk)) return st;
    if (gdr_status st = token_stride(v_stride, vo, &p.ldv)) return st;
    if (rows == 0) return ok();
    NEED(q); NEED(k); NEED(v); NEED(log_decay); NEED(o);
    if (pool) NEED(state);
    if (slots && !aligned_to(slots, 8)) return fail(GDR_ERR_INVALID, "pointer %s is not 8-byte aligned", "slots");
    const Span in[] = {{q, extent(rows, p.ldq, qk), "q"}, {k, extent(rows, p.ldk, qk), "k"}, {v, extent(rows, p.ldv, vo), "v"},
                       {log_decay, sizeof(float) * num_heads, "log_decay"}, {slots, 8 * (size_t)rows, "slots"}};
    const Span out[] = {{o, extent(rows, vo, vo), "o"}, {state, sizeof(float) * (size_t)pool * vo * head_dim, "state"}};
    if (gdr_status st = apart(out, 2, in, 5)) return st;
    p.rows = rows; p.H = num_heads; p.Hk = num_k_heads; p.D = head_dim; p.pool = pool; p.scale = scale;
    p.q = (const __nv_bfloat16*)q; p.k = (const __nv_bfloat16*)k; p.v = (const __nv_bfloat16*)v;
    p.g = log_decay; p.slots = slots; p.state = state; p.o = (__nv_bfloat16*)o;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = timed(GDR_KERNEL_DLA, s, [&] { return launch_dla_step(p, s); }, dla_step_kernels(p));
    return e == cudaSuccess ? ok() : cuda_fail(e, "linear attention step launch");
}

}  // extern "C"
