// Device parts shared by the gated linear recurrence's kernels: pairs of channels, the gate
// function and its chain rule.
//
//   g_t = g_raw_t  (gate "log")   or   -e^{A_log} softplus(g_raw_t + dt_bias)  (gate "softplus")
//   a_t = e^{g_t},   s_t = 1  or  1 - a_t  (complement),   h_t = a_t h_{t-1} + s_t x_t
#pragma once
#include "gdr_block.h"
#include "gdr_common.cuh"

namespace gdr {

enum { GLR_LOG = 0, GLR_SOFTPLUS = 1 };

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// two consecutive channels of a row as loaded, and as fp32
template <class T> struct PairOf;
template <> struct PairOf<__nv_bfloat16> {
    using raw = uint32_t;
    static __device__ __forceinline__ float2 widen(raw r) { return unpack_bf16(r); }
    static __device__ __forceinline__ raw narrow(float2 v) { return pack_bf16(v.x, v.y); }
    static __device__ __forceinline__ raw zero() { return 0u; }
};
template <> struct PairOf<float> {
    using raw = float2;
    static __device__ __forceinline__ float2 widen(raw r) { return r; }
    static __device__ __forceinline__ raw narrow(float2 v) { return v; }
    static __device__ __forceinline__ raw zero() { return make_float2(0.f, 0.f); }
};

// Makes the compiler forget what it derived from a value, so that a later use derives it again
// instead of keeping the result in a register.
__device__ __forceinline__ void forget(uint32_t& v) { asm volatile("" : "+r"(v)); }
__device__ __forceinline__ void forget(float2& v) { asm volatile("" : "+f"(v.x), "+f"(v.y)); }

// The gate is evaluated in base 2: t = g / ln 2, a = 2^t.
//
// 2^t = 2^n (1 + m) with n the integer nearest t and m = 2^f - 1 = f q(f), |f| <= 1/2, q the
// polynomial of degree 5 with the least relative error (1.1e-8; fitted by Lawson's reweighted
// least squares).  A slow channel (t near 0) keeps its state for hundreds of tokens, over which
// an error of a that has one sign grows with the number of tokens; n is 0 there, so a = 1 + m is
// rounded once, and s = 1 - a = -m does not cancel.  No hardware exponential and no branch: 17
// two-lane instructions for two channels.  Decays below 2^-126 count as 2^-126; NaN stays NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void exp2_parts(float2 t, float2& m, float2& scale) {
    t = make_float2(max_nan(t.x, -126.f), max_nan(t.y, -126.f));
    const float2 shifted = __fadd2_rn(t, splat(12582912.f));  // 1.5 * 2^23: n in the low bits
    const float2 f = __fadd2_rn(t, __fadd2_rn(splat(12582912.f), make_float2(-shifted.x, -shifted.y)));
    float2 q = __ffma2_rn(f, splat(1.5403508e-4f), splat(1.3390735e-3f));
    q = __ffma2_rn(f, q, splat(9.6182376e-3f));
    q = __ffma2_rn(f, q, splat(5.5503573e-2f));
    q = __ffma2_rn(f, q, splat(2.4022649e-1f));
    q = __ffma2_rn(f, q, splat(6.9314718e-1f));
    m = __fmul2_rn(f, q);
    scale = make_float2(__uint_as_float((__float_as_uint(shifted.x) << 23) + 0x3f800000u),
                        __uint_as_float((__float_as_uint(shifted.y) << 23) + 0x3f800000u));
}
__device__ __forceinline__ float2 decay(float2 t) {
    float2 m, scale;
    exp2_parts(t, m, scale);
    return __ffma2_rn(scale, m, scale);
}
__device__ __forceinline__ void decay(float2 t, float2& a, float2& s) {  // s = 1 - a
    float2 m, scale;
    exp2_parts(t, m, scale);
    a = __ffma2_rn(scale, m, scale);
    const float2 down = make_float2(-scale.x, -scale.y);
    s = __ffma2_rn(down, m, __fadd2_rn(splat(1.f), down));
}

// softplus(z) = max(z, 0) + log(1 + y), y = e^{-|z|} in (0, 1]; log(1 + y) = y p(y) with the
// polynomial p of degree 8 of the least relative error on [0, 1] (3e-8, fitted likewise), which
// keeps the relative accuracy of the slow channels' small softplus.  Returns y too.
__device__ __forceinline__ float2 softplus2(float2 z, float2& y) {
    y = make_float2(__expf(-fabsf(z.x)), __expf(-fabsf(z.y)));
    float2 q = __ffma2_rn(y, splat(5.2326238e-3f), splat(-2.9504957e-2f));
    q = __ffma2_rn(y, q, splat(7.8225493e-2f));
    q = __ffma2_rn(y, q, splat(-1.3663207e-1f));
    q = __ffma2_rn(y, q, splat(1.9105989e-1f));
    q = __ffma2_rn(y, q, splat(-2.4842978e-1f));
    q = __ffma2_rn(y, q, splat(3.3319095e-1f));
    q = __ffma2_rn(y, q, splat(-4.9999493e-1f));
    q = __ffma2_rn(y, q, splat(9.9999994e-1f));
    return __ffma2_rn(y, q, make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
}

// the gate of two channels: its parameters, the base-2 log gate of raw values, and what a
// gradient of g is multiplied by to give that of the raw value
constexpr float kLog2e = 1.4426950408889634f;
template <int GATE>
struct GlrGate {
    float2 nA, bias;  // -e^{A_log}, dt_bias
    __device__ __forceinline__ void load(const float* A_log, const float* dt_bias, int c) {
        if constexpr (GATE == GLR_SOFTPLUS) {
            const float2 l = *reinterpret_cast<const float2*>(A_log + c);
            nA = make_float2(-expf(l.x), -expf(l.y));
            bias = *reinterpret_cast<const float2*>(dt_bias + c);
        }
    }
    __device__ __forceinline__ float2 log2_gate(float2 raw) const {
        if constexpr (GATE == GLR_LOG) {  // (growth saturates at 2^127)
            const float2 t = __fmul2_rn(raw, splat(kLog2e));
            return make_float2(t.x > 127.f ? 127.f : t.x, t.y > 127.f ? 127.f : t.y);
        } else {
            float2 y;
            return __fmul2_rn(__fmul2_rn(nA, splat(kLog2e)), softplus2(__fadd2_rn(raw, bias), y));
        }
    }
    // dg / d(raw) = -e^{A_log} sigmoid(z): sigmoid = 1 / (1 + y) for z >= 0, y / (1 + y) otherwise
    __device__ __forceinline__ float2 slope(float2 raw) const {
        if constexpr (GATE == GLR_LOG) return splat(1.f);
        const float2 z = __fadd2_rn(raw, bias);
        const float2 y = make_float2(__expf(-fabsf(z.x)), __expf(-fabsf(z.y)));
        const float2 inv = make_float2(__fdividef(1.f, 1.f + y.x), __fdividef(1.f, 1.f + y.y));
        return __fmul2_rn(nA, __fmul2_rn(inv, make_float2(z.x >= 0.f ? 1.f : y.x, z.y >= 0.f ? 1.f : y.y)));
    }
};

// The new state of a token: a h + x, or a h + (1 - a) x with the complement, as x + a (h - x).
template <bool COMP>
__device__ __forceinline__ float2 glr_update(float2 a, float2 h, float2 x) {
    return __ffma2_rn(a, COMP ? __fadd2_rn(h, make_float2(-x.x, -x.y)) : h, x);
}

// ---------------------------------------------------------------------------
// The scan over tokens, y_t = a_t y_{t-1} + b_t with y restarted from a given state at each
// sequence (the forward in the order of time; the backward, whose y is a_t l_t, against it).
//
// The tokens of all sequences are cut into chunks of 8 SUB; a block takes one chunk of 64
// channels, a warp SUB consecutive tokens of it, a lane two channels.  A run of tokens acts on
// the state before it as y -> A y + H.  Each block publishes its chunk's (A, H); the state
// before a chunk is the fold of the runs before it, back to the chunk its sequence begins in.
// So that no block folds many, the last chunk of every 16 also publishes the run of all 16 and
// the last of every 256 the run of those: a chunk reads at most 15 + 15 published runs and one
// for each 256 chunks before.  Which runs are folded, and in which order, depends on the
// position alone, so the results do not depend on the order in which blocks run.
//
// A run that contains a restart does not depend on the state before it: its A is -0 (a product
// of decays is +0 at least), and the fold then takes H as it is, so that no infinity or NaN
// crosses from one sequence into the next.
// ---------------------------------------------------------------------------
constexpr int GLR_WARPS = 8, GLR_MAX_CHUNK = 128, GLR_TILE = 64;
// tokens of a warp: what a thread holds of them as loaded fits 32 registers in the forward and
// 64 in the backward, whatever the type
__host__ __device__ constexpr int glr_sub(bool act_f32) { return act_f32 ? 8 : 16; }
__host__ __device__ inline int glr_chunks(int64_t T, bool act_f32) {  // (T is below 2^36)
    const unsigned chunk = glr_sub(act_f32) * GLR_WARPS;
    return (int)((uint64_t)(T + chunk - 1) / chunk);
}
constexpr int GLR_THREADS = 32 * GLR_WARPS;
constexpr int GLR_GROUP = 16, GLR_SUPER = 256;  // chunks in a published group / super group
constexpr int GLR_SPIN = 1 << 20;               // polls of one published run before giving up

// a run of tokens for two channels
struct Run {
    float2 A, H;
};
__device__ __forceinline__ Run run_identity() { return Run{splat(1.f), splat(0.f)}; }
__device__ __forceinline__ bool run_restarts(float A) { return __float_as_uint(A) == 0x80000000u; }
// the state after a run
__device__ __forceinline__ float2 run_apply(const Run& r, float2 y) {
    return make_float2(run_restarts(r.A.x) ? r.H.x : fmaf(r.A.x, y.x, r.H.x),
                       run_restarts(r.A.y) ? r.H.y : fmaf(r.A.y, y.y, r.H.y));
}
// the run of `first` and then `next`
__device__ __forceinline__ Run run_then(const Run& first, const Run& next) {
    Run o;
    o.H = run_apply(next, first.H);
    o.A = make_float2(run_restarts(next.A.x) ? next.A.x : first.A.x * next.A.x,
                      run_restarts(next.A.y) ? next.A.y : first.A.y * next.A.y);
    return o;
}

// Published runs are polled word by word: the workspace starts at zero and every word is stored
// inverted, so a word is there once it is not zero.  (All bits set, whose inverse is zero, is a
// NaN that no arithmetic gives; a NaN is stored as the usual one.)
__device__ __forceinline__ uint32_t run_word(float v) { return ~(v != v ? 0x7fffffffu : __float_as_uint(v)); }
__device__ __forceinline__ void run_publish(uint4* at, const Run& r) {
    asm volatile("st.relaxed.gpu.global.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"l"(at), "r"(run_word(r.A.x)),
                 "r"(run_word(r.A.y)), "r"(run_word(r.H.x)), "r"(run_word(r.H.y))
                 : "memory");
}
__device__ __forceinline__ uint4 run_poll(const uint4* at) {
    uint4 v;
    asm volatile("ld.relaxed.gpu.global.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ bool run_there(const uint4& v) { return v.x && v.y && v.z && v.w; }
__device__ __forceinline__ Run run_of(const uint4& v) {
    return Run{make_float2(__uint_as_float(~v.x), __uint_as_float(~v.y)),
               make_float2(__uint_as_float(~v.z), __uint_as_float(~v.w))};
}

struct GlrShared {
    uint4 sub[GLR_WARPS][32];   // the warps' runs
    uint4 part[3][GLR_WARPS][32];  // folds of published runs: super groups, groups, chunks
    uint32_t starts[6];         // bit i: token t0 + i begins a sequence (the chunk's end and the end of all tokens count)
    int seq_at_start[GLR_MAX_CHUNK];  // the sequence beginning at token t0 + i, where one does
    int seq0;                   // the sequence of token t0
    int64_t begin0, end1;       // where that sequence begins; where the one of the last token ends
    unsigned ticket;
};
__device__ __forceinline__ uint4 run_bits(const Run& r) {
    return make_uint4(__float_as_uint(r.A.x), __float_as_uint(r.A.y), __float_as_uint(r.H.x), __float_as_uint(r.H.y));
}
__device__ __forceinline__ Run run_from_bits(const uint4& v) {
    return Run{make_float2(__uint_as_float(v.x), __uint_as_float(v.y)),
               make_float2(__uint_as_float(v.z), __uint_as_float(v.w))};
}

// Finds the sequences of a chunk's tokens [t0, t0 + len); all threads of one warp.  Indexes stay
// in range for inconsistent cu_seqlens too.
__device__ __forceinline__ void glr_find_sequences(const GlrParams& p, GlrShared& sm, int64_t t0, int len, int lane) {
    if (lane < 6) sm.starts[lane] = 0;
    for (int i = lane; i < GLR_MAX_CHUNK; i += 32) sm.seq_at_start[i] = 0;
    __syncwarp();
    const int64_t* cu = p.cu_seqlens;
    if (!cu) {
        // t0 / seq_len, from its product with 1 / seq_len, which is off by less than one
        int64_t n0 = (int64_t)((double)t0 * p.inv_len);
        if (n0 * p.seq_len > t0) --n0;
        if ((n0 + 1) * p.seq_len <= t0) ++n0;
        const int64_t begin = n0 * p.seq_len;
        if (lane == 0) {
            sm.seq0 = (int)n0;
            sm.begin0 = begin;
        }
        for (int64_t n = n0 + (begin < t0) + lane, b; (b = n * p.seq_len) <= t0 + len; n += 32) {
            const int i = (int)(b - t0);
            atomicOr(&sm.starts[i >> 5], 1u << (i & 31));
            if (i < GLR_MAX_CHUNK) sm.seq_at_start[i] = (int)n;
        }
        __syncwarp();
        if (lane == 0) {  // the end of the last token's sequence
            int64_t e = begin + p.seq_len;
            if (e < t0 + len)  // (a sequence of over GLR_MAX_CHUNK tokens has one such boundary here)
                e += p.seq_len > GLR_MAX_CHUNK ? p.seq_len : ((unsigned)(t0 + len - 1 - e) / (unsigned)p.seq_len + 1) * p.seq_len;
            sm.end1 = e;
        }
        return;
    }
    // the last sequence that begins at or before t0, by 32 probes at a time
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool before = lane == 0 || (at < hi && cu[at] <= t0);
        lo += (__popc(__ballot_sync(~0u, before)) - 1) * step;
        hi = min(hi, lo + step);
    }
    if (lane == 0) {
        sm.seq0 = lo;
        const int64_t b = cu[lo];
        sm.begin0 = b < 0 ? 0 : (b > t0 ? t0 : b);
        sm.end1 = p.T;
    }
    __syncwarp();
    // the boundaries inside the chunk and at its end, 32 at a time
    for (int n0 = lo; n0 <= p.N; n0 += 32) {
        const int n = n0 + lane;
        const int64_t b = n <= p.N ? cu[n] : p.T;
        const int64_t i = b - t0;
        if (n <= p.N && i >= 0 && i <= len) {
            // of the sequences that begin here the last one is not empty.  (A boundary of inconsistent
            // cu_seqlens gets some sequence's number all the same: no index leaves the states.)
            atomicOr(&sm.starts[i >> 5], 1u << (i & 31));
            if (i < GLR_MAX_CHUNK) atomicMax(&sm.seq_at_start[i], min(n, p.N - 1));
        }
        // the end of the last token's sequence: the first boundary at or past the chunk's end
        const unsigned past = __ballot_sync(~0u, n <= p.N && b >= t0 + len);
        if (past) {
            if (lane == __ffs(past) - 1) sm.end1 = b > p.T ? p.T : b;
            break;
        }
    }
    if (lane == 0 && t0 + len == p.T) atomicOr(&sm.starts[len >> 5], 1u << (len & 31));
    __syncwarp();
}
// start bits of tokens i0 .. i0 + n of the chunk (n <= 16)
__device__ __forceinline__ uint32_t glr_start_bits(const GlrShared& sm, int i0, int n) {
    const uint64_t w = sm.starts[i0 >> 5] | ((uint64_t)sm.starts[(i0 >> 5) + 1] << 32);
    return (uint32_t)(w >> (i0 & 31)) & ((2u << n) - 1u);
}
// the sequence of token t0 + i
__device__ __forceinline__ int glr_seq_at(const GlrShared& sm, int i) {
    uint32_t w = sm.starts[i >> 5] & (0xffffffffu >> (31 - (i & 31)));
    for (int q = i >> 5;;) {
        if (w) return sm.seq_at_start[q * 32 + 31 - __clz(w)];
        if (--q < 0) return sm.seq0;
        w = sm.starts[q];
    }
}

// Where published runs lie in the workspace, after the status word and the ticket counter.
struct GlrRuns {
    uint4 *chunk, *group, *super;  // [..][C / 2]
};
__host__ __device__ inline GlrRuns glr_runs(void* ws, int chunks, int C) {
    GlrRuns r;
    r.chunk = reinterpret_cast<uint4*>(static_cast<unsigned char*>(ws) + 256);
    r.group = r.chunk + (int64_t)chunks * (C / 2);
    r.super = r.group + (int64_t)(chunks / GLR_GROUP) * (C / 2);
    return r;
}
__host__ __device__ inline size_t glr_runs_bytes(int chunks, int C) {  // of one chunk's tokens: none
    return chunks > 1 ? sizeof(uint4) * (size_t)(C / 2) * ((size_t)chunks + chunks / GLR_GROUP + chunks / GLR_SUPER) : 0;
}

// Folds published runs [from, to) of `rows` for this lane's channels in order.  A run that never
// comes (it does: its block holds an earlier ticket) is recorded and left out.
__device__ __forceinline__ Run glr_fold(const uint4* rows, int64_t stride, int from, int to, int* status) {
    Run r = run_identity();
#pragma unroll 1
    for (int i = from; i < to; i += 4) {
        uint4 v[4];
        const int n = min(to - i, 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < n) v[j] = run_poll(rows + (i + j) * stride);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j < n) {
                for (int spin = 0; !run_there(v[j]) && spin < GLR_SPIN; ++spin) v[j] = run_poll(rows + (i + j) * stride);
                if (run_there(v[j])) r = run_then(r, run_of(v[j]));
                else atomicOr(status, ST_MMA_TIMEOUT);
            }
        }
    }
    return r;
}

// After the warps' runs are in sm.sub (a barrier behind them), in the order of the scan: warp 0
// publishes the chunk's run; the state before the chunk is folded from what others published;
// the last chunk of a group (super group) publishes its run.  Returns the state before this
// warp's first token.  `k`: the chunk's number in the order of the scan, `lo`: that of the chunk
// the sequence running into it begins in; `fresh`: the chunk begins with a restart.  `pos`: this
// warp's place in the order of the scan; `c2`: this lane's pair of channels (valid if `live`).
__device__ __forceinline__ float2 glr_carry(const GlrParams& p, GlrShared& sm, int chunks, int k, int lo,
                                            bool fresh, int pos, int lane, int c2, bool live) {
    const int64_t stride = p.C / 2;
    if (chunks > 1) {
        const GlrRuns runs = glr_runs(p.status, chunks, p.C);
        Run own = run_identity();
        if (pos == 0) {
#pragma unroll 1
            for (int w = 0; w < GLR_WARPS; ++w) own = run_then(own, run_from_bits(sm.sub[w][lane]));
            if (live) run_publish(runs.chunk + k * stride + c2, own);
        }
        const int g0 = k / GLR_GROUP * GLR_GROUP, s0 = k / GLR_SUPER * GLR_SUPER;  // first chunk of k's group, super group
        const int cf = lo > g0 ? lo : g0;                                          // chunks [cf, k)
        const int gf = (lo > s0 ? lo : s0) / GLR_GROUP, ge = k / GLR_GROUP;        // groups [gf, ge)
        const int sf = lo / GLR_SUPER, se = k / GLR_SUPER;                         // super groups [sf, se)
        int nc = 0, ng = 0, ns = 0;  // warps that hold a part of each level
        if (!fresh && k > 0) {
            // warps 0-3 fold up to 4 chunks' runs each, warps 4-7 up to 4 groups', all of them the super groups'
            nc = (k - cf + 3) / 4;
            ng = ge > gf ? (ge - gf + 3) / 4 : 0;
            const int per = (se > sf ? se - sf + GLR_WARPS - 1 : 0) / GLR_WARPS;
            ns = per ? (se - sf + per - 1) / (unsigned)per : 0;
            if (live) {
                if (pos < nc) sm.part[2][pos][lane] = run_bits(glr_fold(runs.chunk + c2, stride, cf + 4 * pos, min(k, cf + 4 * pos + 4), p.status));
                const int q = pos - 4;
                if (q >= 0 && q < ng) sm.part[1][q][lane] = run_bits(glr_fold(runs.group + c2, stride, gf + 4 * q, min(ge, gf + 4 * q + 4), p.status));
                if (pos < ns) sm.part[0][pos][lane] = run_bits(glr_fold(runs.super + c2, stride, sf + per * pos, min(se, sf + per * (pos + 1)), p.status));
            }
            __syncthreads();
        }
        float2 y = splat(0.f);
#pragma unroll 1
        for (int q = 0; q < ns; ++q) y = run_apply(run_from_bits(sm.part[0][q][lane]), y);
#pragma unroll 1
        for (int q = 0; q < ng; ++q) y = run_apply(run_from_bits(sm.part[1][q][lane]), y);
#pragma unroll 1
        for (int q = 0; q < nc; ++q) y = run_apply(run_from_bits(sm.part[2][q][lane]), y);
        if (pos == 0 && k % GLR_GROUP == GLR_GROUP - 1 && live) {
            Run r = run_identity();
#pragma unroll 1
            for (int q = 0; q < nc; ++q) r = run_then(r, run_from_bits(sm.part[2][q][lane]));
            r = run_then(r, own);
            run_publish(runs.group + k / GLR_GROUP * stride + c2, r);
            if (k % GLR_SUPER == GLR_SUPER - 1) {
                Run u = run_identity();
#pragma unroll 1
                for (int q = 0; q < ng; ++q) u = run_then(u, run_from_bits(sm.part[1][q][lane]));
                run_publish(runs.super + k / GLR_SUPER * stride + c2, run_then(u, r));
            }
        }
#pragma unroll 1
        for (int w = 0; w < pos; ++w) y = run_apply(run_from_bits(sm.sub[w][lane]), y);
        return y;
    }
    float2 y = splat(0.f);
#pragma unroll 1
    for (int w = 0; w < pos; ++w) y = run_apply(run_from_bits(sm.sub[w][lane]), y);
    return y;
}

// This block's chunk and tile of channels.  With more than one chunk a block takes the next
// ticket, chunks in the order of the scan, so that it waits only for blocks that run already.
__device__ __forceinline__ unsigned glr_ticket(const GlrParams& p, GlrShared& sm, int chunks) {
    if (chunks == 1) return blockIdx.x;
    if (threadIdx.x == 0) sm.ticket = atomicAdd(reinterpret_cast<unsigned*>(p.status) + 1, 1u);
    __syncthreads();
    return sm.ticket;
}

// Empty sequences pass their state through; the first tile's blocks also check cu_seqlens against
// its contract.  Sequences are dealt to the chunks' blocks 32 at a time.  (With one chunk the
// status word is written here, not cleared before.)  One warp.
__device__ __forceinline__ void glr_empty_sequences(const GlrParams& p, const float* from, float* to, int kc,
                                                    int chunks, int c, bool live, bool check) {
    const int64_t* cu = p.cu_seqlens;
    const int lane = threadIdx.x % 32;
    bool bad = false;
    if (cu) {
        if (kc == 0) bad = cu[0] != 0 || cu[p.N] != p.T;
        for (int64_t n0 = (int64_t)kc * 32; n0 < p.N; n0 += (int64_t)chunks * 32) {
            const int64_t n = n0 + lane;
            const int64_t len = n < p.N ? cu[n + 1] - cu[n] : 1;
            bad |= len < 0;
            for (unsigned m = __ballot_sync(~0u, len == 0); m; m &= m - 1) {
                const int64_t at = (n0 + __ffs(m) - 1) * p.C + c;
                if (to && live)
                    *reinterpret_cast<float2*>(to + at) = from ? *reinterpret_cast<const float2*>(from + at) : splat(0.f);
            }
        }
        bad = __any_sync(~0u, bad);
    }
    if (check && lane == 0) {
        if (chunks == 1) *p.status = bad ? ST_BAD_SEQLENS : 0;
        else if (bad) atomicOr(p.status, ST_BAD_SEQLENS);
    }
}

// Calls f.run<TX, TG, GATE, COMP>() for the run-time choice of types, gate
// function and input scale (bf16 / fp32 activations; a bf16 or fp32 gate for bf16 activations).
template <class F>
cudaError_t glr_dispatch(int act_f32, int gate_f32, int gate, int comp, const F& f) {
    using bf = __nv_bfloat16;
#define GLR_PICK(TX, TG)                                                                     \
    do {                                                                                     \
        if (gate == GLR_LOG) return comp ? f.template run<TX, TG, GLR_LOG, true>()            \
                                         : f.template run<TX, TG, GLR_LOG, false>();          \
        return comp ? f.template run<TX, TG, GLR_SOFTPLUS, true>()                            \
                    : f.template run<TX, TG, GLR_SOFTPLUS, false>();                          \
    } while (0)
    if (act_f32) GLR_PICK(float, float);
    if (!gate_f32) GLR_PICK(bf, bf);
    GLR_PICK(bf, float);
#undef GLR_PICK
}

}  // namespace gdr
