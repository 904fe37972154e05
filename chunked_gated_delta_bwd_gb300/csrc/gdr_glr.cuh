// Device parts shared by the gated linear recurrence's kernels: pairs of channels, the gate
// function and its chain rule.
//
//   g_t = g_raw_t  (gate "log")   or   -e^{A_log} softplus(g_raw_t + dt_bias)  (gate "softplus")
//   a_t = e^{g_t},   s_t = 1  or  1 - a_t  (complement),   h_t = a_t h_{t-1} + s_t x_t
#pragma once
#include <atomic>

#include "gdr_block.h"
#include "gdr_common.cuh"
#include "gdr_internal.h"

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
__device__ __forceinline__ void forget(float2& v) { asm volatile("" : "+f"(v.x), "+f"(v.y)); }

// The gate is evaluated in base 2: t = g / ln 2, a = 2^t.
//
// 2^t = 2^n (1 + m) with n the integer nearest t and m = 2^f - 1 = f q(f), |f| <= 1/2, q the
// polynomial of degree 5 with the least relative error (1.1e-8; fitted by Lawson's reweighted
// least squares).  A slow channel (t near 0) keeps its state for hundreds of tokens, over which
// an error of a that has one sign grows with the number of tokens; n is 0 there, so a = 1 + m is
// rounded once, and s = 1 - a = -m does not cancel.  No hardware exponential and no branch: 15
// instructions for two channels.  Decays below 2^-126 count as 2^-126; NaN stays NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void exp2_parts(float2 t, float2& m, float2& scale) {
    t = make_float2(max_nan(t.x, -126.f), max_nan(t.y, -126.f));
    const float2 shifted = __fadd2_rn(t, splat(12582912.f));  // 1.5 * 2^23: n in the low bits
    const float2 f = __ffma2_rn(__fadd2_rn(shifted, splat(-12582912.f)), splat(-1.f), t);
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
    s = __ffma2_rn(__fmul2_rn(scale, m), splat(-1.f), __ffma2_rn(scale, splat(-1.f), splat(1.f)));
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
        if constexpr (GATE == GLR_LOG) {
            return __fmul2_rn(raw, splat(kLog2e));
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
    return __ffma2_rn(a, COMP ? __ffma2_rn(x, splat(-1.f), h) : h, x);
}

// ---------------------------------------------------------------------------
// The scan over tokens, y_t = a_t y_{t-1} + b_t with y restarted from a given state at each
// sequence (the forward in the order of time; the backward, whose y is a_t l_t, against it).
//
// The tokens of all sequences are cut into chunks of 8 SUB; a tile is one chunk of 64 channels,
// a warp takes SUB consecutive tokens of it, a lane two channels.  A run of tokens acts on the
// state before it as y -> A y + H.  Each tile's run (A, H) is published; the state before a chunk
// is the fold of the runs before it, back to the chunk its sequence begins in.  So that no tile
// folds many, the last chunk of every 16 also publishes the run of all 16 and the last of every
// 256 the run of those: a chunk reads at most 15 + 15 published runs and one for each 256 chunks
// before.  Which runs are folded, and in which order, depends on the position alone, so the
// results do not depend on the order in which blocks run.
//
// Blocks stay resident and take tiles by ticket, chunks in the order of the scan: a tile waits
// only for tiles with earlier tickets, which are being worked on.  The loads of the next tile are
// in flight while a tile is worked on; each warp loads its own tokens, so a tile has two barriers.
//
// A run that contains a restart does not depend on the state before it: its A is -0 (a product
// of decays is +0 at least), and a fold that meets it takes H as it is, so that no infinity or
// NaN crosses from one sequence into the next.
// ---------------------------------------------------------------------------
constexpr int GLR_WARPS = 8, GLR_MAX_CHUNK = 128, GLR_TILE = 64;
// tokens of a warp: 32 KB of inputs to a chunk's run at most, whatever the types
__host__ __device__ constexpr int glr_sub(bool act_f32, bool gate_f32) { return act_f32 || gate_f32 ? 8 : 16; }
__host__ __device__ inline int glr_chunks(int64_t T, bool act_f32, bool gate_f32) {  // (T is below 2^36)
    const unsigned chunk = glr_sub(act_f32, gate_f32) * GLR_WARPS;
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
// the run of `first` and then `next`, either of which may contain restarts
__device__ __forceinline__ Run run_then(const Run& first, const Run& next) {
    const bool rx = run_restarts(next.A.x), ry = run_restarts(next.A.y);
    Run o;
    o.H = make_float2(rx ? next.H.x : fmaf(next.A.x, first.H.x, next.H.x),
                      ry ? next.H.y : fmaf(next.A.y, first.H.y, next.H.y));
    o.A = make_float2(rx ? next.A.x : first.A.x * next.A.x, ry ? next.A.y : first.A.y * next.A.y);
    return o;
}
// the same where only `first` may
__device__ __forceinline__ Run run_then_plain(const Run& first, const Run& next) {
    return Run{__fmul2_rn(first.A, next.A), __ffma2_rn(next.A, first.H, next.H)};
}
__device__ __forceinline__ uint4 run_bits(const Run& r) {
    return make_uint4(__float_as_uint(r.A.x), __float_as_uint(r.A.y), __float_as_uint(r.H.x), __float_as_uint(r.H.y));
}
__device__ __forceinline__ Run run_from_bits(const uint4& v) {
    return Run{make_float2(__uint_as_float(v.x), __uint_as_float(v.y)),
               make_float2(__uint_as_float(v.z), __uint_as_float(v.w))};
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

// the sequences of a chunk's tokens
struct GlrInfo {
    uint32_t starts[6];         // bit i: token t0 + i begins a sequence (the chunk's end and the end of all tokens count)
    int seq_at_start[GLR_MAX_CHUNK];  // the sequence beginning at token t0 + i, where one does
    int seq0;                   // the sequence of token t0
    int64_t begin0, end1;       // where that sequence begins; where the one of the last token ends
};
constexpr int GLR_PARTS = 8;
struct GlrShared {
    uint4 sub[GLR_WARPS][32];   // the warps' runs
    uint4 part[GLR_PARTS][32];  // folds of published runs: chunks (4), groups (2), super groups (2)
    GlrInfo info[2];            // of this tile and the next
    unsigned ticket;
};

// Finds the sequences of a chunk's tokens [t0, t0 + len); all threads of one warp.  Indexes stay
// in range for inconsistent cu_seqlens too.
__device__ __forceinline__ void glr_find_sequences(const GlrParams& p, GlrInfo& sm, int64_t t0, int len, int lane) {
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
__device__ __forceinline__ uint32_t glr_start_bits(const GlrInfo& sm, int i0, int n) {
    const uint64_t w = sm.starts[i0 >> 5] | ((uint64_t)sm.starts[(i0 >> 5) + 1] << 32);
    return (uint32_t)(w >> (i0 & 31)) & ((2u << n) - 1u);
}
// the sequence of token t0 + i
__device__ __forceinline__ int glr_seq_at(const GlrInfo& sm, int i) {
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

// Folds published runs [from, to) of `rows` for this lane's channels in order; only the first one
// of all may contain a restart.  A run that never comes (it does: its block holds an earlier
// ticket) is recorded and left out.
__device__ __forceinline__ Run glr_fold(const uint4* rows, int64_t stride, int from, int to, int* status) {
    Run r = run_identity();
#pragma unroll 1
    for (int i = from; i < to; i += 4) {
        uint4 v[4];
        const uint4* at = rows + i * stride;
        const int n = min(to - i, 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < n) v[j] = run_poll(at + j * stride);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j < n) {
#pragma unroll 1
                for (int spin = 0; !run_there(v[j]) && spin < GLR_SPIN; ++spin) v[j] = run_poll(at + j * stride);
                if (run_there(v[j])) r = i + j == from ? run_of(v[j]) : run_then_plain(r, run_of(v[j]));
                else atomicOr(status, ST_MMA_TIMEOUT);
            }
        }
    }
    return r;
}

// A tile's place in the scan: which published runs make up the state before it.
struct GlrPlace {
    int k;                   // the chunk's number in the order of the scan
    int chunk0, group0, group1, super0, super1;  // chunks [chunk0, k), groups [group0, group1), super groups
    int nc, ng, ns;          // parts of each level: 4 runs, 8 runs, half of the runs
    // `lo`: the chunk the sequence running into this one begins in; `fresh`: the chunk begins with a restart
    __device__ __forceinline__ GlrPlace(int k_, int lo, bool fresh) : k(k_) {
        const int g0 = k / GLR_GROUP * GLR_GROUP, s0 = k / GLR_SUPER * GLR_SUPER;
        chunk0 = max(lo, g0);
        group0 = max(lo, s0) / GLR_GROUP;
        group1 = k / GLR_GROUP;
        super0 = lo / GLR_SUPER;
        super1 = k / GLR_SUPER;
        const bool none = fresh || k == 0;
        nc = none ? 0 : (k - chunk0 + 3) / 4;
        ng = none ? 0 : (group1 - group0 + 7) / 8;
        ns = none ? 0 : super1 - super0 > 1 ? 2 : super1 - super0;
    }
};

// Between a tile's barriers.  Warp 0 publishes the tile's run and returns it; warps 1 to 4 fold
// published runs of chunks, 5 and 6 of groups and super groups (warp 7 is left to look ahead).
// `c2`: this lane's pair of channels (valid if `live`).
__device__ __forceinline__ Run glr_exchange(const GlrParams& p, GlrShared& sm, const GlrPlace& at, const GlrRuns& runs, int w,
                                            int lane, int c2, bool live) {
    const int64_t stride = p.C / 2;
    Run own = run_identity();
    if (w == 0) {
#pragma unroll
        for (int i = 0; i < GLR_WARPS; ++i) own = run_then(own, run_from_bits(sm.sub[i][lane]));
        if (live) run_publish(runs.chunk + at.k * stride + c2, own);
    } else if (w <= 4) {
        if (w <= at.nc && live) {
            const int from = at.chunk0 + 4 * (w - 1);
            sm.part[w - 1][lane] = run_bits(glr_fold(runs.chunk + c2, stride, from, min(at.k, from + 4), p.status));
        }
    } else if (w <= 6 && live) {
        const int q = w - 5;
        if (q < at.ng) {
            const int from = at.group0 + 8 * q;
            sm.part[4 + q][lane] = run_bits(glr_fold(runs.group + c2, stride, from, min(at.group1, from + 8), p.status));
        }
        if (q < at.ns) {
            const int half = at.ns == 1 ? 1 : (at.super1 - at.super0) / 2, from = at.super0 + q * half;
            sm.part[6 + q][lane] =
                run_bits(glr_fold(runs.super + c2, stride, from, q == at.ns - 1 ? at.super1 : from + half, p.status));
        }
    }
    return own;
}

// After the second barrier: the state before the chunk.
__device__ __forceinline__ float2 glr_state_before(const GlrShared& sm, const GlrPlace& at, int lane) {
    Run y = run_identity();
#pragma unroll 1
    for (int q = 0; q < at.ns; ++q) y = run_then_plain(y, run_from_bits(sm.part[6 + q][lane]));
#pragma unroll 1
    for (int q = 0; q < at.ng; ++q) y = run_then_plain(y, run_from_bits(sm.part[4 + q][lane]));
#pragma unroll 1
    for (int q = 0; q < at.nc; ++q) y = run_then_plain(y, run_from_bits(sm.part[q][lane]));
    return y.H;
}

// Warp 0 of the last chunk of a group (super group) publishes its run.
__device__ __forceinline__ void glr_publish_groups(const GlrParams& p, const GlrShared& sm, const GlrPlace& at,
                                                   const GlrRuns& runs, const Run& own, int lane, int c2, bool live) {
    if (at.k % GLR_GROUP != GLR_GROUP - 1 || !live) return;
    const int64_t stride = p.C / 2;
    Run r = run_identity();
#pragma unroll 1
    for (int q = 0; q < at.nc; ++q) r = run_then_plain(r, run_from_bits(sm.part[q][lane]));
    r = run_then(r, own);
    run_publish(runs.group + at.k / GLR_GROUP * stride + c2, r);
    if (at.k % GLR_SUPER != GLR_SUPER - 1) return;
    Run u = run_identity();
#pragma unroll 1
    for (int q = 0; q < at.ng; ++q) u = run_then_plain(u, run_from_bits(sm.part[4 + q][lane]));
    run_publish(runs.super + at.k / GLR_SUPER * stride + c2, run_then(u, r));
}

// The run of the warps before this one in the order of the scan (`pos` of them), and the state
// it leaves behind a given one.  `restarts`: the chunk may contain restarts.
__device__ __forceinline__ Run glr_before_warp(const GlrShared& sm, int pos, int lane, bool restarts) {
    Run r = run_identity();
    if (restarts) {
#pragma unroll 1
        for (int i = 0; i < pos; ++i) r = run_then(r, run_from_bits(sm.sub[i][lane]));
    } else {
#pragma unroll 1
        for (int i = 0; i < pos; ++i) r = run_then_plain(r, run_from_bits(sm.sub[i][lane]));
    }
    return r;
}
__device__ __forceinline__ float2 glr_after(const Run& r, float2 y) {
    return run_then(Run{splat(0.f), y}, r).H;
}

// The next tile.  Tickets count in the workspace when there is something to wait for.
__device__ __forceinline__ unsigned glr_next(const GlrParams& p, int chunks, unsigned id) {
    return chunks == 1 ? id + gridDim.x : atomicAdd(reinterpret_cast<unsigned*>(p.status) + 1, 1u);
}

// Asynchronous copies of a warp's rows [0, nt) of 64 channels into shared memory, zeros past them
// and past the `cols` channels there are; rows before `skip` are zeros too.  16 bytes a copy
// where every row of the call's tensors allows it (`wide`), else one pair of channels.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool there) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES), "r"(there ? BYTES : 0) : "memory");
}
template <int SUB, class T>
__device__ __forceinline__ void glr_copy_rows(T* dst, const T* src, int64_t ld, int skip, int nt, int cols, bool wide, int lane,
                                              const T* somewhere) {
    if (wide) {
        constexpr int E = 16 / sizeof(T), S = GLR_TILE / E;  // elements a copy, copies a row
#pragma unroll
        for (int j = 0; j < SUB * S / 32; ++j) {
            const int at = j * 32 + lane, row = at / S, e = at % S * E;
            const bool there = row >= skip && row < nt && e < cols;
            copy_async<16>(dst + row * GLR_TILE + e, there ? src + row * ld + e : somewhere, there);
        }
    } else {
#pragma unroll 4
        for (int row = 0; row < SUB; ++row) {
            const bool there = row >= skip && row < nt && 2 * lane < cols;
            copy_async<2 * sizeof(T)>(dst + row * GLR_TILE + 2 * lane, there ? src + row * ld + 2 * lane : somewhere, there);
        }
    }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the N most recent groups of this thread, then of its warp
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
    __syncwarp();
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

// Launches a scan kernel on as many blocks as are resident at once (or tiles, if fewer).
// `ready`: the devices whose shared-memory limit of this kernel is raised.
template <class K>
cudaError_t glr_launch(K kernel, std::atomic<uint64_t>& ready, size_t smem, int per_sm, const GlrParams& p, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const int64_t all = (int64_t)glr_chunks(p.T, p.act_f32, p.gate_f32) * ((p.C + GLR_TILE - 1) / GLR_TILE);
    const int64_t resident = (int64_t)per_sm * num_sms();
    kernel<<<(unsigned)(all < resident ? all : resident), GLR_THREADS, smem, s>>>(p);
    return cudaGetLastError();
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
