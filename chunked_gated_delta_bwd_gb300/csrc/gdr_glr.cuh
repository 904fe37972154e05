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
#include "gdr_tc.cuh"
#include "gdr_tma.h"

namespace gdr {

enum { GLR_LOG = 0, GLR_SOFTPLUS = 1 };

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// two consecutive channels of a row as loaded, and as fp32
template <class T> struct PairOf;
template <> struct PairOf<__nv_bfloat16> {
    using raw = uint32_t;
    // (a shift and a mask: the conversion function takes three instructions, 3% more time for 30011 x 4096
    // with the softplus gate)
    static __device__ __forceinline__ float2 widen(raw r) {
        return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    }
    static __device__ __forceinline__ raw narrow(float2 v) { return pack_bf16(v.x, v.y); }
    static __device__ __forceinline__ raw zero() { return 0u; }
};
template <> struct PairOf<float> {
    using raw = float2;
    static __device__ __forceinline__ float2 widen(raw r) { return r; }
    static __device__ __forceinline__ raw narrow(float2 v) { return v; }
    static __device__ __forceinline__ raw zero() { return make_float2(0.f, 0.f); }
};

// The gate is evaluated in base 2: t = g / ln 2, a = 2^t.
//
// 2^t = 2^n (1 + m) with n the integer nearest t and m = 2^f - 1 = f q(f), |f| <= 1/2, q the
// polynomial of degree 5 with the least relative error (2.1e-8 with these coefficients; fitted by Lawson's
// reweighted least squares).  A slow channel (t near 0) keeps its state for hundreds of tokens, over which
// an error of a that has one sign grows with the number of tokens; n is 0 there, so a = 1 + m is
// rounded once, and s = 1 - a = -m does not cancel (glr_update).  No hardware exponential and no branch: 15
// instructions for two channels.  Decays below 2^-126 count as 2^-126; NaN stays NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 clamp_exponent(float2 t) { return make_float2(max_nan(t.x, -126.f), max_nan(t.y, -126.f)); }
__device__ __forceinline__ void exp2_parts(float2 t, float2& m, float2& scale) {  // (t clamped)
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

// The decay of a run of tokens, 2^{sum of their t}.  (Not the product of their decays: for a slow channel
// the product of two numbers just below 1 lies the same small part of a last place above the nearest one
// each time, and 5000 tokens of a = 1 - 1e-4 came out 3e-5 too small.)
template <int GATE>
__device__ __forceinline__ float2 run_decay(float2 t) {
    const float2 a = decay(clamp_exponent(t));
    if (GATE == GLR_SOFTPLUS) return a;
    return make_float2(t.x > 127.4f ? INFINITY : a.x, t.y > 127.4f ? INFINITY : a.y);
}

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_ftz(float x) {  // (a result below 2^-126 is zero)
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

// softplus(z) / ln 2 from u = z / ln 2: max(u, 0) + log2(1 + y), y = 2^{-|u|} in (0, 1];
// log2(1 + y) = y p(y) with the polynomial p of degree 7 of the least relative error on [0, 1]
// (2e-7, fitted likewise), which keeps the relative accuracy of the slow channels' small softplus.
__device__ __forceinline__ float2 softplus2(float2 u) {
    const float2 y = make_float2(exp2_ftz(-fabsf(u.x)), exp2_ftz(-fabsf(u.y)));
    float2 q = __ffma2_rn(y, splat(-1.23193122e-02f), splat(6.36073265e-02f));
    q = __ffma2_rn(y, q, splat(-1.55351090e-01f));
    q = __ffma2_rn(y, q, splat(2.56009178e-01f));
    q = __ffma2_rn(y, q, splat(-3.53394642e-01f));
    q = __ffma2_rn(y, q, splat(4.80063642e-01f));
    q = __ffma2_rn(y, q, splat(-7.21310068e-01f));
    q = __ffma2_rn(y, q, splat(1.44269478e+00f));
    return __ffma2_rn(y, q, make_float2(fmaxf(u.x, 0.f), fmaxf(u.y, 0.f)));
}

// the gate of two channels: its parameters, the base-2 log gate of raw values, and what a
// gradient of g is multiplied by to give that of the raw value
template <int GATE>
struct GlrGate {
    float2 nA, bias, inv;  // -e^{A_log}, dt_bias / ln 2, e^{-A_log} (0 where the gate is shut)
    static __device__ __forceinline__ float4 param(float2 A_log, float2 dt_bias) {
        return make_float4(-expf(A_log.x), -expf(A_log.y), kLog2e * dt_bias.x, kLog2e * dt_bias.y);
    }
    __device__ __forceinline__ void set(float4 v) {
        if constexpr (GATE == GLR_SOFTPLUS) {
            nA = make_float2(v.x, v.y);
            bias = make_float2(v.z, v.w);
            inv = make_float2(v.x < -1e-30f ? __fdividef(-1.f, v.x) : 0.f, v.y < -1e-30f ? __fdividef(-1.f, v.y) : 0.f);
        }
    }
    __device__ __forceinline__ void load(const float* A_log, const float* dt_bias, int c) {
        if constexpr (GATE == GLR_SOFTPLUS) {
            const float2 l = *reinterpret_cast<const float2*>(A_log + c), b = *reinterpret_cast<const float2*>(dt_bias + c);
            set(param(l, b));
        }
    }
    __device__ __forceinline__ float2 log2_gate(float2 raw) const {
        if constexpr (GATE == GLR_LOG) {
            // (growth past 2^127 would carry into the sign; the softplus gate's t is never positive)
            const float2 t = clamp_exponent(__fmul2_rn(raw, splat(kLog2e)));
            return make_float2(min_nan(t.x, 127.f), min_nan(t.y, 127.f));
        } else {
            return clamp_exponent(__fmul2_rn(nA, softplus2(__ffma2_rn(raw, splat(kLog2e), bias))));
        }
    }
    // dg / d(raw) = -e^{A_log} sigmoid(z) from the base-2 log gate t = -e^{A_log} softplus(z) / ln 2:
    // sigmoid(z) = 1 - e^{-softplus(z)} = 1 - 2^{t e^{-A_log}}
    __device__ __forceinline__ float2 slope(float2 t) const {
        if constexpr (GATE == GLR_LOG) return splat(1.f);
        float2 a, s;
        decay(clamp_exponent(__fmul2_rn(t, inv)), a, s);
        return __fmul2_rn(nA, s);
    }
};

// The new state of a token, a h + x, or with the complement a h + (1 - a) x, from the number that the
// forward keeps of a token.  1 - a of a slow channel is not to be had from a (rounded, a is off by up to
// 3e-8 whatever 1 - a is: at 1e-4 the states came out 3e-4 off), nor the a of a fast one from 1 - a.  So
// with the complement what is kept is a - 1 (its sign bit set, also for zero) where the integer part of
// -t is 0, and a (at least +0) elsewhere: h + (a - 1) (h - x), or x + a (h - x).  A token with a = 1 leaves
// the state as it is, whatever x.
__device__ __forceinline__ bool keeps_rest(float v) { return __float_as_int(v) < 0; }  // v is a - 1
template <bool COMP>
__device__ __forceinline__ float2 decay_of_kept(float2 v) {
    return COMP ? make_float2(keeps_rest(v.x) ? 1.f + v.x : v.x, keeps_rest(v.y) ? 1.f + v.y : v.y) : v;
}
template <bool COMP>
__device__ __forceinline__ float2 glr_update(float2 v, float2 h, float2 x) {
    if (!COMP) return __ffma2_rn(v, h, x);
    const float2 from = make_float2(keeps_rest(v.x) ? h.x : x.x, keeps_rest(v.y) ? h.y : x.y);
    return __ffma2_rn(v, __ffma2_rn(x, splat(-1.f), h), from);
}
// the same from the base-2 log gate t; returns what is kept.  (The softplus gate's t is -0 at most.)
template <int GATE, bool COMP>
__device__ __forceinline__ float2 glr_update_by_gate(float2 t, float2& h, float2 x) {
    float2 m, scale;
    exp2_parts(t, m, scale);
    float2 v = __ffma2_rn(scale, m, scale), from = x;
    if (!COMP) {
        h = __ffma2_rn(v, h, x);
        return v;
    }
    if (t.x >= -0.5f && (GATE == GLR_SOFTPLUS || t.x <= 0.f)) v.x = -fabsf(m.x), from.x = h.x;
    if (t.y >= -0.5f && (GATE == GLR_SOFTPLUS || t.y <= 0.f)) v.y = -fabsf(m.y), from.y = h.y;
    h = __ffma2_rn(v, __ffma2_rn(x, splat(-1.f), h), from);
    return v;
}

// ---------------------------------------------------------------------------
// The scan over tokens, y_t = a_t y_{t-1} + b_t with y restarted from a given state at each
// sequence (the forward in the order of time; the backward, whose y is a_t l_t, against it).
//
// The tokens of all sequences are cut into chunks of 64; a tile is one chunk of 64 channels, a
// warp takes 64 / (compute warps) consecutive tokens of it, a lane two channels.  A run of tokens acts on the
// state before it as y -> A y + H.  Each tile's run (A, H) is published; the state before a chunk
// is the fold of the runs before it, back to the chunk its sequence begins in.  So that no tile
// folds many, the last chunk of every 8 also publishes the run of all 8, and the last of every 64
// the state after it: a chunk reads at most 7 + 7 published runs and a state, in two rounds of
// loads.  (The states make a chain, one step for 4096 tokens: some 2 us of 7 us that 2048 channels
// of them take to pass; 65536 tokens of 64 channels take 32 us.)  Which runs are folded, and in which
// order, depends on the position alone, so the results do not depend on the order in which blocks
// run.
//
// Blocks stay resident and take tiles by ticket, chunks in the order of the scan: a tile waits
// only for tiles with earlier tickets, which are being worked on.  A block's compute warps walk
// tile j for its run, then tile j - LATE for its results.  One warp takes the tickets and copies
// tiles ahead, three exchange warps, one for every third tile, publish and gather in between
// (GlrRing).  So neither the loads nor the way to the other blocks and back is waited for, and
// what a tile costs besides its tokens (half of the instructions, when each warp copied its own
// rows) does not fall to the warps that work on them.
//
// A run that contains a restart does not depend on the state before it: its A is -0 (a product
// of decays is +0 at least), and a fold that meets it takes H as it is, so that no infinity or
// NaN crosses from one sequence into the next.
// ---------------------------------------------------------------------------
constexpr int GLR_CHUNK = 64, GLR_TILE = 64;
constexpr int GLR_GROUP = 8, GLR_SUPER = 64;  // chunks in a published group; from one published state to the next
// After how many polls waits are given up: for another block's run (a poll takes 0.7 us: 50 ms, once a
// block), of a compute warp for its block's others, and of those (the hardware holds a poll of a barrier for
// some 4 us: 0.5 s and 4 s; each longer than what it waits for may take).
constexpr int GLR_SPIN = 1 << 16, GLR_SPIN_COMPUTE = 1 << 17, GLR_SPIN_LONG = 1 << 20;
__host__ __device__ inline int glr_chunks(const GlrParams& p) { return (int)((uint64_t)(p.T + GLR_CHUNK - 1) / GLR_CHUNK); }

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

// A published run is two 64-bit words, A and H, each stored and loaded at once.  The workspace
// starts at zero and the first half of either word is stored inverted, so a word is there once
// that half is not zero.  (All bits set, whose inverse is zero, is a NaN that no arithmetic
// gives; a NaN is stored as the usual one.)
__device__ __forceinline__ uint32_t run_mark(float v) { return ~(v != v ? 0x7fffffffu : __float_as_uint(v)); }
__device__ __forceinline__ void run_publish(uint4* at, const Run& r) {
    const uint64_t a = run_mark(r.A.x) | ((uint64_t)__float_as_uint(r.A.y) << 32);
    const uint64_t h = run_mark(r.H.x) | ((uint64_t)__float_as_uint(r.H.y) << 32);
    asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};\n" ::"l"(at), "l"(a), "l"(h) : "memory");
}
__device__ __forceinline__ uint4 run_poll(const uint4* at) {
    uint64_t a, h;
    asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];\n" : "=l"(a), "=l"(h) : "l"(at) : "memory");
    return make_uint4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)h, (uint32_t)(h >> 32));
}
__device__ __forceinline__ bool run_there(const uint4& v) { return v.x != 0 && v.z != 0; }
__device__ __forceinline__ Run run_of(const uint4& v) {
    return Run{make_float2(__uint_as_float(~v.x), __uint_as_float(v.y)),
               make_float2(__uint_as_float(~v.z), __uint_as_float(v.w))};
}
// Where published runs lie in the workspace, after the status word and the ticket counter.
struct GlrRuns {
    uint4 *chunk, *group, *state;  // [..][C / 2]
};
__host__ __device__ inline GlrRuns glr_runs(void* ws, int chunks, int C) {
    GlrRuns r;
    r.chunk = reinterpret_cast<uint4*>(static_cast<unsigned char*>(ws) + 256);
    r.group = r.chunk + (int64_t)chunks * (C / 2);
    r.state = r.group + (int64_t)(chunks / GLR_GROUP) * (C / 2);
    return r;
}
__host__ __device__ inline size_t glr_runs_bytes(int chunks, int C) {  // of one chunk's tokens: none
    return chunks > 1 ? sizeof(uint4) * (size_t)(C / 2) * ((size_t)chunks + chunks / GLR_GROUP + chunks / GLR_SUPER) : 0;
}

// a tile's sequences and its place in the scan
struct GlrInfo {
    uint32_t starts[4];         // bit i: token t0 + i begins a sequence (the chunk's end and the end of all tokens count)
    int any;                    // whether any of them does, or restarts the scan
    int seq0;                   // the sequence of token t0
    int seq_at_start[GLR_CHUNK];  // the sequence beginning at token t0 + i, where one does
    // the state before chunk k: the published state after chunk 64 [k / 64] - 1 (if `state`), then the
    // runs of groups [group0, group0 + groups) and of chunks [chunk0, chunk0 + chunks)
    int state, group0, groups, chunk0, chunks;
};

// Works out a chunk's sequences and place; all threads of one warp.  Its tokens are
// [t0, t0 + len), `k` is its number in the order of the scan.  Indexes stay in range for
// inconsistent cu_seqlens too.
template <bool BWD>
__device__ __forceinline__ void glr_find_place(const GlrParams& p, GlrInfo& sm, int chunks, int k, int64_t t0, int len, int lane) {
    if (lane < 4) sm.starts[lane] = 0;
    __syncwarp();
    int64_t begin0, end1;  // where the sequence of token t0 begins; where the one of the last token ends
    const int64_t* cu = p.cu_seqlens;
    bool some = false;
    if (!cu) {
        // t0 / seq_len, from its product with 1 / seq_len, which is off by less than one
        int64_t n0 = (int64_t)((double)t0 * p.inv_len);
        if (n0 * p.seq_len > t0) --n0;
        if ((n0 + 1) * p.seq_len <= t0) ++n0;
        begin0 = n0 * p.seq_len;
        if (lane == 0) sm.seq0 = (int)n0;
        end1 = begin0 + p.seq_len;
        if (begin0 == t0 || end1 <= t0 + len) {
            for (int64_t n = n0 + (begin0 < t0) + lane, b; (b = n * p.seq_len) <= t0 + len; n += 32) {
                const int i = (int)(b - t0);
                atomicOr(&sm.starts[i >> 5], 1u << (i & 31));
                if (i < GLR_CHUNK) sm.seq_at_start[i] = (int)n;
            }
            some = true;
        }
        if (end1 < t0 + len)  // (a sequence of over GLR_CHUNK tokens has one such boundary here)
            end1 += p.seq_len > GLR_CHUNK ? p.seq_len
                                              : ((unsigned)(t0 + len - 1 - end1) / (unsigned)p.seq_len + 1) * p.seq_len;
    } else {
        // the last sequence that begins at or before t0, by 32 probes at a time
        int lo = 0, hi = p.N;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const bool before = lane == 0 || (at < hi && cu[at] <= t0);
            lo += (__popc(__ballot_sync(~0u, before)) - 1) * step;
            hi = min(hi, lo + step);
        }
        if (lane == 0) sm.seq0 = lo;
        begin0 = min(max(cu[lo], (int64_t)0), t0);
        end1 = cu[lo + 1];
        const bool inside = begin0 < t0 && end1 > t0 + len && t0 + len < p.T;  // of one sequence
        end1 = inside ? min(end1, p.T) : p.T;
        if (!inside) {
            for (int i = lane; i < GLR_CHUNK; i += 32) sm.seq_at_start[i] = 0;
            __syncwarp();
        }
        // the boundaries inside the chunk and at its end, 32 at a time
        for (int n0 = inside ? p.N + 1 : lo; n0 <= p.N; n0 += 32) {
            const int n = n0 + lane;
            const int64_t b = n <= p.N ? cu[n] : p.T;
            const int64_t i = b - t0;
            if (n <= p.N && i >= 0 && i <= len) {
                // of the sequences that begin here the last one is not empty.  (A boundary of inconsistent
                // cu_seqlens gets some sequence's number all the same: no index leaves the states.)
                atomicOr(&sm.starts[i >> 5], 1u << (i & 31));
                if (i < GLR_CHUNK) atomicMax(&sm.seq_at_start[i], min(n, p.N - 1));
                some = true;
            }
            // the end of the last token's sequence: the first boundary at or past the chunk's end
            const unsigned past = __ballot_sync(~0u, n <= p.N && b >= t0 + len);
            if (past) {
                end1 = min(__shfl_sync(~0u, b, __ffs(past) - 1), p.T);
                break;
            }
        }
        if (t0 + len == p.T) {
            if (lane == 0) atomicOr(&sm.starts[len >> 5], 1u << (len & 31));
            some = true;
        }
    }
    some = __any_sync(~0u, some);
    __syncwarp();
    if (lane == 0) {
        // the chunk in which the sequence running into this one begins; whether this one begins with a restart
        const int lo = BWD ? chunks - 1 - (int)((uint64_t)(end1 - 1) / GLR_CHUNK) : (int)((uint64_t)begin0 / GLR_CHUNK);
        const bool fresh = BWD ? sm.starts[len >> 5] >> (len & 31) & 1 : sm.starts[0] & 1;
        const int g0 = k / GLR_GROUP * GLR_GROUP, s0 = k / GLR_SUPER * GLR_SUPER;
        const bool none = fresh || k == 0;
        sm.any = some;
        sm.chunk0 = max(lo, g0);
        sm.group0 = max(lo, s0) / GLR_GROUP;
        sm.chunks = none ? 0 : k - sm.chunk0;
        sm.groups = none ? 0 : k / GLR_GROUP - sm.group0;
        sm.state = !none && lo < s0;
    }
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

// A wait has run out: the block's warps wait no more.
__device__ __forceinline__ void glr_give_up(volatile int* over, int* status) {
    *over = 1;
    atomicOr(status, ST_MMA_TIMEOUT);
}

// Up to eight published runs for this lane's channels, all loads in flight at once: one at `first`
// (if `has`), then n <= 7 rows.  Their fold in order; only the first run of all may contain a
// restart (or be a state: A = -0).  Waits for each; one that does not come, whose block holds an earlier
// ticket, is recorded, and what is there is taken (`over` set: without waiting any more).
__device__ __forceinline__ Run glr_fold(const uint4* first, bool has, const uint4* rows, int64_t stride, int n, volatile int* over,
                                        int* status) {
    uint4 v[8];
    bool there = true;
    const uint4* at = rows;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = make_uint4(~__float_as_uint(1.f), __float_as_uint(1.f), ~0u, 0);  // the identity
        if (j == 0 ? has : j <= n) v[j] = run_poll(j == 0 ? first : at);
        if (j > 0) at += stride;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) there &= run_there(v[j]);
    if (!there) {
        int limit = *over ? 1 : GLR_SPIN;
        at = rows;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!run_there(v[j])) {
                int spin = 0;
#pragma unroll 1
                do v[j] = run_poll(j == 0 ? first : at);
                while (!run_there(v[j]) && ++spin < limit);
                if (!run_there(v[j])) {
                    glr_give_up(over, status);
                    limit = 1;
                }
            }
            if (j > 0) at += stride;
        }
    }
    Run r = run_of(v[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) r = run_then_plain(r, run_of(v[j]));
    return r;
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

// The ring through which a block's warps hand tiles to each other; tile j of the block uses slot
// j % 4, or j % (LATE + 1) of what is only needed from its first walk to its second, which comes
// after the first one of tile j + LATE.  CW compute warps, GLR_X exchange warps, one copying warp.
//   tick:  the tile's chunk and channels are known (copying warp)
//   full:  its rows (copying warp), its sequences, place and gate (exchange warp) are there
//   late:  rows that only the second walk needs are there (copying warp)
//   state: the states before each warp's tokens are there (exchange warp)
//   free:  the results are written; the tile's rows may be overwritten (compute warps)
//   runs:  the warps' runs are there (compute warps)
// Every wait is bounded.  The warp whose wait for another warp runs out records it in the status word and in
// `over`, which the exchange warps and the copying one look at while they wait for long, and leaves, storing
// nothing more; so do the others when theirs run out, the copying warp when its copies have landed.
constexpr int GLR_X = 3;
template <int CW_, int LATE_>
struct GlrRing {
    static constexpr int CW = CW_, LATE = LATE_, THREADS = 32 * (CW + GLR_X + 1);
    uint4 sub[LATE + 1][CW][32];  // the warps' runs, in the order of the scan; then the states before them
    GlrInfo info[8];            // (j % 8)
    float4 gate[4][32];         // the gate's parameters (softplus), as GlrGate wants them
    int4 tick[8];               // (j % 8) the tile's chunk in the order of the scan (-1: no more), first channel
    uint64_t bar[7][4];         // (the ticks take two rows: the copying warp is up to eight tiles ahead of who reads them)
    uint64_t never;             // (nothing arrives here: for the test of a wait that runs out)
    int over;                   // a wait has run out
    int looked[GLR_X], left;    // the last tile that each exchange warp has looked at; how many of them have left
};
enum { GLR_TICK = 0, GLR_FULL = 2, GLR_LATE = 3, GLR_STATE = 4, GLR_FREE = 5, GLR_RUNS = 6 };
// tile j's barrier and its phase
template <class Ring>
__device__ __forceinline__ uint32_t glr_bar(Ring& ring, int kind, int j) {
    return smem_u32(&ring.bar[kind][kind == GLR_TICK ? j & 7 : j & 3]);
}
__device__ __forceinline__ uint32_t glr_phase(int kind, int j) { return (kind == GLR_TICK ? j >> 3 : j >> 2) & 1; }

// (rows copied in 16-byte pieces arrive as a count of bytes that one lane announces, others as
// every lane's own copies)
template <class Ring>
__device__ __forceinline__ void glr_ring_init(Ring& ring, bool wide) {
    if (threadIdx.x < 28) {
        const int kind = threadIdx.x / 4, rows = wide ? 1 : 32;
        tc::mbar_init(smem_u32(&ring.bar[kind][threadIdx.x % 4]),
                      kind == GLR_FREE ? Ring::CW : kind == GLR_RUNS ? 32 * Ring::CW : kind == GLR_FULL ? rows + 1 : kind == GLR_LATE ? rows : 1);
    } else if (threadIdx.x == 28) {
        tc::mbar_init(smem_u32(&ring.never), 1);
        for (int i = 0; i < 8; ++i) ring.tick[i] = make_int4(-1, 0, 0, 0);
        for (int i = 0; i < GLR_X; ++i) ring.looked[i] = -1;
        ring.over = ring.left = 0;
    }
    __syncthreads();
}
// The compute warps' wait for tile j's barrier; the thread leaves if it runs out.  (Threads of its warp that
// still saw the phase complete go on, rightly, to their next wait.  What else is done between the polls, or
// called after many, makes every wait end later: with a look at the clock and the flag 30011 x 4096 took
// 275 us instead of 241.)
template <class Ring>
__device__ __forceinline__ void glr_wait(const GlrParams& p, Ring& ring, int kind, int j) {
    if (!tc::mbar_wait(glr_bar(ring, kind, j), glr_phase(kind, j), GLR_SPIN_COMPUTE)) {
        glr_give_up(&ring.over, p.status);
        asm volatile("exit;");
    }
}
// The other warps', who talk across their lanes: false for the whole warp if it or another wait of the block
// has run out.  Their waits are long and not urgent: NAP nanoseconds of sleep between polls (which took a
// quarter of the kernel's instructions).
static __device__ __noinline__ bool glr_wait_on(uint32_t bar, uint32_t parity, volatile int* over, int* status) {
    for (int it = 0; it < GLR_SPIN_LONG / 16 && !*over; ++it)
        if (tc::mbar_wait(bar, parity, 16)) return true;
    glr_give_up(over, status);
    return false;
}
template <int NAP, class Ring>
__device__ __forceinline__ bool glr_wait_long(const GlrParams& p, Ring& ring, int kind, int j) {
    const uint32_t bar = glr_bar(ring, kind, j), parity = glr_phase(kind, j);
    bool there = false;
#pragma unroll 1
    for (int it = 0; it < 1 << 14 && !there; ++it) {
        there = tc::mbar_wait(bar, parity, 1);
        if (!there) __nanosleep(NAP);
    }
    if (!there) there = glr_wait_on(bar, parity, &ring.over, p.status);
    return __all_sync(~0u, there);
}
// What this warp has written for tile j is there.
template <class Ring>
__device__ __forceinline__ void glr_signal(Ring& ring, int kind, int j) {
    __syncwarp();
    if (threadIdx.x % 32 == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(glr_bar(ring, kind, j)) : "memory");
}
// The same for this thread, without waiting for the others of its warp (backward 32768 x 2048: 230 us, 232
// with one arrival a warp).
template <class Ring>
__device__ __forceinline__ void glr_arrive(Ring& ring, int kind, int j) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(glr_bar(ring, kind, j)) : "memory");
}
// The copying warp's end: its copies for tiles [from, to) have landed.  They report to the barrier that the
// tile's exchange warp reports to as well; if that has left before it did, this warp does in its place.
template <class Ring>
__device__ __forceinline__ void glr_landed(const GlrParams& p, Ring& ring, int from, int to) {
    for (int j = max(from, 0); j < to; ++j) {
        if (glr_wait_long<20>(p, ring, GLR_FULL, j)) continue;
        for (int it = 0; *const_cast<volatile int*>(&ring.left) < GLR_X && it < 1 << 24; ++it) __nanosleep(100);
        __syncwarp();
        if (threadIdx.x % 32 == 0 && *const_cast<volatile int*>(&ring.looked[j % GLR_X]) < j)
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(glr_bar(ring, GLR_FULL, j)) : "memory");
        tc::mbar_wait(glr_bar(ring, GLR_FULL, j), glr_phase(GLR_FULL, j), GLR_SPIN_COMPUTE);
    }
}
// An exchange warp leaves.
template <class Ring>
__device__ __forceinline__ void glr_leave(Ring& ring) {
    __syncwarp();
    __threadfence_block();
    if (threadIdx.x % 32 == 0) atomicAdd(&ring.left, 1);
}
// (test hook) A wait of block test_stall - 1 for what never comes.
template <class Ring>
__device__ __forceinline__ bool glr_stalled(const GlrParams& p, Ring& ring, int j) {
    if (p.test_stall != (int)blockIdx.x + 1 || j != 1) return false;
    if (!tc::mbar_wait(smem_u32(&ring.never), 0, 1 << 12)) glr_give_up(&ring.over, p.status);
    return true;
}
// A block's tickets, in the order of its tiles: they count in the workspace when there is something
// to wait for.
__device__ __forceinline__ unsigned glr_ticket(const GlrParams& p, int chunks, int j) {
    return chunks == 1 ? blockIdx.x + j * gridDim.x : atomicAdd(reinterpret_cast<unsigned*>(p.status) + 1, 1u);
}
// An exchange warp's work ahead on tile j: its sequences and place, the gate's parameters.  Returns
// the tile's chunk and first channel (chunk -1: no more tiles, or a wait has run out).
template <bool BWD, class Ring>
__device__ __forceinline__ int4 glr_look(const GlrParams& p, Ring& ring, int chunks, int j, int lane) {
    if (!glr_wait_long<50>(p, ring, GLR_TICK, j)) return make_int4(-1, 0, 0, 0);
    const int4 tick = ring.tick[j & 7];
    const int k = tick.x, kc = BWD ? chunks - 1 - k : k, c = tick.y + 2 * lane;
    if (k >= 0) {
        if (p.gate == GLR_SOFTPLUS) {
            const int at = c < p.C ? c : 0;
            const float2 l = *reinterpret_cast<const float2*>(p.A_log + at), b = *reinterpret_cast<const float2*>(p.dt_bias + at);
            ring.gate[j & 3][lane] = GlrGate<GLR_SOFTPLUS>::param(l, b);
        }
        const int64_t t0 = (int64_t)kc * GLR_CHUNK;
        glr_find_place<BWD>(p, ring.info[j & 7], chunks, k, t0, (int)min((int64_t)GLR_CHUNK, p.T - t0), lane);
    }
    glr_signal(ring, GLR_FULL, j);
    if (lane == 0) *const_cast<volatile int*>(&ring.looked[j % GLR_X]) = j;
    if (k >= 0) glr_empty_sequences(p, BWD ? p.dht : p.h0, BWD ? p.dh0 : p.ht, kc, chunks, c, c < p.C, tick.y == 0);
    return tick;
}

// An exchange warp's work on tile j: its run, published; the states before its warps.  False if its wait
// has run out.
template <bool BWD, class Ring>
__device__ __forceinline__ bool glr_exchange(const GlrParams& p, Ring& ring, const GlrRuns& runs, int chunks, int j, int4 tick,
                                             int lane) {
    constexpr int CW = Ring::CW;
    const int half = j % (Ring::LATE + 1), k = tick.x, c = tick.y + 2 * lane;
    const GlrInfo& at = ring.info[j & 7];
    const bool any = at.any;
    Run y = run_identity();
    if (!glr_wait_long<50>(p, ring, GLR_RUNS, j)) return false;
    if (chunks > 1) {
        const int64_t stride = p.C / 2;
        const int c2 = (c < p.C ? c : 0) / 2;  // (a lane without channels folds channel 0's)
        Run own = run_from_bits(ring.sub[half][0][lane]);
        if (!any) {
            float2 rest = __fadd2_rn(own.A, splat(-1.f));  // A - 1, for the reason at run_decay
#pragma unroll
            for (int i = 1; i < CW; ++i) {
                const Run next = run_from_bits(ring.sub[half][i][lane]);
                const float2 more = __fadd2_rn(next.A, splat(-1.f));
                rest = __ffma2_rn(rest, more, __fadd2_rn(rest, more));
                own = run_then_plain(own, next);
            }
            if (rest.x >= -0.5f && rest.x <= 1.f) own.A.x = 1.f + rest.x;
            if (rest.y >= -0.5f && rest.y <= 1.f) own.A.y = 1.f + rest.y;
        } else {
#pragma unroll 1
            for (int i = 1; i < CW; ++i) own = run_then(own, run_from_bits(ring.sub[half][i][lane]));
        }
        if (c < p.C) run_publish(runs.chunk + k * stride + c2, own);
        // The chunks' runs, of which the last chunk of a group makes the group's; then the state and the
        // groups' runs.  (Nothing is published later than what it is made of allows, for others wait for
        // it: groups published only after the state before them made one chain of everything, four times
        // slower on few channels.  One loop: each copy of the fold's code costs registers.)
        Run near = y;
#pragma unroll 1
        for (int older = 0; older < 2; ++older) {
            const Run r = glr_fold(runs.state + (int64_t)(k / GLR_SUPER - 1) * stride + c2, older && at.state,
                                   (older ? runs.group + at.group0 * stride : runs.chunk + at.chunk0 * stride) + c2, stride,
                                   older ? at.groups : at.chunks, &ring.over, p.status);
            if (older) {
                y = run_then_plain(r, near);
            } else {
                near = r;
                if ((k + 1) % GLR_GROUP == 0 && c < p.C)
                    run_publish(runs.group + k / GLR_GROUP * stride + c2, run_then(near, own));
            }
        }
        if ((k + 1) % GLR_SUPER == 0 && c < p.C)
            run_publish(runs.state + k / GLR_SUPER * stride + c2, Run{splat(-0.f), run_then(Run{splat(-0.f), y.H}, own).H});
    }
    if (!any) {
#pragma unroll
        for (int i = 0; i < CW; ++i) {
            const Run next = run_from_bits(ring.sub[half][i][lane]);
            *reinterpret_cast<float2*>(&ring.sub[half][i][lane]) = y.H;
            y.H = __ffma2_rn(next.A, y.H, next.H);
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < CW; ++i) {
            const Run next = run_from_bits(ring.sub[half][i][lane]);
            *reinterpret_cast<float2*>(&ring.sub[half][i][lane]) = y.H;
            y = run_then(y, next);
        }
    }
    glr_signal(ring, GLR_STATE, j);
    return true;
}

// The copying warp's copies of a tile's rows of one tensor into shared memory.  Where every row of
// the call's tensors is a whole number of aligned 16-byte pieces (`wide`) they go by the tensor's
// map, in boxes of 64 rows, or of 8 where the rows of different warps are to lie 8 x 256 bytes
// apart; they report to the barrier by their bytes.  (A copy of each row by itself kept the copy
// engine busy for longer than the rows took to arrive.)  Else a lane copies a pair of channels of
// each row there is, and reports when all of its copies are done.
// Rows of g lie in their warp's 8 x 256 bytes, which the first walk fills with fp32 values row by
// row: float32 rows in place, bf16 rows in the half that the walk fills last.
template <class TG>
__host__ __device__ constexpr int glr_raw_offset(bool bwd) { return sizeof(TG) == 2 && !bwd ? 1024 : 0; }
struct GlrMaps {
    CUtensorMap g, x, dh, h;
};
// rows t0 .. t0 + 63 (the first `first` of them left out), channels from c0 on.  PITCH: bytes from
// row to row in shared memory, EVERY: from 8 rows to the next 8.
template <int PITCH, int EVERY, class T>
__device__ __forceinline__ void glr_copy_rows(void* to, const CUtensorMap* map, const T* base, int64_t ld, int64_t t0, int first,
                                              int rows, int c0, int cols, bool wide, uint32_t bar, int lane) {
    const uint32_t dst = smem_u32(to);
    if (wide) {
        if (EVERY == 8 * PITCH) {
            if (lane == 0) tc::tma_load_2d(dst, map, c0, (int)t0, bar);
        } else if (lane < 8) {
            tc::tma_load_2d(dst + lane * EVERY, map, c0, (int)t0 + 8 * lane, bar);
        }
    } else if (2 * lane < cols) {
        const T* src = base + t0 * ld + c0 + 2 * lane;
        uint32_t at = dst + 2 * lane * (int)sizeof(T);
        auto copy = [&](int q, const T* row) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(at + q * PITCH), "l"(row), "n"(2 * sizeof(T)) : "memory");
        };
        // (few instructions a row: one warp copies for eight, which wait for it.  32768 x 2050, softplus:
        // forward 197 us, backward 351, an eighth more with the addresses worked out row by row; 2048
        // channels by the tensor maps 132 and 232)
#pragma unroll 1
        for (int i = 0; i < rows; i += 8, at += EVERY) {
            if (i >= first && i + 8 <= rows) {
#pragma unroll
                for (int q = 0; q < 8; ++q, src += ld) copy(q, src);
            } else {
#pragma unroll 1
                for (int q = 0; q < 8; ++q, src += ld)
                    if (i + q >= first && i + q < rows) copy(q, src);
            }
        }
    }
}
// Announces the bytes of tile j's rows (wide), before the copies; after them, the lane's arrival (not wide).
template <class Ring>
__device__ __forceinline__ uint32_t glr_announce(Ring& ring, int kind, int j, bool wide, uint32_t bytes, int lane) {
    const uint32_t bar = glr_bar(ring, kind, j);
    if (wide && lane == 0) tc::mbar_expect_tx(bar, bytes);
    __syncwarp();
    return bar;
}
__device__ __forceinline__ void glr_report(uint32_t bar, bool wide) {
    if (!wide) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

// Blocks of a scan kernel that an SM's 228 KB of shared memory hold (1 KB of it goes with each block): two with bf16
// tiles, one with float32's.
__host__ __device__ constexpr int glr_per_sm(size_t smem) { return 2 * (smem + 1024) <= 228 * 1024 ? 2 : 1; }

// Launches a scan kernel on as many blocks as are resident at once (or tiles, if fewer).
// `ready`: the devices whose shared-memory limit of this kernel is raised.
template <class Tile, class K>
cudaError_t glr_launch(K kernel, std::atomic<uint64_t>& ready, const GlrParams& p, const GlrMaps& maps, cudaStream_t s) {
    constexpr size_t smem = sizeof(Tile);
    constexpr int per_sm = glr_per_sm(smem), threads = decltype(Tile::ring)::THREADS;
    static_assert(per_sm * (smem + 1024) <= 228 * 1024, "a resident block's tiles");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const int64_t all = (int64_t)glr_chunks(p) * ((p.C + GLR_TILE - 1) / GLR_TILE), resident = (int64_t)per_sm * num_sms();
    kernel<<<(unsigned)(all < resident ? all : resident), threads, smem, s>>>(p, maps);
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
