// How the chunks of linear attention with a decay for each head are shared out.
//
// A chain is one (sequence, head): its chunks of 128 tokens in the order in which the state passes through
// them (back to front for the gradients' walk).  All chunks of a call stand in one line, chain after
// chain (sequence by sequence, head by head), and each block takes one range of it: ranges of equal
// length, so that every multiprocessor has the same work whatever the sequences' lengths.  A chain
// takes one place more than it has chunks, ahead of them: its states in and out are as many bytes as a
// chunk's.  (16 sequences of 1 to 60 chunks: the ranges with many short ones were 1.9 times as long.)  A chain that
// crosses from one range into the next hands its state over (gdr_dla.cu); where chains are short
// the ranges end with whole chains instead (`snap`).
#pragma once
#include "gdr_common.cuh"
#include "gdr_dla.h"

namespace gdr {
namespace dla {

constexpr int CHUNK = 128;

// A chunk of the line.
struct Place {
    int seq, head, pos, count;  // the chunk's number in its chain, and the chain's chunks
    int len;                    // the sequence's tokens
    int64_t begin;              // its first token
};

struct Line {
    int N, H;
    int64_t T, seq_len;
    const int64_t* cu;
    int back;

    __device__ __forceinline__ void sequence(Place& p) const {
        p.begin = cu ? cu[p.seq] : p.seq * seq_len;
        p.len = (int)(cu ? cu[p.seq + 1] - p.begin : seq_len);
        p.count = (p.len + CHUNK - 1) / CHUNK;
    }
    // the next chunk, at place f of the line (after the last one `seq` is N)
    __device__ __forceinline__ void next(Place& p, int& f) const {
        ++f;
        if (++p.pos < p.count) return;
        ++f;
        p.pos = 0;
        if (++p.head < H) return;
        p.head = 0;
#pragma unroll 1
        while (++p.seq < N) {
            sequence(p);
            if (p.count) return;
        }
    }
    // tokens of the chain before its chunk `pos`, in the order of the walk
    __device__ __forceinline__ int before(const Place& p, int pos) const {
        if (!back) return min(pos * CHUNK, p.len);
        return pos == 0 ? 0 : p.len - (p.count - pos) * CHUNK;
    }
    __device__ __forceinline__ int first_row(const Place& p) const { return (back ? p.count - 1 - p.pos : p.pos) * CHUNK; }
    __device__ __forceinline__ int rows(const Place& p) const { return min(CHUNK, p.len - first_row(p)); }
    __device__ __forceinline__ int token(const Place& p) const { return (int)p.begin + first_row(p); }
};

// What a block learns before it starts, through shared memory.
struct Plan {
    int total;    // places of the line; -1: the sequences' borders are inconsistent
    int ranges;   // ranges that are not empty (no more than there are places)
    int f0, f1;   // the range
    int f;        // the place of its first chunk
    Place at;     // its first chunk
};

// total r / ranges, in 32 bits (there are a few hundred ranges at most)
__device__ __forceinline__ int range_begin(int total, int r, int ranges) {
    const uint32_t whole = (uint32_t)total / (uint32_t)ranges, rest = (uint32_t)total - whole * ranges;
    return (int)(whole * r + rest * r / (uint32_t)ranges);
}

// places of a chain of that many tokens
__device__ __forceinline__ int places(int64_t tokens) { return tokens > 0 ? (int)((tokens + CHUNK - 1) / CHUNK) + 1 : 0; }
// The first chunk from place f0 of the line on, from the sequence that holds the place and the places of a head before it.
__device__ __forceinline__ void set_first(Plan* out, const Line& line, int seq, int before) {
    Place p;
    p.seq = seq;
    line.sequence(p);
    const int in = out->f0 - before * line.H;
    p.head = in / (p.count + 1);
    p.pos = in - p.head * (p.count + 1) - 1;
    out->f = out->f0;
    if (p.pos < 0) p.pos = 0, ++out->f;
    out->at = p;
}

__device__ __forceinline__ void set_range(Plan* out, int total, int range, int ranges) {
    ranges = max(min(ranges, total), 1);
    out->total = total;
    out->ranges = ranges;
    out->f = out->f0 = total < 0 || range >= ranges ? 0 : range_begin(total, range, ranges);
    out->f1 = total < 0 || range >= ranges ? 0 : range_begin(total, range + 1, ranges);
}

// All THREADS threads of the block; `out` and `scratch` (THREADS / 32 ints) in shared memory.
template <int THREADS>
__device__ __forceinline__ void make_plan(const Line& line, int range, int ranges, int snap, Plan* out, int* scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!line.cu) {
        if (tid == 0) {
            const int per = places(line.seq_len);
            set_range(out, per * line.N * line.H, range, ranges);
            const int seq = out->f0 / (per * line.H);
            set_first(out, line, seq, seq * per);
        }
        __syncthreads();
    } else if (line.N <= 32) {
        // one warp, a sequence a lane
        if (warp == 0) {
            int64_t begin = 0, end = 0;
            if (lane < line.N) begin = line.cu[lane], end = line.cu[lane + 1];
            const int64_t len = end - begin;
            const bool bad = __any_sync(~0u, lane < line.N && (len < 0 || len > line.T || (lane == 0 && begin != 0) || (lane == line.N - 1 && end != line.T)));
            const int mine = lane < line.N && !bad ? places(len) : 0;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int u = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += u;
            }
            const int total = bad ? -1 : __shfl_sync(~0u, upto, 31) * line.H;
            if (lane == 0) set_range(out, total, range, ranges);
            __syncwarp();
            const int at = out->f0 / line.H, before = upto - mine;
            if (out->f0 < out->f1 && mine && before <= at && at < upto) set_first(out, line, lane, before);
        }
        __syncthreads();
    } else {
        // every block adds up the sequences' places: N reads, all of them hits in the second-level cache
        int sum = 0;
        bool bad = line.cu[0] != 0 || line.cu[line.N] != line.T;
#pragma unroll 1
        for (int i = tid; i < line.N; i += THREADS) {
            const int64_t len = line.cu[i + 1] - line.cu[i];
            bad |= len < 0 || len > line.T;
            sum += places(len);
        }
        // (borders that never decrease from 0 to T are all inside)
        bad = __syncthreads_or(bad);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == 0) scratch[warp] = sum;
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) total += scratch[i];
        if (tid == 0) set_range(out, bad ? -1 : total * line.H, range, ranges);
        __syncthreads();
        const int f0 = out->f0;
        // the sequence that holds place f0 (none where the range is empty)
        int base = 0;
#pragma unroll 1
        for (int i0 = 0; f0 < out->f1 && i0 < line.N; i0 += THREADS) {
            const int i = i0 + tid;
            const int mine = i < line.N ? places(line.cu[i + 1] - line.cu[i]) : 0;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int u = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += u;
            }
            __syncthreads();
            if (lane == 31) scratch[warp] = upto;
            __syncthreads();
            int strip = 0;
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) {
                if (w < warp) upto += scratch[w];
                strip += scratch[w];
            }
            const int before = base + upto - mine;
            if (mine && before <= f0 / line.H && f0 / line.H < before + mine) set_first(out, line, i, before);
            base += strip;
            if (base > f0 / line.H) break;
        }
        __syncthreads();
    }
    if (snap && tid == 0 && out->f0 < out->f1) {
        // whole chains: the first that begins in the range, to the end of the last that does
        if (out->f - out->at.pos - 1 < out->f0) {
            out->f += out->at.count - 1 - out->at.pos;
            out->at.pos = out->at.count - 1;
            if (out->f + 1 < out->f1) line.next(out->at, out->f);
            else out->f1 = out->f0;  // (none does)
        }
    }
    if (snap) __syncthreads();
}

// whether the walk of a range goes on at `p`, place f of the line
__device__ __forceinline__ bool more(const Plan& plan, const Place& p, int f, int snap) {
    return plan.f0 < plan.f1 && f < plan.total && (snap ? p.pos != 0 || f - 1 < plan.f1 : f < plan.f1);
}

// The log decay of a head.  (Below -10^4 no token remembers another; an infinite one would make 0 times infinity.)
__device__ __forceinline__ float log_decay(const float* g, int head) {
    const float x = __ldg(g + head);
    return x < -1e4f ? -1e4f : x;
}
// e^(g n)
__device__ __forceinline__ float power(float g, int n) { return expf(g * (float)n); }
// e^(g n) S + t as c.y S + (c.x S + t): a decay near 1 is held by its distance from 1, so that its rounding
// does not add up over thousands of chunks.
__device__ __forceinline__ float2 carry(float g, int n) {
    const float a = g * (float)n;
    return a > -0.5f && a < 0.5f ? make_float2(expm1f(a), 1.f) : make_float2(expf(a), 0.f);
}

}  // namespace dla
}  // namespace gdr
