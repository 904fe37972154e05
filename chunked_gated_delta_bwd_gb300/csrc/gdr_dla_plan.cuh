// How the chunks of linear attention with a decay for each head are shared out.
//
// A chain is one (sequence, head): its chunks of 128 tokens in the order in which the state passes through
// them (back to front for the gradients' walk).  A chain takes one place more than it has chunks, ahead of
// them: its states in and out are as many bytes as a chunk's.
//
// Long chains stand in one line, chain after chain (sequence by sequence, head by head), and a block takes
// one range of it: ranges of equal length, so that every multiprocessor has the same work whatever the
// sequences' lengths.  (16 sequences of 1 to 60 chunks, ranges of as many chains each: the longest took 1.9
// times the mean.)  A chain that crosses from one range into the next hands its state over, for which its
// last part is read twice (gdr_dla.cu).
//
// Chains that are short beside a block's share stand in a queue, the longest first: blocks take one whole
// when they have nothing left, and nothing is handed over.
#pragma once
#include "gdr_common.cuh"
#include "gdr_dla.h"

namespace gdr {
namespace dla {

constexpr int CHUNK = 128;

// What the blocks are asked for: ranges, and a queue where packed sequences allow it (the longest first where they are
// few, 32: a sequence a lane); ranges of whole chains (SNAP: packed sequences of a few chunks); all chains from the queue (WHOLE: sequences of one length).
enum Mode { RANGES, SNAP, WHOLE };

// A chunk of the line or the queue.
struct Place {
    int rank, seq;              // the sequence, and its number in the line
    int head, pos, count;       // the chunk's number in its chain, and the chain's chunks
    int len;                    // the sequence's tokens
    int64_t begin;              // its first token
};

// What a block learns before it starts, through shared memory.
struct Plan {
    int total;      // places of the line; -1: the sequences' borders are inconsistent
    int ranges;     // ranges that are not empty (no more than there are places)
    int f0, f1;     // the range
    int f;          // the place of its first chunk
    int cut;        // sequences of the line; those behind them in the order are the queue's
    int chains;     // of the queue
    int order[32];  // the sequences that have tokens, the longest first, where the call has 32 at most
    Place at;       // the block's first chunk
};

struct Line {
    int N, H;
    int64_t T, seq_len;
    const int64_t* cu;
    int back;
    const Plan* plan;

    __device__ __forceinline__ void sequence(Place& p) const {
        p.seq = cu && N <= 32 ? plan->order[p.rank] : p.rank;
        p.begin = cu ? cu[p.seq] : p.seq * seq_len;
        p.len = (int)(cu ? cu[p.seq + 1] - p.begin : seq_len);
        p.count = (p.len + CHUNK - 1) / CHUNK;
    }
    // the next chunk, at place f of the line (after the last one `rank` is the line's number of sequences)
    __device__ __forceinline__ void next(Place& p, int& f) const {
        ++f;
        if (++p.pos < p.count) return;
        ++f;
        p.pos = 0;
        if (++p.head < H) return;
        p.head = 0;
#pragma unroll 1
        while (++p.rank < plan->cut) {
            sequence(p);
            if (p.count) return;
        }
    }
    // the first chunk of chain `c` of the queue
    __device__ __forceinline__ Place chain(int c) const {
        Place p;
        p.rank = plan->cut + c / H;
        p.head = c % H;
        p.pos = 0;
        sequence(p);
        return p;
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

// Whether chains are short enough for the queue: the time at which the last block would end, in places, beside the
// mean.  Ranges read their last chains' inputs twice and take two more launches; the queue leaves blocks idle at its
// end, but what they leave of the memory's rate the others have.  8192 tokens in one sequence of so many heads of 128,
// ranges and whole chains (1 / mean):
//   96 (1.58) 213 and 199 us   90 (1.69) 202 and 198   84 (1.81) 189 and 198   76 (2) 168 and 197
// the backward (50 blocks a walk):  32 (1.56) 192 and 199   28 (1.79) 175 and 175, 24 (2.08) 159 and 197
// 16 sequences of up to 70 chunks, 32 heads: all ranges 254, queue up to 1.25 of the mean 244, up to 1.8 227.
__host__ __device__ inline bool short_enough(int64_t end, int64_t mean) { return 5 * end <= 9 * mean; }

// total r / ranges, in 32 bits (there are a few hundred ranges at most)
__device__ __forceinline__ int range_begin(int total, int r, int ranges) {
    const uint32_t whole = (uint32_t)total / (uint32_t)ranges, rest = (uint32_t)total - whole * ranges;
    return (int)(whole * r + rest * r / (uint32_t)ranges);
}

// places of a chain of that many tokens
__device__ __forceinline__ int places(int64_t tokens) { return tokens > 0 ? (int)((tokens + CHUNK - 1) / CHUNK) + 1 : 0; }
// The first chunk from place f0 of the line on, from the sequence (its number in the line) that holds the place and the
// places of a head before it.
__device__ __forceinline__ void set_first(Plan* out, const Line& line, int rank, int before) {
    Place p;
    p.rank = rank;
    line.sequence(p);
    const int in = out->f0 - before * line.H;
    p.head = in / (p.count + 1);
    p.pos = in - p.head * (p.count + 1) - 1;
    out->f = out->f0;
    if (p.pos < 0) p.pos = 0, ++out->f;
    out->at = p;
}

// (`cut`, `chains`: sequences of the line, chains of the queue)
__device__ __forceinline__ void set_range(Plan* out, int total, int range, int ranges, int cut, int chains) {
    ranges = max(min(ranges, total), 0);
    out->cut = cut;
    out->chains = chains;
    out->total = total;
    out->ranges = ranges;
    out->f = out->f0 = total < 0 || range >= ranges ? 0 : range_begin(total, range, ranges);
    out->f1 = total < 0 || range >= ranges ? 0 : range_begin(total, range + 1, ranges);
}

// All THREADS threads of the block; `out` and `scratch` (THREADS / 32 ints) in shared memory.
template <int THREADS>
__device__ __forceinline__ void make_plan(const Line& line, int range, int ranges, int mode, Plan* out, int* scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!line.cu) {
        if (tid == 0) {
            const int per = places(line.seq_len), all = line.N * line.H;
            if (mode == WHOLE) {
                set_range(out, 0, range, ranges, 0, all);
            } else {
                set_range(out, per * all, range, ranges, line.N, 0);
                const int seq = out->f0 / (per * line.H);
                if (out->f0 < out->f1) set_first(out, line, seq, seq * per);
            }
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
            // its number in the order of lengths, the places ahead of it (of a head)
            int rank = 0, ahead = 0, all = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const int u = __shfl_sync(~0u, mine, j);
                if (u > mine || (u == mine && j < lane)) ++rank, ahead += u;
                all += u;
            }
            out->order[rank] = lane;
            __syncwarp();
            // The line takes sequences up to the last that is not short: its last chain begins, at the latest, when the
            // blocks have shared out evenly what is ahead of it.
            const int sequences = __popc(__ballot_sync(~0u, mine));
            int cut = sequences;
            if (mode == RANGES) {
                const int64_t ends = ((int64_t)(ahead + mine) * line.H - mine) / ranges + mine;
                cut = mine && !short_enough(ends, (int64_t)all * line.H / ranges) ? rank + 1 : 0;
#pragma unroll
                for (int o = 16; o; o >>= 1) cut = max(cut, __shfl_xor_sync(~0u, cut, o));
            }
            // places of the line, of a head; blocks for it: no range longer than the mean
            int in_line = rank < cut ? mine : 0;
#pragma unroll
            for (int o = 16; o; o >>= 1) in_line += __shfl_xor_sync(~0u, in_line, o);
            const int blocks = all ? (int)(((int64_t)in_line * ranges + all - 1) / all) : 0;
            if (lane == 0) set_range(out, bad ? -1 : in_line * line.H, range, blocks, cut, (sequences - cut) * line.H);
            __syncwarp();
            const int at = out->f0 / line.H;
            if (out->f0 < out->f1 && mine && ahead <= at && at < ahead + mine) set_first(out, line, rank, ahead);
        }
        __syncthreads();
    } else {
        // every block adds up the sequences' places: N reads, all of them hits in the second-level cache
        int sum = 0, longest = 0;
        bool holes = false;
        bool bad = line.cu[0] != 0 || line.cu[line.N] != line.T;
#pragma unroll 1
        for (int i = tid; i < line.N; i += THREADS) {
            const int64_t len = line.cu[i + 1] - line.cu[i];
            bad |= len < 0 || len > line.T;
            sum += places(len);
            longest = max(longest, places(len));
            holes |= len == 0;
        }
        // (borders that never decrease from 0 to T are all inside)
        bad = __syncthreads_or(bad);
        holes = __syncthreads_or(holes);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o), longest = max(longest, __shfl_xor_sync(~0u, longest, o));
        if (lane == 0) scratch[warp] = sum;
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) total += scratch[i];
        __syncthreads();
        if (lane == 0) scratch[warp] = longest;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) longest = max(longest, scratch[i]);
        // (not in the order of lengths: the last block ends at most one chain after the blocks have shared out all evenly;
        // a queue with empty sequences would have to skip them one by one)
        const int64_t mean = (int64_t)total * line.H / ranges;
        const bool queue = mode == RANGES && !bad && !holes && short_enough(mean + longest, mean);
        if (tid == 0) {
            if (queue) set_range(out, 0, range, ranges, 0, line.N * line.H);
            else set_range(out, bad ? -1 : total * line.H, range, ranges, line.N, 0);
        }
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
    if (mode == SNAP && tid == 0 && out->f0 < out->f1) {
        // whole chains: the first that begins in the range, to the end of the last that does
        if (out->f - out->at.pos - 1 < out->f0) {
            out->f += out->at.count - 1 - out->at.pos;
            out->at.pos = out->at.count - 1;
            if (out->f + 1 < out->f1) line.next(out->at, out->f);
            else out->f1 = out->f0;  // (none does)
        }
    }
    if (mode == SNAP) __syncthreads();
}

// whether the walk of a range goes on at place f of the line, `p`
__device__ __forceinline__ bool more(const Plan& plan, const Place& p, int f, int mode) {
    return f < plan.total && plan.f0 < plan.f1 && (mode == SNAP ? p.pos != 0 || f - 1 < plan.f1 : f < plan.f1);
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
