// qmixer_scan.cuh -- the selective scan of prompts: what its kernels share.
//
// Segments.  A scan is one chain per (sequence, head).  Where these are fewer
// than the SMs hold at once, or unequal, every sequence is cut into segments of
// seg_len tokens that are scanned side by side, in three launches:
//   1. the state that each segment but a sequence's last adds, from zero, and
//      the product of its decays;
//   2. the chain over each sequence's segments: the state in front of each;
//   3. the scan of every segment from the state in front of it.
// Launch 1 costs about half of launch 3, so the cut is made only where the
// chains would leave SMs idle for longer than that (scan_plan).  One sequence of
// 16001 tokens, 16 heads of 128 x 128, runs in nine segments of 1792 tokens, two rounds
// of CTAs: 137.5 us (of the three launches, cold and one by one, 53, 8 and 90); in four
// of 4096, one round, 137.5 too, in eight 149.5.
#pragma once

#include "qmixer_common.cuh"

namespace qm {

struct ScanParams {
    const void* x;
    int64_t xs;
    const void* dt;
    int64_t dts;
    const float* A;
    const void* B;
    int64_t Bs;
    const void* C;
    int64_t Cs;
    const float* D;
    const float* dt_bias;
    float* state;
    void* y;
    int64_t ys;
    Sequences seq;
    int heads, per_group, dv;
    bool dt_bf16, softplus, initial;
    int64_t seg_len;            // tokens a segment, at least 1
    int64_t segments;           // room for so many in seg_state
    bool cut;                   // more than one segment a sequence may be there
    float* seg_state;           // [segments][heads][d_k][d_v], where cut
    float* seg_decay;           // [segments][heads]
    uint32_t polls;             // of a wait, before it is given up
    int32_t drop_from;          // chunks from this one on are never loaded; -1: off
};

constexpr uint32_t kWaitPolls = 1u << 24;      // several seconds

constexpr int kBatchTokens = 16;   // the recurrent form's segments are whole batches,
constexpr int kChunk = 128;        // the chunked form's whole chunks

struct Segment {
    int sequence;
    int64_t from, to;           // tokens
    bool last;                  // of its sequence
};

__device__ __forceinline__ int64_t segments_of(const ScanParams& p, int s) {
    const int64_t n = p.seq.start(s + 1) - p.seq.start(s);
    return n <= p.seg_len ? 1 : (n + p.seg_len - 1) / p.seg_len;
}

// Segment number g, counted over the sequences in order; false behind the last.
// Called by whole warps.
__device__ __forceinline__ bool find_segment(const ScanParams& p, int64_t g, Segment& o) {
    int64_t k;
    int s;
    if (!p.cut) {
        if (g >= p.seq.n) return false;
        s = (int)g;
        k = 0;
    } else if (!p.seq.starts) {
        const int64_t each = segments_of(p, 0);
        if (g >= each * p.seq.n) return false;
        s = (int)(g / each);
        k = g % each;
    } else {
        const int lane = threadIdx.x & 31;
        int64_t before = 0;
        s = -1;
        for (int base = 0; base < p.seq.n && s < 0; base += 32) {
            int64_t c = base + lane < p.seq.n ? segments_of(p, base + lane) : 0, sum = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t u = __shfl_up_sync(~0u, sum, d);
                if (lane >= d) sum += u;
            }
            const unsigned past = __ballot_sync(~0u, before + sum > g);
            if (past) {
                const int at = __ffs(past) - 1;
                s = base + at;
                k = g - (before + __shfl_sync(~0u, sum - c, at));
            } else {
                before += __shfl_sync(~0u, sum, 31);
            }
        }
        if (s < 0) return false;
    }
    const int64_t from = p.seq.start(s), end = p.seq.start(s + 1);
    o.sequence = s;
    o.from = from + k * p.seg_len;
    o.to = p.cut && o.from + p.seg_len < end ? o.from + p.seg_len : end;
    o.last = o.to == end || end <= from;
    return true;
}

// The kernels of the recurrent form (binary32) and of the chunked form (bfloat16,
// tensor cores): states only (launch 1) or the whole scan.  False, with nothing
// launched and no error left behind, where a launch cannot be prepared.
bool launch_scan_rec(const ScanParams& p, int dk, int64_t segments, bool states_only, cudaStream_t st);
bool launch_scan_chunk(const ScanParams& p, int dk, int64_t segments, bool states_only, cudaStream_t st);
// CTAs of the chunked form on the current device that gave up a wait, once `st` has run.
bool scan_timeouts(uint64_t* count, cudaStream_t st);

}  // namespace qm
