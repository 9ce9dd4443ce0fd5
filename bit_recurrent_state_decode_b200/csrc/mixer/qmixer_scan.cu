// qmixer_scan.cu -- the prompt scan's plan, the chain over segments, and its
// C entries.
#include "qmixer_scan.cuh"

namespace qm {

// Launch 2 of a cut scan: seg_state holds what each segment adds and becomes the
// state in front of it.  One thread per four elements of a (sequence, head)
// state; the loads of the next segment do not wait for this one's sum.
__global__ void __launch_bounds__(256) join_kernel(const ScanParams p, int dk) {
    const int s = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31;
    const int64_t tile = (int64_t)dk * p.dv, at = (blockIdx.z * (int64_t)blockDim.x + threadIdx.x) * 4;
    int64_t before = 0;
    if (p.seq.starts) {
        for (int i = lane; i < s; i += 32) before += segments_of(p, i);
#pragma unroll
        for (int d = 16; d; d >>= 1) before += __shfl_xor_sync(~0u, before, d);
    } else {
        before = segments_of(p, 0) * s;
    }
    if (at >= tile) return;
    const int64_t n = segments_of(p, s);
    if (before + n > p.segments) return;         // starts that do not ascend
    float4 S = make_float4(0, 0, 0, 0);
    if (p.initial) S = *reinterpret_cast<const float4*>(p.state + ((int64_t)s * p.heads + h) * tile + at);
    float* seg = p.seg_state + (before * p.heads + h) * tile + at;
    const float* decay = p.seg_decay + before * p.heads + h;
    const int64_t step = p.heads * tile;
    for (int64_t k = 0; k + 1 < n; k += 4) {
        float4 add[4];
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (k + i + 1 < n) {
                add[i] = *reinterpret_cast<const float4*>(seg + (k + i) * step);
                a[i] = decay[(k + i) * p.heads];
            }
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (k + i + 1 < n) {
                *reinterpret_cast<float4*>(seg + (k + i) * step) = S;
                S.x = fmaf(S.x, a[i], add[i].x);
                S.y = fmaf(S.y, a[i], add[i].y);
                S.z = fmaf(S.z, a[i], add[i].z);
                S.w = fmaf(S.w, a[i], add[i].w);
            }
    }
    *reinterpret_cast<float4*>(seg + (n - 1) * step) = S;
}

struct ScanPlan {
    int64_t seg_len, segments;   // segments: most that there can be
    bool cut;
    int64_t state_bytes, bytes;  // of the workspace
};

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 148;
    }
    return n;
}

// Where to cut, by an estimate of the time in tokens of one CTA's chain.
// `resident` chains run at once; a CTA of the recurrent form takes a batch's time
// before its first token (of 0 to 256 tokens tried for either form, this gave the
// least over ragged and single prompts); launch 1 takes `states` of launch 3 (measured: 0.41 of the
// chunked form, 0.6 of the recurrent one), and cutting two launches more.
//   equal sequences: whole rounds of resident CTAs, each as long as a segment
//   unequal ones:    the work spread evenly, and the last segment behind it; the
//                    longest uncut sequence is taken as four times the mean (the
//                    lengths lie on the device)
ScanPlan scan_plan(int sequences, int64_t tokens, int heads, int dk, int dv, int dtype, bool ragged, int sms) {
    const bool chunked = dtype == QSTATE_BF16;
    const int64_t unit = chunked ? kChunk : kBatchTokens;
    const int64_t chains = (int64_t)heads * (dv / 64), resident = (chunked ? 1 : dk == 64 ? 3 : 2) * (int64_t)sms;
    const double states = chunked ? 0.41 : 0.6, launches = chunked ? 4 * kChunk : 2 * kBatchTokens;
    const int64_t start = chunked ? 0 : kBatchTokens;
    const int64_t mean = tokens / sequences, longest = ragged ? (4 * mean < tokens ? 4 * mean : tokens) : mean;
    ScanPlan o{};
    o.seg_len = tokens > 0 ? tokens : 1;
    double best = 0.0;
    for (int k = 1; k <= 64; k++) {
        // k segments of the longest sequence
        const int64_t len = ((longest + k - 1) / k + unit - 1) / unit * unit;
        if (k > 1 && len < 2 * unit) break;
        const int64_t each = len > 0 ? (mean + len - 1) / len : 1;
        double time;
        if (ragged) time = (double)tokens * chains / resident * (len + start) / (len > 0 ? len : 1) + 0.5 * len;
        else time = (double)((sequences * chains * each + resident - 1) / resident) * (len + start);
        if (ragged && time < len) time = (double)len;
        if (k > 1) time = time * (1.0 + states) + launches;
        if (k == 1 || time < best) {
            best = time;
            o.cut = k > 1;
            if (k > 1) o.seg_len = len;
        }
    }
    o.segments = o.cut ? tokens / o.seg_len + sequences : sequences;
    if (o.cut) {
        o.state_bytes = o.segments * heads * dk * dv * 4;
        o.bytes = o.state_bytes + (o.segments * heads * 4 + 15) / 16 * 16;
    }
    return o;
}

int check_scan(int sequences, int64_t tokens, int heads, int groups, int dk, int dv, int dtype) {
    if (!known(dtype) || sequences < 0 || tokens < 0 || tokens > INT32_MAX || heads < 1 || groups < 1 ||
        heads % groups || dk < 1 || dv < 1)
        return QSTATE_EINVAL;
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128) || (int64_t)heads * (dv / 64) > 65535)
        return QSTATE_EUNSUPPORTED;
    return QSTATE_OK;
}

// What qmixer_debug_set set for the scans after it.
std::atomic<uint32_t> wait_polls{kWaitPolls};
std::atomic<int32_t> drop_from{-1};

}  // namespace qm

extern "C" {

int qmixer_scan_timeouts(uint64_t* count, qstate_stream stream) {
    if (!count) return QSTATE_EINVAL;
    return qm::scan_timeouts(count, (cudaStream_t)stream) ? QSTATE_OK : QSTATE_ECUDA;
}

int qmixer_debug_set(int32_t drop_from_chunk, uint32_t wait_polls) {
    if (drop_from_chunk < -1 || !wait_polls) return QSTATE_EINVAL;
    qm::drop_from.store(drop_from_chunk, std::memory_order_relaxed);
    qm::wait_polls.store(wait_polls, std::memory_order_relaxed);
    return QSTATE_OK;
}

int64_t qmixer_scan_workspace(int32_t sequences, int64_t tokens, int32_t heads, int32_t groups, int32_t d_k,
                              int32_t d_v, int32_t dtype) {
    const int rc = qm::check_scan(sequences, tokens, heads, groups, d_k, d_v, dtype);
    if (rc != QSTATE_OK) return rc;
    if (!sequences) return 0;
    const int sms = qm::sm_count();
    const int64_t a = qm::scan_plan(sequences, tokens, heads, d_k, d_v, dtype, true, sms).bytes;
    const int64_t b = qm::scan_plan(sequences, tokens, heads, d_k, d_v, dtype, false, sms).bytes;
    return a > b ? a : b;
}

int qmixer_scan(const qmixer_scan_args* args, qstate_stream stream) {
    if (!args) return QSTATE_EINVAL;
    const qmixer_scan_args& a = *args;
    const int rc = qm::check_scan(a.sequences, a.tokens, a.heads, a.groups, a.d_k, a.d_v, a.dtype);
    if (rc == QSTATE_EINVAL) return rc;
    if (!qm::known(a.dt_dtype) || (a.flags & ~(QMIXER_INITIAL | QMIXER_SOFTPLUS))) return QSTATE_EINVAL;
    if (a.x_stride < (int64_t)a.heads * a.d_v || a.y_stride < (int64_t)a.heads * a.d_v || a.dt_stride < a.heads ||
        a.B_stride < (int64_t)a.groups * a.d_k || a.C_stride < (int64_t)a.groups * a.d_k)
        return QSTATE_EINVAL;
    const int size = qm::size_of(a.dtype), unit = 16 / size;
    if (a.x_stride % unit || a.B_stride % unit || a.C_stride % unit || !qm::aligned(a.x, 16) || !qm::aligned(a.B, 16) ||
        !qm::aligned(a.C, 16) || !qm::aligned(a.state, 16) || !qm::aligned(a.workspace, 16) || !qm::aligned(a.y, size) ||
        !qm::aligned(a.dt, qm::size_of(a.dt_dtype)) || !qm::aligned(a.A, 4) || !qm::aligned(a.D, 4) ||
        !qm::aligned(a.dt_bias, 4) || !qm::aligned(a.seq_starts, 4))
        return QSTATE_EINVAL;
    if (!a.seq_starts && a.sequences && a.tokens % a.sequences) return QSTATE_EINVAL;
    if ((a.flags & QMIXER_INITIAL) && !a.state && a.sequences) return QSTATE_EINVAL;
    if (rc != QSTATE_OK) return rc;
    if (!a.sequences || (!a.tokens && !a.state)) return QSTATE_OK;
    if (!a.A || (a.tokens && (!a.x || !a.dt || !a.B || !a.C || !a.y))) return QSTATE_EINVAL;
    const qm::ScanPlan plan = qm::scan_plan(a.sequences, a.tokens, a.heads, a.d_k, a.d_v, a.dtype, a.seq_starts != nullptr, qm::sm_count());
    if (plan.bytes && (!a.workspace || a.workspace_bytes < plan.bytes)) return QSTATE_EINVAL;
    if (plan.segments > INT32_MAX) return QSTATE_EUNSUPPORTED;
    qm::ScanParams p{a.x, a.x_stride, a.dt, a.dt_stride, a.A, a.B, a.B_stride, a.C, a.C_stride, a.D, a.dt_bias, a.state, a.y, a.y_stride,
                     {a.seq_starts, a.sequences, a.tokens, a.tokens / a.sequences}, a.heads, a.heads / a.groups, a.d_v,
                     a.dt_dtype == QSTATE_BF16, (a.flags & QMIXER_SOFTPLUS) != 0, (a.flags & QMIXER_INITIAL) != 0,
                     plan.seg_len, plan.segments, plan.cut, static_cast<float*>(a.workspace),
                     plan.cut ? reinterpret_cast<float*>(static_cast<char*>(a.workspace) + plan.state_bytes) : nullptr,
                     qm::wait_polls.load(std::memory_order_relaxed), qm::drop_from.load(std::memory_order_relaxed)};
    const cudaStream_t st = (cudaStream_t)stream;
    // (without tokens only states are set: any form does)
    const bool chunked = a.dtype == QSTATE_BF16 && a.tokens > 0;
    auto launch = [&](bool states_only) {
        return chunked ? qm::launch_scan_chunk(p, a.d_k, plan.segments, states_only, st)
                       : qm::launch_scan_rec(p, a.d_k, plan.segments, states_only, st);
    };
    if (plan.cut) {
        if (!launch(true)) return QSTATE_ECUDA;
        const dim3 grid((unsigned)a.sequences, (unsigned)a.heads, (unsigned)(a.d_k * a.d_v / 1024));
        qm::join_kernel<<<grid, 256, 0, st>>>(p, a.d_k);
    }
    if (!launch(false)) return QSTATE_ECUDA;
    return qm::launched();
}

}  // extern "C"
