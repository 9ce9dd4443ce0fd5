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

// Cut or not, by an estimate in tokens of one CTA's chain.  Uncut: the longest
// chain, taken as up to four times the mean where the lengths are not known
// here, or the whole work over the resident CTAs.  Cut: the work with launch 1
// on top.
ScanPlan scan_plan(int sequences, int64_t tokens, int heads, int dk, int dv, bool ragged, int sms) {
    const int64_t unit = kBatchTokens;
    const int64_t chains = (int64_t)heads * (dv / 64), resident = 2 * sms;
    const int64_t mean = tokens / sequences, longest = ragged ? (4 * mean < tokens ? 4 * mean : tokens) : mean;
    const int64_t even = tokens * chains / resident;
    ScanPlan o{};
    o.seg_len = tokens > 0 ? tokens : 1;
    int64_t len = (even + unit - 1) / unit * unit;
    if (len < 2 * unit) len = 2 * unit;
    if (16 * len + 8 * unit < 10 * longest) {        // 1.6 times the work, two launches
        o.cut = true;
        o.seg_len = len;
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
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128) || heads * (dv / 64) > 65535) return QSTATE_EUNSUPPORTED;
    return QSTATE_OK;
}

}  // namespace qm

extern "C" {

int64_t qmixer_scan_workspace(int32_t sequences, int64_t tokens, int32_t heads, int32_t groups, int32_t d_k,
                              int32_t d_v, int32_t dtype) {
    const int rc = qm::check_scan(sequences, tokens, heads, groups, d_k, d_v, dtype);
    if (rc != QSTATE_OK) return rc;
    if (!sequences) return 0;
    const int sms = qm::sm_count();
    const int64_t a = qm::scan_plan(sequences, tokens, heads, d_k, d_v, true, sms).bytes;
    const int64_t b = qm::scan_plan(sequences, tokens, heads, d_k, d_v, false, sms).bytes;
    return a > b ? a : b;
}

int qmixer_scan(const void* x, int64_t x_stride, const void* dt, int64_t dt_stride, const float* A, const void* B,
                int64_t B_stride, const void* C, int64_t C_stride, const float* D, const float* dt_bias,
                float* state, void* y, int64_t y_stride, const int32_t* seq_starts, int32_t sequences,
                int64_t tokens, int32_t heads, int32_t groups, int32_t d_k, int32_t d_v, int32_t dtype,
                int32_t dt_dtype, int32_t flags, void* workspace, int64_t workspace_bytes, qstate_stream stream) {
    const int rc = qm::check_scan(sequences, tokens, heads, groups, d_k, d_v, dtype);
    if (rc == QSTATE_EINVAL) return rc;
    if (!qm::known(dt_dtype) || (flags & ~(QMIXER_INITIAL | QMIXER_SOFTPLUS))) return QSTATE_EINVAL;
    if (x_stride < (int64_t)heads * d_v || y_stride < (int64_t)heads * d_v || dt_stride < heads ||
        B_stride < (int64_t)groups * d_k || C_stride < (int64_t)groups * d_k)
        return QSTATE_EINVAL;
    const int size = qm::size_of(dtype), unit = 16 / size;
    if (x_stride % unit || B_stride % unit || C_stride % unit || !qm::aligned(x, 16) || !qm::aligned(B, 16) ||
        !qm::aligned(C, 16) || !qm::aligned(state, 16) || !qm::aligned(workspace, 16) || !qm::aligned(y, size) ||
        !qm::aligned(dt, qm::size_of(dt_dtype)) || !qm::aligned(A, 4) || !qm::aligned(D, 4) ||
        !qm::aligned(dt_bias, 4) || !qm::aligned(seq_starts, 4))
        return QSTATE_EINVAL;
    if (!seq_starts && sequences && tokens % sequences) return QSTATE_EINVAL;
    if ((flags & QMIXER_INITIAL) && !state && sequences) return QSTATE_EINVAL;
    if (rc != QSTATE_OK) return rc;
    if (!sequences || (!tokens && !state)) return QSTATE_OK;
    if (!A || (tokens && (!x || !dt || !B || !C || !y))) return QSTATE_EINVAL;
    const qm::ScanPlan plan = qm::scan_plan(sequences, tokens, heads, d_k, d_v, seq_starts != nullptr, qm::sm_count());
    if (plan.bytes && (!workspace || workspace_bytes < plan.bytes)) return QSTATE_EINVAL;
    if (plan.segments > INT32_MAX) return QSTATE_EUNSUPPORTED;
    qm::ScanParams p{x, x_stride, dt, dt_stride, A, B, B_stride, C, C_stride, D, dt_bias, state, y, y_stride,
                     {seq_starts, sequences, tokens, tokens / sequences}, heads, heads / groups, d_v,
                     dt_dtype == QSTATE_BF16, (flags & QMIXER_SOFTPLUS) != 0, (flags & QMIXER_INITIAL) != 0,
                     plan.seg_len, plan.segments, plan.cut, static_cast<float*>(workspace),
                     plan.cut ? reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.state_bytes) : nullptr};
    const cudaStream_t st = (cudaStream_t)stream;
    if (plan.cut) {
        qm::launch_scan_rec(p, dtype, d_k, plan.segments, true, st);
        const dim3 grid((unsigned)sequences, (unsigned)heads, (unsigned)(d_k * d_v / 1024));
        qm::join_kernel<<<grid, 256, 0, st>>>(p, d_k);
    }
    qm::launch_scan_rec(p, dtype, d_k, plan.segments, false, st);
    return qm::launched();
}

}  // extern "C"
