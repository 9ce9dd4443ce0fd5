// qmixer_scan_rec.cu -- the prompt scan of binary32 inputs, token by token, in
// binary32 throughout:
// S <- a S + (dt x) B^T, y = S^T C + D x.
//
// A CTA takes 64 value columns of one head over one segment, with the state in
// registers: a thread holds 8 rows x 4 columns as pairs of rows, so that B and C
// come from shared memory as the pairs that the packed binary32 instructions take
// (sm_100 issues two operations of a pair at once).  Inside a batch of kBatch tokens
// the state is kept divided by c_t, the product of the batch's decays up to t:
//   S_t / c_t = S_{t-1} / c_{t-1} + (dt x / c_t) B^T,  y = c_t (S_t / c_t)^T C + D x
// which spares the decay's multiplication of every element (a third of the
// instructions).  It must not cost range: what is divided by c may not overflow where
// the plain form would not.  So it holds while c_t >= 2^-40, decays are at most 1 and
// finite inputs are moderate: |x|, |B|, |C| < 2^13, |dt| < 2^7, the state in front of the
// segment below 2^64.  A token then adds less than 2^33 to an element, the fewer than
// 2^31 tokens of a sequence less than 2^64, and the largest value that is formed, a sum
// of y over 128 rows, stays below 2^13 2^65 2^7 2^40 = 2^125.  From the first token on
// whose c leaves its range the batch takes the plain form, from the first that breaks
// another of these bounds on all of the segment: whatever a later token holds, an
// earlier one is computed alike.
//
// A token then costs 32 packed instructions and five 16-byte shared loads a thread.
// kBatch tokens are staged at a time while the next ones are on their way to registers.
// The 8 or 16 threads of a column leave their parts of y in shared memory, where they
// are added once per batch (shuffles within the token took a fifth of the instructions
// and most of the waiting).  Eight sequences of 1024 tokens, 32 heads of 128 x 64, take
// 344 us (367 with the decay in every token, 333 without the range's checks).  No pipe
// bounds it: the multipliers are busy for 49% of the time and 43% of the issue slots are
// used; 13 of 64 warps are there, which wait for shared loads, the two barriers of a
// batch and one another's results, a warp 1.8, 1.5 and 1.4 times as long as it issues.
#include <type_traits>

#include "qmixer_scan.cuh"

namespace qm {

constexpr int kBatch = kBatchTokens;
constexpr float kLeast = 0x1p-40f, kMostInput = 0x1p13f, kMostStep = 0x1p7f, kMostState = 0x1p64f;

// Whether a finite one of eight values reaches `limit`.  (Infinities and NaN are the
// same in either form, and leave the rest of their token as it is.)
__device__ __forceinline__ bool large(const float (&v)[8], float limit) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(v[j]));
    if (m < limit) return false;
    bool any = false;
#pragma unroll
    for (int j = 0; j < 8; j++) any |= fabsf(v[j]) >= limit && fabsf(v[j]) < INFINITY;
    return any;
}

template <int N, bool OUT> struct RecSmem {
    static constexpr int kOut = OUT ? kBatch : 1;
    // all but the last are read 16 bytes at a time
    alignas(16) float k[2][kBatch][N];
    alignas(16) float x[2][kBatch][64];
    alignas(16) float q[2][kOut][N];
    alignas(16) float part[kOut][N / 8][68];     // a row of 64 shifted by four banks against the next
    alignas(16) float2 ad[2][kBatch];            // decay and time step
    alignas(16) float2 cd[2][kBatch];            // product of the batch's decays, time step / it
    int scaled[2];               // so many leading tokens in the scaled form, as far as c goes
    int plain;                   // the segment's first token from which on no form but the plain one will do
};

template <int N, bool OUT>
__global__ void __launch_bounds__(N * 2, N == 128 ? 2 : 3) rec_kernel(const ScanParams p) {
    constexpr int kThreads = N * 2, kL = N / 8;      // threads of one column group
    extern __shared__ __align__(16) unsigned char raw[];
    RecSmem<N, OUT>& sm = *reinterpret_cast<RecSmem<N, OUT>*>(raw);
    const int tid = threadIdx.x;
    Segment seg;
    if (!find_segment(p, blockIdx.x, seg)) return;
    if (!OUT && seg.last) return;
    const int parts = p.dv / 64, h = blockIdx.y / parts, c0 = blockIdx.y % parts * 64;
    const int g = h / p.per_group, r4 = tid % kL * 4, pg = tid / kL * 4;
    const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f, D = OUT && p.D ? p.D[h] : 0.0f;

    if (tid == 0) sm.plain = INT32_MAX;
    __syncthreads();
    // rows r4 .. r4+3 and N/2 + r4 .. : four pairs of rows, four columns
    f2 S[4][4];
    const float* from = nullptr;
    if (OUT && p.cut) from = p.seg_state + ((int64_t)blockIdx.x * p.heads + h) * N * p.dv;
    else if (OUT && p.initial) from = p.state + ((int64_t)seg.sequence * p.heads + h) * N * p.dv;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = (i / 2) * (N / 2) + r4 + i % 2 * 2;
        float4 lo = make_float4(0, 0, 0, 0), hi = lo;
        if (from) {
            lo = *reinterpret_cast<const float4*>(from + (int64_t)r * p.dv + c0 + pg);
            hi = *reinterpret_cast<const float4*>(from + (int64_t)(r + 1) * p.dv + c0 + pg);
        }
        S[i][0] = pair(lo.x, hi.x);
        S[i][1] = pair(lo.y, hi.y);
        S[i][2] = pair(lo.z, hi.z);
        S[i][3] = pair(lo.w, hi.w);
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        if (large(v, kMostState)) atomicMin(&sm.plain, 0);
    }

    // staging: thread t brings eight elements of k and q (row t / (N/8)) and,
    // below 128, of x (row t / 8); below kBatch a token's decay
    const int kr = tid / (N / 8), kc = tid % (N / 8) * 8, xr = tid / 8, xc = tid % 8 * 8;
    float nk[8], nq[8], nx[8], na = 1.0f, nd = 0.0f;
    auto fetch = [&](int64_t t0) {
#pragma unroll
        for (int j = 0; j < 8; j++) nk[j] = nq[j] = nx[j] = 0.0f;
        na = 1.0f;
        nd = 0.0f;
        if (t0 + kr < seg.to) {
            load8(static_cast<const float*>(p.B) + (t0 + kr) * p.Bs + (int64_t)g * N + kc, nk);
            if (OUT) load8(static_cast<const float*>(p.C) + (t0 + kr) * p.Cs + (int64_t)g * N + kc, nq);
        }
        if (tid < 128 && t0 + xr < seg.to)
            load8(static_cast<const float*>(p.x) + (t0 + xr) * p.xs + (int64_t)h * p.dv + c0 + xc, nx);
        if (tid < kBatch && t0 + tid < seg.to) {
            nd = time_step(load_dt(p.dt, (t0 + tid) * p.dts + h, p.dt_bf16), bias, p.softplus);
            na = expf(nd * A);
        }
    };
    // the batch that starts at token t0 of the segment
    auto stage = [&](int b, int t0) {
        if (large(nk, kMostInput) || (OUT && large(nq, kMostInput))) atomicMin(&sm.plain, t0 + kr);
        if (large(nx, kMostInput)) atomicMin(&sm.plain, t0 + xr);
        store8(&sm.k[b][kr][kc], nk);
        if (OUT) store8(&sm.q[b][kr][kc], nq);
        if (tid < 128) store8(&sm.x[b][xr][xc], nx);
        if (tid < 32) {
            // c_t, the product of the batch's decays up to token t
            float c = na;
#pragma unroll
            for (int d = 1; d < kBatch; d <<= 1) {
                const float u = __shfl_up_sync(~0u, c, d);
                if (tid >= d) c *= u;
            }
            const int first = __ffs(__ballot_sync(~0u, !(c >= kLeast) || tid >= kBatch)) - 1;
            if (!(na <= 1.0f && fabsf(nd) < kMostStep)) atomicMin(&sm.plain, t0 + tid);
            if (tid < kBatch) {
                sm.ad[b][tid] = make_float2(na, nd);
                sm.cd[b][tid] = make_float2(c, __fdiv_rn(nd, c));
            }
            if (tid == 0) sm.scaled[b] = first;
        }
    };

    float total = 1.0f;
    int b = 0;
    fetch(seg.from);
    stage(0, 0);
    __syncthreads();
    for (int64_t t0 = seg.from; t0 < seg.to; t0 += kBatch, b ^= 1) {
        fetch(t0 + kBatch);
        const int n = seg.to - t0 < kBatch ? (int)(seg.to - t0) : kBatch;
        const int at = (int)(t0 - seg.from);
        int scaled = sm.scaled[b] < n ? sm.scaled[b] : n;
        // (what a thread already ahead finds in the next batch changes nothing here)
        const int plain = *const_cast<volatile int*>(&sm.plain) - at;
        if (plain < scaled) scaled = plain > 0 ? plain : 0;
        auto token = [&](int t, auto scaled_form) {
            constexpr bool kScaled = decltype(scaled_form)::value;
            const float2 ad = kScaled ? sm.cd[b][t] : sm.ad[b][t];
            const float4 xv = *reinterpret_cast<const float4*>(&sm.x[b][t][pg]);
            const ulonglong2 k0 = *reinterpret_cast<const ulonglong2*>(&sm.k[b][t][r4]);
            const ulonglong2 k1 = *reinterpret_cast<const ulonglong2*>(&sm.k[b][t][N / 2 + r4]);
            const f2 k[4] = {k0.x, k0.y, k1.x, k1.y};
            const f2 a = pair(ad.x, ad.x);
            const f2 v[4] = {pair(xv.x * ad.y, xv.x * ad.y), pair(xv.y * ad.y, xv.y * ad.y),
                             pair(xv.z * ad.y, xv.z * ad.y), pair(xv.w * ad.y, xv.w * ad.y)};
            if (!OUT && !kScaled) total *= ad.x;
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) S[i][j] = fma2(k[i], v[j], kScaled ? S[i][j] : mul2(S[i][j], a));
            if constexpr (OUT) {
                const ulonglong2 q0 = *reinterpret_cast<const ulonglong2*>(&sm.q[b][t][r4]);
                const ulonglong2 q1 = *reinterpret_cast<const ulonglong2*>(&sm.q[b][t][N / 2 + r4]);
                const f2 q[4] = {q0.x, q0.y, q1.x, q1.y};
                float o[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    f2 s = mul2(q[0], S[0][j]);
#pragma unroll
                    for (int i = 1; i < 4; i++) s = fma2(q[i], S[i][j], s);
                    const float2 u = unpair(s);
                    o[j] = u.x + u.y;
                }
                *reinterpret_cast<float4*>(&sm.part[t][tid % kL][pg]) = make_float4(o[0], o[1], o[2], o[3]);
            }
        };
#pragma unroll 4
        for (int t = 0; t < scaled; t++) token(t, std::true_type{});
        if (scaled) {
            const float c = sm.cd[b][scaled - 1].x;
            if (!OUT) total *= c;
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) S[i][j] = mul2(S[i][j], pair(c, c));
        }
#pragma unroll 2
        for (int t = scaled; t < n; t++) token(t, std::false_type{});
        stage(b ^ 1, at + kBatch);
        __syncthreads();
        if constexpr (OUT) {
            // token and four columns a thread, in 256 / kThreads rounds
#pragma unroll
            for (int e = 0; e < 256 / kThreads; e++) {
                const int t = (e * kThreads + tid) / 16, c = tid % 16 * 4;
                if (t >= n) continue;
                const float4 x4 = *reinterpret_cast<const float4*>(&sm.x[b][t][c]);
                float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int l = 0; l < kL; l++) {
                    const float4 v = *reinterpret_cast<const float4*>(&sm.part[t][l][c]);
                    u.x += v.x;
                    u.y += v.y;
                    u.z += v.z;
                    u.w += v.w;
                }
                const float c1 = t < scaled ? sm.cd[b][t].x : 1.0f;
                u.x = fmaf(D, x4.x, u.x * c1);
                u.y = fmaf(D, x4.y, u.y * c1);
                u.z = fmaf(D, x4.z, u.z * c1);
                u.w = fmaf(D, x4.w, u.w * c1);
                float* const y = static_cast<float*>(p.y) + (t0 + t) * p.ys + (int64_t)h * p.dv + c0 + c;
                if ((reinterpret_cast<uintptr_t>(y) & 15) == 0) {
                    *reinterpret_cast<float4*>(y) = u;
                } else {
                    y[0] = u.x;
                    y[1] = u.y;
                    y[2] = u.z;
                    y[3] = u.w;
                }
            }
            __syncthreads();             // parts and x have been read
        }
    }
    float* to = nullptr;
    if (!OUT) to = p.seg_state + ((int64_t)blockIdx.x * p.heads + h) * N * p.dv;
    else if (seg.last && p.state) to = p.state + ((int64_t)seg.sequence * p.heads + h) * N * p.dv;
    if (to) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int r = (i / 2) * (N / 2) + r4 + i % 2 * 2;
            const float2 s0 = unpair(S[i][0]), s1 = unpair(S[i][1]), s2 = unpair(S[i][2]), s3 = unpair(S[i][3]);
            *reinterpret_cast<float4*>(to + (int64_t)r * p.dv + c0 + pg) = make_float4(s0.x, s1.x, s2.x, s3.x);
            *reinterpret_cast<float4*>(to + (int64_t)(r + 1) * p.dv + c0 + pg) = make_float4(s0.y, s1.y, s2.y, s3.y);
        }
    }
    if (!OUT && tid == 0 && c0 == 0) p.seg_decay[(int64_t)blockIdx.x * p.heads + h] = total;
}

template <int N, bool OUT>
bool launch_rec(const ScanParams& p, int64_t segments, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(reinterpret_cast<const void*>(rec_kernel<N, OUT>), sizeof(RecSmem<N, OUT>), done)) return false;
    const dim3 grid((unsigned)segments, (unsigned)(p.heads * (p.dv / 64)));
    rec_kernel<N, OUT><<<grid, N * 2, sizeof(RecSmem<N, OUT>), st>>>(p);
    return true;
}

template <int N>
bool launch_rec(const ScanParams& p, int64_t segments, bool states_only, cudaStream_t st) {
    return states_only ? launch_rec<N, false>(p, segments, st) : launch_rec<N, true>(p, segments, st);
}

bool launch_scan_rec(const ScanParams& p, int dk, int64_t segments, bool states_only, cudaStream_t st) {
    return dk == 64 ? launch_rec<64>(p, segments, states_only, st) : launch_rec<128>(p, segments, states_only, st);
}

}  // namespace qm
