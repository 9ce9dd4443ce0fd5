// qmixer_norm.cu -- root-mean-square norm of a row, y = h / sqrt(mean(h^2) +
// eps) * weight, with h = x + residual or x silu(gate) formed on the way in and
// y rounded once on the way out: to the inputs' type, or to 8-bit codes with a
// binary32 scale per row or per group of columns.
//
// Bound: memory (x and the second operand read once, y written once).  A warp, 128
// or 512 threads hold one row in registers between the sum of squares and the
// output, so nothing is read twice; each thread takes eight consecutive columns at a
// time, all loads of a row in flight together.  The groups of the 8-bit scales are
// powers of two of at most 256 columns: 32 lanes or fewer of one warp, joined by
// shuffles.  Measured on 16384 rows of 2048 bfloat16: residual, output in type 42 us
// (6.3 TB/s, 97% of the copy rate); gate to e4m3 in groups of 128 43 us (3.9 TB/s) and
// int8 of whole rows 27.5 us (3.7 TB/s): what a code costs beside its bytes, 2.5 and
// 0.3 us of it for the quotients' correct rounding.
#include "qmixer_common.cuh"

namespace qm {

struct NormParams {
    const void* x;
    int64_t xs;
    void* other;
    int64_t os;
    const void* w;
    void* y;
    int64_t ys;
    float* scales;
    int64_t rows;
    int columns, group;
    float eps, per_column;      // per_column = 1 / columns
    int before, out;
};


__device__ __forceinline__ void floats(const f2 (&h)[4], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = unpair(h[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// Eight elements as they lie in memory: all of a row's loads are issued before
// the first is converted.
template <class T, bool VEC> struct Eight;
template <> struct Eight<bf16, true> {
    uint4 r;
    __device__ __forceinline__ void load(const bf16* p, int) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(f2 (&v)[4]) const {
        v[0] = bf_pair(r.x); v[1] = bf_pair(r.y); v[2] = bf_pair(r.z); v[3] = bf_pair(r.w);
    }
};
template <> struct Eight<float, true> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p, int) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void get(f2 (&v)[4]) const {
        v[0] = pair(a.x, a.y); v[1] = pair(a.z, a.w); v[2] = pair(b.x, b.y); v[3] = pair(b.z, b.w);
    }
};
template <class T> struct Eight<T, false> {
    float f[8];
    __device__ __forceinline__ void load(const T* p, int left) {
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = i < left ? to_f32<T>(p[i]) : 0.0f;
    }
    __device__ __forceinline__ void get(f2 (&v)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = pair(f[2 * i], f[2 * i + 1]);
    }
};

template <class T, bool VEC>
__device__ __forceinline__ void put8(T* p, int left, const f2 (&h)[4]) {
    float v[8];
    floats(h, v);
    if constexpr (VEC) {
        store8(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < left) p[i] = from_f32<T>(v[i]);
    }
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The largest magnitude of eight, as bits.
__device__ __forceinline__ uint32_t largest(const f2 (&h)[4]) {
    float v[8];
    floats(h, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// The scale of a group from its largest magnitude (as bits: an integer maximum
// keeps a NaN) and the codes of eight of its values.  scale = most / Qmax and the
// quotient y / scale are the correctly rounded ones: a product with the rounded
// reciprocal, then one correction by the exact remainder (Markstein's scheme).
struct Codes {
    float scale, inv;
    bool odd;            // not a number, zero, or so small that a remainder may not be exact
    // `unit`: RN(1 / qmax)
    __device__ __forceinline__ Codes(uint32_t most, float qmax, float unit) {
        const float m = __uint_as_float(most), q = m * unit;
        scale = most >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : fmaf(fmaf(-q, qmax, m), unit, q);
        odd = !(scale >= 0x1p-80f);
        if (odd && most < 0x7f800000u) scale = __fdiv_rn(m, qmax);
        const float near = rcp_approx(scale);
        inv = fmaf(fmaf(-scale, near, 1.0f), near, near);        // one step of Newton's
    }
    __device__ __forceinline__ void divide(const f2 (&y)[4], f2 (&z)[4]) const {
        const f2 by = pair(inv, inv), less = pair(-scale, -scale);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const f2 q = mul2(y[i], by);
            z[i] = fma2(fma2(q, less, y[i]), by, q);
        }
        if (odd) {
            // (a scale below the normal numbers is far off its quotient: clamped)
            float v[8];
            floats(y, v);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = scale > 0.0f ? fminf(fmaxf(__fdiv_rn(v[i], scale), -448.0f), 448.0f) : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; i++) z[i] = pair(v[2 * i], v[2 * i + 1]);
        }
    }
    __device__ __forceinline__ uint2 int8(const f2 (&y)[4]) const {
        f2 z[4];
        float f[8];
        uint32_t c[8];
        divide(y, z);
        // 1.5 * 2^23: rounds half to even.  (No quotient rounds beyond 127 but an odd
        // one's, which is clamped.)
#pragma unroll
        for (int i = 0; i < 4; i++) z[i] = add2(z[i], pair(12582912.0f, 12582912.0f));
        floats(z, f);
        if (odd)
#pragma unroll
            for (int i = 0; i < 8; i++) f[i] = fminf(fmaxf(f[i], 12582785.0f), 12583039.0f);
#pragma unroll
        for (int i = 0; i < 8; i++) c[i] = __float_as_uint(f[i]);
        return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x40), __byte_perm(c[2], c[3], 0x40), 0x5410),
                          __byte_perm(__byte_perm(c[4], c[5], 0x40), __byte_perm(c[6], c[7], 0x40), 0x5410));
    }
    __device__ __forceinline__ uint2 e4m3(const f2 (&y)[4]) const {
        f2 q[4];
        float z[8];
        divide(y, q);
        floats(q, z);
        return make_uint2(e4m3x2(z[0], z[1]) | e4m3x2(z[2], z[3]) << 16, e4m3x2(z[4], z[5]) | e4m3x2(z[6], z[7]) << 16);
    }
};

template <class T, bool VEC, int BEFORE, int THREADS, int N>
__global__ void __launch_bounds__(THREADS < 128 ? 128 : THREADS, THREADS == 128 && N <= 2 ? 12 : 1) norm_kernel(const NormParams p) {
    constexpr int kBlock = THREADS < 128 ? 128 : THREADS;
    constexpr int kWarps = THREADS / 32;
    __shared__ float sums[kWarps];
    __shared__ uint32_t tops[kWarps];
    const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = THREADS == 32 ? blockIdx.x * (int64_t)(kBlock / 32) + threadIdx.x / 32 : blockIdx.x;
    if (row >= p.rows) return;                   // THREADS > 32: one row per block, never taken
    const T* const x = static_cast<const T*>(p.x) + row * p.xs;
    T* const other = static_cast<T*>(p.other) + row * p.os;
    const T* const w = static_cast<const T*>(p.w);

    f2 h[N][4];
    {
        Eight<T, VEC> xr[N], orow[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int c = (i * THREADS + tid) * 8, left = p.columns - c;
            if (left > 0) {
                xr[i].load(x + c, left);
                if (BEFORE != QMIXER_BEFORE_NONE) orow[i].load(other + c, left);
            }
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int c = (i * THREADS + tid) * 8, left = p.columns - c;
#pragma unroll
            for (int j = 0; j < 4; j++) h[i][j] = 0;
            if (left <= 0) continue;
            xr[i].get(h[i]);
            if constexpr (BEFORE != QMIXER_BEFORE_NONE) {
                f2 o[4];
                orow[i].get(o);
#pragma unroll
                for (int j = 0; j < 4; j++)
                    h[i][j] = BEFORE == QMIXER_BEFORE_RESIDUAL ? add2(h[i][j], o[j]) : mul2(h[i][j], silu2<T>(o[j]));
                if (BEFORE == QMIXER_BEFORE_RESIDUAL) put8<T, VEC>(other + c, left, h[i]);
            }
        }
    }
    f2 squares = 0;
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) squares = fma2(h[i][j], h[i][j], squares);
    float sum = unpair(squares).x + unpair(squares).y;
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
    if constexpr (THREADS > 32) {
        if ((tid & 31) == 0) sums[tid / 32] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; i++) sum += sums[i];
    }
    const float r = rsqrtf(fmaf(sum, p.per_column, p.eps));         // 2 units of binary32
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int c = (i * THREADS + tid) * 8, left = p.columns - c;
        if (left <= 0) continue;
        f2 g[4];
        Eight<T, VEC> wr;
        wr.load(w + c, left);
        wr.get(g);
#pragma unroll
        for (int j = 0; j < 4; j++) h[i][j] = mul2(mul2(h[i][j], pair(r, r)), g[j]);
        if (p.out != QMIXER_OUT_SAME && !p.group) most = max(most, largest(h[i]));
    }
    if (p.out == QMIXER_OUT_SAME) {
        T* const y = static_cast<T*>(p.y) + row * p.ys;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int c = (i * THREADS + tid) * 8, left = p.columns - c;
            if (left > 0) put8<T, VEC>(y + c, left, h[i]);
        }
        return;
    }
    uint8_t* const y = static_cast<uint8_t*>(p.y) + row * p.ys;
    const float qmax = p.out == QMIXER_OUT_INT8 ? 127.0f : 448.0f;
    const float unit = p.out == QMIXER_OUT_INT8 ? 1.0f / 127.0f : 1.0f / 448.0f;
    if (!p.group) {
        most = __reduce_max_sync(~0u, most);
        if constexpr (THREADS > 32) {
            if ((tid & 31) == 0) tops[tid / 32] = most;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kWarps; i++) most = max(most, tops[i]);
        }
    }
    const int lanes = p.group >> 3, ngroups = p.group ? p.columns / p.group : 1;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int c = (i * THREADS + tid) * 8, left = p.columns - c;
        uint32_t m = most;
        if (p.group) {
            m = left > 0 ? largest(h[i]) : 0;
            for (int d = 1; d < lanes; d <<= 1) m = max(m, __shfl_xor_sync(~0u, m, d));
        }
        if (left <= 0) continue;
        const Codes q(m, qmax, unit);
        if (p.group ? (c & (p.group - 1)) == 0 : c == 0)
            p.scales[row * ngroups + (p.group ? c / p.group : 0)] = q.scale;
        const uint2 b = p.out == QMIXER_OUT_INT8 ? q.int8(h[i]) : q.e4m3(h[i]);
        if constexpr (VEC) {
            *reinterpret_cast<uint2*>(y + c) = b;
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (j < left) y[c + j] = (uint8_t)((j < 4 ? b.x : b.y) >> (j % 4 * 8));
        }
    }
}

template <class T, bool VEC, int BEFORE, int THREADS, int N> void launch_norm(const NormParams& p, cudaStream_t st) {
    constexpr int kBlock = THREADS < 128 ? 128 : THREADS;
    const int64_t per = kBlock / THREADS;
    norm_kernel<T, VEC, BEFORE, THREADS, N><<<(unsigned)((p.rows + per - 1) / per), kBlock, 0, st>>>(p);
}

// Up to 1024 columns in a warp of its own where there are rows enough to fill the
// SMs, else 128 threads a row (2048 columns in a warp took 84 us where 128 threads
// take 45); beyond 4096 columns 512.
template <class T, bool VEC, int BEFORE> void by_columns(const NormParams& p, cudaStream_t st) {
    const int v = (p.columns + 7) / 8;
    const bool few = p.rows < 148 * 8;
    if (v <= 32) launch_norm<T, VEC, BEFORE, 32, 1>(p, st);
    else if (!few && v <= 64) launch_norm<T, VEC, BEFORE, 32, 2>(p, st);
    else if (!few && v <= 128) launch_norm<T, VEC, BEFORE, 32, 4>(p, st);
    else if (v <= 128) launch_norm<T, VEC, BEFORE, 128, 1>(p, st);
    else if (v <= 256) launch_norm<T, VEC, BEFORE, 128, 2>(p, st);
    else if (v <= 512) launch_norm<T, VEC, BEFORE, 128, 4>(p, st);
    else if (v <= 1024) launch_norm<T, VEC, BEFORE, 512, 2>(p, st);
    else if (v <= 2048) launch_norm<T, VEC, BEFORE, 512, 4>(p, st);
    else launch_norm<T, VEC, BEFORE, 512, 8>(p, st);
}

template <class T, bool VEC> void dispatch_norm(const NormParams& p, cudaStream_t st) {
    if (p.before == QMIXER_BEFORE_NONE) by_columns<T, VEC, QMIXER_BEFORE_NONE>(p, st);
    else if (p.before == QMIXER_BEFORE_RESIDUAL) by_columns<T, VEC, QMIXER_BEFORE_RESIDUAL>(p, st);
    else by_columns<T, VEC, QMIXER_BEFORE_GATE>(p, st);
}

}  // namespace qm

extern "C" int qmixer_norm(const qmixer_norm_args* args, qstate_stream stream) {
    if (!args) return QSTATE_EINVAL;
    const qmixer_norm_args& a = *args;
    if (!qm::known(a.dtype) || a.rows < 0 || a.columns < 1 || a.group < 0 || !(a.eps >= 0.0f) || a.eps > 3.4e38f)
        return QSTATE_EINVAL;
    if (a.before < QMIXER_BEFORE_NONE || a.before > QMIXER_BEFORE_GATE || a.out < QMIXER_OUT_SAME || a.out > QMIXER_OUT_E4M3)
        return QSTATE_EINVAL;
    if (a.x_stride < a.columns || a.y_stride < a.columns || (a.before && a.other_stride < a.columns)) return QSTATE_EINVAL;
    if (a.group && (a.out == QMIXER_OUT_SAME || a.columns % a.group)) return QSTATE_EINVAL;
    const int size = qm::size_of(a.dtype), ysize = a.out == QMIXER_OUT_SAME ? size : 1;
    if (!qm::aligned(a.x, size) || !qm::aligned(a.other, size) || !qm::aligned(a.weight, size) || !qm::aligned(a.y, ysize) ||
        !qm::aligned(a.scales, 4))
        return QSTATE_EINVAL;
    if (a.columns > 32768 || a.rows > INT32_MAX) return QSTATE_EUNSUPPORTED;
    if (a.group && (a.group < 8 || a.group > 256 || (a.group & (a.group - 1)))) return QSTATE_EUNSUPPORTED;
    if (!a.rows) return QSTATE_OK;
    if (!a.x || !a.weight || !a.y || (a.before && !a.other) || (a.out && !a.scales)) return QSTATE_EINVAL;
    const qm::NormParams p{a.x, a.x_stride, a.other, a.other_stride, a.weight, a.y, a.y_stride, a.scales,
                           a.rows, a.columns, a.group, a.eps, 1.0f / (float)a.columns, a.before, a.out};
    // eight a.columns at a time where a.columns, strides and bases allow 16-byte
    // accesses (8-byte ones of codes); else element by element
    const int unit = 16 / size;
    const bool vec = a.columns % 8 == 0 && a.x_stride % unit == 0 && qm::aligned(a.x, 16) && qm::aligned(a.weight, 16) &&
                     (!a.before || (a.other_stride % unit == 0 && qm::aligned(a.other, 16))) &&
                     (a.out ? a.y_stride % 8 == 0 && qm::aligned(a.y, 8) : a.y_stride % unit == 0 && qm::aligned(a.y, 16));
    const cudaStream_t st = (cudaStream_t)stream;
    if (a.dtype == QSTATE_BF16) {
        if (vec) qm::dispatch_norm<qm::bf16, true>(p, st);
        else qm::dispatch_norm<qm::bf16, false>(p, st);
    } else {
        if (vec) qm::dispatch_norm<float, true>(p, st);
        else qm::dispatch_norm<float, false>(p, st);
    }
    return qm::launched();
}
