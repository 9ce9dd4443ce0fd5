// qmixer_common.cuh -- what the mixer kernels share: typed loads and stores of
// eight elements, the gate functions, and where a CTA finds its sequence.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "qmixer.h"

namespace qm {

using bf16 = __nv_bfloat16;

template <class T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<bf16>(bf16 v) { return __bfloat162float(v); }

template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 from_f32<bf16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight consecutive elements on a 16-byte boundary.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf(v[0], v[1]), pack_bf(v[2], v[3]),
                                              pack_bf(v[4], v[5]), pack_bf(v[6], v[7]));
}

// Two binary32 in one register pair: sm_100 issues an operation on both at once,
// each half rounded as the scalar instruction rounds it.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 bf_pair(uint32_t u) { return pair(bf_lo(u), bf_hi(u)); }
__device__ __forceinline__ uint32_t pack_bf(f2 v) {
    const float2 f = unpair(v);
    return pack_bf(f.x, f.y);
}

__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// z / (1 + e^-z).  For bfloat16 results the hardware's exponential and reciprocal,
// off by a few units of binary32: far inside the rounding that follows (and the
// results that they flush to zero are below 2^-119).  Binary32 results take the
// full functions.
template <class T> __device__ __forceinline__ f2 silu2(f2 z) {
    if constexpr (sizeof(T) == 2) {
        const float2 t = unpair(mul2(z, pair(-1.44269504f, -1.44269504f)));
        const float2 d = unpair(add2(pair(ex2_approx(t.x), ex2_approx(t.y)), pair(1.0f, 1.0f)));
        return mul2(z, pair(rcp_approx(d.x), rcp_approx(d.y)));
    } else {
        const float2 v = unpair(z);
        return pair(__fdiv_rn(v.x, 1.0f + expf(-v.x)), __fdiv_rn(v.y, 1.0f + expf(-v.y)));
    }
}

// dt = softplus(z) = max(z, 0) + log(1 + e^-|z|): no overflow on either side.
__device__ __forceinline__ float time_step(float raw, float bias, bool softplus) {
    const float z = raw + bias;
    return softplus ? fmaxf(z, 0.0f) + log1pf(expf(-fabsf(z))) + (z != z ? z : 0.0f) : z;
}

__device__ __forceinline__ float load_dt(const void* dt, int64_t i, bool is_bf16) {
    return is_bf16 ? __bfloat162float(static_cast<const bf16*>(dt)[i]) : static_cast<const float*>(dt)[i];
}

// The first token of sequence i (i = sequences: the end), inside [0, tokens].
struct Sequences {
    const int32_t* starts;      // NULL: equal sequences
    int n;
    int64_t tokens;
    int64_t each;               // tokens / n, for equal sequences

    __device__ __forceinline__ int64_t start(int i) const {
        if (!starts) return each * i;
        const int64_t v = __ldg(starts + i);
        return v < 0 ? 0 : v > tokens ? tokens : v;
    }
};

// The last sequence that starts at or before token t (0 if none does).
__device__ __forceinline__ int sequence_at(const Sequences& q, int64_t t) {
    if (!q.starts) {
        if (q.each == 0) return q.n - 1;
        const uint32_t i = (uint32_t)t / (uint32_t)q.each;      // tokens are below 2^31
        return i < (uint32_t)q.n ? (int)i : q.n - 1;
    }
    int lo = 0, hi = q.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (q.start(mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool known(int32_t dtype) { return dtype == QSTATE_F32 || dtype == QSTATE_BF16; }
inline int size_of(int32_t dtype) { return dtype == QSTATE_BF16 ? 2 : 4; }
// Let a kernel take more dynamic shared memory than 48 KB, once per device.
// `done` is the kernel's own mask of devices.  (A failure leaves no error behind
// that the next call's launched() would take for its own.)
inline bool allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError(), false;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return cudaGetLastError(), false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}
inline int launched() { return cudaGetLastError() == cudaSuccess ? QSTATE_OK : QSTATE_ECUDA; }

}  // namespace qm
