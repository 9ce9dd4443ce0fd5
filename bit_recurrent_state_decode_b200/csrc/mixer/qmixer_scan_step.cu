// qmixer_scan_step.cu -- one token of each sequence: the selective step on
// binary32 states, and the operands and output of the same step on a low-bit
// state (qstate_step).
//
// The step reads and writes a state of d_k x d_v binary32 per head and does
// five operations an element: memory is its bound.  A CTA takes one (sequence,
// head) tile; a thread holds four neighbouring columns of kRows rows, all loaded
// before the first is used, so that an SM has its CTAs' whole tiles in flight.
// y = S^T C is summed over a thread's rows, over the warp's row groups by
// shuffles, and over the warps through shared memory.  2048 states of 128 x 64 take
// 22.8 us (5.9 TB/s, 90% of the copy rate); one sequence of two 64 x 64 states 2.5 us,
// the latency of its chain of loads.
#include "qmixer_common.cuh"

namespace qm {

struct StepParams {
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
    int heads, per_group;      // heads per group
    bool dt_bf16, softplus;
};

template <class T, int N, int P>
__global__ void __launch_bounds__(256) scan_step_kernel(const StepParams p) {
    constexpr int kCols = P / 4;                 // threads across a row
    constexpr int kStep = 256 / kCols;           // rows side by side
    constexpr int kRows = N / kStep;
    __shared__ float part[8][P];
    const int64_t b = blockIdx.x / p.heads;
    const int h = blockIdx.x % p.heads, g = h / p.per_group;
    const int col = threadIdx.x % kCols * 4, row = threadIdx.x / kCols;
    float* const S = p.state + (int64_t)blockIdx.x * (N * P) + row * P + col;
    float4 s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; i++) s[i] = __ldcs(reinterpret_cast<const float4*>(S + (int64_t)i * kStep * P));
    const T* const x = static_cast<const T*>(p.x) + b * p.xs + (int64_t)h * P;
    const T* const B = static_cast<const T*>(p.B) + b * p.Bs + (int64_t)g * N + row;
    const T* const C = static_cast<const T*>(p.C) + b * p.Cs + (int64_t)g * N + row;
    float k[kRows], q[kRows], xv[4];
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        k[i] = to_f32<T>(B[i * kStep]);
        q[i] = to_f32<T>(C[i * kStep]);
    }
#pragma unroll
    for (int j = 0; j < 4; j++) xv[j] = to_f32<T>(x[col + j]);
    const float dt = time_step(load_dt(p.dt, b * p.dts + h, p.dt_bf16), p.dt_bias ? p.dt_bias[h] : 0.0f, p.softplus);
    const float a = expf(dt * p.A[h]);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        const float kd = k[i] * dt;
        s[i].x = fmaf(kd, xv[0], s[i].x * a);
        s[i].y = fmaf(kd, xv[1], s[i].y * a);
        s[i].z = fmaf(kd, xv[2], s[i].z * a);
        s[i].w = fmaf(kd, xv[3], s[i].w * a);
        o.x = fmaf(q[i], s[i].x, o.x);
        o.y = fmaf(q[i], s[i].y, o.y);
        o.z = fmaf(q[i], s[i].z, o.z);
        o.w = fmaf(q[i], s[i].w, o.w);
        __stcs(reinterpret_cast<float4*>(S + (int64_t)i * kStep * P), s[i]);
    }
#pragma unroll
    for (int d = kCols; d < 32; d <<= 1) {
        o.x += __shfl_xor_sync(~0u, o.x, d);
        o.y += __shfl_xor_sync(~0u, o.y, d);
        o.z += __shfl_xor_sync(~0u, o.z, d);
        o.w += __shfl_xor_sync(~0u, o.w, d);
    }
    if ((threadIdx.x & 31) < kCols) *reinterpret_cast<float4*>(&part[threadIdx.x / 32][col]) = o;
    __syncthreads();
    if (threadIdx.x < P) {
        float v = p.D ? p.D[h] * to_f32<T>(x[threadIdx.x]) : 0.0f;
#pragma unroll
        for (int w = 0; w < 8; w++) v += part[w][threadIdx.x];
        static_cast<T*>(p.y)[b * p.ys + (int64_t)h * P + threadIdx.x] = from_f32<T>(v);
    }
}

template <class T> void launch_scan_step(const StepParams& p, int64_t tiles, int dk, int dv, cudaStream_t st) {
    const unsigned n = (unsigned)tiles;
    if (dk == 64 && dv == 64) scan_step_kernel<T, 64, 64><<<n, 256, 0, st>>>(p);
    else if (dk == 64) scan_step_kernel<T, 64, 128><<<n, 256, 0, st>>>(p);
    else if (dv == 64) scan_step_kernel<T, 128, 64><<<n, 256, 0, st>>>(p);
    else scan_step_kernel<T, 128, 128><<<n, 256, 0, st>>>(p);
}

// ------------------------------------------------- the low-bit state's operands
struct OperandParams {
    StepParams s;
    void *q, *k, *v, *gates;
    int64_t tiles;
    int dk, dv;
    bool out_bf16, gate_bf16;
};

__device__ __forceinline__ void put(void* p, int64_t i, float v, bool is_bf16) {
    if (is_bf16) static_cast<bf16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(p)[i] = v;
}

template <class T> __global__ void __launch_bounds__(128) operands_kernel(const OperandParams p) {
    const int64_t tile = blockIdx.x;
    const int64_t b = tile / p.s.heads;
    const int h = tile % p.s.heads, g = h / p.s.per_group, t = threadIdx.x;
    const float dt = time_step(load_dt(p.s.dt, b * p.s.dts + h, p.s.dt_bf16),
                               p.s.dt_bias ? p.s.dt_bias[h] : 0.0f, p.s.softplus);
    if (t < p.dk) {
        put(p.q, tile * p.dk + t, to_f32<T>(static_cast<const T*>(p.s.C)[b * p.s.Cs + (int64_t)g * p.dk + t]), p.out_bf16);
        put(p.k, tile * p.dk + t, to_f32<T>(static_cast<const T*>(p.s.B)[b * p.s.Bs + (int64_t)g * p.dk + t]), p.out_bf16);
    }
    if (t < p.dv)
        put(p.v, tile * p.dv + t, dt * to_f32<T>(static_cast<const T*>(p.s.x)[b * p.s.xs + (int64_t)h * p.dv + t]), p.out_bf16);
    if (t == 0) put(p.gates, tile, expf(dt * p.s.A[h]), p.gate_bf16);
}

template <class T>
__global__ void __launch_bounds__(256) output_kernel(const float* out, const T* x, int64_t xs, const float* D, T* y,
                                                     int64_t ys, int64_t n, int heads, int dv) {
    const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int64_t row = i / ((int64_t)heads * dv);
    const int c = int(i % ((int64_t)heads * dv));
    float v = out[i];
    if (D) v = fmaf(D[c / dv], to_f32<T>(x[row * xs + c]), v);
    y[row * ys + c] = from_f32<T>(v);
}

int check_step(const void* x, int64_t xs, const void* dt, int64_t dts, const float* A, const void* B, int64_t Bs,
               const void* C, int64_t Cs, int batch, int heads, int groups, int dk, int dv, int dtype, int dt_dtype,
               int flags) {
    if (!known(dtype) || !known(dt_dtype) || batch < 0 || heads < 1 || groups < 1 || heads % groups || dk < 1 || dv < 1)
        return QSTATE_EINVAL;
    if (flags & ~QMIXER_SOFTPLUS) return QSTATE_EINVAL;
    if (xs < (int64_t)heads * dv || dts < heads || Bs < (int64_t)groups * dk || Cs < (int64_t)groups * dk)
        return QSTATE_EINVAL;
    const int unit = 16 / size_of(dtype);
    if (xs % unit || Bs % unit || Cs % unit || !aligned(x, 16) || !aligned(B, 16) || !aligned(C, 16) ||
        !aligned(dt, size_of(dt_dtype)) || !aligned(A, 4))
        return QSTATE_EINVAL;
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128) || (int64_t)batch * heads > INT32_MAX)
        return QSTATE_EUNSUPPORTED;
    if (batch && (!x || !dt || !A || !B || !C)) return QSTATE_EINVAL;
    return QSTATE_OK;
}

}  // namespace qm

extern "C" {

int qmixer_scan_step(const qmixer_scan_step_args* args, qstate_stream stream) {
    if (!args) return QSTATE_EINVAL;
    const qmixer_scan_step_args& a = *args;
    const int rc = qm::check_step(a.x, a.x_stride, a.dt, a.dt_stride, a.A, a.B, a.B_stride, a.C, a.C_stride, a.batch, a.heads, a.groups, a.d_k,
                                  a.d_v, a.dtype, a.dt_dtype, a.flags);
    if (rc != QSTATE_OK) return rc;
    if (a.y_stride < (int64_t)a.heads * a.d_v || !qm::aligned(a.state, 16) || !qm::aligned(a.y, qm::size_of(a.dtype)) ||
        !qm::aligned(a.D, 4) || !qm::aligned(a.dt_bias, 4))
        return QSTATE_EINVAL;
    if (!a.batch) return QSTATE_OK;
    if (!a.state || !a.y) return QSTATE_EINVAL;
    const qm::StepParams p{a.x, a.x_stride, a.dt, a.dt_stride, a.A, a.B, a.B_stride, a.C, a.C_stride, a.D, a.dt_bias, a.state, a.y, a.y_stride,
                           a.heads, a.heads / a.groups, a.dt_dtype == QSTATE_BF16, (a.flags & QMIXER_SOFTPLUS) != 0};
    if (a.dtype == QSTATE_BF16) qm::launch_scan_step<qm::bf16>(p, (int64_t)a.batch * a.heads, a.d_k, a.d_v, (cudaStream_t)stream);
    else qm::launch_scan_step<float>(p, (int64_t)a.batch * a.heads, a.d_k, a.d_v, (cudaStream_t)stream);
    return qm::launched();
}

int qmixer_step_operands(const qmixer_step_operands_args* args, qstate_stream stream) {
    if (!args) return QSTATE_EINVAL;
    const qmixer_step_operands_args& a = *args;
    const int rc = qm::check_step(a.x, a.x_stride, a.dt, a.dt_stride, a.A, a.B, a.B_stride, a.C, a.C_stride, a.batch, a.heads, a.groups, a.d_k,
                                  a.d_v, a.dtype, a.dt_dtype, a.flags);
    if (rc != QSTATE_OK) return rc;
    if (!qm::known(a.qkv_dtype) || !qm::known(a.gate_dtype) || !qm::aligned(a.dt_bias, 4)) return QSTATE_EINVAL;
    if (!qm::aligned(a.q, 4) || !qm::aligned(a.k, 4) || !qm::aligned(a.v, 4) || !qm::aligned(a.gates, 4)) return QSTATE_EINVAL;
    if (!a.batch) return QSTATE_OK;
    if (!a.q || !a.k || !a.v || !a.gates) return QSTATE_EINVAL;
    qm::OperandParams p{};
    p.s = {a.x, a.x_stride, a.dt, a.dt_stride, a.A, a.B, a.B_stride, a.C, a.C_stride, nullptr, a.dt_bias, nullptr, nullptr, 0,
           a.heads, a.heads / a.groups, a.dt_dtype == QSTATE_BF16, (a.flags & QMIXER_SOFTPLUS) != 0};
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.gates = a.gates;
    p.tiles = (int64_t)a.batch * a.heads;
    p.dk = a.d_k;
    p.dv = a.d_v;
    p.out_bf16 = a.qkv_dtype == QSTATE_BF16;
    p.gate_bf16 = a.gate_dtype == QSTATE_BF16;
    if (a.dtype == QSTATE_BF16) qm::operands_kernel<qm::bf16><<<(unsigned)p.tiles, 128, 0, (cudaStream_t)stream>>>(p);
    else qm::operands_kernel<float><<<(unsigned)p.tiles, 128, 0, (cudaStream_t)stream>>>(p);
    return qm::launched();
}

int qmixer_step_output(const qmixer_step_output_args* args, qstate_stream stream) {
    if (!args) return QSTATE_EINVAL;
    const qmixer_step_output_args& a = *args;
    if (!qm::known(a.dtype) || a.batch < 0 || a.heads < 1 || a.d_v < 1) return QSTATE_EINVAL;
    const int64_t row = (int64_t)a.heads * a.d_v, n = a.batch * row;
    if (row > INT32_MAX || a.y_stride < row || (a.D && a.x_stride < row)) return QSTATE_EINVAL;
    const int size = qm::size_of(a.dtype);
    if (!qm::aligned(a.out, 4) || !qm::aligned(a.D, 4) || !qm::aligned(a.x, size) || !qm::aligned(a.y, size)) return QSTATE_EINVAL;
    if (!n) return QSTATE_OK;
    if (!a.out || !a.y || (a.D && !a.x)) return QSTATE_EINVAL;
    if ((n + 255) / 256 > INT32_MAX) return QSTATE_EUNSUPPORTED;
    const unsigned blocks = (unsigned)((n + 255) / 256);
    if (a.dtype == QSTATE_BF16)
        qm::output_kernel<<<blocks, 256, 0, (cudaStream_t)stream>>>(a.out, (const qm::bf16*)a.x, a.x_stride, a.D, (qm::bf16*)a.y,
                                                                    a.y_stride, n, a.heads, a.d_v);
    else
        qm::output_kernel<<<blocks, 256, 0, (cudaStream_t)stream>>>(a.out, (const float*)a.x, a.x_stride, a.D, (float*)a.y,
                                                                    a.y_stride, n, a.heads, a.d_v);
    return qm::launched();
}

}  // extern "C"
