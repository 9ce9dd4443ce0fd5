// qmixer_quantize.cu -- binary32 states into the codes and scales of a low-bit
// object: what stands between a prompt's scan and the first decode step.
//
// The arithmetic is the dynamic rule of qstate.h on a fresh state (scale =
// cvt(max / Qmax), code = clamp(round_half_even(S * inv)), the product exact),
// bit for bit.  Bound: memory (four bytes read, bits / 8 written an element).  A
// CTA takes a tile, or a part of one where groups lie inside a row, and holds it in
// registers: a thread eight consecutive columns at a time, so that one scale of a
// whole tile (group 0) costs no second read.  A group's lanes are joined by shuffles.
// 2048 tiles of 128 x 64 to int8 take 16 us (5.4 TB/s, 82% of the copy rate); with the
// copies into the object 21.
#include "qmixer_common.cuh"

namespace qm {

constexpr int kMaxMixedHeads = 512;

struct QuantParams {
    const float* S;
    uint8_t* codes;
    void* scales;
    float* ref;
    int heads, group, bits;
    bool scale_f32, rotate, mixed;
    int64_t row_bytes, tile_bytes;
    uint8_t head_bits[kMaxMixedHeads];
    uint32_t head_off[kMaxMixedHeads];
};

// x * inv rounded half to even from the exact product, as the low bits of the
// result: one fused multiply-add to 1.5 * 2^23 rounds it once.
__device__ __forceinline__ uint32_t code_of(float x, float inv, float qmax) {
    constexpr float kMagic = 12582912.0f;
    return __float_as_uint(fminf(fmaxf(fmaf(x, inv, kMagic), kMagic - qmax), kMagic + qmax));
}

// PARTS: CTAs that share a tile (one where a scale is of the whole tile).
template <int DK, int DV, int PARTS>
__global__ void __launch_bounds__(256) quantize_kernel(const __grid_constant__ QuantParams p) {
    constexpr int kEach = DK * DV / 8 / 256 / PARTS, kRow = DV / 8;
    __shared__ uint32_t tops[8];                    // the warps' maxima
    const int64_t tile = blockIdx.x / PARTS;
    const int u0 = (int)(blockIdx.x % PARTS) * (kEach * 256) + threadIdx.x;     // its first eight columns
    const int h = int(tile % p.heads);
    const int64_t row = tile / p.heads;
    const int bits = p.mixed ? p.head_bits[h] : p.bits;
    uint8_t* const codes = p.codes + row * p.row_bytes + (p.mixed ? (int64_t)p.head_off[h] : h * p.tile_bytes);
    const float* const S = p.S + tile * (DK * DV);
    float v[kEach][8];
#pragma unroll
    for (int i = 0; i < kEach; i++) load8(S + (i * 256 + u0) * 8, v[i]);
    if (p.rotate) {
        // the butterfly of qstate.h along d_v, one rounding per sum; a row is
        // kRow neighbouring lanes of eight columns
#pragma unroll
        for (int i = 0; i < kEach; i++) {
#pragma unroll
            for (int s = 1; s < 8; s <<= 1)
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (!(j & s)) {
                        const float a = v[i][j], b = v[i][j | s];
                        v[i][j] = a + b;
                        v[i][j | s] = a - b;
                    }
            for (int s = 1; s < kRow; s <<= 1) {
                const bool high = threadIdx.x & s;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float o = __shfl_xor_sync(~0u, v[i][j], s);
                    v[i][j] = high ? o - v[i][j] : v[i][j] + o;
                }
            }
        }
    }
    if (p.ref) {
#pragma unroll
        for (int i = 0; i < kEach; i++) store8(p.ref + tile * (DK * DV) + (i * 256 + u0) * 8, v[i]);
    }
    if (bits == 32) {
#pragma unroll
        for (int i = 0; i < kEach; i++)
            store8(reinterpret_cast<float*>(codes) + (i * 256 + u0) * 8, v[i]);
        return;
    }
    uint32_t m[kEach];
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        m[i] = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) m[i] = max(m[i], __float_as_uint(v[i][j]) & 0x7fffffffu);
    }
    const int lanes = p.group / 8;
    if (!p.group) {
        uint32_t all = 0;
#pragma unroll
        for (int i = 0; i < kEach; i++) all = max(all, m[i]);
        all = __reduce_max_sync(~0u, all);
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x / 32] = all;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; w++) all = max(all, tops[w]);
#pragma unroll
        for (int i = 0; i < kEach; i++) m[i] = all;
    } else {
        // a group divides d_v: a power of two of lanes
        for (int d = 1; d < lanes; d <<= 1)
#pragma unroll
            for (int i = 0; i < kEach; i++) m[i] = max(m[i], __shfl_xor_sync(~0u, m[i], d));
    }
    const float qmax = (float)((1 << (bits - 1)) - 1);
    const int per_row = p.group ? DV / p.group : 1;
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        const int u = i * 256 + u0, r = u / kRow, c8 = u % kRow;
        float scale = __fdiv_rn(__uint_as_float(m[i]), qmax);
        if (!p.scale_f32) {
            // an infinite half saturates, as in a step; one that is not a number stays so,
            // and with it every value of its group
            const __half hs = __float2half_rn(scale);
            scale = __hisinf(hs) ? 65504.0f : __half2float(hs);
        }
        const float inv = scale == 0.0f ? 0.0f : __frcp_rn(scale);
        const bool first = p.group ? c8 % lanes == 0 : u == 0;
        if (first) {
            const int64_t at = p.group ? (tile * DK + r) * per_row + c8 / lanes : tile;
            if (p.scale_f32) static_cast<float*>(p.scales)[at] = scale;
            else static_cast<__half*>(p.scales)[at] = __float2half_rn(scale);
        }
        uint32_t c[8];
#pragma unroll
        for (int j = 0; j < 8; j++) c[j] = code_of(v[i][j], inv, qmax);
        uint32_t lo = 0, hi = 0;
        if (bits == 8) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                lo |= (c[j] & 255) << (8 * j);
                hi |= (c[j + 4] & 255) << (8 * j);
            }
            *reinterpret_cast<uint2*>(codes + u * 8) = make_uint2(lo, hi);
        } else if (bits == 2) {
#pragma unroll
            for (int j = 0; j < 8; j++) lo |= (c[j] & 3) << (2 * j);
            *reinterpret_cast<uint16_t*>(codes + u * 2) = (uint16_t)lo;
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                lo |= (c[j] & 15) << (4 * j);
                hi |= ((c[j] >> 4) & 3) << (2 * j);
            }
            *reinterpret_cast<uint32_t*>(codes + u * 4) = lo;
            if (bits == 6) *reinterpret_cast<uint16_t*>(codes + DK * DV / 2 + u * 2) = (uint16_t)hi;
        }
    }
}

// Groups are of a row: a tile then falls into pieces of 256 threads, for as many
// loads in flight as may be (and one small tile over several SMs).
template <int DK, int DV> void launch_quantize(const QuantParams& p, int64_t tiles, cudaStream_t st) {
    constexpr int kParts = DK * DV / 8 / 256;
    if (p.group) quantize_kernel<DK, DV, kParts><<<(unsigned)(tiles * kParts), 256, 0, st>>>(p);
    else quantize_kernel<DK, DV, 1><<<(unsigned)tiles, 256, 0, st>>>(p);
}

bool width_ok(int b) { return b == 2 || b == 4 || b == 6 || b == 8; }

}  // namespace qm

extern "C" int qmixer_quantize(const qmixer_quantize_args* args, qstate_stream stream) {
    if (!args) return QSTATE_EINVAL;
    const qmixer_quantize_args& a = *args;
    if (a.rows < 0 || a.heads < 1 || a.d_k < 8 || a.d_v < 8 || a.d_k % 8 || a.d_v % 8) return QSTATE_EINVAL;
    if (a.rows > INT32_MAX || a.rows * a.heads > INT32_MAX) return QSTATE_EINVAL;
    if (a.group < 0 || (a.group && (a.group % 8 || a.d_v % a.group))) return QSTATE_EINVAL;
    if (a.scale_dtype != QSTATE_F16 && a.scale_dtype != QSTATE_F32) return QSTATE_EINVAL;
    if (a.rotation != 0 && a.rotation != 1) return QSTATE_EINVAL;
    if (a.head_bits) {
        for (int i = 0; i < a.heads; i++)
            if (!qm::width_ok(a.head_bits[i])) return QSTATE_EINVAL;
    } else if (!qm::width_ok(a.bits) && a.bits != 32) {
        return QSTATE_EINVAL;
    }
    if (!qm::aligned(a.S, 16) || !qm::aligned(a.codes, 16) || !qm::aligned(a.ref, 16) || !qm::aligned(a.scales, 4))
        return QSTATE_EINVAL;
    if ((a.d_k != 64 && a.d_k != 128) || (a.d_v != 64 && a.d_v != 128)) return QSTATE_EUNSUPPORTED;
    if (a.head_bits && a.heads > qm::kMaxMixedHeads) return QSTATE_EUNSUPPORTED;
    if (!a.rows) return QSTATE_OK;
    if (!a.S || !a.codes || ((a.head_bits || a.bits != 32) && !a.scales)) return QSTATE_EINVAL;
    qm::QuantParams p{};
    p.S = a.S;
    p.codes = static_cast<uint8_t*>(a.codes);
    p.scales = a.scales;
    p.ref = a.ref;
    p.heads = a.heads;
    p.group = a.group;
    p.bits = a.bits;
    p.scale_f32 = a.scale_dtype == QSTATE_F32;
    p.rotate = a.rotation == 1;
    p.mixed = a.head_bits != nullptr;
    p.tile_bytes = (int64_t)a.d_k * a.d_v * a.bits / 8;
    p.row_bytes = p.tile_bytes * a.heads;
    if (a.head_bits) {
        uint32_t off = 0;
        for (int i = 0; i < a.heads; i++) {
            p.head_bits[i] = a.head_bits[i];
            p.head_off[i] = off;
            off += (uint32_t)(a.d_k * a.d_v * a.head_bits[i] / 8);
        }
        p.row_bytes = off;
        p.tile_bytes = 0;
    }
    const int64_t tiles = a.rows * a.heads;
    const cudaStream_t st = (cudaStream_t)stream;
    if (tiles * (a.d_k * a.d_v / 2048) > INT32_MAX) return QSTATE_EUNSUPPORTED;
    if (a.d_k == 64 && a.d_v == 64) qm::launch_quantize<64, 64>(p, tiles, st);
    else if (a.d_k == 64) qm::launch_quantize<64, 128>(p, tiles, st);
    else if (a.d_v == 64) qm::launch_quantize<128, 64>(p, tiles, st);
    else qm::launch_quantize<128, 128>(p, tiles, st);
    return qm::launched();
}
