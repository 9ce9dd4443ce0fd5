// qmixer_scan_chunk.cu -- the prompt scan of bfloat16 inputs in chunks of 128
// tokens, on the tensor cores.
//
// Mathematics.  With a_t the decay of token t, P(i, j) = a_{j+1} .. a_i, S the
// state in front of the chunk and i, j tokens of it:
//   G = C B^T                                            128 x 128, over d_k
//   M_ij = G_ij P(i, j) dt_j for j <= i, else 0
//   y = M X + diag(P(i, 0)) (C S) + D x
//   S <- P(128, 0) S + B^T (w X),  w_j = P(128, j) dt_j
// Every decay enters as a product of the a_t, never as the exponential of a
// difference of sums: no cancellation, zeros and underflow are exact, and a
// non-finite time step touches its own and later tokens only.  P(i, j) of two
// different 32-token blocks is (product in i's block) (whole blocks between)
// (product behind j in j's block).
//
// Rounding.  The tensor cores take bfloat16 factors and add in binary32.  B, C
// and X are bfloat16 already.  M and the copy of S that C multiplies are rounded
// once: both enter y alone, which is rounded to bfloat16 itself, and their errors
// are of that size and independent of it.  w X is not rounded, since the state
// is binary32 and carried on: it is split into three bfloat16 terms, 24 bits.
// The state itself lives in binary32 registers.
//
// Work.  A CTA of eight warps takes 64 value columns of one head over one
// segment; two CTAs share an SM, so that one computes while the other waits for
// its loads or products.  Tensor memory, 256 columns a CTA: G (128), later Y and
// the state's increment; C S (64); M (64, as the A operand of M X).  Shared
// memory: C, B, X as TMA lays them down (128-byte swizzle), S.  w X takes C's and
// S's places once G and C S are done.  B serves twice, by rows for G and by
// columns (transposed descriptor) for B^T.
#include <cuda.h>

#include "qmixer_scan.cuh"

namespace qm {

constexpr uint32_t kPolls = 1u << 24;      // several seconds

// ------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_at(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_at(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity) {
    for (uint32_t i = 0; i < kPolls; i++) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(smem_at(b)), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}
__device__ __forceinline__ void tma_load(void* to, const CUtensorMap* map, int x, int y, uint64_t* b) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_at(to)),
        "l"(map), "r"(x), "r"(y), "r"(smem_at(b))
        : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_at(b))
                 : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: start, the stride between
// 64-element blocks along rows of a column-major operand (`lead`), and the stride
// between groups of eight rows (1024 bytes).
__device__ __forceinline__ uint64_t mat(uint32_t at, uint32_t lead) {
    return (uint64_t)((at & 0x3ffff) >> 4) | (uint64_t)((lead >> 4) & 0x3fff) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Instruction descriptor: bfloat16 factors, binary32 sums, 128 x n.
__host__ __device__ constexpr uint32_t ins(int n, bool a_by_columns, bool b_by_columns) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)a_by_columns << 15 | (uint32_t)b_by_columns << 16 |
           (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void tm_load32(uint32_t at, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tm_store16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// ------------------------------------------------------------ shared memory
// A token's decays and time step, per chunk.
struct Scalars {
    float a[kChunk], dt[kChunk];
    float upto[kChunk];          // product of its block's decays up to it
    float behind[kChunk];        // product of its block's decays behind it, times dt
    float block[4];              // product of a block's decays
};

template <int N, bool OUT> struct ChunkSmem {
    static constexpr int kOp = N * kChunk * 2;               // bytes of B or C
    static constexpr int kX = 64 * kChunk * 2;
    // offsets in the 1024-byte aligned part.  w X: three parts of kX.
    static constexpr int kB = 0, kXs = kB + kOp, kC = kXs + kX;
    static constexpr int kW0 = kC, kW1 = kC + kX;            // in C's place (N = 128) or behind it
    static constexpr int kS = kC + 2 * kX, kW2 = kS;
    static constexpr int kEnd = kS + kX;
    static constexpr int kBytes = kEnd + 1024 + 2 * (int)sizeof(Scalars) + 64 * 4 + 64;
};

// Byte offset of 16-byte piece c of row r in rows of 128 bytes, swizzled.
__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

template <int N, bool OUT>
__global__ void __launch_bounds__(256, 2)
chunk_kernel(const __grid_constant__ ScanParams p, const __grid_constant__ CUtensorMap mx,
             const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mc) {
    using L = ChunkSmem<N, OUT>;
    extern __shared__ unsigned char raw[];
    unsigned char* const sm = raw + ((1024 - (smem_at(raw) & 1023)) & 1023);
    Scalars* const scal = reinterpret_cast<Scalars*>(sm + L::kEnd);
    int* const bad = reinterpret_cast<int*>(scal + 2);            // first non-finite token of a column
    uint64_t* const bars = reinterpret_cast<uint64_t*>(bad + 64);  // loads, products a, products b
    uint32_t* const tm_slot = reinterpret_cast<uint32_t*>(bars + 3);
    constexpr uint32_t kTmem = OUT ? 256 : 64;
    constexpr uint32_t kG = 0, kD = 0, kY = 64, kYo = 128, kM = 192;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, quad = warp & 3, half = warp >> 2;
    Segment seg;
    if (!find_segment(p, blockIdx.x, seg)) return;
    if (!OUT && seg.last) return;
    const int parts = p.dv / 64, h = blockIdx.y / parts, c0 = blockIdx.y % parts * 64, g = h / p.per_group;
    const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f, D = OUT && p.D ? p.D[h] : 0.0f;

    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 3; i++) bar_init(bars + i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    if (tid < 64) bad[tid] = kChunk;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(tm_slot)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncthreads();
    const uint32_t tm = *reinterpret_cast<volatile uint32_t*>(tm_slot);
    const uint32_t tq = tm + ((uint32_t)(quad * 32) << 16);

    // the state: row n, columns half * 32 ..
    const int row = quad * 32 + lane;
    const bool holds = row < N;
    float S[32];
    {
        const float* from = nullptr;
        if (OUT && p.cut) from = p.seg_state + ((int64_t)blockIdx.x * p.heads + h) * N * p.dv;
        else if (OUT && p.initial) from = p.state + ((int64_t)seg.sequence * p.heads + h) * N * p.dv;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            float4 v = make_float4(0, 0, 0, 0);
            if (from && holds) v = *reinterpret_cast<const float4*>(from + (int64_t)row * p.dv + c0 + half * 32 + i);
            S[i] = v.x; S[i + 1] = v.y; S[i + 2] = v.z; S[i + 3] = v.w;
        }
    }
    auto put_state = [&] {
        if (OUT && holds) {
#pragma unroll
            for (int c = 0; c < 4; c++)
                *reinterpret_cast<uint4*>(sm + L::kS + swz(row, half * 4 + c)) =
                    make_uint4(pack_bf(S[c * 8], S[c * 8 + 1]), pack_bf(S[c * 8 + 2], S[c * 8 + 3]),
                               pack_bf(S[c * 8 + 4], S[c * 8 + 5]), pack_bf(S[c * 8 + 6], S[c * 8 + 7]));
        }
        fence_async();
    };
    auto load = [&](int64_t t0) {           // thread 0
        const int t = (int)t0;
        bar_expect(bars, (OUT ? 2 : 1) * L::kOp + L::kX);
#pragma unroll
        for (int i = 0; i < N / 64; i++) {
            tma_load(sm + L::kB + i * 16384, &mb, g * N + i * 64, t, bars);
            if (OUT) tma_load(sm + L::kC + i * 16384, &mc, g * N + i * 64, t, bars);
        }
        tma_load(sm + L::kXs, &mx, h * p.dv + c0, t, bars);
    };
    float raw_dt = 0.0f;
    auto fetch_dt = [&](int64_t t0) {       // threads below 128
        raw_dt = tid < kChunk && t0 + tid < seg.to ? load_dt(p.dt, (t0 + tid) * p.dts + h, p.dt_bf16) : 0.0f;
    };
    auto scalars = [&](int64_t t0, Scalars& s) {
        if (tid >= kChunk) return;
        const bool in = t0 + tid < seg.to;
        const float dt = in ? time_step(raw_dt, bias, p.softplus) : 0.0f, a = in ? expf(dt * A) : 1.0f;
        float up = a, down = a;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const float u = __shfl_up_sync(~0u, up, d), v = __shfl_down_sync(~0u, down, d);
            if (lane >= d) up *= u;
            if (lane + d < 32) down *= v;
        }
        float behind = __shfl_down_sync(~0u, down, 1);
        if (lane == 31) behind = 1.0f;
        s.a[tid] = a;
        s.dt[tid] = dt;
        s.upto[tid] = up;
        s.behind[tid] = behind * dt;
        if (lane == 31) s.block[warp] = up;
    };

    bool ok = true;
    float total = 1.0f;
    int64_t t0 = seg.from;
    if (t0 < seg.to) {
        if (tid == 0) load(t0);
        fetch_dt(t0);
        scalars(t0, scal[0]);
        put_state();
        if (t0 + kChunk < seg.to) fetch_dt(t0 + kChunk);
    }
    for (uint32_t it = 0; t0 < seg.to; t0 += kChunk, it++) {
        const uint32_t par = it & 1;
        const Scalars& sc = scal[par];
        const int valid = seg.to - t0 < kChunk ? (int)(seg.to - t0) : kChunk;
        ok = bar_wait(bars, par);
        if (valid < kChunk) {
            // rows of other sequences or of nothing: zero, whatever they hold
            for (int i = tid; i < (kChunk - valid) * (N / 8 + 8); i += 256) {
                const int r = valid + i / (N / 8 + 8), c = i % (N / 8 + 8);
                unsigned char* at = c < N / 8 ? sm + L::kB + c / 8 * 16384 + r * 128 + c % 8 * 16
                                              : sm + L::kXs + r * 128 + (c - N / 8) * 16;
                *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
            }
            fence_async();
        }
        tc_before();
        if (!__syncthreads_and(ok)) { ok = false; break; }
        if (OUT && tid == 0) {
            tc_after();
            const uint32_t c = smem_at(sm + L::kC), b = smem_at(sm + L::kB), s = smem_at(sm + L::kS);
#pragma unroll
            for (int k = 0; k < N / 16; k++)
                mma_ss(tm + kG, mat(c + k / 4 * 16384 + k % 4 * 32, 16), mat(b + k / 4 * 16384 + k % 4 * 32, 16),
                       ins(128, false, false), k > 0);
#pragma unroll
            for (int k = 0; k < N / 16; k++)
                mma_ss(tm + kYo, mat(c + k / 4 * 16384 + k % 4 * 32, 16), mat(s + k * 2048, 16384),
                       ins(64, false, true), k > 0);
            tc_commit(bars + 1);
        }
        if (OUT) {
            ok = bar_wait(bars + 1, par);
            tc_after();
        }
        // w X in three parts: row r, pieces half * 4 ..
        {
            const int r = tid & 127, blk = r / 32;
            float w = sc.behind[r];
#pragma unroll
            for (int u = 1; u < 4; u++)
                if (u > blk) w *= sc.block[u];
            float probe = 0.0f;
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const int at = swz(r, half * 4 + c);
                const uint4 v = *reinterpret_cast<const uint4*>(sm + L::kXs + at);
                const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                uint32_t o[3][4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float xa = bf_lo(in[i]), xb = bf_hi(in[i]);
                    probe = fmaf(xa, 0.0f, probe);
                    probe = fmaf(xb, 0.0f, probe);
                    float pa = w * xa, pb = w * xb;
                    o[0][i] = pack_bf(pa, pb);
                    pa -= bf_lo(o[0][i]);
                    pb -= bf_hi(o[0][i]);
                    o[1][i] = pack_bf(pa, pb);
                    pa -= bf_lo(o[1][i]);
                    pb -= bf_hi(o[1][i]);
                    o[2][i] = pack_bf(pa, pb);
                }
                *reinterpret_cast<uint4*>(sm + L::kW0 + at) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
                *reinterpret_cast<uint4*>(sm + L::kW1 + at) = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
                *reinterpret_cast<uint4*>(sm + L::kW2 + at) = make_uint4(o[2][0], o[2][1], o[2][2], o[2][3]);
            }
            if (OUT && probe != probe) {
                // a non-finite x must not reach earlier rows through M's zeros: it
                // leaves X, and its column becomes NaN from its row on
                for (int c = 0; c < 4; c++)
                    for (int i = 0; i < 8; i++) {
                        uint16_t* e = reinterpret_cast<uint16_t*>(sm + L::kXs + swz(r, half * 4 + c)) + i;
                        if ((*e & 0x7f80) == 0x7f80) {
                            *e = 0;
                            atomicMin(bad + half * 32 + c * 8 + i, r);
                        }
                    }
            }
        }
        if (OUT) {
            // M, two 32 x 32 blocks a warp: row `row`, columns b * 32 ..
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int b = e * 2 + half;
                uint32_t m[16];
                if (b > quad) {
#pragma unroll
                    for (int i = 0; i < 16; i++) m[i] = 0;
                } else {
                    float v[32];
                    tm_load32(tq + kG + b * 32, v);
                    if (b == quad) {
                        float f = 1.0f;                   // P(row, j) for j = 31 .. 0
#pragma unroll
                        for (int j = 31; j >= 0; j--) {
                            const float fd = f * sc.dt[b * 32 + j];
                            v[j] = j <= lane ? v[j] * fd : 0.0f;
                            f = j <= lane ? f * sc.a[b * 32 + j] : f;
                        }
                    } else {
                        float f = sc.upto[row];
#pragma unroll
                        for (int u = 1; u < 3; u++)
                            if (u > b && u < quad) f *= sc.block[u];
#pragma unroll
                        for (int j = 0; j < 32; j++) v[j] *= f * sc.behind[b * 32 + j];
                    }
#pragma unroll
                    for (int i = 0; i < 16; i++) m[i] = pack_bf(v[2 * i], v[2 * i + 1]);
                }
                tm_store16(tq + kM + b * 16, m);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        fence_async();
        tc_before();
        if (!__syncthreads_and(ok)) { ok = false; break; }
        if (tid == 0) {
            tc_after();
            const uint32_t b = smem_at(sm + L::kB), x = smem_at(sm + L::kXs);
            const uint32_t w[3] = {smem_at(sm + L::kW0), smem_at(sm + L::kW1), smem_at(sm + L::kW2)};
            if (OUT)
#pragma unroll
                for (int k = 0; k < 8; k++)
                    mma_ts(tm + kY, tm + kM + k * 8, mat(x + k * 2048, 16384), ins(64, false, true), k > 0);
#pragma unroll
            for (int i = 2; i >= 0; i--)
#pragma unroll
                for (int k = 0; k < 8; k++)
                    mma_ss(tm + kD, mat(b + k * 2048, 16384), mat(w[i] + k * 2048, 16384), ins(64, true, true),
                           i < 2 || k > 0);
            tc_commit(bars + 2);
        }
        // while the products run: the next chunk's decays, and x for D x
        const bool more = t0 + kChunk < seg.to;
        if (more) scalars(t0 + kChunk, scal[par ^ 1]);
        if (t0 + 2 * kChunk < seg.to) fetch_dt(t0 + 2 * kChunk);
        uint4 xr[4];
        if (OUT)
#pragma unroll
            for (int c = 0; c < 4; c++) xr[c] = *reinterpret_cast<const uint4*>(sm + L::kXs + swz(row, half * 4 + c));
        __syncthreads();                       // X has been read
        ok = bar_wait(bars + 2, par);
        tc_after();
        if (ok && more && tid == 0) load(t0 + kChunk);
        {
            float v[32];
            tm_load32(tq + kD + half * 32, v);
            const float dec = sc.block[0] * sc.block[1] * (sc.block[2] * sc.block[3]);
            if (!OUT) total *= dec;
#pragma unroll
            for (int i = 0; i < 32; i++) S[i] = fmaf(S[i], dec, v[i]);
            if (more) put_state();
        }
        if (OUT) {
            float v[32], o[32];
            tm_load32(tq + kY + half * 32, v);
            tm_load32(tq + kYo + half * 32, o);
            float f = sc.upto[row];
#pragma unroll
            for (int u = 0; u < 3; u++)
                if (u < quad) f *= sc.block[u];
#pragma unroll
            for (int i = 0; i < 32; i++) v[i] = fmaf(f, o[i], v[i]);
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const uint32_t in[4] = {xr[c].x, xr[c].y, xr[c].z, xr[c].w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    v[c * 8 + 2 * i] = fmaf(D, bf_lo(in[i]), v[c * 8 + 2 * i]);
                    v[c * 8 + 2 * i + 1] = fmaf(D, bf_hi(in[i]), v[c * 8 + 2 * i + 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 32; i++)
                if (row >= bad[half * 32 + i]) v[i] = __uint_as_float(0x7fc00000u);
            if (row < valid) {
                bf16* const y = static_cast<bf16*>(p.y) + (t0 + row) * p.ys + (int64_t)h * p.dv + c0 + half * 32;
                if ((reinterpret_cast<uintptr_t>(y) & 15) == 0) {
#pragma unroll
                    for (int c = 0; c < 4; c++)
                        *reinterpret_cast<uint4*>(y + c * 8) =
                            make_uint4(pack_bf(v[c * 8], v[c * 8 + 1]), pack_bf(v[c * 8 + 2], v[c * 8 + 3]),
                                       pack_bf(v[c * 8 + 4], v[c * 8 + 5]), pack_bf(v[c * 8 + 6], v[c * 8 + 7]));
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i++) y[i] = __float2bfloat16_rn(v[i]);
                }
            }
        }
    }
    const bool all = __syncthreads_and(ok);
    if (!all) {
        // a wait ran out (a GPU preempted for seconds): what is left is NaN
        for (int i = 0; i < 32; i++) S[i] = total = __uint_as_float(0x7fc00000u);
        if (OUT)
            for (int64_t t = t0 + (tid & 127); t < seg.to; t += kChunk)
                for (int i = 0; i < 32; i++)
                    static_cast<bf16*>(p.y)[t * p.ys + (int64_t)h * p.dv + c0 + half * 32 + i] = __float2bfloat16_rn(S[0]);
    }
    tc_before();
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kTmem) : "memory");
    float* to = nullptr;
    if (!OUT) to = p.seg_state + ((int64_t)blockIdx.x * p.heads + h) * N * p.dv;
    else if (seg.last && p.state) to = p.state + ((int64_t)seg.sequence * p.heads + h) * N * p.dv;
    if (to && holds) {
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(to + (int64_t)row * p.dv + c0 + half * 32 + i) =
                make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
    }
    if (!OUT && tid == 0 && c0 == 0) p.seg_decay[(int64_t)blockIdx.x * p.heads + h] = total;
}

// ------------------------------------------------------------ host
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static std::atomic<EncodeFn> fn{nullptr};
    EncodeFn f = fn.load(std::memory_order_acquire);
    if (!f) {
        void* at = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        f = reinterpret_cast<EncodeFn>(at);
        fn.store(f, std::memory_order_release);
    }
    return f;
}

// Rows of `width` bfloat16, `tokens` of them, in boxes of 64 x 128.
bool encode(CUtensorMap* m, const void* at, int64_t width, int64_t stride, int64_t tokens) {
    const EncodeFn f = encoder();
    if (!f) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)tokens}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, kChunk}, ones[2] = {1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(at), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int N, bool OUT>
bool launch_chunk(const ScanParams& p, const CUtensorMap (&m)[3], int64_t segments, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    constexpr int bytes = ChunkSmem<N, OUT>::kBytes;
    if (!allow_smem(reinterpret_cast<const void*>(chunk_kernel<N, OUT>), bytes, done)) return false;
    const dim3 grid((unsigned)segments, (unsigned)(p.heads * (p.dv / 64)));
    chunk_kernel<N, OUT><<<grid, 256, bytes, st>>>(p, m[0], m[1], m[2]);
    return true;
}

bool launch_scan_chunk(const ScanParams& p, int dk, int64_t segments, bool states_only, cudaStream_t st) {
    const int groups = p.heads / p.per_group;
    CUtensorMap m[3];
    if (!encode(&m[0], p.x, (int64_t)p.heads * p.dv, p.xs, p.seq.tokens) ||
        !encode(&m[1], p.B, (int64_t)groups * dk, p.Bs, p.seq.tokens) ||
        !encode(&m[2], p.C, (int64_t)groups * dk, p.Cs, p.seq.tokens))
        return false;
    if (dk == 64)
        return states_only ? launch_chunk<64, false>(p, m, segments, st) : launch_chunk<64, true>(p, m, segments, st);
    return states_only ? launch_chunk<128, false>(p, m, segments, st) : launch_chunk<128, true>(p, m, segments, st);
}

}  // namespace qm
