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
// Work.  A CTA takes 64 value columns of one head over one segment and fills an
// SM.  Only S chains one chunk to the next, so its warps have roles that run a
// chunk ahead of each other and meet at mbarriers:
//   load     C, B, X of two chunks by TMA (128-byte swizzle)
//   product  two warps: C S and the increment B^T (w X), which the next chunk waits
//            for, and G and M X, which no chunk waits for
//   M        eight warps: the decays two chunks ahead; G from tensor memory, M back
//            to it (as the A operand)
//   W        eight warps: w X in three parts to shared memory
//   E        eight warps: S, half a row a thread in registers, from the increment,
//            its bfloat16 copy to shared memory; then y
// Tensor memory: G (128 columns), C S (2 x 64), M X (64), M (64), the increment (128:
// the first two parts of w X are one product of 128 columns, for reading B^T from
// shared memory bounds it).  Shared memory: two stages of C, B, X, two parts of w X,
// and one place that holds S, then, once C S is done, the third part.  B serves
// twice, by rows for G and by columns (transposed descriptor) for B^T.  Loops are
// unrolled no further than they have to be: the roles share the instruction cache,
// and with all of it unrolled a chunk took twice as long.
//
// Measured: eight sequences of 2048 tokens, 32 heads of 128 x 64, 88 us, 4000 cycles a
// chunk and SM.  The products take 2100 of them (48 cycles each at 64 columns, 64 at
// 128: operand reads from shared memory), instructions issue in half of the slots;
// what bounds a chunk is the chain S, C S, third part, increment, S, with two waits
// for tensor memory and two for shared memory on it, and 256 chains on 148 SMs take
// two rounds.  All warps in step, two CTAs an SM, took 137 us.
#include <cuda.h>

#include "qmixer_scan.cuh"

namespace qm {

// Every wait is bounded: by ScanParams::polls, or, for a CTA's own copies and products,
// which end by themselves, by kWaitPolls.  A wait that runs out (a GPU preempted for
// seconds) ends its role; what waits for that role runs out in turn, no copy or product
// outlives the CTA, its segment's y and state become NaN, and it is counted here.
__device__ unsigned long long lost_ctas;

// ------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_at(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_at(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_at(b)), "r"(parity)
        : "memory");
    return ok;
}
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, uint32_t polls) {
    for (uint32_t i = 0; i < polls; i++) {
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
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* b) {
    asm volatile(
        "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_at(b))
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
// Called by a whole warp, so that the descriptors stay in uniform registers; one
// elected lane issues.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// Sixteen columns at two places, on their way together.
__device__ __forceinline__ void tm_load16(uint32_t at, uint32_t at2, float (&v)[16], float (&w)[16]) {
    uint32_t r[16], q[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%32];\n"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%33];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
          "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
          "=&r"(q[0]), "=&r"(q[1]), "=&r"(q[2]), "=&r"(q[3]), "=&r"(q[4]), "=&r"(q[5]), "=&r"(q[6]), "=&r"(q[7]),
          "=&r"(q[8]), "=&r"(q[9]), "=&r"(q[10]), "=&r"(q[11]), "=&r"(q[12]), "=&r"(q[13]), "=&r"(q[14]), "=&r"(q[15])
        : "r"(at), "r"(at2)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) {
        v[i] = __uint_as_float(r[i]);
        w[i] = __uint_as_float(q[i]);
    }
}
__device__ __forceinline__ void tm_load8(uint32_t at, uint32_t at2, float (&v)[8], float (&w)[8]) {
    uint32_t r[8], q[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
          "=&r"(q[0]), "=&r"(q[1]), "=&r"(q[2]), "=&r"(q[3]), "=&r"(q[4]), "=&r"(q[5]), "=&r"(q[6]), "=&r"(q[7])
        : "r"(at), "r"(at2)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; i++) {
        v[i] = __uint_as_float(r[i]);
        w[i] = __uint_as_float(q[i]);
    }
}
__device__ __forceinline__ void tm_store8(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
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
    static constexpr int kX = 64 * kChunk * 2;               // bytes of X, of a part of w X, room of S
    // offsets in the 1024-byte aligned part; a stage is B, X, C.  (The products
    // read 128 columns of B by columns: for N = 64 the second half is X, and rows
    // of tensor memory that nothing reads.)
    static constexpr int kB = 0, kXs = kOp, kC = kOp + kX;
    static constexpr int kStage = kOp + kX + (OUT ? kOp : 0);
    static constexpr int kW0 = 2 * kStage, kW1 = kW0 + kX, kW2 = kW1 + kX, kS = kW2;
    static constexpr int kEnd = kW2 + kX;
    static constexpr int kBytes = kEnd + 1024 + 3 * (int)sizeof(Scalars) + 2 * 64 * 4 + 22 * 8 + 16;
};
static_assert(ChunkSmem<128, true>::kBytes <= 232448, "shared memory of a CTA");

// mbarriers.  No waiter may fall two phases behind; those with more places take turns
// by chunk (three: by threes), where a phase may end before all have waited for the
// one in front of it.
enum { B_FULL = 0, B_SC = 2, B_E = 5, B_W01 = 7, B_G = 9, B_D = 11, B_Y = 13, B_YO, B_W2, B_M, B_S, B_WSYNC, B_DRAIN, kBars = B_DRAIN + 2 };

// Byte offset of 16-byte piece c of row r in rows of 128 bytes, swizzled.
__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__device__ __forceinline__ void bar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(b)) : "memory");
}
// One arrival of a warp whose lanes are done (their own fences come before).
__device__ __forceinline__ void warp_arrive(uint64_t* b, int lane) {
    __syncwarp();
    if (lane == 0) bar_arrive(b);
}
__device__ __forceinline__ void store32(bf16* p, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// warps 0 to 7: E, 8 to 15: M, 16 to 23: W, 24 and 25: products, 26: load
constexpr int kThreads = 864;
constexpr uint32_t kG = 0, kYo = 128, kY = 256, kM = 320, kD = 384;      // tensor memory columns

template <int N, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
chunk_kernel(const __grid_constant__ ScanParams p, const __grid_constant__ CUtensorMap mx,
             const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mc) {
    using L = ChunkSmem<N, OUT>;
    extern __shared__ unsigned char raw[];
    unsigned char* const sm = raw + ((1024 - (smem_at(raw) & 1023)) & 1023);
    Scalars* const scal = reinterpret_cast<Scalars*>(sm + L::kEnd);
    int* const bad = reinterpret_cast<int*>(scal + 3);            // [2][64]: a column's first non-finite token, by chunk
    uint64_t* const bars = reinterpret_cast<uint64_t*>(bad + 128);
    uint32_t* const tm_slot = reinterpret_cast<uint32_t*>(bars + 22);
    volatile uint32_t* const lost = tm_slot + 1;                  // set by a role that gave up
    static_assert(kBars <= 22, "room");
    constexpr uint32_t kTmem = 512;

    // the same in all lanes, and known to be: only then do the products' descriptors
    // live in uniform registers (else each product takes 135 cycles to issue, not 48)
    auto uniform = [](uint32_t v) { return __shfl_sync(~0u, v, 0); };
    const int tid = threadIdx.x, warp = (int)uniform(tid / 32), lane = tid & 31, quad = warp & 3;
    Segment seg;
    if (!find_segment(p, blockIdx.x, seg)) return;
    if (!OUT && seg.last) return;
    const int parts = p.dv / 64, h = blockIdx.y / parts, c0 = blockIdx.y % parts * 64, g = h / p.per_group;
    // (seg.to may lie below seg.from)
    const int chunks = (int)uniform((uint32_t)(seg.to > seg.from ? (seg.to - seg.from + kChunk - 1) / kChunk : 0));

    if (tid == 0) {
        *lost = 0;
        for (int i = 0; i < 2; i++) {
            bar_init(bars + B_FULL + i, 2);
            bar_init(bars + B_G + i, 1);
            bar_init(bars + B_D + i, 1);
            bar_init(bars + B_E + i, 8);
            bar_init(bars + B_W01 + i, 8);
            bar_init(bars + B_DRAIN + i, 1);
        }
        bar_init(bars + B_YO, 1);
        bar_init(bars + B_W2, 8);
        bar_init(bars + B_M, 8);
        bar_init(bars + B_S, 8);
        bar_init(bars + B_WSYNC, 8);
        for (int i = 0; i < 3; i++) bar_init(bars + B_SC + i, 4);
        bar_init(bars + B_Y, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    if (tid < 128) bad[tid] = kChunk;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(tm_slot)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncthreads();
    const uint32_t tm = uniform(*reinterpret_cast<volatile uint32_t*>(tm_slot));
    const uint32_t tq = tm + ((uint32_t)(quad * 32) << 16);
    bool ok = true;
    // wait for phase `k` of a barrier, or for chunk c's of two or three that take turns
    // (lanes of a warp may differ in when they give up: all do when one does)
    auto wait = [&](int b, int k) { return ok = ok && __all_sync(~0u, bar_wait(bars + b, k & 1, p.polls)); };
    auto wait2 = [&](int b, int c) { return ok = ok && __all_sync(~0u, bar_wait(bars + b + (c & 1), (c >> 1) & 1, p.polls)); };
    auto wait3 = [&](int b, int c) { return ok = ok && __all_sync(~0u, bar_wait(bars + b + c % 3, c / 3 & 1, p.polls)); };

    if (warp == 26) {
        // ---------------------------------------------------- load
        int issued = 0, half = 0;
        for (int c = 0; c < chunks; c++) {
            unsigned char* const st = sm + (c & 1) * L::kStage;
            uint64_t* const full = bars + B_FULL + (c & 1);
            const int t = (int)(seg.from + (int64_t)c * kChunk);
            if (p.drop_from >= 0 && c >= p.drop_from) break;      // (for tests: these never come)
            // B and C as soon as the products have read the last ones, X when y has
            if (c >= 2 && (!wait2(B_D, c - 2) || (OUT && !wait2(B_G, c - 2)))) break;
            if (lane == 0) {
                bar_expect(full, (OUT ? 2 : 1) * L::kOp);
#pragma unroll
                for (int i = 0; i < N / 64; i++) tma_load(st + L::kB + i * 16384, &mb, g * N + i * 64, t, full);
                if (OUT)
#pragma unroll
                    for (int i = 0; i < N / 64; i++) tma_load(st + L::kC + i * 16384, &mc, g * N + i * 64, t, full);
            }
            half = 1;
            if (c >= 2 && !wait2(B_E, c - 2)) break;
            if (lane == 0) {
                bar_expect(full, L::kX);
                tma_load(st + L::kXs, &mx, h * p.dv + c0, t, full);
                // the chunk that has no stage yet: from DRAM to L2 (C and B come for the
                // first of their heads only)
                if (c + 2 < chunks) tma_prefetch(&mx, h * p.dv + c0, t + 2 * kChunk);
            }
            half = 0;
            issued = c + 1;
        }
        // no copy may outlive the CTA, whatever became of its readers
        if (lane == 0) {
            if (!ok) *lost = 1;          // in front of the arrival that stands for an X that never came
            if (half) bar_arrive(bars + B_FULL + (issued & 1));
        }
        issued += half;
        for (int c = issued > 2 ? issued - 2 : 0; c < issued; c++)
            ok = bar_wait(bars + B_FULL + (c & 1), (c >> 1) & 1, kWaitPolls) && ok;
    } else if (warp >= 24) {
        // ---------------------------------------------------- products
        // descriptors of the first stage; what follows adds multiples of 16 bytes
        const uint64_t bk = mat(smem_at(sm + L::kB), 16), ck = mat(smem_at(sm + L::kC), 16);
        const uint64_t bn = mat(smem_at(sm + L::kB), 16384), xn = mat(smem_at(sm + L::kXs), 16384);
        const uint64_t sn = mat(smem_at(sm + L::kS), 16384), wn = mat(smem_at(sm + L::kW0), 16384);
        bool any = false;                // a product was issued
        if (warp == 24) {
            // what the states wait for: C S and the increment
            for (int c = 0; c < chunks; c++) {
                const uint64_t at = (uint64_t)((c & 1) * (L::kStage / 16));
                const uint32_t yo = tm + kYo + (c & 1) * 64;
                if (!wait2(B_FULL, c) || !wait(B_S, c)) break;   // S in shared memory, the increment read
                tc_after();
                any = true;
                if (OUT) {
#pragma unroll 4
                    for (int k = 0; k < N / 16; k++)
                        mma_ss(yo, ck + at + k / 4 * 1024 + k % 4 * 2, sn + k * 128, ins(64, false, true), k > 0);
                    tc_commit(bars + B_YO);
                }
                if (!wait2(B_W01, c)) break;
                tc_after();
#pragma unroll 4
                for (int k = 0; k < 8; k++)
                    mma_ss(tm + kD, bn + at + k * 128, wn + k * 128, ins(128, true, true), k > 0);
                if (!wait(B_W2, c)) break;
                tc_after();
#pragma unroll 4
                for (int k = 0; k < 8; k++)
                    mma_ss(tm + kD, bn + at + k * 128, wn + 2 * (L::kX / 16) + k * 128, ins(64, true, true), 1);
                tc_commit(bars + B_D + (c & 1));
            }
        } else if (OUT && chunks > 0) {
            // M X of a chunk and G of the next: G first, which M waits for, where its
            // operands are there
            auto make_g = [&](int c) {
                const uint64_t at = (uint64_t)((c & 1) * (L::kStage / 16));
                if (!wait2(B_FULL, c)) return;
                tc_after();
                any = true;
#pragma unroll 4
                for (int k = 0; k < N / 16; k++)
                    mma_ss(tm + kG, ck + at + k / 4 * 1024 + k % 4 * 2, bk + at + k / 4 * 1024 + k % 4 * 2,
                           ins(128, false, false), k > 0);
                tc_commit(bars + B_G + (c & 1));
            };
            make_g(0);
            for (int c = 0; c < chunks; c++) {
                // M is there and G has been read; X's rows behind the last token are
                // zero; the last y has been read
                if (!wait(B_M, c)) break;
                tc_after();
                const bool next = c + 1 < chunks;
                const bool early = next && __all_sync(~0u, bar_test(bars + B_FULL + (c + 1 & 1), (c + 1) >> 1 & 1));
                if (early) make_g(c + 1);
                if (!wait2(B_W01, c) || (c > 0 && !wait2(B_E, c - 1))) break;
                tc_after();
                const uint64_t at = (uint64_t)((c & 1) * (L::kStage / 16));
#pragma unroll 4
                for (int k = 0; k < 8; k++)
                    mma_ts(tm + kY, tm + kM + k * 8, xn + at + k * 128, ins(64, false, true), k > 0);
                tc_commit(bars + B_Y);
                if (next && !early) make_g(c + 1);
            }
        }
        // products in flight end before tensor memory is given back, whoever waited for them
        if (any) {
            __syncwarp();
            tc_commit(bars + B_DRAIN + (warp & 1));
            ok = bar_wait(bars + B_DRAIN + (warp & 1), 0, kWaitPolls) && ok;
        }
    } else if (warp >= 16) {
        // ---------------------------------------------------- W: half of row `r` of X
        const int wt = tid - 16 * 32, r = wt & 127, half = wt >> 7;
        constexpr int kPieces = 4;                               // 16-byte pieces of half a row
        for (int c = 0; c < chunks; c++) {
            const int64_t t0 = seg.from + (int64_t)c * kChunk;
            const int valid = seg.to - t0 < kChunk ? (int)(seg.to - t0) : kChunk;
            const Scalars& sc = scal[c % 3];
            if (!wait3(B_SC, c) || !wait2(B_FULL, c)) break;
            unsigned char* const st = sm + (c & 1) * L::kStage;
            if (valid < kChunk) {
                // rows of other sequences or of nothing: zero, whatever they hold
                for (int i = wt; i < (kChunk - valid) * (N / 8 + 8); i += 256) {
                    const int q = valid + i / (N / 8 + 8), e = i % (N / 8 + 8);
                    unsigned char* at = e < N / 8 ? st + L::kB + e / 8 * 16384 + q * 128 + e % 8 * 16
                                                  : st + L::kXs + q * 128 + (e - N / 8) * 16;
                    *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
                }
                // the last chunk: the one phase of this barrier
                fence_async();
                warp_arrive(bars + B_WSYNC, lane);
                if (!wait(B_WSYNC, 0)) break;
            }
            float w = sc.behind[r];
#pragma unroll
            for (int u = 1; u < 4; u++)
                if (u > r / 32) w *= sc.block[u];
            // part k of the piece `v` (each remainder is exact), and a probe that is NaN
            // where x is not a finite number
            f2 probe = 0;
            auto split = [&](const uint4& v, uint4 (&o)[3]) {
                const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                uint32_t q[3][4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const f2 xv = bf_pair(in[i]);
                    probe = fma2(xv, 0ull, probe);
                    f2 t = mul2(xv, pair(w, w));
                    q[0][i] = pack_bf(t);
                    t = fma2(bf_pair(q[0][i]), pair(-1.0f, -1.0f), t);
                    q[1][i] = pack_bf(t);
                    q[2][i] = pack_bf(fma2(bf_pair(q[1][i]), pair(-1.0f, -1.0f), t));
                }
#pragma unroll
                for (int k = 0; k < 3; k++) o[k] = make_uint4(q[k][0], q[k][1], q[k][2], q[k][3]);
            };
            if (c >= 1 && !wait2(B_D, c - 1)) break;              // the last parts have been multiplied
            uint4 lo[kPieces];
#pragma unroll
            for (int e = 0; e < kPieces; e++) {
                const int at = swz(r, half * 4 + e);
                uint4 o[3];
                split(*reinterpret_cast<const uint4*>(st + L::kXs + at), o);
                *reinterpret_cast<uint4*>(sm + L::kW0 + at) = o[0];
                *reinterpret_cast<uint4*>(sm + L::kW1 + at) = o[1];
                lo[e] = o[2];
            }
            const float2 pr = unpair(probe);
            if (OUT && pr.x + pr.y != 0.0f) {
                // a non-finite x must not reach earlier rows through M's zeros: it
                // leaves X, and its column becomes NaN from its row on
                for (int e = 0; e < kPieces; e++)
                    for (int i = 0; i < 8; i++) {
                        uint16_t* at = reinterpret_cast<uint16_t*>(st + L::kXs + swz(r, half * 4 + e)) + i;
                        if ((*at & 0x7f80) == 0x7f80) {
                            *at = 0;
                            atomicMin(bad + (c & 1) * 64 + (half * 4 + e) * 8 + i, r);
                        }
                    }
            }
            fence_async();
            warp_arrive(bars + B_W01 + (c & 1), lane);
            // the third part's place is S's until S has been multiplied
            if (OUT && !wait(B_YO, c)) break;
#pragma unroll
            for (int e = 0; e < kPieces; e++) *reinterpret_cast<uint4*>(sm + L::kW2 + swz(r, half * 4 + e)) = lo[e];
            fence_async();
            warp_arrive(bars + B_W2, lane);
        }
    } else if (warp >= 8) {
        // ---------------------------------------------------- M: row `row`
        // (warps 8 to 11: the blocks left of its own; 12 to 15: its own, and the decays)
        const int row = quad * 32 + lane;
        const bool own = warp >= 12;
        const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
        auto fetch = [&](int c) {
            const int64_t t = seg.from + (int64_t)c * kChunk + row;
            // as it lies in memory: a conversion here would wait for the load
            if (t >= seg.to) return 0u;
            const int64_t i = t * p.dts + h;
            return p.dt_bf16 ? (uint32_t)__ldg(static_cast<const uint16_t*>(p.dt) + i) : __ldg(static_cast<const uint32_t*>(p.dt) + i);
        };
        uint32_t raw_dt = fetch(0);
        auto decays = [&](int c) {
            Scalars& sc = scal[c % 3];
            const bool in = seg.from + (int64_t)c * kChunk + row < seg.to;
            const float raw = __uint_as_float(p.dt_bf16 ? raw_dt << 16 : raw_dt);
            const float dt = in ? time_step(raw, bias, p.softplus) : 0.0f, a = in ? expf(dt * A) : 1.0f;
            float up = a, down = a;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float u = __shfl_up_sync(~0u, up, d), v = __shfl_down_sync(~0u, down, d);
                if (lane >= d) up *= u;
                if (lane + d < 32) down *= v;
            }
            float behind = __shfl_down_sync(~0u, down, 1);
            if (lane == 31) behind = 1.0f;
            sc.a[row] = a;
            sc.dt[row] = dt;
            sc.upto[row] = up;
            sc.behind[row] = behind * dt;
            if (lane == 31) sc.block[quad] = up;
            warp_arrive(bars + B_SC + c % 3, lane);
            raw_dt = fetch(c + 1);
        };
        for (int c = 0; c < 2 && c < chunks && own; c++) decays(c);
        // M of a chunk, then the decays two chunks ahead (three places: no one reads
        // this one any more)
        for (int c = 0; c < chunks; c++) {
            if constexpr (OUT) {
                const Scalars& sc = scal[c % 3];
                if (!wait3(B_SC, c) || !wait2(B_G, c) || (c > 0 && !wait(B_Y, c - 1))) break;
                tc_after();
#pragma unroll 1
                for (int b = 0; b < quad && !own; b++) {
                    float f = sc.upto[row];
#pragma unroll 1
                    for (int u = b + 1; u < quad; u++) f *= sc.block[u];
                    float v[2][16];
                    tm_load16(tq + kG + b * 32, tq + kG + b * 32 + 16, v[0], v[1]);
                    const float4* behind = reinterpret_cast<const float4*>(sc.behind + b * 32);
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        uint32_t o[8];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const float4 q = behind[e * 4 + j];
                            o[2 * j] = pack_bf(mul2(pair(v[e][4 * j], v[e][4 * j + 1]), mul2(pair(f, f), pair(q.x, q.y))));
                            o[2 * j + 1] = pack_bf(mul2(pair(v[e][4 * j + 2], v[e][4 * j + 3]), mul2(pair(f, f), pair(q.z, q.w))));
                        }
                        tm_store8(tq + kM + b * 16 + e * 8, o);
                    }
                }
                if (own) {
                    // its own block, from the right: P(row, j) for j = 31 .. 0
                    float v[2][16], e = 1.0f;
                    tm_load16(tq + kG + quad * 32, tq + kG + quad * 32 + 16, v[0], v[1]);
#pragma unroll
                    for (int b = 1; b >= 0; b--) {
                        const float4* dts = reinterpret_cast<const float4*>(sc.dt + quad * 32 + b * 16);
                        const float4* as = reinterpret_cast<const float4*>(sc.a + quad * 32 + b * 16);
                        uint32_t o[8];
#pragma unroll
                        for (int j = 3; j >= 0; j--) {
                            const float4 t4 = dts[j], a4 = as[j];
                            const float t[4] = {t4.x, t4.y, t4.z, t4.w}, a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                            for (int i = 3; i >= 0; i--) {
                                const bool in = b * 16 + 4 * j + i <= lane;
                                float& u = v[b][4 * j + i];
                                u = in ? u * (e * t[i]) : 0.0f;
                                e = in ? e * a[i] : e;
                            }
                            o[2 * j] = pack_bf(v[b][4 * j], v[b][4 * j + 1]);
                            o[2 * j + 1] = pack_bf(v[b][4 * j + 2], v[b][4 * j + 3]);
                        }
                        tm_store8(tq + kM + quad * 16 + b * 8, o);
                    }
                    {
                        const uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
                        for (int b = 2 * quad + 2; b < 8; b++) tm_store8(tq + kM + b * 8, o);
                    }
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_before();
                warp_arrive(bars + B_M, lane);
            }
            if (own && c + 2 < chunks) {
                if (c >= 1 && !wait2(B_E, c - 1)) break;
                decays(c + 2);
            }
        }
    } else {
        // ---------------------------------------------------- E: half of row `row` of S and of y
        const int row = quad * 32 + lane, half = warp >> 2;
        const bool holds = row < N;
        const float D = OUT && p.D ? p.D[h] : 0.0f;
        const int64_t tile = (int64_t)N * p.dv, mine = (int64_t)row * p.dv + c0 + half * 32;
        f2 S[16];
        {
            const float* from = nullptr;
            if (OUT && p.cut) from = p.seg_state + ((int64_t)blockIdx.x * p.heads + h) * tile + mine;
            else if (OUT && p.initial) from = p.state + ((int64_t)seg.sequence * p.heads + h) * tile + mine;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                float4 v = make_float4(0, 0, 0, 0);
                if (from && holds) v = *reinterpret_cast<const float4*>(from + 2 * i);
                S[i] = pair(v.x, v.y);
                S[i + 1] = pair(v.z, v.w);
            }
        }
        auto put_state = [&] {
            if (OUT && holds)
#pragma unroll
                for (int c = 0; c < 4; c++)
                    *reinterpret_cast<uint4*>(sm + L::kS + swz(row, half * 4 + c)) =
                        make_uint4(pack_bf(S[c * 4]), pack_bf(S[c * 4 + 1]), pack_bf(S[c * 4 + 2]), pack_bf(S[c * 4 + 3]));
            fence_async();
            tc_before();
            warp_arrive(bars + B_S, lane);
        };
        put_state();
        float total = 1.0f;
        for (int c = 0; c < chunks; c++) {
            const Scalars& sc = scal[c % 3];
            if (!wait3(B_SC, c) || !wait2(B_D, c)) break;
            tc_after();
            const float dec = sc.block[0] * sc.block[1] * (sc.block[2] * sc.block[3]);
            if (!OUT) total *= dec;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float v[16], o[16];
                tm_load16(tq + kD + half * 32 + e * 16, tq + kD + 64 + half * 32 + e * 16, v, o);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    S[e * 8 + i] = fma2(S[e * 8 + i], pair(dec, dec),
                                        add2(pair(v[2 * i], v[2 * i + 1]), pair(o[2 * i], o[2 * i + 1])));
            }
            put_state();
            if (!OUT) {
                // (not before the next decays: M, which no product waits for here, may
                // then not fall two phases of B_E behind)
                if (c + 1 < chunks && !wait3(B_SC, c + 1)) break;
                warp_arrive(bars + B_E + (c & 1), lane);
                continue;
            }
            float f = sc.upto[row];
#pragma unroll
            for (int u = 0; u < 3; u++)
                if (u < quad) f *= sc.block[u];
            // (the first two have passed; X is read here, as they left it)
            if (!wait2(B_FULL, c) || !wait2(B_W01, c) || !wait(B_Y, c)) break;
            tc_after();
            const unsigned char* const xs = sm + (c & 1) * L::kStage + L::kXs;
            const int64_t t = seg.from + (int64_t)c * kChunk + row;
            bf16* const y = static_cast<bf16*>(p.y) + t * p.ys + (int64_t)h * p.dv + c0 + half * 32;
            const bool wide = (reinterpret_cast<uintptr_t>(y) & 31) == 0;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                uint32_t out[8];
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    float v[8], o[8];
                    const uint32_t col = half * 32 + e * 16 + q * 8;
                    tm_load8(tq + kYo + (c & 1) * 64 + col, tq + kY + col, o, v);
                    const uint4 x4 = *reinterpret_cast<const uint4*>(xs + swz(row, half * 4 + e * 2 + q));
                    const uint32_t in[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const f2 u = fma2(pair(f, f), pair(o[2 * i], o[2 * i + 1]), pair(v[2 * i], v[2 * i + 1]));
                        out[q * 4 + i] = pack_bf(fma2(pair(D, D), bf_pair(in[i]), u));
                    }
                }
                if (t >= seg.to) continue;
                if (wide) {
                    store32(y + e * 16, out);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        reinterpret_cast<uint16_t*>(y)[e * 16 + 2 * i] = (uint16_t)out[i];
                        reinterpret_cast<uint16_t*>(y)[e * 16 + 2 * i + 1] = (uint16_t)(out[i] >> 16);
                    }
                }
            }
            // columns with a non-finite x, from its row on (128: none)
            const int b0 = bad[(c & 1) * 64 + half * 32 + lane];
            uint32_t nans = 0;                                   // of this row
            if (__any_sync(~0u, b0 < kChunk)) {
#pragma unroll 1
                for (int j = 0; j < 32; j++) nans |= (uint32_t)(row >= __shfl_sync(~0u, b0, j)) << j;
            }
            tc_before();
            warp_arrive(bars + B_E + (c & 1), lane);             // stage, decays, C S and M X have been read
            if (t < seg.to) {
#pragma unroll 1
                for (; nans; nans &= nans - 1) reinterpret_cast<uint16_t*>(y)[__ffs((int)nans) - 1] = 0x7fc0;
            }
        }
        if (!ok || *lost) {
            // a wait ran out: all of the segment is NaN
            total = __uint_as_float(0x7fc00000u);
#pragma unroll
            for (int i = 0; i < 16; i++) S[i] = pair(total, total);
            if (OUT)
                for (int64_t t = seg.from + row; t < seg.to; t += kChunk)
                    for (int i = 0; i < 32; i++)
                        static_cast<bf16*>(p.y)[t * p.ys + (int64_t)h * p.dv + c0 + half * 32 + i] = __float2bfloat16_rn(total);
        }
        float* to = nullptr;
        if (!OUT) to = p.seg_state + ((int64_t)blockIdx.x * p.heads + h) * tile + mine;
        else if (seg.last && p.state) to = p.state + ((int64_t)seg.sequence * p.heads + h) * tile + mine;
        if (to && holds) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 u = unpair(S[i]), v = unpair(S[i + 1]);
                *reinterpret_cast<float4*>(to + 2 * i) = make_float4(u.x, u.y, v.x, v.y);
            }
        }
        if (!OUT && tid == 0 && c0 == 0) p.seg_decay[(int64_t)blockIdx.x * p.heads + h] = total;
        tc_before();
    }
    if (!ok && lane == 0) *lost = 1;
    __syncthreads();
    if (tid == 0 && *lost) atomicAdd(&lost_ctas, 1ull);
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kTmem) : "memory");
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
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();          // none is left for the next call
            return nullptr;
        }
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
    chunk_kernel<N, OUT><<<grid, kThreads, bytes, st>>>(p, m[0], m[1], m[2]);
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

bool scan_timeouts(uint64_t* count, cudaStream_t st) {
    unsigned long long n = 0;
    if (cudaMemcpyFromSymbolAsync(&n, lost_ctas, sizeof(n), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    *count = n;
    return true;
}

}  // namespace qm
