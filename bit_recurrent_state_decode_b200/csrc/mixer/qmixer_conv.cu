// qmixer_conv.cu -- the short causal convolution over the channels of a layer,
// z_t = bias + sum_k w_k x_{t-W+1+k}, y = silu(z), for prompts and for single
// tokens.
//
// Bound: memory (each x read once, each y written once; 2 W + 4 operations an
// element).  A thread owns 16 bytes of channels (eight bf16, four binary32) of a
// walk of kWalk tokens, and has all of the walk's rows and the W - 1 in front of
// it on their way before the first is used; a warp holds 32 such neighbours, a CTA
// 4 walks in a row, so that the rows in front of a walk come from L1.  Eight prompts
// of 2048 tokens by 2304 channels take 34 us (4.4 TB/s); with 16 neighbours 36, with
// walks of 4 tokens 39 to 43, of 12 tokens 37; walks of 16 to 64 tokens with a moving
// window and four rows on their way took 41 to 53.
//
// State.  Sequence s continues from state[s] and leaves its last W - 1 rows
// there, in place.  One thread does both for its channels: the walk in which a
// sequence starts.  It also computes the sequence's first W - 1 tokens where
// they reach past its end, since no other thread may read a history that this
// one overwrites.
#include "qmixer_common.cuh"

namespace qm {

constexpr int kWalk = 8, kAcross = 32, kDown = 128 / kAcross;

struct ConvParams {
    const void* x;
    int64_t xs;
    const void* w;
    const void* bias;
    void* state;
    void* y;
    int64_t ys;
    Sequences seq;
    int channels, vecs;
    unsigned across;            // CTAs across the channels
    int64_t walks;
    bool initial, act;
    bool wide_taps;             // weight and bias on 16-byte boundaries
};

// V channels as they lie in memory: V * sizeof(T) = 16 bytes, or V = 1 for any
// alignment.
template <class T, int V> struct Raw;
template <> struct Raw<bf16, 8> {
    uint4 r;
    __device__ __forceinline__ void load(const bf16* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(f2 (&v)[4]) const {
        v[0] = bf_pair(r.x); v[1] = bf_pair(r.y); v[2] = bf_pair(r.z); v[3] = bf_pair(r.w);
    }
    __device__ static __forceinline__ void put(bf16* p, const f2 (&v)[4]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf(v[0]), pack_bf(v[1]), pack_bf(v[2]), pack_bf(v[3]));
    }
};
template <> struct Raw<float, 4> {
    float4 r;
    __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void get(f2 (&v)[2]) const {
        v[0] = pair(r.x, r.y);
        v[1] = pair(r.z, r.w);
    }
    __device__ static __forceinline__ void put(float* p, const f2 (&v)[2]) {
        const float2 a = unpair(v[0]), b = unpair(v[1]);
        *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
    }
};
template <class T> struct Raw<T, 1> {
    T r;
    __device__ __forceinline__ void load(const T* p) { r = *p; }
    __device__ __forceinline__ void get(f2 (&v)[1]) const { v[0] = pair(to_f32<T>(r), 0.0f); }
    __device__ static __forceinline__ void put(T* p, const f2 (&v)[1]) { *p = from_f32<T>(unpair(v[0]).x); }
};

// The same as pairs of binary32.
template <class T, int V> struct Vec {
    static constexpr int kP = (V + 1) / 2;
    f2 v[kP];
    __device__ __forceinline__ void from(const Raw<T, V>& r) { r.get(v); }
    __device__ __forceinline__ void load(const T* p) {
        Raw<T, V> r;
        r.load(p);
        r.get(v);
    }
    __device__ __forceinline__ void store(T* p) const { Raw<T, V>::put(p, v); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kP; i++) v[i] = 0;
    }
};

template <class T, int V, int W> struct Taps {
    static constexpr int kP = Vec<T, V>::kP;
    f2 w[W][kP], b[kP];
    __device__ __forceinline__ void load(const ConvParams& p, int c0) {
        const T* wt = static_cast<const T*>(p.w) + (int64_t)c0 * W;
        const T* bt = static_cast<const T*>(p.bias);
        float f[V * W], g[V];
        if (V > 1 && p.wide_taps) {
            // V W consecutive weights, 16 bytes at a time
#pragma unroll
            for (int i = 0; i < W; i++) {
                Vec<T, V> v;
                v.load(wt + i * V);
#pragma unroll
                for (int j = 0; j < V; j++) f[i * V + j] = j & 1 ? unpair(v.v[j / 2]).y : unpair(v.v[j / 2]).x;
            }
            Vec<T, V> v;
            v.zero();
            if (bt) v.load(bt + c0);
#pragma unroll
            for (int j = 0; j < V; j++) g[j] = j & 1 ? unpair(v.v[j / 2]).y : unpair(v.v[j / 2]).x;
        } else {
#pragma unroll
            for (int i = 0; i < V * W; i++) f[i] = to_f32<T>(wt[i]);
#pragma unroll
            for (int j = 0; j < V; j++) g[j] = bt ? to_f32<T>(bt[c0 + j]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kP; i++) {
            constexpr bool two = V > 1;
#pragma unroll
            for (int k = 0; k < W; k++) w[k][i] = pair(f[2 * i * W + k], two ? f[(two ? 2 * i + 1 : 0) * W + k] : 0.0f);
            b[i] = pair(g[2 * i], two ? g[two ? 2 * i + 1 : 0] : 0.0f);
        }
    }
    // rows h[0 .. W-2], then x
    __device__ __forceinline__ Vec<T, V> apply(const Vec<T, V> (&h)[W - 1], const Vec<T, V>& x, bool act) const {
        Vec<T, V> o;
#pragma unroll
        for (int i = 0; i < kP; i++) {
            f2 z = b[i];
#pragma unroll
            for (int k = 0; k < W - 1; k++) z = fma2(w[k][i], h[k].v[i], z);
            z = fma2(w[W - 1][i], x.v[i], z);
            o.v[i] = act ? silu2<T>(z) : z;
        }
        return o;
    }
};

template <class T, int V, int W>
__global__ void __launch_bounds__(128, 4) conv_kernel(const ConvParams p) {
    const int vec = int(blockIdx.x % p.across) * kAcross + threadIdx.x % kAcross;
    const int64_t walk = (int64_t)(blockIdx.x / p.across) * kDown + threadIdx.x / kAcross;
    if (vec >= p.vecs) return;
    const int c0 = vec * V;
    T* const st = static_cast<T*>(p.state);
    if (walk >= p.walks) {
        // one thread per sequence and channels: an empty sequence that starts
        // from zeros leaves zeros (no walk holds a token of it)
        const int64_t s = walk - p.walks;
        if (s < p.seq.n && st && !p.initial && p.seq.start((int)s + 1) <= p.seq.start((int)s)) {
            Vec<T, V> z;
            z.zero();
#pragma unroll
            for (int r = 0; r < W - 1; r++) z.store(st + (s * (W - 1) + r) * (int64_t)p.channels + c0);
        }
        return;
    }
    const T* const x = static_cast<const T*>(p.x) + c0;
    T* const y = static_cast<T*>(p.y) + c0;
    const int64_t stop = p.seq.start(p.seq.n);
    const int64_t t0 = walk * kWalk;
    int64_t t1 = t0 + kWalk < stop ? t0 + kWalk : stop;
    if (t0 >= t1) return;
    int s = sequence_at(p.seq, t0);
    int64_t t = t0, from = p.seq.start(s), to = p.seq.start(s + 1);
    Taps<T, V, W> taps;
    if (t - from >= W - 1 && t + kWalk <= to && t + kWalk <= stop) {
        // a whole walk inside its sequence
        Raw<T, V> r[kWalk + W - 1];
#pragma unroll
        for (int i = 0; i < kWalk + W - 1; i++) r[i].load(x + (t - (W - 1) + i) * p.xs);
        taps.load(p, c0);
        Vec<T, V> h[W - 1];
#pragma unroll
        for (int k = 0; k < W - 1; k++) h[k].from(r[k]);
#pragma unroll
        for (int i = 0; i < kWalk; i++) {
            Vec<T, V> v;
            v.from(r[W - 1 + i]);
            taps.apply(h, v, p.act).store(y + (t + i) * p.ys);
#pragma unroll
            for (int k = 0; k + 1 < W - 1; k++) h[k] = h[k + 1];
            h[W - 2] = v;
        }
        return;
    }
    taps.load(p, c0);
    if (t < from) t = from;              // tokens in front of the first sequence
    Vec<T, V> h[W - 1];
    if (t > from && t < to) {
        // inside a sequence: its first W - 1 tokens belong to the walk it starts in
        if (t - from < W - 1) t = from + W - 1 < to ? from + W - 1 : to;
#pragma unroll
        for (int r = 0; r < W - 1; r++) {
            const int64_t at = t - (W - 1) + r;
            if (t < t1 && at >= from) h[r].load(x + at * p.xs);
            else h[r].zero();
        }
    }
    while (t < t1) {
        while (t >= to && s + 1 < p.seq.n) {        // the next sequence that holds a token
            s++;
            from = p.seq.start(s);
            to = p.seq.start(s + 1);
            if (t < from) t = from;
        }
        if (t >= to || t >= t1) return;
        int64_t end = to < t1 ? to : t1;
        if (t == from) {
            T* const own = st ? st + (int64_t)s * (W - 1) * p.channels + c0 : nullptr;
#pragma unroll
            for (int r = 0; r < W - 1; r++) {
                if (p.initial) h[r].load(own + (int64_t)r * p.channels);
                else h[r].zero();
            }
            if (own) {
                Vec<T, V> last[W - 1];
#pragma unroll
                for (int r = 0; r < W - 1; r++) {
                    const int64_t at = to - (W - 1) + r;
                    if (at >= from) last[r].load(x + at * p.xs);
                    else {
                        last[r].zero();
#pragma unroll
                        for (int q = 0; q < W - 1; q++)     // row at - from of the history, from its end
                            if (at - from + (W - 1) == q) last[r] = h[q];
                    }
                }
#pragma unroll
                for (int r = 0; r < W - 1; r++) last[r].store(own + (int64_t)r * p.channels);
            }
            // its first W - 1 tokens, also past the end of this walk
            const int64_t least = from + W - 1 < to ? from + W - 1 : to;
            if (end < least) end = least;
        }
        for (; t < end; t++) {
            Vec<T, V> r;
            r.load(x + t * p.xs);
            taps.apply(h, r, p.act).store(y + t * p.ys);
#pragma unroll
            for (int k = 0; k + 1 < W - 1; k++) h[k] = h[k + 1];
            h[W - 2] = r;
        }
    }
}

// One token of each sequence: the state moves on by one row.
template <class T, int V, int W>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvParams p) {
    const int64_t id = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    const int64_t b = id / p.vecs;
    if (b >= p.seq.n) return;
    const int c0 = int(id % p.vecs) * V;
    T* const st = static_cast<T*>(p.state) + b * (W - 1) * p.channels + c0;
    Vec<T, V> h[W - 1], x;
#pragma unroll
    for (int r = 0; r < W - 1; r++) h[r].load(st + (int64_t)r * p.channels);
    x.load(static_cast<const T*>(p.x) + b * p.xs + c0);
    Taps<T, V, W> taps;
    taps.load(p, c0);
    taps.apply(h, x, p.act).store(static_cast<T*>(p.y) + b * p.ys + c0);
#pragma unroll
    for (int r = 0; r + 1 < W - 1; r++) h[r + 1].store(st + (int64_t)r * p.channels);
    x.store(st + (int64_t)(W - 2) * p.channels);
}

template <class T, int V, int W> void launch(const ConvParams& p, bool step, cudaStream_t st) {
    const int64_t walks = p.walks + (p.state && !p.initial ? p.seq.n : 0);
    const int64_t blocks = step ? ((int64_t)p.seq.n * p.vecs + 127) / 128 : (walks + kDown - 1) / kDown * p.across;
    if (!blocks) return;
    if (step) conv_step_kernel<T, V, W><<<(unsigned)blocks, 128, 0, st>>>(p);
    else conv_kernel<T, V, W><<<(unsigned)blocks, 128, 0, st>>>(p);
}

template <class T, int V> void launch_w(const ConvParams& p, int width, bool step, cudaStream_t st) {
    if (width == 2) launch<T, V, 2>(p, step, st);
    else if (width == 3) launch<T, V, 3>(p, step, st);
    else launch<T, V, 4>(p, step, st);
}

int conv_any(ConvParams& p, int width, int dtype, bool step, cudaStream_t st) {
    const int wide = dtype == QSTATE_BF16 ? 8 : 4;
    // 16-byte accesses need the channels, both strides and all bases to allow
    // them; else element by element
    const bool vec = p.channels % wide == 0 && p.xs % wide == 0 && p.ys % wide == 0 && aligned(p.x, 16) &&
                     aligned(p.y, 16) && aligned(p.state, 16);
    p.vecs = vec ? p.channels / wide : p.channels;
    p.wide_taps = aligned(p.w, 16) && aligned(p.bias, 16);
    p.walks = (p.seq.tokens + kWalk - 1) / kWalk;
    p.across = (unsigned)(((int64_t)p.vecs + kAcross - 1) / kAcross);
    if (((p.walks + p.seq.n) / kDown + 1) * p.across > INT32_MAX || (int64_t)p.seq.n * p.vecs / 128 >= INT32_MAX)
        return QSTATE_EUNSUPPORTED;
    if (dtype == QSTATE_BF16) {
        if (vec) launch_w<bf16, 8>(p, width, step, st);
        else launch_w<bf16, 1>(p, width, step, st);
    } else {
        if (vec) launch_w<float, 4>(p, width, step, st);
        else launch_w<float, 1>(p, width, step, st);
    }
    return launched();
}

}  // namespace qm

extern "C" {

int qmixer_conv(const qmixer_conv_args* args, qstate_stream stream) {
    if (!args) return QSTATE_EINVAL;
    const qmixer_conv_args& a = *args;
    if (!qm::known(a.dtype) || a.sequences < 0 || a.tokens < 0 || a.tokens > INT32_MAX || a.channels < 1 || a.width < 1)
        return QSTATE_EINVAL;
    if (a.flags & ~(QMIXER_INITIAL | QMIXER_SILU)) return QSTATE_EINVAL;
    if (a.x_stride < a.channels || a.y_stride < a.channels) return QSTATE_EINVAL;
    if (!a.seq_starts && a.sequences && a.tokens % a.sequences) return QSTATE_EINVAL;
    if ((a.flags & QMIXER_INITIAL) && !a.state && a.sequences) return QSTATE_EINVAL;
    const int size = qm::size_of(a.dtype);
    if (!qm::aligned(a.x, size) || !qm::aligned(a.y, size) || !qm::aligned(a.weight, size) || !qm::aligned(a.bias, size) ||
        !qm::aligned(a.state, size) || !qm::aligned(a.seq_starts, 4))
        return QSTATE_EINVAL;
    if (a.width < 2 || a.width > 4) return QSTATE_EUNSUPPORTED;
    if (!a.sequences || (!a.tokens && !a.state)) return QSTATE_OK;
    if (!a.weight || (a.tokens && (!a.x || !a.y))) return QSTATE_EINVAL;
    qm::ConvParams p{a.x, a.x_stride, a.weight, a.bias, a.state, a.y, a.y_stride,
                     {a.seq_starts, a.sequences, a.tokens, a.tokens / a.sequences}, a.channels, 0, 0, 0,
                     (a.flags & QMIXER_INITIAL) != 0, (a.flags & QMIXER_SILU) != 0, false};
    return qm::conv_any(p, a.width, a.dtype, false, (cudaStream_t)stream);
}

int qmixer_conv_step(const qmixer_conv_step_args* args, qstate_stream stream) {
    if (!args) return QSTATE_EINVAL;
    const qmixer_conv_step_args& a = *args;
    if (!qm::known(a.dtype) || a.batch < 0 || a.channels < 1 || a.width < 1 || (a.flags & ~QMIXER_SILU)) return QSTATE_EINVAL;
    if (a.x_stride < a.channels || a.y_stride < a.channels) return QSTATE_EINVAL;
    const int size = qm::size_of(a.dtype);
    if (!qm::aligned(a.x, size) || !qm::aligned(a.y, size) || !qm::aligned(a.weight, size) || !qm::aligned(a.bias, size) ||
        !qm::aligned(a.state, size))
        return QSTATE_EINVAL;
    if (a.width < 2 || a.width > 4) return QSTATE_EUNSUPPORTED;
    if (!a.batch) return QSTATE_OK;
    if (!a.x || !a.y || !a.weight || !a.state) return QSTATE_EINVAL;
    qm::ConvParams p{a.x, a.x_stride, a.weight, a.bias, a.state, a.y, a.y_stride, {nullptr, a.batch, a.batch, 1}, a.channels, 0, 0, 0,
                     false, (a.flags & QMIXER_SILU) != 0, false};
    return qm::conv_any(p, a.width, a.dtype, true, (cudaStream_t)stream);
}

}  // extern "C"
