// recurrence.cu -- the gated linear recurrence over time: forward, backward and one token.
//
//   ra = sigmoid(gate_a), rx = sigmoid(gate_x), a = exp(-kappa softplus(decay) ra),
//   h[t] = a[t] h[t-1] + sqrt(1 - a[t]^2) rx[t] x[t]
//
// per channel.  A run of rows acts on the state before it as h -> A h + H, with A the product
// of its a's and H its result from a zero state, and two runs join by
// (A1, H1), (A2, H2) -> (A1 A2, A2 H1 + H2): so the time axis is split.
//
// One work item is kRecChunk rows of kRecTile channels.  Its warps take equal runs of rows, a
// lane two channels; each scans its run from zero in registers, the runs' (A, H) meet in shared
// memory, and once the state in front of the item is known each warp scans again and writes.
// Items are handed out by a counter, early rows first, so an item only waits for items that are
// already running.  An item publishes its (A, H) as soon as it has them and the state behind
// it as soon as it knows the one before; the next item takes the nearest published state and
// applies the (A, H) after it, oldest first -- the same operations in the same order whichever
// state it found, so the result does not depend on timing.  A value is its own flag: both arrays
// start as all ones bits, which no published value has.
//
// Sequence starts inside an item are cuts: there A = 0, and joining selects instead of
// multiplying, so what a sequence holds (infinities and NaN too) never reaches its neighbour.
#include "ptx.cuh"
#include "sequence.cuh"

namespace conv2d_b200 {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// ----------------------------------------------------------- element access ---
// The two channels of a lane: adjacent (kVec: one load; even C, strides and base), or 32 apart.
template <typename T, bool kVec>
struct Lane2 {
    int c0, c1;
    bool ok0, ok1;
    __device__ Lane2(int tile, int C) {
        const int lane = threadIdx.x & 31;
        c0 = tile * kRecTile + (kVec ? 2 * lane : lane);
        c1 = c0 + (kVec ? 1 : 32);
        ok0 = c0 < C;
        ok1 = c1 < C;
    }
};

template <typename T> struct Raw2;
template <> struct Raw2<float> {
    float2 v;
    __device__ float2 get() const { return v; }
};
template <> struct Raw2<__nv_bfloat16> {
    uint32_t v;
    __device__ float2 get() const { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
};

template <typename T, bool kVec>
__device__ __forceinline__ Raw2<T> load2(const T *row, const Lane2<T, kVec> &l) {
    Raw2<T> r;
    if constexpr (sizeof(T) == 4) {
        if constexpr (kVec) {
            r.v = l.ok0 ? __ldcs(reinterpret_cast<const float2 *>(row + l.c0)) : make_float2(0.f, 0.f);
        } else {
            r.v.x = l.ok0 ? __ldcs(row + l.c0) : 0.f;
            r.v.y = l.ok1 ? __ldcs(row + l.c1) : 0.f;
        }
    } else {
        if constexpr (kVec) {
            r.v = l.ok0 ? __ldcs(reinterpret_cast<const uint32_t *>(row + l.c0)) : 0u;
        } else {
            const uint16_t *u = reinterpret_cast<const uint16_t *>(row);
            r.v = (l.ok0 ? u[l.c0] : 0u) | (l.ok1 ? static_cast<uint32_t>(u[l.c1]) << 16 : 0u);
        }
    }
    return r;
}

template <typename T, bool kVec>
__device__ __forceinline__ void store2(T *row, float2 f, const Lane2<T, kVec> &l) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (kVec) {
            if (l.ok0) __stcs(reinterpret_cast<float2 *>(row + l.c0), f);
        } else {
            if (l.ok0) row[l.c0] = f.x;
            if (l.ok1) row[l.c1] = f.y;
        }
    } else {
        if constexpr (kVec) {
            const __nv_bfloat162 h = __float22bfloat162_rn(f);
            if (l.ok0) __stcs(reinterpret_cast<uint32_t *>(row + l.c0), *reinterpret_cast<const uint32_t *>(&h));
        } else {
            if (l.ok0) row[l.c0] = __float2bfloat16_rn(f.x);
            if (l.ok1) row[l.c1] = __float2bfloat16_rn(f.y);
        }
    }
}

template <typename T, bool kVec>
__device__ __forceinline__ float2 load_f32(const float *row, const Lane2<T, kVec> &l) {
    return row ? make_float2(l.ok0 ? row[l.c0] : 0.f, l.ok1 ? row[l.c1] : 0.f) : make_float2(0.f, 0.f);
}
template <typename T, bool kVec>
__device__ __forceinline__ void store_f32(float *row, float2 f, const Lane2<T, kVec> &l) {
    if (l.ok0) row[l.c0] = f.x;
    if (l.ok1) row[l.c1] = f.y;
}

// ----------------------------------------------------------------- the gates ---
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// log2(a) per unit of ra: -kappa softplus(decay) log2(e).
template <typename T, bool kVec>
__device__ __forceinline__ float2 decay_rate(const float *decay, float kappa, const Lane2<T, kVec> &l) {
    const float2 d = load_f32(decay, l);
    return make_float2(-kappa * kLog2e * softplus(d.x), -kappa * kLog2e * softplus(d.y));
}

__device__ __forceinline__ float2 sigmoid2(float2 z) {
    const float2 t = mul2(z, splat(-kLog2e));
    const float2 d = add2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), splat(1.f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

// 2^y - 1 for y <= 0, exact to a few units of the result also where it is small: with
// y = n + f, |f| <= 1/2, it is 2^n (2^f - 1) + (2^n - 1).  2^f - 1 is f times the polynomial of
// degree 5 that interpolates (2^f - 1)/f at the Chebyshev points of [-1/2, 1/2] (2e-8 off).
// A decay a = 1 + p that is a little below 1 is applied thousands of times, so an approximate
// exponential, biased by a unit or two, would not do.  (No special-function unit is used either:
// the sigmoids keep that one busy.)
__device__ __forceinline__ float2 exp2m1(float2 y) {
    y = make_float2(fmaxf(y.x, -126.f), fmaxf(y.y, -126.f));
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number in the low bits
    const float2 r = add2(y, splat(kRound));
    const float2 f = add2(y, mul2(add2(r, splat(-kRound)), splat(-1.f)));
    const float2 s = make_float2(__int_as_float((__float_as_int(r.x) << 23) + 0x3f800000),
                                 __int_as_float((__float_as_int(r.y) << 23) + 0x3f800000));
    float2 q = fma2(f, splat(0.00015453163f), splat(0.0013390863f));
    q = fma2(f, q, splat(0.009618083f));
    q = fma2(f, q, splat(0.05550357f));
    q = fma2(f, q, splat(0.2402265f));
    q = fma2(f, q, splat(0.6931472f));
    q = mul2(f, q);
    return fma2(s, q, add2(s, splat(-1.f)));
}

// From p = a - 1: beta = sqrt(1 - a^2) and its reciprocal.  1 - a^2 = -p (2 + p) has no
// cancellation.  Both are 0 where a is 1 to within 1e-37: such a row adds nothing.
__device__ __forceinline__ void beta_of(float2 p, float2 &beta, float2 &inv) {
    const float2 v = mul2(mul2(p, splat(-1.f)), add2(p, splat(2.f)));
    inv = make_float2(v.x > 1e-37f ? rsqrt_approx(v.x) : 0.f, v.y > 1e-37f ? rsqrt_approx(v.y) : 0.f);
    if (v.x != v.x) inv.x = v.x;
    if (v.y != v.y) inv.y = v.y;
    beta = mul2(v, inv);
}

// ------------------------------------------------------------------ joining ---
// The state behind a run (A, H) that h enters; a run with a cut (A = 0) forgets h, whatever it is.
__device__ __forceinline__ float after(float A, float H, float h) { return A == 0.f ? H : fmaf(A, h, H); }

__device__ __forceinline__ float no_flag(float v) { return v == v ? v : __int_as_float(0x7fc00000); }

__device__ __forceinline__ void publish(float *at, float v) {
    asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(at), "f"(no_flag(v)) : "memory");
}
__device__ __forceinline__ void publish(float2 *at, float a, float h) {
    const uint64_t w = static_cast<uint64_t>(__float_as_uint(no_flag(h))) << 32 | __float_as_uint(no_flag(a));
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(at), "l"(w) : "memory");
}
__device__ __forceinline__ uint32_t peek(const float *at) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t peek(const float2 *at) {
    uint64_t v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(at) : "memory");
    return v;
}

// Waits, as one warp, for what item `chunk` has published: its carry (returned with A = 0), or
// its (A, H) unless only the carry will do.  After the time limit it reports and returns zeros.
template <typename T, bool kVec>
__device__ __forceinline__ float4 await_item(const RecParams &p, int chunk, bool carry_only, const Lane2<T, kVec> &l) {
    const size_t at = static_cast<size_t>(chunk) * p.Cpad;
    uint64_t start = 0;
    for (unsigned i = 0;; ++i) {
        const uint32_t c0 = peek(p.carry + at + l.c0), c1 = peek(p.carry + at + l.c1);
        const uint64_t a0 = peek(p.aggregate + at + l.c0), a1 = peek(p.aggregate + at + l.c1);
        if (__all_sync(kFull, c0 != kFull && c1 != kFull))
            return make_float4(0.f, __uint_as_float(c0), 0.f, __uint_as_float(c1));
        if (!carry_only && __all_sync(kFull, static_cast<uint32_t>(a0) != kFull && static_cast<uint32_t>(a1) != kFull))
            return make_float4(__uint_as_float(static_cast<uint32_t>(a0)), __uint_as_float(a0 >> 32),
                               __uint_as_float(static_cast<uint32_t>(a1)), __uint_as_float(a1 >> 32));
        if ((i & 63u) == 63u) {
            const uint64_t now = __shfl_sync(kFull, ptx::globaltimer_ns(), 0);
            if (!start) start = now;
            else if (now - start > static_cast<uint64_t>(p.timeout_ns)) {
                if ((threadIdx.x & 31) == 0) atomicExch(p.status, kDevTimeoutCarry);
                return make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    }
}

// What the rows row0 .. row0+L-1 of one warp are, a bit each; `seq` of lane j is row j's sequence.
struct Run {
    unsigned in, start, end;
    int seq;
};

template <int L>
__device__ __forceinline__ Run run_of(const Sequences &q, int row0) {
    const int lane = threadIdx.x & 31, row = row0 + lane;
    Run r;
    r.seq = 0;
    bool in = false, start = false, end = false;
    if (lane < L && row < q.rows) {
        const int s = seq_of(q, row);
        if (s >= 0) {
            const int b = seq_begin(q, s), e = seq_begin(q, s + 1);
            in = row < e;
            start = in && row == b;
            end = in && row + 1 == e;
            r.seq = s;
        }
    }
    r.in = __ballot_sync(kFull, in);
    r.start = __ballot_sync(kFull, start);
    r.end = __ballot_sync(kFull, end);
    return r;
}

// Whether a sequence begins or ends inside the chunk, or rows of it belong to none: then its rows are looked at one by
// one.  The same for all threads of the block.
__device__ __forceinline__ bool has_edges(const Sequences &q, int chunk) {
    const int row0 = chunk * kRecChunk, s = seq_of(q, row0);
    return s < 0 || seq_begin(q, s) >= row0 || seq_begin(q, s + 1) <= row0 + kRecChunk;
}

__device__ __forceinline__ const float *seq_row(const float *base, const Run &r, int j, int C) {
    const int s = __shfl_sync(kFull, r.seq, j);
    return base ? base + static_cast<size_t>(s) * C : nullptr;
}

// Takes the next item; all threads of the block get it.  Without a counter (one chunk: nothing
// waits for anything) the items are dealt out in turn.
__device__ __forceinline__ unsigned take_item(const RecParams &p, unsigned *shared) {
    __syncthreads();
    if (threadIdx.x == 0) {
        if (p.ticket) *shared = atomicAdd(p.ticket, 1u) + 1u;
        else *shared += gridDim.x;
    }
    __syncthreads();
    return *shared;
}

// The state that enters a chunk: the nearest published carry of the `n` chunks in front of it
// (the warps wait for one each), and the (A, H) of those after it, oldest first.  step: +1 where
// the chunk in front of chunk k is k-1, -1 where it is k+1.
template <typename T, bool kVec, int W>
__device__ __forceinline__ float2 carry_in(const RecParams &p, int chunk, int before, int step, float4 (*s_prev)[32],
                                           int *s_known, const Lane2<T, kVec> &l) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float4 got = make_float4(0.f, 0.f, 0.f, 0.f);
    if (warp < before) got = await_item(p, chunk - step * (warp + 1), warp == W - 1, l);
    s_prev[warp][lane] = got;
    const bool known = __all_sync(kFull, got.x == 0.f && got.z == 0.f);
    if (lane == 0) s_known[warp] = known;
    __syncthreads();
    int j = 0;
    while (j < W - 1 && !s_known[j]) ++j;
    float2 h = splat(0.f);
    for (; j >= 0; --j) {
        const float4 r = s_prev[j][lane];
        h = make_float2(after(r.x, r.y, h.x), after(r.z, r.w, h.y));
    }
    return h;
}

// ------------------------------------------------------------------ forward ---
template <typename T, bool kVec, int W, int L, bool kEdge>
__device__ __forceinline__ void forward_item(const RecParams &p, int chunk, const Lane2<T, kVec> &l, const Run &run,
                                             float4 (*s_run)[32], float4 (*s_prev)[32], int *s_known) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = chunk * kRecChunk + warp * L;
    const T *px = static_cast<const T *>(p.x) + static_cast<size_t>(row0) * p.ldx;
    const T *pa = static_cast<const T *>(p.ga) + static_cast<size_t>(row0) * p.lda;
    const T *pg = static_cast<const T *>(p.gx) + static_cast<size_t>(row0) * p.ldg;
    Raw2<T> rx[L], ra[L], rg[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
        if (!kEdge || (run.in >> j & 1u)) {
            ra[j] = load2<T, kVec>(pa + j * p.lda, l);
            rg[j] = load2<T, kVec>(pg + j * p.ldg, l);
            rx[j] = load2<T, kVec>(px + j * p.ldx, l);
        }
    }
    const float2 rate = decay_rate(p.decay, p.kappa, l);
    float2 a[L], b[L];
    float2 A = splat(1.f), H = splat(0.f);
#pragma unroll
    for (int j = 0; j < L; ++j) {
        if (kEdge && !(run.in >> j & 1u)) {
            a[j] = b[j] = A = H = splat(0.f);
            continue;
        }
        const float2 pm = exp2m1(mul2(rate, sigmoid2(ra[j].get())));
        float2 beta, inv;
        beta_of(pm, beta, inv);
        a[j] = add2(pm, splat(1.f));
        b[j] = mul2(mul2(beta, sigmoid2(rg[j].get())), rx[j].get());
        if (kEdge && (run.start >> j & 1u)) {
            const float2 h0 = load_f32(seq_row(p.state, run, j, p.C), l);
            b[j] = fma2(a[j], h0, b[j]);
            A = splat(0.f);
            H = b[j];
        } else {
            A = mul2(A, a[j]);
            H = fma2(a[j], H, b[j]);
        }
    }
    s_run[warp][lane] = make_float4(A.x, H.x, A.y, H.y);
    if (warp == 0 && lane == 0) s_known[W] = chunk > 0 && (run.in & 1u) && !(run.start & 1u);
    __syncthreads();
    const bool needed = s_known[W];  // whether the state of the rows in front enters this chunk
    const size_t at = static_cast<size_t>(chunk) * p.Cpad;
    float4 all = make_float4(1.f, 0.f, 1.f, 0.f);
    if (warp == W - 1 && chunk + 1 < p.chunks) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float4 r = s_run[w][lane];
            all = make_float4(all.x * r.x, after(r.x, r.y, all.y), all.z * r.z, after(r.z, r.w, all.w));
        }
        if (needed && !p.starve) {
            publish(p.aggregate + at + l.c0, all.x, all.y);
            publish(p.aggregate + at + l.c1, all.z, all.w);
        }
    }
    float2 h = splat(0.f);
    if (needed) h = carry_in<T, kVec, W>(p, chunk, chunk, 1, s_prev, s_known, l);
    if (warp == W - 1 && chunk + 1 < p.chunks && !p.starve) {
        publish(p.carry + at + l.c0, after(all.x, all.y, h.x));
        publish(p.carry + at + l.c1, after(all.z, all.w, h.y));
    }
    for (int w = 0; w < warp; ++w) {
        const float4 r = s_run[w][lane];
        h = make_float2(after(r.x, r.y, h.x), after(r.z, r.w, h.y));
    }
    T *py = static_cast<T *>(p.y) + static_cast<size_t>(row0) * p.ldy;
#pragma unroll
    for (int j = 0; j < L; ++j) {
        if (kEdge && !(run.in >> j & 1u)) continue;
        h = kEdge && (run.start >> j & 1u) ? b[j] : fma2(a[j], h, b[j]);
        store2<T, kVec>(py + j * p.ldy, h, l);
        if (kEdge && (run.end >> j & 1u) && p.final_state)
            store_f32(const_cast<float *>(seq_row(p.final_state, run, j, p.C)), h, l);
    }
}

// What a state leaves of an empty sequence: itself.
template <typename T, bool kVec>
__device__ __forceinline__ void copy_empty(const Sequences &q, const float *from, float *to, int C, const Lane2<T, kVec> &l) {
    if (!to) return;
    for (int s = threadIdx.x >> 5; s < q.nseq; s += blockDim.x >> 5)
        if (seq_begin(q, s + 1) <= seq_begin(q, s))
            store_f32(to + static_cast<size_t>(s) * C, load_f32(from ? from + static_cast<size_t>(s) * C : nullptr, l), l);
}

template <typename T, bool kVec, int W, int L>
__global__ void __launch_bounds__(W * 32, 1) rec_forward_kernel(const __grid_constant__ RecParams p) {
    static_assert(W * L == kRecChunk, "a run of L rows per warp");
    __shared__ float4 s_run[W][32], s_prev[W][32];
    __shared__ int s_known[W + 1];
    __shared__ unsigned s_item;
    if (threadIdx.x == 0) s_item = blockIdx.x - gridDim.x;
    const int warp = threadIdx.x >> 5;
    for (;;) {
        const unsigned item = take_item(p, &s_item);
        if (item >= static_cast<unsigned>(p.chunks) * p.tiles) break;
        const int chunk = item / p.tiles, tile = item - chunk * p.tiles;
        const Lane2<T, kVec> l(tile, p.C);
        if (item == 0) check_offsets(p.seq, p.status);
        if (chunk == 0) copy_empty<T, kVec>(p.seq, p.state, p.final_state, p.C, l);
        if (has_edges(p.seq, chunk))
            forward_item<T, kVec, W, L, true>(p, chunk, l, run_of<L>(p.seq, chunk * kRecChunk + warp * L), s_run, s_prev,
                                              s_known);
        else
            forward_item<T, kVec, W, L, false>(p, chunk, l, Run{~0u, 0u, 0u, 0}, s_run, s_prev, s_known);
    }
}

// ----------------------------------------------------------------- backward ---
// With g[t] the gradient of h[t] through everything after it, G[t] = a[t] g[t] is what enters row
// t-1: G[t] = a[t] (dh[t] + G[t+1]), the same kind of recurrence backwards.  The states are
// computed again from the forward pass's carries.  Per row, with w = ra d/d(log a):
//   dx = g beta rx, d_gate_x = g beta x rx (1-rx), w = a g (h[t-1] - a rx x / beta) ra,
//   d_gate_a = -kappa softplus(decay) w (1-ra), d_decay = -kappa sigmoid(decay) sum w.
template <typename T, bool kVec, int W, int L, bool kEdge>
__device__ __forceinline__ float2 backward_item(const RecParams &p, int chunk, const Lane2<T, kVec> &l, const Run &run,
                                                float4 (*s_run)[32], float4 (*s_back)[32], float4 (*s_prev)[32],
                                                int *s_known) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = chunk * kRecChunk + warp * L;
    const T *px = static_cast<const T *>(p.x) + static_cast<size_t>(row0) * p.ldx;
    const T *pa = static_cast<const T *>(p.ga) + static_cast<size_t>(row0) * p.lda;
    const T *pg = static_cast<const T *>(p.gx) + static_cast<size_t>(row0) * p.ldg;
    const T *pd = static_cast<const T *>(p.dy) + static_cast<size_t>(row0) * p.lddy;
    const size_t at = static_cast<size_t>(chunk) * p.Cpad;
    Raw2<T> x[L], dh[L];
    float2 pm[L], ra[L], rx[L], bh[L];  // a - 1, the gates, and first b, then h[t-1]
    {
        Raw2<T> qa[L], qg[L];
#pragma unroll
        for (int j = 0; j < L; ++j) {
            if (!kEdge || (run.in >> j & 1u)) {
                qa[j] = load2<T, kVec>(pa + j * p.lda, l);
                qg[j] = load2<T, kVec>(pg + j * p.ldg, l);
                x[j] = load2<T, kVec>(px + j * p.ldx, l);
                dh[j] = load2<T, kVec>(pd + j * p.lddy, l);
            }
        }
        const float2 rate = decay_rate(p.decay, p.kappa, l);
#pragma unroll
        for (int j = 0; j < L; ++j) {
            if (kEdge && !(run.in >> j & 1u)) continue;
            ra[j] = sigmoid2(qa[j].get());
            rx[j] = sigmoid2(qg[j].get());
            pm[j] = exp2m1(mul2(rate, ra[j]));
            float2 beta, inv;
            beta_of(pm[j], beta, inv);
            bh[j] = mul2(mul2(beta, rx[j]), x[j].get());
        }
    }
    float2 A = splat(1.f), H = splat(0.f), B = splat(1.f), S = splat(0.f);
#pragma unroll
    for (int j = 0; j < L; ++j) {
        if (kEdge && !(run.in >> j & 1u)) {
            A = H = splat(0.f);
            continue;
        }
        const float2 a = add2(pm[j], splat(1.f));
        if (kEdge && (run.start >> j & 1u)) {
            H = fma2(a, load_f32(seq_row(p.state, run, j, p.C), l), bh[j]);
            A = splat(0.f);
        } else {
            H = fma2(a, H, bh[j]);
            A = mul2(A, a);
        }
    }
    if (!kEdge) B = A;
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
        if (kEdge && !(run.in >> j & 1u)) {
            B = S = splat(0.f);
            continue;
        }
        const float2 a = add2(pm[j], splat(1.f));
        if (kEdge && (run.end >> j & 1u)) {
            S = mul2(a, add2(dh[j].get(), load_f32(seq_row(p.d_final, run, j, p.C), l)));
            B = splat(0.f);
        } else {
            S = mul2(a, add2(dh[j].get(), S));
            if (kEdge) B = mul2(B, a);
        }
    }
    s_run[warp][lane] = make_float4(A.x, H.x, A.y, H.y);
    s_back[warp][lane] = make_float4(B.x, S.x, B.y, S.y);
    if (lane == 0) {
        if (warp == 0) s_known[W + 1] = chunk > 0 && (run.in & 1u) && !(run.start & 1u);
        if (warp == W - 1) s_known[W] = chunk + 1 < p.chunks && (run.in >> (L - 1) & 1u) && !(run.end >> (L - 1) & 1u);
    }
    __syncthreads();
    const bool needed = s_known[W];  // whether the rows behind this chunk send a gradient into it
    float4 all = make_float4(1.f, 0.f, 1.f, 0.f);
    if (warp == 0 && chunk > 0) {
#pragma unroll
        for (int w = W - 1; w >= 0; --w) {
            const float4 r = s_back[w][lane];
            all = make_float4(all.x * r.x, after(r.x, r.y, all.y), all.z * r.z, after(r.z, r.w, all.w));
        }
        if (needed && !p.starve) {
            publish(p.aggregate + at + l.c0, all.x, all.y);
            publish(p.aggregate + at + l.c1, all.z, all.w);
        }
    }
    // the states again
    float2 h = splat(0.f);
    if (s_known[W + 1]) {
        const float *saved = p.saved + at - p.Cpad;
        h = make_float2(saved[l.c0], saved[l.c1]);
    }
    for (int w = 0; w < warp; ++w) {
        const float4 r = s_run[w][lane];
        h = make_float2(after(r.x, r.y, h.x), after(r.z, r.w, h.y));
    }
#pragma unroll
    for (int j = 0; j < L; ++j) {
        if (kEdge && !(run.in >> j & 1u)) continue;
        if (kEdge && (run.start >> j & 1u)) h = load_f32(seq_row(p.state, run, j, p.C), l);
        const float2 b = bh[j];
        bh[j] = h;
        h = fma2(add2(pm[j], splat(1.f)), h, b);
    }
    float2 G = splat(0.f);
    if (needed) G = carry_in<T, kVec, W>(p, chunk, p.chunks - 1 - chunk, -1, s_prev, s_known, l);
    if (warp == 0 && chunk > 0 && !p.starve) {
        publish(p.carry + at + l.c0, after(all.x, all.y, G.x));
        publish(p.carry + at + l.c1, after(all.z, all.w, G.y));
    }
    for (int w = W - 1; w > warp; --w) {
        const float4 r = s_back[w][lane];
        G = make_float2(after(r.x, r.y, G.x), after(r.z, r.w, G.y));
    }
    const float2 rate = mul2(decay_rate(p.decay, p.kappa, l), splat(1.f / kLog2e));
    T *ox = static_cast<T *>(p.y) + static_cast<size_t>(row0) * p.ldy;
    T *oa = static_cast<T *>(p.dga) + static_cast<size_t>(row0) * p.ld_da;
    T *og = static_cast<T *>(p.dgx) + static_cast<size_t>(row0) * p.ld_dg;
    float2 sum = splat(0.f);
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
        if (kEdge && !(run.in >> j & 1u)) continue;
        if (kEdge && (run.end >> j & 1u)) G = load_f32(seq_row(p.d_final, run, j, p.C), l);
        const float2 a = add2(pm[j], splat(1.f));
        const float2 g = add2(dh[j].get(), G);
        G = mul2(a, g);
        float2 beta, inv;
        beta_of(pm[j], beta, inv);
        const float2 xv = x[j].get();
        const float2 dx = mul2(g, mul2(beta, rx[j]));
        const float2 minus_ra = mul2(ra[j], splat(-1.f)), minus_rx = mul2(rx[j], splat(-1.f));
        const float2 dg = mul2(mul2(dx, xv), add2(minus_rx, splat(1.f)));
        const float2 w = mul2(mul2(G, ra[j]), fma2(mul2(a, inv), mul2(minus_rx, xv), bh[j]));
        sum = add2(sum, w);
        const float2 da = mul2(mul2(rate, w), add2(minus_ra, splat(1.f)));
        store2<T, kVec>(ox + j * p.ldy, dx, l);
        store2<T, kVec>(oa + j * p.ld_da, da, l);
        store2<T, kVec>(og + j * p.ld_dg, dg, l);
        if (kEdge && (run.start >> j & 1u) && p.d_state)
            store_f32(const_cast<float *>(seq_row(p.d_state, run, j, p.C)), G, l);
    }
    return sum;
}

template <typename T, bool kVec, int W, int L>
__global__ void __launch_bounds__(W * 32, 1) rec_backward_kernel(const __grid_constant__ RecParams p) {
    static_assert(W * L == kRecChunk, "a run of L rows per warp");
    __shared__ float4 s_run[W][32], s_back[W][32], s_prev[W][32];
    __shared__ float2 s_sum[W][32];
    __shared__ int s_known[W + 2];
    __shared__ unsigned s_item;
    if (threadIdx.x == 0) s_item = blockIdx.x - gridDim.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (;;) {
        const unsigned item = take_item(p, &s_item);
        if (item >= static_cast<unsigned>(p.chunks) * p.tiles) break;
        const int chunk = p.chunks - 1 - static_cast<int>(item / p.tiles), tile = item % p.tiles;
        const Lane2<T, kVec> l(tile, p.C);
        if (item == 0) check_offsets(p.seq, p.status);
        if (chunk == 0) copy_empty<T, kVec>(p.seq, p.d_final, p.d_state, p.C, l);
        if (has_edges(p.seq, chunk))
            s_sum[warp][lane] = backward_item<T, kVec, W, L, true>(
                p, chunk, l, run_of<L>(p.seq, chunk * kRecChunk + warp * L), s_run, s_back, s_prev, s_known);
        else
            s_sum[warp][lane] = backward_item<T, kVec, W, L, false>(p, chunk, l, Run{~0u, 0u, 0u, 0}, s_run, s_back,
                                                                    s_prev, s_known);
        __syncthreads();
        if (warp == 0) {  // the chunk's sum of w, its warps' in order
            float2 sum = splat(0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) sum = add2(sum, s_sum[w][lane]);
            float *out = p.decay_partial + static_cast<size_t>(chunk) * p.Cpad;
            out[l.c0] = sum.x;
            out[l.c1] = sum.y;
        }
    }
}

// d_decay[c] = -kappa sigmoid(decay[c]) times the sum over chunks, in 64 bits: 32 channels and 32 groups of chunks
// per block.
__global__ void __launch_bounds__(1024) rec_decay_kernel(const float *partial, const float *decay, float kappa,
                                                         float *d_decay, int chunks, int C, int Cpad) {
    __shared__ double s_sum[32][33];
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    double sum = 0.0;
    if (c < C)
        for (int k = group; k < chunks; k += 32) sum += partial[static_cast<size_t>(k) * Cpad + c];
    s_sum[group][lane] = sum;
    __syncthreads();
    sum = s_sum[lane][group];
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    const int out = blockIdx.x * 32 + group;
    if (lane == 0 && out < C) {
        const double v = decay[out];
        d_decay[out] = static_cast<float>(-static_cast<double>(kappa) * sum / (1.0 + exp(-v)));
    }
}

// All ones in the counter and the arrays whose values are their own flags.
__global__ void __launch_bounds__(256) rec_init_kernel(uint32_t *a, size_t na, uint32_t *b, size_t nb) {
    const size_t step = static_cast<size_t>(gridDim.x) * blockDim.x;
    for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < na + nb; i += step)
        (i < na ? a : b - na)[i] = kFull;
}

// One token: a block takes 256 channels of one row.
template <typename T, bool kVec>
__global__ void __launch_bounds__(128) rec_step_kernel(const __grid_constant__ RecStepParams p) {
    const int b = blockIdx.x / p.tiles;
    const Lane2<T, kVec> l(blockIdx.x % p.tiles * 4 + (threadIdx.x >> 5), p.C);
    const int slot = p.slots ? p.slots[b] : b;
    const float2 x = load2<T, kVec>(static_cast<const T *>(p.x) + static_cast<size_t>(b) * p.ldx, l).get();
    const float2 ga = load2<T, kVec>(static_cast<const T *>(p.ga) + static_cast<size_t>(b) * p.lda, l).get();
    const float2 gx = load2<T, kVec>(static_cast<const T *>(p.gx) + static_cast<size_t>(b) * p.ldg, l).get();
    const float2 rate = decay_rate(p.decay, p.kappa, l);
    if (slot < 0 || slot >= p.pool) return;
    float *state = p.state + static_cast<size_t>(slot) * p.C;
    const float2 h0 = load_f32(state, l);
    if (p.slots && slot_named_before(p.slots, b, slot)) {
        if (threadIdx.x == 0) atomicExch(p.status, kDevBadSlot);
        return;
    }
    const float2 pm = exp2m1(mul2(rate, sigmoid2(ga)));
    float2 beta, inv;
    beta_of(pm, beta, inv);
    const float2 h = fma2(add2(pm, splat(1.f)), h0, mul2(mul2(beta, sigmoid2(gx)), x));
    store2<T, kVec>(static_cast<T *>(p.y) + static_cast<size_t>(b) * p.ldy, h, l);
    store_f32(state, h, l);
}

template <typename K>
cudaError_t launch_items(K kernel, const RecParams &p, int threads, int sms, cudaStream_t s) {
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0);
    if (e != cudaSuccess) return e;
    const long long items = static_cast<long long>(p.chunks) * p.tiles;
    const long long room = static_cast<long long>(per_sm < 1 ? 1 : per_sm) * sms;
    kernel<<<static_cast<int>(items < room ? items : room), threads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rec_init(const RecParams &p, size_t words, float *carry, size_t carry_words, cudaStream_t s) {
    const size_t blocks = (words + carry_words + 1023) / 1024;
    rec_init_kernel<<<static_cast<int>(blocks < 592 ? blocks : 592), 256, 0, s>>>(
        p.ticket, words, reinterpret_cast<uint32_t *>(carry), carry_words);
    return cudaGetLastError();
}

cudaError_t launch_rec_forward(const RecParams &p, bool f32, bool vec, int sms, cudaStream_t s) {
    if (f32) return vec ? launch_items(rec_forward_kernel<float, true, 16, 8>, p, 512, sms, s)
                        : launch_items(rec_forward_kernel<float, false, 16, 8>, p, 512, sms, s);
    return vec ? launch_items(rec_forward_kernel<__nv_bfloat16, true, 16, 8>, p, 512, sms, s)
               : launch_items(rec_forward_kernel<__nv_bfloat16, false, 16, 8>, p, 512, sms, s);
}

cudaError_t launch_rec_backward(const RecParams &p, bool f32, bool vec, int sms, cudaStream_t s) {
    if (f32) return vec ? launch_items(rec_backward_kernel<float, true, 16, 8>, p, 512, sms, s)
                        : launch_items(rec_backward_kernel<float, false, 16, 8>, p, 512, sms, s);
    return vec ? launch_items(rec_backward_kernel<__nv_bfloat16, true, 16, 8>, p, 512, sms, s)
               : launch_items(rec_backward_kernel<__nv_bfloat16, false, 16, 8>, p, 512, sms, s);
}

cudaError_t launch_rec_decay(const float *partial, const float *decay, float kappa, float *d_decay, int chunks, int C,
                             int Cpad, cudaStream_t s) {
    rec_decay_kernel<<<(C + 31) / 32, 1024, 0, s>>>(partial, decay, kappa, d_decay, chunks, C, Cpad);
    return cudaGetLastError();
}

cudaError_t launch_rec_step(const RecStepParams &p, bool f32, bool vec, cudaStream_t s) {
    if (f32) {
        if (vec) rec_step_kernel<float, true><<<p.B * p.tiles, 128, 0, s>>>(p);
        else rec_step_kernel<float, false><<<p.B * p.tiles, 128, 0, s>>>(p);
    } else {
        if (vec) rec_step_kernel<__nv_bfloat16, true><<<p.B * p.tiles, 128, 0, s>>>(p);
        else rec_step_kernel<__nv_bfloat16, false><<<p.B * p.tiles, 128, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace conv2d_b200
