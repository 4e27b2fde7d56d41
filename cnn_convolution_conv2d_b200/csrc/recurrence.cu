// recurrence.cu -- the gated linear recurrence over time: forward, backward and one token.
//
//   ra = sigmoid(gate_a), rx = sigmoid(gate_x), a = exp(-kappa softplus(decay) ra),
//   h[t] = a[t] h[t-1] + sqrt(1 - a[t]^2) rx[t] x[t]
//
// per channel.  A run of rows acts on the state before it as h -> A h + H, with A the product
// of its a's and H its result from a zero state, and two runs join by
// (A1, H1), (A2, H2) -> (A1 A2, A2 H1 + H2): so the time axis is split.
//
// One work item is a chunk of rows of kRecTile channels.  Its working warps take two runs of rows each, half a warp
// a run, a lane two channels; it scans its run from zero in registers and leaves the run's (A, H) in shared memory.  A
// joining warp joins them, finds the state that enters the chunk, and hands every run the state
// that enters it; then the warps write their results.  Two blocks an SM, so that one works
// while the other's runs are joined.
// Items are handed out by a counter, early rows first, so an item only waits for items that are
// already running.  An item publishes its (A, H) as soon as it has them and the state behind
// it as soon as it knows the one before; the next item takes the nearest published state and
// applies the (A, H) after it, oldest first -- the same operations in the same order whichever
// state it found, so the result does not depend on timing.  A value is its own flag: both arrays
// start as all ones bits, which no published value has.
//
// Sequence starts inside an item are cuts: there A = 0, and joining selects instead of
// multiplying, so what a sequence holds (infinities and NaN too) never reaches its neighbour.  Where
// there is no cut, A is kept above 0, so that a NaN reaches every later row of its sequence.
// Only the warps whose rows a sequence begins or ends in look at their rows one by one.
//
// Bound by HBM (8 bytes an element forward, 14 backward in bf16) with the arithmetic close
// behind: two sigmoids, an exponential and a square root an element.  Hence two channels to an
// instruction, and rows that travel by TMA, the next items' tiles while an item is at work, and
// back from the same places in shared memory: with loads and stores of its own each thread spent
// more on addresses than on the recurrence.  Tensors whose base or row stride is no multiple of
// 16 bytes take the same item code with copies by the warps.
// What the time goes into: about 70 instructions for a lane's two channels, backward 140 (not quite an issue slot in two is used), the
// special-function unit (56% busy forward), 18 warps an SM that wait for one another at the joining, and with one long sequence
// the chain of states, a link some 0.7 us.  So tiles are narrow and chunks long (64 channels of half the rows: half as many
// chains with twice the links, 197 us where these took 158 for 32768 rows of 2048 channels).
// 16384 rows of 4096 channels in bf16: forward 143 us (3.7 TB/s), backward 282 us (3.3 TB/s); 2048 channels in fp32:
// 100 us (5.3 TB/s) and 194 us (4.8 TB/s); one sequence of 32768 x 2048 in bf16: 160 and 293 us; 12 packed ones of 16384 x
// 2560: 139 and 223 us; 3 x 777 x 1001 in fp32, whose rows TMA does not take: 35 and 51 us.  (With a formed as
// 1 + p these took 141 and 279, 100 and 184 us, and the gradients of fast decays were wrong.)
#include <atomic>

#include "ptx.cuh"
#include "sequence.cuh"

namespace conv2d_b200 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxKnown = 64;  // devices whose launch shapes are remembered

// Two channels to an instruction.  (A product that a sum takes up right away is written as fma2: the
// compiler fuses the two in some kernels and not in others, and results should not depend on that.)
__device__ __forceinline__ uint64_t pair(float2 v) { return static_cast<uint64_t>(__float_as_uint(v.y)) << 32 | __float_as_uint(v.x); }
__device__ __forceinline__ float2 unpair(uint64_t v) {
    return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a)), "l"(pair(b)));
    return unpair(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a)), "l"(pair(b)));
    return unpair(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pair(a)), "l"(pair(b)), "l"(pair(c)));
    return unpair(d);
}
__device__ __forceinline__ float2 add1(float2 a, float c) { return add2(a, splat(c)); }
__device__ __forceinline__ float2 one_minus(float2 a) { return fma2(a, splat(-1.f), splat(1.f)); }
__device__ __forceinline__ float2 negative(float2 a) { return make_float2(-a.x, -a.y); }

// ----------------------------------------------------------- element access ---
// Half a warp (16 lanes) takes the channels of a tile, and the two halves of a warp take runs of their own.
__device__ __forceinline__ int lane16() { return threadIdx.x & 15; }
__device__ __forceinline__ int half() { return threadIdx.x >> 4 & 1; }

// The two channels of a lane: of a tile, adjacent ones.
struct Lane2 {
    int c0, c1;
    bool ok0, ok1;
    __device__ Lane2(int c0_, int c1_, int C) : c0(c0_), c1(c1_), ok0(c0_ < C), ok1(c1_ < C) {}
    __device__ Lane2(int tile, int C) : Lane2(tile * kRecTile + 2 * lane16(), tile * kRecTile + 2 * lane16() + 1, C) {}
};

template <typename T>
__device__ __forceinline__ float2 load2(const T *row, const Lane2 &l) {
    return make_float2(l.ok0 ? to_float(row[l.c0]) : 0.f, l.ok1 ? to_float(row[l.c1]) : 0.f);
}
template <typename T>
__device__ __forceinline__ void store2(T *row, float2 f, const Lane2 &l) {
    if (l.ok0) row[l.c0] = from_float<T>(f.x);
    if (l.ok1) row[l.c1] = from_float<T>(f.y);
}
__device__ __forceinline__ float2 load_f32(const float *row, const Lane2 &l) {
    return row ? load2<float>(row, l) : make_float2(0.f, 0.f);
}

// The tensors of an item, by their place in its tile.
enum : int { kX = 0, kGateA = 1, kGateX = 2, kDy = 3 };

// The rows of a half warp's run in a tile in shared memory, where the results take the places of the
// inputs (same tensor, same thread).  By TMA they leave by one bulk store for a warp and tensor -- unless some rows of
// the warp's runs belong to no sequence: those must not be written, so the others go out one by one.  Otherwise
// the warp copies its rows in and out itself, a lane a channel.
// (In bf16 the two halves meet in the same 16 banks: their rows lie an even number of 64 bytes apart.)
template <typename T, int kRows, int L, bool kTma>
struct TileRun {
    static constexpr int kRun = L, kTwo = 2 * L;
    static constexpr int kRow = kRecTile * sizeof(T), kTensor = kRows * kRow;
    static constexpr unsigned kAll = ~0u >> (32 - kTwo);
    const RecParams &p;
    const CUtensorMap *maps;  // of the outputs, boxes of 2 L rows
    uint8_t *first;  // the warp's first row
    uint8_t *base;   // this half's
    int tile, row0, saved;  // row0: the warp's first row
    unsigned present;       // a bit for each of the warp's rows: it belongs to a sequence
    Lane2 l;
    __device__ TileRun(const RecParams &p_, const CUtensorMap *maps_, uint8_t *stage, int warp, int tile_, int row0_, int saved_)
        : p(p_), maps(maps_), first(stage + warp * kTwo * kRow), base(first + half() * L * kRow), tile(tile_), row0(row0_),
          saved(saved_), present(kAll), l(tile_, p_.C) {}
    __device__ uint8_t *at(int tensor, int j) const {
        return base + tensor * kTensor + j * kRow + lane16() * 2 * static_cast<int>(sizeof(T));
    }
    __device__ T *output(int tensor) const { return static_cast<T *>(tensor == 0 ? p.y : tensor == 1 ? p.dga : p.dgx); }
    __device__ long long stride(int tensor) const { return tensor == 0 ? p.ldy : tensor == 1 ? p.ld_da : p.ld_dg; }
    __device__ float2 get(int tensor, int j) const {
        if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float2 *>(at(tensor, j));
        const uint32_t v = *reinterpret_cast<const uint32_t *>(at(tensor, j));
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    // A value of the lane's own in the places of a row's two gates.
    __device__ void keep(int j, float2 f) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float2 *>(at(kGateA, j)) = f;
        } else {
            *reinterpret_cast<float *>(at(kGateA, j)) = f.x;
            *reinterpret_cast<float *>(at(kGateX, j)) = f.y;
        }
    }
    __device__ float2 kept(int j) const {
        if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float2 *>(at(kGateA, j));
        return make_float2(*reinterpret_cast<const float *>(at(kGateA, j)), *reinterpret_cast<const float *>(at(kGateX, j)));
    }
    __device__ void put(int tensor, int j, float2 f) {
        if (kTma && present != kAll) {
            store2<T>(output(tensor) + static_cast<size_t>(row0 + half() * L + j) * stride(tensor), f, l);
        } else if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float2 *>(at(tensor, j)) = f;
        } else {
            *reinterpret_cast<__nv_bfloat162 *>(at(tensor, j)) = __float22bfloat162_rn(f);
        }
    }
    // Sends the results of the first n tensors; by TMA, the tile is free once lane 0's bulk reads are done.  (The barrier
    // comes first also where nothing is sent: lane 0 frees the tile for the next loads, so all lanes must have read it.)
    __device__ void done(int n) {
        if constexpr (kTma) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (present != kAll) return;
            if ((threadIdx.x & 31) == 0) {
                for (int i = 0; i < n; ++i) ptx::tma_store_2d(maps + i, first + i * kTensor, tile * kRecTile, row0);
                ptx::bulk_commit_group();
            }
        } else {
            __syncwarp();
            const int lane = threadIdx.x & 31, c = tile * kRecTile + lane;
            for (int i = 0; i < n; ++i) {
                T *out = output(i) + static_cast<size_t>(row0) * stride(i) + c;
                const T *from = reinterpret_cast<const T *>(first + i * kTensor) + lane;
#pragma unroll 8
                for (int r = 0; r < kTwo; ++r)
                    if ((present >> r & 1u) && c < p.C) out[r * stride(i)] = from[r * kRecTile];
            }
            __syncwarp();
        }
    }
    // Copies the warp's rows of the first n tensors in, asynchronously where the copy instruction has the size (4 bytes).
    __device__ void fetch(int n) {
        const int lane = threadIdx.x & 31, c = tile * kRecTile + lane, rows = min(p.seq.rows - row0, kTwo);
        for (int i = 0; i < n; ++i) {
            const long long ld = i == kX ? p.ldx : i == kGateA ? p.lda : i == kGateX ? p.ldg : p.lddy;
            const T *from = static_cast<const T *>(i == kX ? p.x : i == kGateA ? p.ga : i == kGateX ? p.gx : p.dy) +
                            static_cast<size_t>(row0) * ld + c;
            T *to = reinterpret_cast<T *>(first + i * kTensor) + lane;
            if (c >= p.C) continue;
            if constexpr (sizeof(T) == 4) {
#pragma unroll 4
                for (int r = 0; r < rows; ++r) cp_async_4(to + r * kRecTile, from + r * ld);
            } else {
#pragma unroll 8
                for (int r = 0; r < rows; ++r) to[r * kRecTile] = from[r * ld];
            }
        }
        cp_async_commit();
    }
};

// ----------------------------------------------------------------- the gates ---
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// log2(a) per unit of ra: -kappa softplus(decay) log2(e).
__device__ __forceinline__ float decay_rate(float decay, float kappa) { return -kappa * kLog2e * softplus(decay); }

__device__ __forceinline__ float2 decay_rate(const RecParams &p, const Lane2 &l) {
    if (p.rates) return load2<float>(p.rates, l);
    const float2 d = load2<float>(p.decay, l);
    return make_float2(decay_rate(d.x, p.kappa), decay_rate(d.y, p.kappa));
}

__device__ __forceinline__ float2 sigmoid2(float2 z) {
    const float2 t = mul2(z, splat(-kLog2e));
    const float2 d = add2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), splat(1.f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// A decay a = 2^y for y <= 0, and p = a - 1, each exact to a few units of itself: with
// y = n + f, |f| <= 1/2, they are 2^n q + 2^n and 2^n q + (2^n - 1), q = 2^f - 1.  q is f times the polynomial of
// degree 5 that interpolates (2^f - 1)/f at the Chebyshev points of [-1/2, 1/2] (2e-8 off).
// A decay a little below 1 is applied thousands of times, so an approximate
// exponential, biased by a unit or two, would not do; a small one is a factor of d_gate_a, d_decay and the state's gradient,
// so 1 + p, exact to 2^-25 of 1 only, would not do either.  (No special-function unit is used either:
// the sigmoids keep that one busy.)  y below -126 counts as -126: a is above 0.
struct Decay {
    float2 a, p;
};
__device__ __forceinline__ Decay decay_of(float2 y) {
    y = make_float2(max_or_nan(y.x, -126.f), max_or_nan(y.y, -126.f));
    constexpr float kRound = 12582912.f + 127.f;  // 1.5 * 2^23 and the exponent's bias: adding it leaves n + 127 in the low bits
    const float2 r = add2(y, splat(kRound));
    const float2 f = fma2(add2(r, splat(-kRound)), splat(-1.f), y);
    const float2 s = make_float2(__int_as_float(__float_as_int(r.x) << 23), __int_as_float(__float_as_int(r.y) << 23));
    float2 q = fma2(f, splat(0.00015453163f), splat(0.0013390863f));
    q = fma2(f, q, splat(0.009618083f));
    q = fma2(f, q, splat(0.05550357f));
    q = fma2(f, q, splat(0.2402265f));
    q = fma2(f, q, splat(0.6931472f));
    q = mul2(f, q);
    return Decay{fma2(s, q, s), fma2(s, q, add1(s, -1.f))};
}

// From p = a - 1: minus v, v = 1 - a^2.  -p (2 + p) has no cancellation.
__device__ __forceinline__ float2 minus_v(float2 p) { return mul2(p, add1(p, 2.f)); }
// b = beta rx x.  Where a is 1, beta is 0: such a row adds nothing.
__device__ __forceinline__ float2 contribution(float2 p, float2 rx, float2 x) {
    const float2 mv = minus_v(p);
    return mul2(make_float2(sqrt_approx(-mv.x), sqrt_approx(-mv.y)), mul2(rx, x));
}

// ------------------------------------------------------------------ joining ---
// The product of two runs' decays.  Only a cut makes it 0: a product that falls below the smallest number is that
// number, and of a NaN (which H has too) the smallest number is left.
constexpr float kLeast = 1.4e-45f;
__device__ __forceinline__ float product(float A, float B) { return A == 0.f || B == 0.f ? 0.f : fmaxf(A * B, kLeast); }
__device__ __forceinline__ float2 product(float2 A, float2 B) { return make_float2(product(A.x, B.x), product(A.y, B.y)); }
__device__ __forceinline__ float2 no_cut(float2 a) { return make_float2(fmaxf(a.x, kLeast), fmaxf(a.y, kLeast)); }

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

// What the chunks in front of a chunk have published, read by one warp: the nearest kWindow ones.
constexpr int kWindow = 3;
struct Published {
    uint64_t a0[kWindow], a1[kWindow];
    uint32_t c0[kWindow], c1[kWindow];
    // step: +1 where the chunk in front of chunk k is k-1, -1 where it is k+1; `before` of them exist
    __device__ __forceinline__ void read(const RecParams &p, int chunk, int before, int step, const Lane2 &l) {
#pragma unroll
        for (int i = 0; i < kWindow; ++i) {
            a0[i] = a1[i] = 0;
            c0[i] = c1[i] = 0;
            if (i < before) {
                const ptrdiff_t at = static_cast<ptrdiff_t>(chunk - step * (i + 1)) * p.Cpad;
                c0[i] = peek(p.carry + at + l.c0);
                c1[i] = peek(p.carry + at + l.c1);
                a0[i] = peek(p.aggregate + at + l.c0);
                a1[i] = peek(p.aggregate + at + l.c1);
            }
        }
    }
    // The state that enters the chunk, if it can be told: the nearest carry, and the (A, H) of the
    // chunks after it, oldest first.
    __device__ __forceinline__ bool state(float2 &h) const {
        bool told = true;  // whether all nearer chunks' (A, H) are there
        int found = -1;
#pragma unroll
        for (int i = 0; i < kWindow; ++i) {
            if (found < 0 && told && __all_sync(kFull, c0[i] != kFull && c1[i] != kFull)) found = i;
            told = told && __all_sync(kFull, static_cast<uint32_t>(a0[i]) != kFull && static_cast<uint32_t>(a1[i]) != kFull);
        }
        if (found < 0) return false;
#pragma unroll
        for (int i = kWindow - 1; i >= 0; --i) {
            if (i == found) h = make_float2(__uint_as_float(c0[i]), __uint_as_float(c1[i]));
            if (i < found)
                h = make_float2(after(__uint_as_float(static_cast<uint32_t>(a0[i])), __uint_as_float(a0[i] >> 32), h.x),
                                after(__uint_as_float(static_cast<uint32_t>(a1[i])), __uint_as_float(a1[i] >> 32), h.y));
        }
        return true;
    }
};

// An item.
struct Item {
    int chunk;  // -1: no more items
    int tile, row0;
    int saved;  // saved_place of its first run
    int flags;
    int seq, last;  // the sequences of its first and its last row
};
// An item is the first of all; a sequence begins or ends inside it, or rows of it belong to none; else its rows are the
// first, the last of their sequence; the rows in front of it (against the order of time: behind it) reach into it.
enum : int { kFirst = 1, kEdges = 2, kStarts = 4, kEnds = 8, kNeedsFront = 16 };

// What the rows of a half warp's run are, a bit each; `seq` of lane j is the sequence of the warp's row j.  In a chunk
// of one sequence: whether the run begins or ends it, and the sequence.
struct Run {
    unsigned in, start, end;
    int seq;
};
template <int L>
__device__ __forceinline__ Run run_of(const Sequences &q, const Item &item, int row0, int limit) {
    const int lane = threadIdx.x & 31, row = row0 + lane;
    Run r;
    r.seq = 0;
    bool in = false, start = false, end = false;
    if (lane < 2 * L && row < limit) {
        const int s = seq_of(q, row, item.seq, item.last);
        if (s >= 0) {
            const int b = seq_begin(q, s), e = seq_begin(q, s + 1);
            in = row < e;
            start = in && row == b;
            end = in && row + 1 == e;
            r.seq = s;
        }
    }
    const auto bits = [](bool v) { return __ballot_sync(kFull, v) >> (half() * L) & ((1u << L) - 1u); };
    r.in = bits(in);
    r.start = bits(start);
    r.end = bits(end);
    return r;
}

// The channels of the sequence of a run's row j.  Called by the whole warp.
template <int L>
__device__ __forceinline__ const float *seq_row(const float *base, const Run &r, int j, int C) {
    const int s = __shfl_sync(kFull, r.seq, half() * L + j);
    return base ? base + static_cast<size_t>(s) * C : nullptr;
}

// The next item of the block, by one thread.  Without a counter (one chunk: nothing waits for
// anything) the items are dealt out in turn.
__device__ __forceinline__ unsigned next_item(const RecParams &p, unsigned &dealt) {
    if (p.ticket) return atomicAdd(p.ticket, 1u) + 1u;
    const unsigned item = dealt;
    dealt += gridDim.x;
    return item;
}

// Shared memory of an item's joining: the runs, and the states that enter them.
template <int W, bool kBack>
struct Joins {
    float4 run[W][32];    // the run of lane l's half of warp w
    float2 start[W][32];
    float2 sum[2][kBack ? W : 1][32];  // backward: the runs' sums of w, of this item and the one before
    int stop;
};

// The meetings of the W working warps and the joining warp: the working warps announce their runs, and wait for
// the states that enter them (false: the block has to stop).
constexpr int kRunsIn = 1, kStartsIn = 2, kEnd = 3;
template <int W, bool kBack>
__device__ __forceinline__ bool exchange(Joins<W, kBack> &s, float4 run, int warp) {
    s.run[warp][threadIdx.x & 31] = run;
    __syncwarp();
    named_barrier_arrive(kRunsIn, (W + 1) * 32);
    ptx::named_barrier(kStartsIn, (W + 1) * 32);
    return *static_cast<volatile int *>(&s.stop) == 0;
}

// Joins a run (A0, H0, A1, H1) to what lies in front of it; without a cut in the chunk a product will do.
template <bool kEdge>
__device__ __forceinline__ float4 join(float4 all, float4 r) {
    if (kEdge) return make_float4(product(all.x, r.x), after(r.x, r.y, all.y), product(all.z, r.z), after(r.z, r.w, all.w));
    const float2 A = make_float2(r.x, r.z), H = fma2(A, make_float2(all.y, all.w), make_float2(r.y, r.w));
    const float2 P = mul2(make_float2(all.x, all.z), A);
    return make_float4(P.x, H.x, P.y, H.y);
}
template <bool kEdge>
__device__ __forceinline__ float2 step_over(float4 r, float2 h) {
    if (kEdge) return make_float2(after(r.x, r.y, h.x), after(r.z, r.w, h.y));
    return fma2(make_float2(r.x, r.z), h, make_float2(r.y, r.w));
}

// The joining warp's part of an item: publishes the chunk's (A, H), finds the state that enters the chunk,
// publishes the one that leaves it, and hands out those that enter the runs.
template <bool kEdge, bool kForward, int W>
__device__ __forceinline__ void join_runs(const RecParams &p, int chunk, bool needed, float2 h, Published &front, bool &gave_up,
                                          const float4 (*runs)[32], float2 (*start)[32], const Lane2 &l) {
    constexpr int kStep = kForward ? 1 : -1;
    const int lane = threadIdx.x & 31;
    const int before = kForward ? chunk : p.chunks - 1 - chunk;
    const bool sends = (kForward ? chunk + 1 < p.chunks : chunk > 0) && !p.starve;
    const size_t at = static_cast<size_t>(chunk) * p.Cpad;
    // half the lanes join the first half of the runs, the others the second
    const auto place = [&](int i) { return kForward ? half() * W + i : 2 * W - 1 - (half() * W + i); };
    const auto run = [&](int i) { return runs[place(i) >> 1][(place(i) & 1) * 16 + lane16()]; };
    const auto from_half = [&](const float4 &v, int h) {
        return make_float4(__shfl_sync(kFull, v.x, h * 16 + lane16()), __shfl_sync(kFull, v.y, h * 16 + lane16()),
                           __shfl_sync(kFull, v.z, h * 16 + lane16()), __shfl_sync(kFull, v.w, h * 16 + lane16()));
    };
    float4 mine = run(0);
#pragma unroll
    for (int i = 1; i < W; ++i) mine = join<kEdge>(mine, run(i));
    const float4 first = from_half(mine, 0);
    float4 all = join<kEdge>(first, from_half(mine, 1));
    if (!kEdge) {
        all.x = fmaxf(all.x, kLeast);
        all.z = fmaxf(all.z, kLeast);
    }
    if (sends && needed && half() == 0) {
        publish(p.aggregate + at + l.c0, all.x, all.y);
        publish(p.aggregate + at + l.c1, all.z, all.w);
    }
    if (needed) {
        uint64_t began = 0;
        for (unsigned i = 1; !front.state(h); ++i) {
            if ((i & 63u) == 0) {
                const uint64_t now = __shfl_sync(kFull, ptx::globaltimer_ns(), 0);
                if (!began) began = now;
                else if (gave_up || now - began > static_cast<uint64_t>(p.timeout_ns)) {  // report, and go on with zeros
                    gave_up = true;  // the block's next waits are short
                    if (lane == 0) atomicExch(p.status, kDevTimeoutCarry);
                    h = splat(0.f);
                    break;
                }
            }
            front.read(p, chunk, before, kStep, l);
        }
    }
    if (sends && half() == 0) {
        publish(p.carry + at + l.c0, after(all.x, all.y, h.x));
        publish(p.carry + at + l.c1, after(all.z, all.w, h.y));
    }
    if (half()) h = step_over<kEdge>(first, h);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        start[place(i) >> 1][(place(i) & 1) * 16 + lane16()] = h;
        h = step_over<kEdge>(run(i), h);
    }
}

// ------------------------------------------------------------------ forward ---
// A working warp's part of an item.  The run from a zero state: the states H of its rows, and the products A of
// its decays up to each; with the state h that enters it, A h + H, as the joining has it.
// `halfway` runs in between, when what was sent before has left.
template <bool kEdge, int W, typename Rows, typename Halfway>
__device__ __forceinline__ bool forward_item(const RecParams &p, Rows &rows, const Run &run, Joins<W, false> &s, int warp,
                                             Halfway halfway) {
    constexpr int L = Rows::kRun, kUnroll = kEdge ? 1 : L;
    constexpr int kGroup = kEdge ? 4 : L;  // rows whose gates are worked out together
    float2 A[L], H[L];
    const float2 rate = decay_rate(p, rows.l);
#pragma unroll kUnroll
    for (int j0 = 0; j0 < L; j0 += kGroup) {
        float2 a[kGroup], b[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const int j = j0 + i;
            if (j == L / 2) halfway();
            const Decay d = decay_of(mul2(rate, sigmoid2(rows.get(kGateA, j))));
            b[i] = contribution(d.p, sigmoid2(rows.get(kGateX, j)), rows.get(kX, j));
            a[i] = d.a;
            if (!kEdge) {
                A[j] = j ? mul2(A[j ? j - 1 : 0], a[i]) : a[i];
                H[j] = j ? fma2(a[i], H[j ? j - 1 : 0], b[i]) : b[i];
            }
        }
        if constexpr (kEdge) {
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                const int j = j0 + i;
                const float *from = seq_row<L>(p.state, run, j, p.C);
                float2 before = j ? H[j ? j - 1 : 0] : splat(0.f), kept = j ? A[j ? j - 1 : 0] : splat(1.f);
                if (run.start >> j & 1u) {
                    before = load_f32(from, rows.l);
                    kept = splat(0.f);
                }
                const bool in = run.in >> j & 1u;
                A[j] = in ? product(kept, no_cut(a[i])) : splat(0.f);
                H[j] = in ? fma2(a[i], before, b[i]) : splat(0.f);
            }
        }
    }
    const float2 all = kEdge ? A[L - 1] : no_cut(A[L - 1]);
    if (!exchange(s, make_float4(all.x, H[L - 1].x, all.y, H[L - 1].y), warp)) return false;
    const float2 h = s.start[warp][threadIdx.x & 31];
    float2 y = h;
#pragma unroll kUnroll
    for (int j = 0; j < L; ++j) {
        const float *to = kEdge ? seq_row<L>(p.final_state, run, j, p.C) : nullptr;
        if (kEdge && !(run.in >> j & 1u)) continue;
        if (j % kRecRun == 0 && p.saved) store2(p.saved + static_cast<size_t>(rows.saved + j / kRecRun) * p.Cpad, y, rows.l);
        y = kEdge ? make_float2(after(A[j].x, H[j].x, h.x), after(A[j].y, H[j].y, h.y)) : fma2(A[j], h, H[j]);
        rows.put(0, j, y);
        if (kEdge && (run.end >> j & 1u) && p.final_state)
            store2(const_cast<float *>(to), y, rows.l);
    }
    if (!kEdge && run.end && p.final_state) store2(p.final_state + static_cast<size_t>(run.seq) * p.C, y, rows.l);
    rows.done(1);
    return true;
}

// What a state leaves of an empty sequence: itself.
template <int kWarps>
__device__ __forceinline__ void copy_empty(const Sequences &q, const float *from, float *to, int C, const Lane2 &l) {
    if (!to) return;
    for (int s = threadIdx.x >> 4; s < q.nseq; s += 2 * kWarps)
        if (seq_begin(q, s + 1) <= seq_begin(q, s))
            store2(to + static_cast<size_t>(s) * C, load_f32(from ? from + static_cast<size_t>(s) * C : nullptr, l), l);
}

// ----------------------------------------------------------------- backward ---
// With g[t] the gradient of h[t] through everything after it, G[t] = a[t] g[t] is what enters row
// t-1: G[t] = a[t] (dh[t] + G[t+1]), the same kind of recurrence backwards.  The states are
// computed again from those that the forward pass kept.  Per row, with w = ra d/d(log a):
//   dx = g beta rx, d_gate_x = g beta x rx (1-rx), w = a g (h[t-1] - a rx x / beta) ra,
//   d_gate_a = -kappa softplus(decay) w (1-ra), d_decay = -kappa sigmoid(decay) sum w.
template <bool kEdge, int W, typename Rows, typename Halfway>
__device__ __forceinline__ bool backward_item(const RecParams &p, Rows &rows, const Run &run, Joins<W, true> &s,
                                              float2 (*s_sum)[32], int warp, Halfway halfway) {
    constexpr int L = Rows::kRun, kUnroll = kEdge ? 1 : L;
    static_assert(L == kRecRun, "a saved state for each run");
    float2 h = splat(0.f);  // what enters the run
    if (!kEdge && run.start) h = load_f32(p.state ? p.state + static_cast<size_t>(run.seq) * p.C : nullptr, rows.l);
    else if (!kEdge || (run.in & 1u)) h = load2<float>(p.saved + static_cast<size_t>(rows.saved) * p.Cpad, rows.l);
    const float2 rate = decay_rate(p, rows.l);
    // The gates' places in the tile take h[t-1] once the gates are worked out: registers would not hold it beside a and a - 1.
    float2 as[L], pm[L], ra[L], rx[L];  // a, a - 1, the gates
#pragma unroll kUnroll
    for (int j = 0; j < L; ++j) {
        if (j == L / 2) halfway();
        const float *from = kEdge ? seq_row<L>(p.state, run, j, p.C) : nullptr;
        if (kEdge && !(run.in >> j & 1u)) continue;
        ra[j] = sigmoid2(rows.get(kGateA, j));
        rx[j] = sigmoid2(rows.get(kGateX, j));
        const Decay d = decay_of(mul2(rate, ra[j]));
        as[j] = d.a;
        pm[j] = d.p;
        if (kEdge && (run.start >> j & 1u)) h = load_f32(from, rows.l);
        rows.keep(j, h);
        h = fma2(d.a, h, contribution(d.p, rx[j], rows.get(kX, j)));
    }
    // g from zero behind the run, the a of the row after, and the product of all a's so far
    float2 g = splat(0.f), a = splat(0.f), B = splat(1.f);
#pragma unroll kUnroll
    for (int j = L - 1; j >= 0; --j) {
        const float *behind = kEdge ? seq_row<L>(p.d_final, run, j, p.C) : nullptr;
        if (kEdge && !(run.in >> j & 1u)) {
            g = a = B = splat(0.f);
            continue;
        }
        const float2 dh = rows.get(kDy, j);
        if (kEdge && (run.end >> j & 1u)) {
            g = add2(dh, load_f32(behind, rows.l));
            B = splat(0.f);
        } else {
            g = j < L - 1 ? fma2(a, g, dh) : dh;
        }
        a = as[j];
        B = kEdge ? product(B, no_cut(a)) : mul2(B, a);
    }
    const float2 S = mul2(a, g);
    if (!kEdge) B = no_cut(B);
    if (!exchange(s, make_float4(B.x, S.x, B.y, S.y), warp)) return false;
    const float2 G = s.start[warp][threadIdx.x & 31];
    const float2 natural = mul2(decay_rate(p, rows.l), splat(1.f / kLog2e));
    float2 sum = splat(0.f);
    g = a = splat(0.f);
#pragma unroll kUnroll
    for (int j = L - 1; j >= 0; --j) {
        const float *behind = kEdge ? seq_row<L>(p.d_final, run, j, p.C) : nullptr;
        const float *to = kEdge ? seq_row<L>(p.d_state, run, j, p.C) : nullptr;
        if (kEdge && !(run.in >> j & 1u)) {
            g = a = splat(0.f);
            continue;
        }
        const float2 dh = rows.get(kDy, j), x = rows.get(kX, j);
        if (kEdge && (run.end >> j & 1u)) g = add2(dh, load_f32(behind, rows.l));
        else g = j < L - 1 ? fma2(a, g, dh) : add2(dh, G);
        a = as[j];
        const float2 back = mul2(a, g), ga = mul2(ra[j], back), bx = mul2(rx[j], x);
        // 1 / beta; 1e-37 under the root keeps it finite where a is 1 and ra, beta and so all but dh's share are 0
        const float2 mv = minus_v(pm[j]);
        const float2 under = fma2(mv, splat(-1.f), splat(1e-37f));
        const float2 inv = make_float2(rsqrt_approx(under.x), rsqrt_approx(under.y));
        const float2 dx = mul2(mul2(g, rx[j]), negative(mul2(mv, inv)));
        const float2 dg = mul2(mul2(dx, x), one_minus(rx[j]));
        const float2 inner = fma2(negative(mul2(a, inv)), bx, rows.kept(j));
        const float2 w = mul2(ga, inner);
        sum = fma2(ga, inner, sum);
        const float2 da = mul2(mul2(natural, w), one_minus(ra[j]));
        rows.put(0, j, dx);
        rows.put(1, j, da);
        rows.put(2, j, dg);
        if (kEdge && (run.start >> j & 1u) && p.d_state)
            store2(const_cast<float *>(to), back, rows.l);
        if (!kEdge && j == 0 && run.start && p.d_state) store2(p.d_state + static_cast<size_t>(run.seq) * p.C, back, rows.l);
    }
    rows.done(3);
    s_sum[warp][threadIdx.x & 31] = sum;
    return true;
}

template <bool kEdge, int W, bool kBack, typename Rows, typename Halfway>
__device__ __forceinline__ bool work_item(const RecParams &p, Rows &rows, const Run &run, Joins<W, kBack> &s, float2 (*s_sum)[32],
                                          int warp, Halfway halfway) {
    if constexpr (kBack) return backward_item<kEdge, W>(p, rows, run, s, s_sum, warp, halfway);
    else return forward_item<kEdge, W>(p, rows, run, s, warp, halfway);
}
// The form for rows with edges, as a call (inlined, it would take registers from the other) and in loops: unrolled, the
// instructions of both forms together did not stay in the cache, and a packed batch took twice the time.
template <int W, bool kBack, typename Rows, typename Halfway>
__device__ __noinline__ bool work_item_edges(const RecParams &p, Rows rows, Run run, Joins<W, kBack> &s, float2 (*s_sum)[32],
                                             int warp, Halfway halfway) {
    return work_item<true, W, kBack>(p, rows, run, s, s_sum, warp, halfway);
}

// The chunk's sum of w, its halves' and their warps' in order.
template <int W>
__device__ __forceinline__ void store_sum(const RecParams &p, int chunk, const float2 (*s_sum)[32], const Lane2 &l) {
    float2 sum = splat(0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) sum = add2(sum, s_sum[w][threadIdx.x & 31]);
    sum.x += __shfl_xor_sync(kFull, sum.x, 16);
    sum.y += __shfl_xor_sync(kFull, sum.y, 16);
    if (half()) return;
    float *out = p.decay_partial + static_cast<size_t>(chunk) * p.Cpad;
    out[l.c0] = sum.x;
    out[l.c1] = sum.y;
}

// ------------------------------------------------------------------ kernels ---
// Where the chunks lie.  Either they follow one another over all rows, or each sequence has its own
// (p.per_seq of them): then the items go round the sequences, and a chunk follows the one in front of it so
// many items later that it hardly ever waits.
__device__ __forceinline__ int chunk_row(const RecParams &p, int chunk, int chunk_rows) {
    if (!p.per_seq) return chunk * chunk_rows;
    const int s = chunk / p.per_seq;
    return s * p.seq.T + (chunk - s * p.per_seq) * chunk_rows;
}
// The end of the rows that a chunk may have.
__device__ __forceinline__ int chunk_limit(const RecParams &p, int chunk) {
    return p.per_seq ? (chunk / p.per_seq + 1) * p.seq.T : p.seq.rows;
}

// The place of the first saved state of a run: one for every kRecRun rows, counted in each sequence if it has chunks of its own.
__device__ __forceinline__ int saved_place(const RecParams &p, int chunk, int row0) {
    if (!p.per_seq) return row0 / kRecRun;
    const int s = chunk / p.per_seq;
    return s * ((p.seq.T + kRecRun - 1) / kRecRun) + (row0 - s * p.seq.T) / kRecRun;
}

__device__ __forceinline__ Item item_of(const RecParams &p, unsigned item, int chunk_rows, bool back) {
    if (item >= static_cast<unsigned>(p.chunks) * p.tiles) return Item{-1, 0, 0, 0, 0, 0, 0};
    const int turn = item / p.tiles, tile = item - turn * p.tiles;
    int chunk = back ? p.chunks - 1 - turn : turn;
    if (p.per_seq) {
        const int k = turn / p.seq.nseq, s = turn - k * p.seq.nseq;
        chunk = s * p.per_seq + (back ? p.per_seq - 1 - k : k);
    }
    const int row0 = chunk_row(p, chunk, chunk_rows);
    const int seq = seq_of(p.seq, row0), begin = seq < 0 ? 0 : seq_begin(p.seq, seq), end = seq < 0 ? 0 : seq_begin(p.seq, seq + 1);
    int flags = item == 0 ? kFirst : 0;
    const int row1 = row0 + chunk_rows;
    int last = seq;
    bool front = back ? chunk + 1 < p.chunks : chunk > 0;
    if (begin > row0 || end < row1) {
        flags |= kEdges;
        last = seq_of(p.seq, row1 - 1);
        if (p.per_seq) front = (back ? chunk + 1 : chunk) % p.per_seq != 0;
        else if (back) front = front && last >= 0 && row1 < seq_begin(p.seq, last + 1);
        else front = front && begin < row0 && row0 < end;
    } else {
        flags |= (begin == row0 ? kStarts : 0) | (end == row1 ? kEnds : 0);
        front = front && (back ? end != row1 : begin != row0);
    }
    if (front) flags |= kNeedsFront;
    return Item{chunk, tile, row0, saved_place(p, chunk, row0), flags, seq, last};
}

// Which of a warp's rows belong to a sequence, from its two runs.
template <int L>
__device__ __forceinline__ unsigned present_rows(const Run &run) {
    return __shfl_sync(kFull, run.in, 0) | __shfl_sync(kFull, run.in, 16) << L;
}

// Whether a sequence begins or ends in a warp's rows, or some belong to none: then they are looked at one by one.
template <int L>
__device__ __forceinline__ bool row_by_row(const Item &item, const Run &run) {
    return item.flags & kEdges && __any_sync(kFull, run.in != (1u << L) - 1u || run.start || run.end);
}

// A run of a chunk of one sequence.
template <int W>
__device__ __forceinline__ Run whole_run(const Item &item) {
    const int place = threadIdx.x >> 4;
    return Run{~0u, (item.flags & kStarts) && place == 0, (item.flags & kEnds) && place == 2 * W - 1, item.seq};
}

// The joining warp's work on an item: first, while the runs are still at work, it looks for what is in front.
template <int W, int L, bool kBack>
struct Joining {
    Published front;
    float2 h;  // what enters the chunk where no rows in front of it do
    bool &gave_up;
    __device__ explicit Joining(bool &gave_up_) : gave_up(gave_up_) {}
    __device__ __forceinline__ void look(const RecParams &p, const Item &item, const Lane2 &l) {
        const int chunk = item.chunk;
        h = splat(0.f);
        if (item.flags & (kBack ? kEnds : kStarts)) {
            const float *from = kBack ? p.d_final : p.state;
            h = load_f32(from ? from + static_cast<size_t>(item.seq) * p.C : nullptr, l);
        }
        if (item.flags & kNeedsFront) front.read(p, chunk, kBack ? p.chunks - 1 - chunk : chunk, kBack ? -1 : 1, l);
    }
    __device__ __forceinline__ void join(const RecParams &p, const Item &item, const float4 (*runs)[32], float2 (*start)[32],
                                         const Lane2 &l) {
        if (item.flags & kEdges) join_runs<true, !kBack, W>(p, item.chunk, item.flags & kNeedsFront, h, front, gave_up, runs, start, l);
        else join_runs<false, !kBack, W>(p, item.chunk, item.flags & kNeedsFront, h, front, gave_up, runs, start, l);
    }
};

// Items whose rows the warps copy themselves, for tensors that TMA does not take: the next item's while one is at work.
template <typename T, int W, int L, bool kBack>
__global__ void __launch_bounds__((W + 1) * 32, 2) rec_plain_kernel(const __grid_constant__ RecParams p) {
    using Tile = TileRun<T, 2 * W * L, L, false>;
    constexpr int kIn = kBack ? 4 : 3, kAll = (W + 1) * 32;
    extern __shared__ __align__(128) uint8_t s_tiles[];
    __shared__ Joins<W, kBack> s;
    __shared__ Item s_item[2];
    const int warp = threadIdx.x >> 5;
    unsigned dealt = blockIdx.x;
    const auto tile_of = [&](const Item &item, int stage) {
        return Tile(p, nullptr, s_tiles + stage * kIn * Tile::kTensor, warp, item.tile, item.row0 + warp * 2 * L,
                    item.saved + (warp * 2 + half()) * (L / kRecRun));
    };
    Item ahead{-1, 0, 0, 0, 0, 0, 0};  // one thread's: the next item, taken while nothing waits for it
    const auto take = [&] {
        if (threadIdx.x == W * 32) ahead = item_of(p, next_item(p, dealt), 2 * W * L, kBack);
    };
    take();
    if (threadIdx.x == W * 32) {
        s.stop = 0;
        s_item[0] = ahead;
    }
    take();
    __syncthreads();
    bool gave_up = false;  // the joining warp's: a wait for what is in front ran out
    if (warp < W && s_item[0].chunk >= 0) tile_of(s_item[0], 0).fetch(kIn);
    for (unsigned n = 0;; ++n) {
        const Item item = s_item[n & 1];
        if (item.chunk < 0) break;
        if (threadIdx.x == W * 32) s_item[~n & 1] = ahead;
        __syncthreads();
        if (item.flags & kFirst) check_offsets(p.seq, p.status);
        if (item.chunk == 0)
            copy_empty<W + 1>(p.seq, kBack ? p.d_final : p.state, kBack ? p.d_state : p.final_state, p.C, Lane2(item.tile, p.C));
        auto nothing = [] {};
        if (warp == W) {
            const Lane2 l(item.tile, p.C);
            Joining<W, L, kBack> joining(gave_up);
            joining.look(p, item, l);
            ptx::named_barrier(kRunsIn, kAll);
            joining.join(p, item, s.run, s.start, l);
            __syncwarp();
            named_barrier_arrive(kStartsIn, kAll);
            take();
        } else {
            const Item next = s_item[~n & 1];
            if (next.chunk >= 0) {
                tile_of(next, ~n & 1).fetch(kIn);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
            __syncwarp();
            Tile rows = tile_of(item, n & 1);
            const Run run = item.flags & kEdges ? run_of<L>(p.seq, item, rows.row0, chunk_limit(p, item.chunk)) : whole_run<W>(item);
            if (row_by_row<L>(item, run)) {
                rows.present = present_rows<L>(run);
                work_item_edges<W, kBack>(p, rows, run, s, s.sum[0], warp, nothing);
            } else {
                work_item<false, W, kBack>(p, rows, run, s, s.sum[0], warp, nothing);
            }
        }
        if constexpr (kBack) {
            __syncthreads();
            if (warp == W) store_sum<W>(p, item.chunk, s.sum[0], Lane2(item.tile, p.C));
        }
    }
}

// Items in tiles that travel by TMA through S stages of shared memory.  The joining warp also takes the items and
// issues their loads.
template <typename T, int W, int L, int S, bool kBack, int kBlocks>
__global__ void __launch_bounds__((W + 1) * 32, kBlocks) rec_tile_kernel(const __grid_constant__ RecTiles q) {
    static_assert(S >= 2, "one item at work, one on its way");
    using Tile = TileRun<T, 2 * W * L, L, true>;
    constexpr int kIn = kBack ? 4 : 3, kAll = (W + 1) * 32;
    constexpr int kStage = kIn * Tile::kTensor;
    extern __shared__ __align__(128) uint8_t s_tiles[];
    __shared__ Joins<W, kBack> s;
    __shared__ uint64_t s_full[S], s_free;  // a stage's loads have come; the last item's results have left
    __shared__ Item s_item[S];
    __shared__ int s_abort;
    const RecParams &p = q.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s_abort = s.stop = 0;
        for (int i = 0; i < S; ++i) ptx::mbar_init(&s_full[i], 1);
        ptx::mbar_init(&s_free, W);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    const ptx::Watchdog wd{&s_abort, p.status, static_cast<uint64_t>(p.timeout_ns)};
    if (warp == W) {
        unsigned dealt = blockIdx.x;
        Item ahead{-1, 0, 0, 0, 0, 0, 0};  // lane 0: the item to be loaded next, taken while nothing waits for it
        auto take = [&] {
            if (lane == 0) ahead = item_of(p, next_item(p, dealt), 2 * W * L, kBack);
        };
        auto issue = [&](int stage) {  // its loads
            if (lane == 0) {
                s_item[stage] = ahead;
                if (ahead.chunk < 0) {
                    ptx::mbar_arrive(&s_full[stage]);
                } else {
                    ptx::fence_proxy_async_smem();
                    ptx::mbar_arrive_expect_tx(&s_full[stage], kStage);
#pragma unroll
                    for (int i = 0; i < kIn; ++i)
                        ptx::tma_load_2d(s_tiles + stage * kStage + i * Tile::kTensor, &q.in[i], &s_full[stage],
                                         ahead.tile * kRecTile, ahead.row0);
                }
            }
            __syncwarp();
        };
        for (int i = 0; i < S; ++i) {
            take();
            issue(i);
        }
        take();
        int2 one = make_int2(-1, 0);  // chunk and tile of the item before
        unsigned n = 0;
        bool stop = false, gave_up = false;  // a load did not come; a wait for what is in front ran out
        for (;; ++n) {
            const Item item = s_item[n % S];
            if (item.chunk < 0) break;
            const Lane2 l(item.tile, p.C);
            if (item.flags & kFirst) check_offsets(p.seq, p.status, lane, 32);
            ptx::mbar_wait(&s_free, n & 1u, wd, kDevTimeoutEmpty);
            if (n > 0) issue((n - 1) % S);
            Joining<W, L, kBack> joining(gave_up);
            joining.look(p, item, l);
            ptx::named_barrier(kRunsIn, kAll);
            stop = *static_cast<volatile int *>(&s_abort) != 0;
            if (stop) s.stop = 1;
            else joining.join(p, item, s.run, s.start, l);
            __syncwarp();
            named_barrier_arrive(kStartsIn, kAll);
            if (stop) break;
            if constexpr (kBack) {
                if (one.x >= 0) store_sum<W>(p, one.x, s.sum[~n & 1], Lane2(one.y, p.C));
            }
            if (n > 0) take();
            one = make_int2(item.chunk, item.tile);
        }
        if (stop) {
            if (lane == 0) {  // a load did not come: wait, within the limit, for those in flight
                s_abort = 0;
                const unsigned issued = n ? n + S : S;  // turns whose loads were issued
                for (unsigned i = n; i < issued; ++i) ptx::mbar_wait(&s_full[i % S], i / S & 1u, wd, kDevTimeoutFull);
            }
        } else if constexpr (kBack) {
            ptx::named_barrier(kEnd, kAll);
            if (one.x >= 0) store_sum<W>(p, one.x, s.sum[~n & 1], Lane2(one.y, p.C));
        }
        return;
    }
    // the results of the item before have left its stage
    auto halfway = [&] {
        if (lane == 0) {
            ptx::bulk_wait_group_read<0>();
            ptx::mbar_arrive(&s_free);
        }
    };
    int stage = 0;
    unsigned parity = 0;
    bool fine = true;
    for (unsigned n = 0;; ++n) {
        ptx::mbar_wait(&s_full[stage], parity, wd, kDevTimeoutFull);  // a failure stops the block at the joining
        const Item item = s_item[stage];
        if (item.chunk < 0) break;
        const int row0 = item.row0 + warp * 2 * L;
        const Run run = item.flags & kEdges ? run_of<L>(p.seq, item, row0, chunk_limit(p, item.chunk)) : whole_run<W>(item);
        Tile rows(p, q.out, s_tiles + stage * kStage, warp, item.tile, row0, item.saved + (warp * 2 + half()) * (L / kRecRun));
        const bool edges = row_by_row<L>(item, run);
        if (edges) rows.present = present_rows<L>(run);
        if (item.chunk == 0)
            copy_empty<W>(p.seq, kBack ? p.d_final : p.state, kBack ? p.d_state : p.final_state, p.C, rows.l);
        fine = edges ? work_item_edges<W, kBack>(p, rows, run, s, s.sum[n & 1], warp, halfway)
                     : work_item<false, W, kBack>(p, rows, run, s, s.sum[n & 1], warp, halfway);
        if (!fine) break;
        if (++stage == S) {
            stage = 0;
            parity ^= 1u;
        }
    }
    if (lane == 0) ptx::bulk_wait_group_read<0>();
    if constexpr (kBack) {
        if (fine) ptx::named_barrier(kEnd, kAll);
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

// All ones in the counter and the arrays whose values are their own flags; the decay rates of the channels.
__global__ void __launch_bounds__(256) rec_init_kernel(uint4 *words, size_t n, const float *decay, float kappa, float *rates,
                                                       int C) {
    const size_t step = static_cast<size_t>(gridDim.x) * blockDim.x, i0 = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x;
    for (size_t i = i0; i < n; i += step) words[i] = make_uint4(kFull, kFull, kFull, kFull);
    for (size_t c = i0; c < static_cast<size_t>(C); c += step) rates[c] = decay_rate(decay[c], kappa);
}

// One token: a block takes kRecStepTile channels of one row.  Bound by the launch and two waits for memory, one behind the
// other (a slot's number, its state): one row of 2048 channels 6 us, 64 rows of 4096 8 us, the launch of a graph included.
template <typename T>
__global__ void __launch_bounds__(kRecStepTile / 2) rec_step_kernel(const __grid_constant__ RecStepParams p) {
    const int b = blockIdx.x / p.tiles;
    const int c = blockIdx.x % p.tiles * kRecStepTile + threadIdx.x;
    const Lane2 l(c, c + kRecStepTile / 2, p.C);
    const int slot = p.slots ? p.slots[b] : b;
    const float2 x = load2<T>(static_cast<const T *>(p.x) + static_cast<size_t>(b) * p.ldx, l);
    const float2 ga = load2<T>(static_cast<const T *>(p.ga) + static_cast<size_t>(b) * p.lda, l);
    const float2 gx = load2<T>(static_cast<const T *>(p.gx) + static_cast<size_t>(b) * p.ldg, l);
    const float2 decay = load2<float>(p.decay, l);
    if (slot < 0 || slot >= p.pool) return;
    float *state = p.state + static_cast<size_t>(slot) * p.C;
    const float2 h0 = load2<float>(state, l);
    if (p.slots && slot_named_before(p.slots, b, slot)) {
        if (threadIdx.x == 0) atomicExch(p.status, kDevBadSlot);
        return;
    }
    const float2 rate = make_float2(decay_rate(decay.x, p.kappa), decay_rate(decay.y, p.kappa));
    const Decay d = decay_of(mul2(rate, sigmoid2(ga)));
    const float2 h = fma2(d.a, h0, contribution(d.p, sigmoid2(gx), x));
    store2<T>(static_cast<T *>(p.y) + static_cast<size_t>(b) * p.ldy, h, l);
    store2<float>(state, h, l);
}

// Resident blocks of a kernel, looked up once per device, when its shared memory is allowed.
template <typename K>
cudaError_t resident_blocks(K kernel, int threads, size_t smem, std::atomic<int> *known, int *blocks) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    *blocks = dev < kMaxKnown ? known[dev].load(std::memory_order_relaxed) : 0;
    if (*blocks) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    int per_sm = 0, sms = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    *blocks = (per_sm < 1 ? 1 : per_sm) * sms;
    if (dev < kMaxKnown) known[dev].store(*blocks, std::memory_order_relaxed);
    return cudaSuccess;
}

int grid_of(const RecParams &p, int blocks) {
    const long long items = static_cast<long long>(p.chunks) * p.tiles;
    return static_cast<int>(items < blocks ? items : blocks);
}

template <typename T, bool kBack>
cudaError_t launch_plain(const RecParams &p, cudaStream_t s) {
    constexpr RecShape k = rec_shape(sizeof(T), kBack);
    constexpr size_t smem = 2 * static_cast<size_t>(kBack ? 4 : 3) * TileRun<T, k.rows(), k.run, false>::kTensor;
    static std::atomic<int> known[kMaxKnown];
    int blocks = 0;
    const auto kernel = rec_plain_kernel<T, k.warps, k.run, kBack>;
    const cudaError_t e = resident_blocks(kernel, (k.warps + 1) * 32, smem, known, &blocks);
    if (e != cudaSuccess) return e;
    kernel<<<grid_of(p, blocks), (k.warps + 1) * 32, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T, bool kBack>
cudaError_t launch_tiles(const RecTiles &q, cudaStream_t s) {
    constexpr RecShape k = rec_shape(sizeof(T), kBack);
    constexpr size_t smem = static_cast<size_t>(k.stages) * (kBack ? 4 : 3) * TileRun<T, k.rows(), k.run, true>::kTensor;
    static std::atomic<int> known[kMaxKnown];
    int blocks = 0;
    const auto kernel = rec_tile_kernel<T, k.warps, k.run, k.stages, kBack, k.blocks>;
    const cudaError_t e = resident_blocks(kernel, (k.warps + 1) * 32, smem, known, &blocks);
    if (e != cudaSuccess) return e;
    kernel<<<grid_of(q.p, blocks), (k.warps + 1) * 32, smem, s>>>(q);
    return cudaGetLastError();
}

}  // namespace

// `words`: a multiple of 4.
cudaError_t launch_rec_init(const RecParams &p, size_t words, float *rates, cudaStream_t s) {
    const size_t blocks = (words / 4 + 255) / 256;
    rec_init_kernel<<<static_cast<int>(blocks < 592 ? blocks : 592), 256, 0, s>>>(reinterpret_cast<uint4 *>(p.ticket), words / 4,
                                                                                  p.decay, p.kappa, rates, p.C);
    return cudaGetLastError();
}

cudaError_t launch_rec_plain(const RecParams &p, bool f32, bool back, cudaStream_t s) {
    if (f32) return back ? launch_plain<float, true>(p, s) : launch_plain<float, false>(p, s);
    return back ? launch_plain<__nv_bfloat16, true>(p, s) : launch_plain<__nv_bfloat16, false>(p, s);
}

cudaError_t launch_rec_tiles(const RecTiles &q, bool f32, bool back, cudaStream_t s) {
    if (f32) return back ? launch_tiles<float, true>(q, s) : launch_tiles<float, false>(q, s);
    return back ? launch_tiles<__nv_bfloat16, true>(q, s) : launch_tiles<__nv_bfloat16, false>(q, s);
}

cudaError_t launch_rec_decay(const float *partial, const float *decay, float kappa, float *d_decay, int chunks, int C,
                             int Cpad, cudaStream_t s) {
    rec_decay_kernel<<<(C + 31) / 32, 1024, 0, s>>>(partial, decay, kappa, d_decay, chunks, C, Cpad);
    return cudaGetLastError();
}

cudaError_t launch_rec_step(const RecStepParams &p, bool f32, cudaStream_t s) {
    if (f32) rec_step_kernel<float><<<p.B * p.tiles, kRecStepTile / 2, 0, s>>>(p);
    else rec_step_kernel<__nv_bfloat16><<<p.B * p.tiles, kRecStepTile / 2, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace conv2d_b200
