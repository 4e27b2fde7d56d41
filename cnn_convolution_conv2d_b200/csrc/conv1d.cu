// conv1d.cu -- the causal depthwise convolution over time: forward, backward and one token.
//
//   z[t] = bias + sum_{k<K} w[k] x[t-K+1+k],  y = z or z sigmoid(z)
//
// per channel, t counted inside a sequence, rows before it taken from a carried window.
// All three are bound by HBM: 2K + ~10 operations for 4 to 8 bytes.  A warp takes a strip of
// rows of 32*V channels and slides down it with the last K-1 rows in registers, so each row
// is read once (plus K-1 rows in front of a strip, which the neighbouring warp brings into L2).
// Rows travel ahead of their use in a ring in shared memory that is the warp's own: no block
// barriers, and no registers or load counters held meanwhile (with prefetched rows in registers a
// warp waited for its newest load at every row, 2.4 times slower, or spilled).  Where TMA takes the
// tensors, a lane loads a batch of rows with one instruction, the results take the places of the rows and
// leave the same way: half the instructions of copies and stores by every thread, which is the form for
// other strides and alignments.
// What the time goes into: forward, the rows' travel: with K = 2 and no SiLU it takes 51 us of the 55 below (a copy of those
// bytes takes 41), while the special-function unit is 65% busy and not the limit.  Backward the
// same least work takes 82 us (its bytes 62, with K-1 rows read twice a strip, the sums' reduction and 16 warps an SM); what bf16
// takes above that, up to 98, are instructions whose latency so few warps do not hide (an issue slot in two is used).
// 16384 rows of 4096 channels in bf16, K = 4, SiLU: forward 55 us (4.9 TB/s, 74% of a copy's rate), backward 98 us
// (4.1 TB/s); without SiLU 53 and 86 us; K = 8: 74 and 158 us; 2048 channels in fp32: 55 and 82 us (4.9 TB/s); 32768 rows of
// 1001 channels in bf16, whose rows TMA does not take: 61 and 121 us.
#include <atomic>
#include <type_traits>

#include "ptx.cuh"
#include "sequence.cuh"

namespace conv2d_b200 {
namespace {

// V channels of a row as floats.  kVec: adjacent ones in one load (rows and base aligned to
// V elements, C a multiple of V); else lane + 32*v, for any alignment and any C.
template <typename T, int V, bool kVec>
struct Chan {
    int c;  // first channel of this lane
    int C;
    __device__ Chan(int tile, int C_) : C(C_) {
        const int lane = threadIdx.x & 31;
        c = tile * 32 * V + (kVec ? lane * V : lane);
    }
    __device__ int at(int v) const { return kVec ? c + v : c + 32 * v; }
    __device__ bool has(int v) const { return at(v) < C; }
    __device__ bool any() const { return c < C; }
};

template <typename T, int V> struct alignas(sizeof(T) * V) Raw { T v[V]; };

template <typename T, int V, bool kVec>
__device__ __forceinline__ Raw<T, V> load_raw(const T *row, const Chan<T, V, kVec> &ch) {
    Raw<T, V> r;
    if constexpr (kVec) {
        static_assert(sizeof(r) == 4 || sizeof(r) == 8 || sizeof(r) == 16, "one load");
        if constexpr (sizeof(r) == 16) *reinterpret_cast<uint4 *>(&r) = ch.any() ? *reinterpret_cast<const uint4 *>(row + ch.c) : uint4{0, 0, 0, 0};
        else if constexpr (sizeof(r) == 8) *reinterpret_cast<uint2 *>(&r) = ch.any() ? *reinterpret_cast<const uint2 *>(row + ch.c) : uint2{0, 0};
        else *reinterpret_cast<uint32_t *>(&r) = ch.any() ? *reinterpret_cast<const uint32_t *>(row + ch.c) : 0u;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) r.v[v] = ch.has(v) ? row[ch.at(v)] : from_float<T>(0.f);
    }
    return r;
}

// Copies a lane's channels of a row to its place in the ring, asynchronously where the copy
// instruction has the size (4 bytes).
template <typename T, int V>
__device__ __forceinline__ void copy_ahead(Raw<T, V> *to, const T *row, const Chan<T, V, false> &ch) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (ch.has(v)) cp_async_4(&to->v[v], row + ch.at(v));
    } else {
        *to = load_raw<T, V, false>(row, ch);
    }
}

constexpr int kRing = 3;  // batches in the ring: one at work, two on their way

// A warp's ring of batches of U rows of N tensors.
template <typename T, int V, int U, int N, bool kTma>
struct Ring {
    Raw<T, V> (*rows)[N][U][32];  // [kRing]
    uint64_t *full;               // [kRing], TMA
    int *abort;                   // the block's flag of waits that ran out
    int slot = 0;
    unsigned parity = 0;
    int coming = 0;               // batches fetched and not waited for

    // The batch of rows from `row` on, into the slot `ahead` places on; none from row1 on.
    __device__ __forceinline__ void fetch(const CUtensorMap *maps, const T *const (&from)[N], const long long (&ld)[N], int row,
                                          int row1, int tile, int ahead, const Chan<T, V, kTma> &ch) {
        const int to = slot + ahead >= kRing ? slot + ahead - kRing : slot + ahead;
        if (row < row1) ++coming;
        if constexpr (kTma) {
            __syncwarp();
            if (row < row1 && (threadIdx.x & 31) == 0) {
                ptx::bulk_wait_group_read<0>();  // what left from this slot
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive_expect_tx(&full[to], N * U * 32 * sizeof(Raw<T, V>));
#pragma unroll
                for (int i = 0; i < N; ++i) ptx::tma_load_2d(&rows[to][i][0][0], maps + i, &full[to], tile * 32 * V, row);
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (row + u < row1) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        copy_ahead<T, V>(&rows[to][i][u][threadIdx.x & 31], from[i] + static_cast<size_t>(row + u) * ld[i], ch);
                }
            cp_async_commit();
        }
    }
    __device__ __forceinline__ bool wait(const Conv1dParams &p) {
        if constexpr (kTma) {
            const ptx::Watchdog wd{abort, p.status, static_cast<uint64_t>(p.timeout_ns)};
            if (!ptx::mbar_wait(&full[slot], parity, wd, kDevTimeoutFull)) return false;
        } else {
            cp_async_wait<1>();
        }
        --coming;
        return true;
    }
    // Nothing may be on its way into or out of the ring when its block ends.
    __device__ __forceinline__ void drain(const Conv1dParams &p) {
        if constexpr (kTma) {
            for (; coming > 0; next()) {  // a wait ran out: once more, and for the others, within the limit
                *abort = 0;
                if (!wait(p)) --coming;
            }
            if ((threadIdx.x & 31) == 0) ptx::bulk_wait_group_read<0>();
        }
    }
    __device__ __forceinline__ Raw<T, V> &at(int i, int u) { return rows[slot][i][u][threadIdx.x & 31]; }
    __device__ __forceinline__ void next() {
        if (++slot == kRing) {
            slot = 0;
            parity ^= 1u;
        }
    }
    // Sends the batch's first tensor, whose rows are results now, to the rows from `row` on.
    __device__ __forceinline__ void send(const CUtensorMap *map, int tile, int row) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            ptx::tma_store_2d(map, &rows[slot][0][0][0], tile * 32 * V, row);
            ptx::bulk_commit_group();
        }
    }
};

// The block's rings in shared memory.
template <typename T, int V, int U, int N, bool kTma>
__device__ __forceinline__ Ring<T, V, U, N, kTma> make_ring(Raw<T, V> (*s_rows)[kRing][N][U][32]) {
    __shared__ uint64_t s_full[kConvWarps][kRing];
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5;
    if constexpr (kTma) {
        if (threadIdx.x % 32 == 0) s_abort = 0;  // (every warp the same)
        if ((threadIdx.x & 31) < kRing) ptx::mbar_init(&s_full[warp][threadIdx.x & 31], 1);
        ptx::fence_mbar_init();
        __syncwarp();
    }
    return Ring<T, V, U, N, kTma>{s_rows[warp], s_full[warp], &s_abort};
}

// V channels as pairs: the arithmetic runs two channels to an instruction.
template <int V> struct Pairs { float2 p[V / 2]; };

template <int V>
__device__ __forceinline__ Pairs<V> zero_pairs() {
    Pairs<V> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.p[i] = make_float2(0.f, 0.f);
    return r;
}
template <typename T, int V>
__device__ __forceinline__ Pairs<V> pairs(const Raw<T, V> &raw) {
    Pairs<V> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.p[i] = make_float2(to_float(raw.v[2 * i]), to_float(raw.v[2 * i + 1]));
    return r;
}
template <int V>
__device__ __forceinline__ Pairs<V> pairs(const float (&f)[V]) {
    Pairs<V> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.p[i] = make_float2(f[2 * i], f[2 * i + 1]);
    return r;
}
template <int V>
__device__ __forceinline__ void add_product(Pairs<V> &sum, const Pairs<V> &a, const Pairs<V> &b) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) sum.p[i] = __ffma2_rn(a.p[i], b.p[i], sum.p[i]);
}
// 1 / (1 + e^-z).  Where e^-z passes the largest float, 1/inf = 0 is the right value.
template <int V>
__device__ __forceinline__ Pairs<V> sigmoid(const Pairs<V> &z) {
    Pairs<V> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 t = __fmul2_rn(z.p[i], make_float2(-kLog2e, -kLog2e));
        const float2 d = __fadd2_rn(make_float2(ex2_approx(t.x), ex2_approx(t.y)), make_float2(1.f, 1.f));
        r.p[i] = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    }
    return r;
}
template <int V>
__device__ __forceinline__ Pairs<V> mul(const Pairs<V> &a, const Pairs<V> &b) {
    Pairs<V> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.p[i] = __fmul2_rn(a.p[i], b.p[i]);
    return r;
}
// The derivative of z sigmoid(z) is s (1 + z (1 - s)) with s = sigmoid(z).
template <int V>
__device__ __forceinline__ Pairs<V> silu_slope(const Pairs<V> &z) {
    const Pairs<V> s = sigmoid<V>(z);
    Pairs<V> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const float2 one = make_float2(1.f, 1.f);
        const float2 rest = __ffma2_rn(s.p[i], make_float2(-1.f, -1.f), one);
        r.p[i] = __fmul2_rn(s.p[i], __ffma2_rn(z.p[i], rest, one));
    }
    return r;
}

template <typename T, int V, bool kVec>
__device__ __forceinline__ Pairs<V> load(const T *row, const Chan<T, V, kVec> &ch) {
    return pairs<T, V>(load_raw<T, V, kVec>(row, ch));
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> pack(const Pairs<V> &f) {
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<__nv_bfloat162 *>(&r.v[2 * i]) = __float22bfloat162_rn(f.p[i]);
        } else {
            r.v[2 * i] = f.p[i].x;
            r.v[2 * i + 1] = f.p[i].y;
        }
    }
    return r;
}

template <typename T, int V, bool kVec>
__device__ __forceinline__ void store(T *row, const Pairs<V> &f, const Chan<T, V, kVec> &ch) {
    Raw<T, V> r = pack<T, V>(f);
    if constexpr (kVec) {
        if (ch.any()) {
            if constexpr (sizeof(r) == 16) *reinterpret_cast<uint4 *>(row + ch.c) = *reinterpret_cast<uint4 *>(&r);
            else if constexpr (sizeof(r) == 8) *reinterpret_cast<uint2 *>(row + ch.c) = *reinterpret_cast<uint2 *>(&r);
            else *reinterpret_cast<uint32_t *>(row + ch.c) = *reinterpret_cast<uint32_t *>(&r);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (ch.has(v)) row[ch.at(v)] = r.v[v];
    }
}

template <typename T, int K, int V, bool kVec>
__device__ __forceinline__ void load_weights(Pairs<V> (&w)[K], Pairs<V> &b, const void *wp, const void *bp,
                                             const Chan<T, V, kVec> &ch) {
    const T *wt = static_cast<const T *>(wp), *bt = static_cast<const T *>(bp);
    float f[V];
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = ch.has(v) && bt ? to_float(bt[ch.at(v)]) : 0.f;
    b = pairs<V>(f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = ch.has(v) ? to_float(wt[static_cast<size_t>(ch.at(v)) * K + k]) : 0.f;
        w[k] = pairs<V>(f);
    }
}

// Row `before` rows ahead of a sequence's first one (1 <= before <= K-1).
template <typename T, int K, int V, bool kVec>
__device__ __forceinline__ Pairs<V> load_state(const void *state, int s, int before, const Chan<T, V, kVec> &ch) {
    if (!state) return zero_pairs<V>();
    return load<T, V, kVec>(static_cast<const T *>(state) + (static_cast<size_t>(s) * (K - 1) + (K - 1 - before)) * ch.C, ch);
}

// Where a strip stands among the sequences.
struct Cursor {
    int s;      // current sequence; -1 ahead of the first, nseq behind the last
    int begin;  // its first row
    int end;    // its end; the cursor moves on when a row reaches it
    __device__ void place(const Sequences &q, int row) {
        s = seq_of(q, row);
        if (s < 0) {
            begin = 0;
            end = seq_begin(q, 0);
        } else {
            begin = seq_begin(q, s);
            end = seq_begin(q, s + 1);
            if (row >= end) outside(q);
        }
    }
    __device__ void outside(const Sequences &q) {
        s = q.nseq;
        end = 0x7fffffff;
    }
    // The sequence that begins at `row`: the next one that is not empty.
    __device__ void next(const Sequences &q, int row) {
        ++s;
        while (s < q.nseq && seq_begin(q, s + 1) <= row) ++s;
        if (s >= q.nseq) {
            outside(q);
        } else {
            begin = row;
            end = seq_begin(q, s + 1);
        }
    }
    __device__ bool inside(const Sequences &q) const { return s >= 0 && s < q.nseq; }
};

// The K-1 rows in front of row `row`: of its sequence, or of the window ahead of it.
template <typename T, int K, int V, bool kVec>
__device__ __forceinline__ void load_window(Pairs<V> (&win)[K - 1], const Conv1dParams &p, const Cursor &cur, int row,
                                            const Chan<T, V, kVec> &ch) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int back = K - 1 - j;
        if (!cur.inside(p.seq)) win[j] = zero_pairs<V>();
        else if (row - back >= cur.begin)
            win[j] = load<T, V, kVec>(static_cast<const T *>(p.x) + static_cast<size_t>(row - back) * p.ldx, ch);
        else win[j] = load_state<T, K, V, kVec>(p.state, cur.s, back - (row - cur.begin), ch);
    }
}

// final_state[s]: the last K-1 rows of (window, x).  One block of the grid for a tile and a sequence.
template <typename T, int K, int V, bool kVec>
__device__ __forceinline__ void copy_final(const Conv1dParams &p, int s, const Chan<T, V, kVec> &ch) {
    const int begin = seq_begin(p.seq, s), n = max(0, seq_begin(p.seq, s + 1) - begin);
    for (int j = threadIdx.x >> 5; j < K - 1; j += kConvWarps) {
        const int place = n - (K - 1) + j;
        const Pairs<V> f = place >= 0
                               ? load<T, V, kVec>(static_cast<const T *>(p.x) + static_cast<size_t>(begin + place) * p.ldx, ch)
                               : load_state<T, K, V, kVec>(p.state, s, -place, ch);
        store<T, V, kVec>(static_cast<T *>(p.final_state) + (static_cast<size_t>(s) * (K - 1) + j) * p.C, f, ch);
    }
}

// Moves a window of rows on by one.
template <int N, int V>
__device__ __forceinline__ void shift_in(Pairs<V> (&win)[N], const Pairs<V> &row) {
#pragma unroll
    for (int j = 0; j + 1 < N; ++j) win[j] = win[j + 1];
    win[N - 1] = row;
}

template <typename T, int K, int V, bool kVec>
__global__ void __launch_bounds__(kConvWarps * 32, kConvBlocks) conv1d_forward_kernel(const __grid_constant__ Conv1dTiles q) {
    constexpr int U = kConvBatch / sizeof(T);
    const Conv1dParams &p = q.p;
    const int tile = blockIdx.x % p.tiles, block = blockIdx.x / p.tiles;  // neighbours share rows
    const Chan<T, V, kVec> ch(tile, p.C);
    if (blockIdx.x == 0) check_offsets(p.seq, p.status);
    if (block >= p.row_blocks) {
        copy_final<T, K, V, kVec>(p, block - p.row_blocks, ch);
        return;
    }
    const long long first = (static_cast<long long>(block) * kConvWarps + (threadIdx.x >> 5)) * p.strip;
    if (first >= p.seq.rows) return;
    const int row0 = static_cast<int>(first), row1 = min(p.seq.rows - row0, p.strip) + row0;
    const T *x = static_cast<const T *>(p.x);
    T *y = static_cast<T *>(p.y);
    __shared__ __align__(128) Raw<T, V> s_rows[kConvWarps][kRing][1][U][32];
    auto ring = make_ring<T, V, U, 1, kVec>(s_rows);
    auto fetch = [&](int row, int ahead) { ring.fetch(&q.in[0], {x}, {p.ldx}, row, row1, tile, ahead, ch); };
    fetch(row0, 0);
    fetch(row0 + U, 1);
    Pairs<V> w[K], b, win[K - 1];
    load_weights<T, K, V, kVec>(w, b, p.w, p.bias, ch);
    Cursor cur;
    cur.place(p.seq, row0);
    load_window<T, K, V, kVec>(win, p, cur, row0, ch);
    auto result = [&](const Pairs<V> *rows) {  // from the K rows that end with the result's own
        Pairs<V> z = b;
#pragma unroll
        for (int k = 0; k < K; ++k) add_product<V>(z, w[k], rows[k]);
        return p.silu ? mul<V>(z, sigmoid<V>(z)) : z;
    };
    for (int row = row0; row < row1; row += U, ring.next()) {
        if (!ring.wait(p)) break;
        if (cur.inside(p.seq) && row + U <= min(cur.end, row1)) {
            Pairs<V> all[K - 1 + U];
#pragma unroll
            for (int j = 0; j < K - 1; ++j) all[j] = win[j];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u == U / 2) fetch(row + 2 * U, 2);  // by now what the last batch left has gone
                Raw<T, V> &at = ring.at(0, u);
                all[K - 1 + u] = pairs<T, V>(at);
                if constexpr (kVec) at = pack<T, V>(result(all + u));
                else store<T, V, kVec>(y + static_cast<size_t>(row + u) * p.ldy, result(all + u), ch);
            }
            if constexpr (kVec) ring.send(&q.out, tile, row);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) win[j] = all[U + j];
        } else {  // a sequence or the strip ends here: row by row
            fetch(row + 2 * U, 2);
#pragma unroll 1
            for (int u = 0; u < U && row + u < row1; ++u) {
                if (row + u >= cur.end) {
                    cur.next(p.seq, row + u);
                    load_window<T, K, V, kVec>(win, p, cur, row + u, ch);
                }
                Pairs<V> all[K];
#pragma unroll
                for (int j = 0; j < K - 1; ++j) all[j] = win[j];
                all[K - 1] = pairs<T, V>(ring.at(0, u));
                if (cur.inside(p.seq)) store<T, V, kVec>(y + static_cast<size_t>(row + u) * p.ldy, result(all), ch);
                shift_in<K - 1, V>(win, all[K - 1]);
            }
        }
    }
    ring.drain(p);
}

// Backward.  Going down the rows, row t's dz completes the gradient of row t-(K-1):
// dx[t-(K-1)] = sum_j w[K-1-j] dz[t-(K-1)+j], from the last K-1 dz's in registers (zeros ahead of the
// sequence; a target ahead of the sequence is a row of the carried window).  K-1 rows behind the strip
// are read for the dz's that its last rows still need.
template <typename T, int K, int V, bool kVec>
__global__ void __launch_bounds__(kConvWarps * 32, kConvBlocksBack) conv1d_backward_kernel(const __grid_constant__ Conv1dTiles q) {
    constexpr int U = kConvBatch / sizeof(T);
    const Conv1dParams &p = q.p;
    const int tile = blockIdx.x % p.tiles, block = blockIdx.x / p.tiles;  // neighbours share rows
    const Chan<T, V, kVec> ch(tile, p.C);
    if (blockIdx.x == 0) check_offsets(p.seq, p.status);
    const int warp = threadIdx.x >> 5;
    if (block >= p.row_blocks) {  // d_state of an empty sequence: d_final itself
        const int s = block - p.row_blocks;
        if (seq_begin(p.seq, s + 1) > seq_begin(p.seq, s)) return;
        for (int j = warp; j < K - 1; j += kConvWarps)
            store<T, V, kVec>(static_cast<T *>(p.d_state) + (static_cast<size_t>(s) * (K - 1) + j) * p.C,
                              load_state<T, K, V, kVec>(p.d_final, s, K - 1 - j, ch), ch);
        return;
    }
    extern __shared__ __align__(128) uint8_t s_dynamic[];
    auto s_rows = reinterpret_cast<Raw<T, V> (*)[kRing][2][U][32]>(s_dynamic);
    float2 (*s_sum)[16 * V] = reinterpret_cast<float2 (*)[16 * V]>(s_dynamic);  // once the rings are done with
    auto ring = make_ring<T, V, U, 2, kVec>(s_rows);
    Pairs<V> w[K], b, dw[K], db = zero_pairs<V>();
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k] = zero_pairs<V>();
    const long long first = (static_cast<long long>(block) * kConvWarps + warp) * p.strip;
    if (first < p.seq.rows) {
        const int row0 = static_cast<int>(first), row1 = min(p.seq.rows - row0, p.strip) + row0;
        const int last = min(p.seq.rows - row1, K - 1) + row1;  // rows read
        const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
        T *dx = static_cast<T *>(p.y);
        auto fetch = [&](int row, int ahead) { ring.fetch(&q.in[0], {x, dy}, {p.ldx, p.lddy}, row, last, tile, ahead, ch); };
        fetch(row0, 0);
        fetch(row0 + U, 1);
        load_weights<T, K, V, kVec>(w, b, p.w, p.bias, ch);
        Pairs<V> win[K - 1], past[K - 1];  // x and dz of the K-1 rows before
        Cursor cur;
        cur.place(p.seq, row0);
        load_window<T, K, V, kVec>(win, p, cur, row0, ch);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) past[j] = zero_pairs<V>();
        // dz of a row from its dy, and the K rows of x that end with it
        auto slope = [&](const Pairs<V> &d, const Pairs<V> *rows) {
            if (!p.silu) return d;
            Pairs<V> z = b;
#pragma unroll
            for (int k = 0; k < K; ++k) add_product<V>(z, w[k], rows[k]);
            return mul<V>(d, silu_slope<V>(z));
        };
        auto sums = [&](const Pairs<V> &d, const Pairs<V> *rows) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) db.p[i] = __fadd2_rn(db.p[i], d.p[i]);
#pragma unroll
            for (int k = 0; k < K; ++k) add_product<V>(dw[k], d, rows[k]);
        };
        auto gradient = [&](const Pairs<V> *dz) {  // of the first of K rows, from their dz
            Pairs<V> g = mul<V>(w[K - 1], dz[0]);
#pragma unroll
            for (int j = 1; j < K; ++j) add_product<V>(g, w[K - 1 - j], dz[j]);
            return g;
        };
        // The gradient of the row K-1 rows ahead of row t of sequence `cur`, to where it belongs.
        auto emit = [&](int t, const Pairs<V> &g) {
            const int target = t - (K - 1);
            if (target >= cur.begin) {
                if (target >= row0 && target < row1) store<T, V, kVec>(dx + static_cast<size_t>(target) * p.ldy, g, ch);
            } else if (p.d_state && cur.begin >= row0 && cur.begin < row1) {
                store<T, V, kVec>(static_cast<T *>(p.d_state) +
                                      (static_cast<size_t>(cur.s) * (K - 1) + (target - cur.begin + K - 1)) * p.C, g, ch);
            }
        };
        // Behind a sequence's last row: its last K-1 rows, with what d_final sends them, are finished.
        auto flush = [&]() {
#pragma unroll 1
            for (int i = 0; i < K - 1; ++i) {
                Pairs<V> g = load_state<T, K, V, kVec>(p.d_final, cur.s, K - 1 - i, ch);
#pragma unroll
                for (int j = 0; j < K - 1; ++j) add_product<V>(g, w[K - 1 - j], past[j]);
                emit(cur.end + i, g);
                shift_in<K - 1, V>(past, zero_pairs<V>());
            }
        };
        // U rows of one sequence, all of whose gradients belong to it too.  kWhole: those of the strip, sent together
        // (without the checks of the other form: 102 -> 98 us).
        auto batch = [&](int row, auto whole) {
            constexpr bool kWhole = decltype(whole)::value;
            Pairs<V> all[K - 1 + U], dz[K - 1 + U];
            const int target = row - (K - 1);  // the first of the rows whose gradients are finished
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                all[j] = win[j];
                dz[j] = past[j];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u == U / 2) fetch(row + 2 * U, 2);
                Raw<T, V> &at = ring.at(0, u);
                all[K - 1 + u] = pairs<T, V>(at);
                dz[K - 1 + u] = slope(pairs<T, V>(ring.at(1, u)), all + u);
                if (kWhole || row + u < row1) sums(dz[K - 1 + u], all + u);
                const Pairs<V> g = gradient(dz + u);
                if (kWhole) at = pack<T, V>(g);
                else if (target + u >= row0 && target + u < row1)  // (rows behind `last` hold nothing, and end here)
                    store<T, V, kVec>(dx + static_cast<size_t>(target + u) * p.ldy, g, ch);
            }
            if (kWhole) ring.send(&q.out, tile, target);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                win[j] = all[U + j];
                past[j] = dz[U + j];
            }
        };
        bool done = false;
        for (int row = row0; row < last; row += U, ring.next()) {
            if (!ring.wait(p)) break;
            if (done) continue;  // (two batches at most: K-1 rows behind the strip)
            if (cur.inside(p.seq) && row + U <= cur.end && row - (K - 1) >= cur.begin) {
                if (kVec && row - (K - 1) >= row0 && row + U <= row1) batch(row, std::true_type{});
                else batch(row, std::false_type{});
            } else {  // a sequence begins or ends here: row by row
                fetch(row + 2 * U, 2);
#pragma unroll 1
                for (int u = 0; u < U && row + u < last; ++u) {
                    const int t = row + u;
                    if (t >= cur.end) {
                        if (cur.inside(p.seq)) flush();
                        cur.next(p.seq, t);
                        load_window<T, K, V, kVec>(win, p, cur, t, ch);
                        // what follows the strip's last sequence is none of the strip's
                        if (t >= row1) cur.outside(p.seq);
                    }
                    if (!cur.inside(p.seq)) {
                        if (t >= row1) {
                            done = true;
                            break;
                        }
                        continue;
                    }
                    Pairs<V> all[K], dz[K];
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) {
                        all[j] = win[j];
                        dz[j] = past[j];
                    }
                    all[K - 1] = pairs<T, V>(ring.at(0, u));
                    dz[K - 1] = slope(pairs<T, V>(ring.at(1, u)), all);
                    if (t < row1) sums(dz[K - 1], all);
                    emit(t, gradient(dz));
                    shift_in<K - 1, V>(win, all[K - 1]);
                    shift_in<K - 1, V>(past, dz[K - 1]);
                }
            }
        }
        // the rows ended with this sequence
        if (!done && cur.inside(p.seq) && last >= cur.end) flush();
        ring.drain(p);
    }
    // The block's sums of dw and db: its warps' in order, so that equal inputs give equal bits.
#pragma unroll
    for (int k = 0; k < K + 1; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V / 2; ++i) s_sum[warp][i * 32 + (threadIdx.x & 31)] = k < K ? dw[k < K ? k : 0].p[i] : db.p[i];
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * V; i += kConvWarps * 32) {
            const int v = i >> 5 << 1, lane = i & 31;
            const int c = tile * 32 * V + (kVec ? lane * V + v : lane + 32 * v);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int q = 0; q < kConvWarps; ++q) sum = __fadd2_rn(sum, s_sum[q][i]);
            float *out = p.partial + (static_cast<size_t>(block) * (K + 1) + k) * p.C;
            if (c < p.C) out[c] = sum.x;
            if (c + (kVec ? 1 : 32) < p.C) out[c + (kVec ? 1 : 32)] = sum.y;
        }
    }
}

// dw[c][k] and db[c] from the row blocks' sums.  A block: 32 channels of one k, 32 groups of row blocks.
template <typename T>
__global__ void __launch_bounds__(1024) conv1d_reduce_kernel(const float *partial, T *dw, T *db, int row_blocks, int C,
                                                             int K) {
    __shared__ float s_sum[32][33];
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
    float sum = 0.f;
    if (c < C)
        for (int r = group; r < row_blocks; r += 32) sum += partial[(static_cast<size_t>(r) * (K + 1) + k) * C + c];
    s_sum[group][lane] = sum;
    __syncthreads();
    // lane l of warp g now holds group l's sum of channel g
    sum = s_sum[lane][group];
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const int out = blockIdx.x * 32 + group;
    if (lane == 0 && out < C) {
        if (k < K) dw[static_cast<size_t>(out) * K + k] = from_float<T>(sum);
        else if (db) db[out] = from_float<T>(sum);
    }
}

// One token: a warp takes 32 * V channels of one row.  Bound by the launch and two waits for memory, one behind the other (a
// slot's number, its window): 64 rows of 4096 channels 8 us, the launch of a graph included.
template <typename T, int K, int V, bool kVec>
__global__ void __launch_bounds__(128) conv1d_step_kernel(const __grid_constant__ Conv1dStepParams p) {
    const Chan<T, V, kVec> ch(blockIdx.x % p.tiles * 4 + (threadIdx.x >> 5), p.C);
    const int b = blockIdx.x / p.tiles;
    const int slot = p.slots ? p.slots[b] : b;
    const Pairs<V> x = load<T, V, kVec>(static_cast<const T *>(p.x) + static_cast<size_t>(b) * p.ldx, ch);
    Pairs<V> w[K], z, win[K - 1];
    load_weights<T, K, V, kVec>(w, z, p.w, p.bias, ch);
    if (slot < 0 || slot >= p.pool) return;  // the whole block: b names no window
    T *state = static_cast<T *>(p.state) + static_cast<size_t>(slot) * (K - 1) * p.C;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) win[j] = load<T, V, kVec>(state + static_cast<size_t>(j) * p.C, ch);
    if (p.slots && slot_named_before(p.slots, b, slot)) {
        if (threadIdx.x == 0) atomicExch(p.status, kDevBadSlot);
        return;
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k) add_product<V>(z, w[k], win[k]);
    add_product<V>(z, w[K - 1], x);
    if (p.silu) z = mul<V>(z, sigmoid<V>(z));
    store<T, V, kVec>(static_cast<T *>(p.y) + static_cast<size_t>(b) * p.ldy, z, ch);
#pragma unroll
    for (int j = 0; j + 1 < K - 1; ++j) store<T, V, kVec>(state + static_cast<size_t>(j) * p.C, win[j + 1], ch);
    store<T, V, kVec>(state + static_cast<size_t>(K - 2) * p.C, x, ch);
}

// Channels of one lane: few enough that weights, window and gradient sums stay in registers.
constexpr int lane_channels(int K) { return K <= 4 ? 4 : 2; }

template <typename T, bool kVec, int K>
cudaError_t forward_k(const Conv1dTiles &q, cudaStream_t s) {
    constexpr int V = lane_channels(K);
    const Conv1dParams &p = q.p;
    const int grid = p.tiles * (p.row_blocks + (p.final_state ? p.seq.nseq : 0));
    conv1d_forward_kernel<T, K, V, kVec><<<grid, kConvWarps * 32, 0, s>>>(q);
    return cudaGetLastError();
}

template <typename T, bool kVec, int K>
cudaError_t backward_k(const Conv1dTiles &q, cudaStream_t s) {
    constexpr int V = lane_channels(K);
    const Conv1dParams &p = q.p;
    const int grid = p.tiles * (p.row_blocks + (p.d_state ? p.seq.nseq : 0));
    constexpr size_t smem = kConvWarps * kRing * 2 * (kConvBatch / sizeof(T)) * 32 * sizeof(Raw<T, V>);
    const auto kernel = conv1d_backward_kernel<T, K, V, kVec>;
    static std::atomic<uint64_t> allowed{0};  // a bit for each device on which the kernel may have that much
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    kernel<<<grid, kConvWarps * 32, smem, s>>>(q);
    return cudaGetLastError();
}

template <typename T, bool kVec, int K>
cudaError_t step_k(const Conv1dStepParams &p, cudaStream_t s) {
    constexpr int V = lane_channels(K);
    conv1d_step_kernel<T, K, V, kVec><<<p.tiles * p.B, 128, 0, s>>>(p);
    return cudaGetLastError();
}

#define CONV1D_BY_K(fn, k, p, s)                \
    switch (k) {                                \
        case 2: return fn<T, kVec, 2>(p, s);    \
        case 3: return fn<T, kVec, 3>(p, s);    \
        case 4: return fn<T, kVec, 4>(p, s);    \
        case 5: return fn<T, kVec, 5>(p, s);    \
        case 6: return fn<T, kVec, 6>(p, s);    \
        case 7: return fn<T, kVec, 7>(p, s);    \
        case 8: return fn<T, kVec, 8>(p, s);    \
        default: return cudaErrorInvalidValue;  \
    }

template <typename T, bool kVec> cudaError_t forward_t(const Conv1dTiles &q, cudaStream_t s) { CONV1D_BY_K(forward_k, q.p.K, q, s) }
template <typename T, bool kVec> cudaError_t backward_t(const Conv1dTiles &q, cudaStream_t s) { CONV1D_BY_K(backward_k, q.p.K, q, s) }
template <typename T, bool kVec> cudaError_t step_t(const Conv1dStepParams &p, cudaStream_t s) { CONV1D_BY_K(step_k, p.K, p, s) }

}  // namespace

int conv1d_channels_per_block(int K) { return 32 * lane_channels(K); }

// Rows of a warp's strip, a multiple of 8.  Forward: 64, fewer where that leaves SMs without a block.  Backward, which
// has fewer warps on an SM: up to 128, so that the rounds of blocks on the device, each as long as a strip and what it
// costs to begin one (some 12 rows' time), take the least together.  At 16384 rows of 4096 channels the last round of
// strips of 64 is mostly empty: backward 115 -> 102 us, while forward, whose warps wait for memory, loses (55 -> 57 us).
int conv1d_strip(int rows, int C, int K, int sms, bool back) {
    const long long tiles = (C + conv1d_channels_per_block(K) - 1) / conv1d_channels_per_block(K);
    const auto blocks = [&](int strip) { return tiles * ((rows + kConvWarps * strip - 1LL) / (kConvWarps * strip)); };
    int best = 64;
    if (!back || sms < 1) {
        while (best > 8 && blocks(best) < 4LL * sms) best >>= 1;
        return best;
    }
    const long long resident = static_cast<long long>(sms) * kConvBlocksBack;
    const auto time = [&](int strip) { return (blocks(strip) + resident - 1) / resident * (strip + 12); };
    for (int strip = 8; strip <= 128; strip += 8)
        if (time(strip) < time(best) || (time(strip) == time(best) && strip > best)) best = strip;
    return best;
}

cudaError_t launch_conv1d_forward(const Conv1dTiles &q, bool f32, bool tma, cudaStream_t s) {
    if (f32) return tma ? forward_t<float, true>(q, s) : forward_t<float, false>(q, s);
    return tma ? forward_t<__nv_bfloat16, true>(q, s) : forward_t<__nv_bfloat16, false>(q, s);
}

cudaError_t launch_conv1d_backward(const Conv1dTiles &q, bool f32, bool tma, cudaStream_t s) {
    if (f32) return tma ? backward_t<float, true>(q, s) : backward_t<float, false>(q, s);
    return tma ? backward_t<__nv_bfloat16, true>(q, s) : backward_t<__nv_bfloat16, false>(q, s);
}

cudaError_t launch_conv1d_reduce(const float *partial, void *dw, void *db, int row_blocks, int C, int K, bool f32,
                                 cudaStream_t s) {
    const dim3 grid((C + 31) / 32, K + 1);
    if (f32)
        conv1d_reduce_kernel<float><<<grid, 1024, 0, s>>>(partial, static_cast<float *>(dw), static_cast<float *>(db),
                                                          row_blocks, C, K);
    else
        conv1d_reduce_kernel<__nv_bfloat16><<<grid, 1024, 0, s>>>(partial, static_cast<__nv_bfloat16 *>(dw),
                                                                  static_cast<__nv_bfloat16 *>(db), row_blocks, C, K);
    return cudaGetLastError();
}

cudaError_t launch_conv1d_step(const Conv1dStepParams &p, bool f32, bool vec, cudaStream_t s) {
    if (f32) return vec ? step_t<float, true>(p, s) : step_t<float, false>(p, s);
    return vec ? step_t<__nv_bfloat16, true>(p, s) : step_t<__nv_bfloat16, false>(p, s);
}

}  // namespace conv2d_b200
