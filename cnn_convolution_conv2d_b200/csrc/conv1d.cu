// conv1d.cu -- the causal depthwise convolution over time: forward, backward and one token.
//
//   z[t] = bias + sum_{k<K} w[k] x[t-K+1+k],  y = z or z sigmoid(z)
//
// per channel, t counted inside a sequence, rows before it taken from a carried window.
// All three are bound by HBM: 2K + ~10 operations for 4 to 8 bytes.  A warp takes a strip of
// rows of 32*V channels and slides down it with the last K-1 rows in registers, so each row
// is read once (plus K-1 rows in front of a strip, which the neighbouring warp brings into L2).
// Rows are loaded U at a time ahead of the arithmetic to keep enough bytes in flight.
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

template <typename T, int V> struct Raw { T v[V]; };

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

template <typename T, int V, bool kVec>
__device__ __forceinline__ void load(float (&f)[V], const T *row, const Chan<T, V, kVec> &ch) {
    const Raw<T, V> r = load_raw<T, V, kVec>(row, ch);
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = to_float(r.v[v]);
}

template <typename T, int V, bool kVec>
__device__ __forceinline__ void store(T *row, const float (&f)[V], const Chan<T, V, kVec> &ch) {
    Raw<T, V> r;
#pragma unroll
    for (int v = 0; v < V; ++v) r.v[v] = from_float<T>(f[v]);
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
__device__ __forceinline__ void load_weights(float (&w)[K][V], float (&b)[V], const void *wp, const void *bp,
                                             const Chan<T, V, kVec> &ch) {
    const T *wt = static_cast<const T *>(wp), *bt = static_cast<const T *>(bp);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool has = ch.has(v);
        b[v] = has && bt ? to_float(bt[ch.at(v)]) : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][v] = has ? to_float(wt[static_cast<size_t>(ch.at(v)) * K + k]) : 0.f;
    }
}

// Row `before` rows ahead of a sequence's first one (1 <= before <= K-1).
template <typename T, int K, int V, bool kVec>
__device__ __forceinline__ void load_state(float (&f)[V], const void *state, int s, int before,
                                           const Chan<T, V, kVec> &ch) {
    if (state) {
        load<T, V, kVec>(f, static_cast<const T *>(state) + (static_cast<size_t>(s) * (K - 1) + (K - 1 - before)) * ch.C, ch);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = 0.f;
    }
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

// final_state[s]: the last K-1 rows of (window, x).  One block of the grid for a tile and a sequence.
template <typename T, int K, int V, bool kVec>
__device__ __forceinline__ void copy_final(const Conv1dParams &p, int s, const Chan<T, V, kVec> &ch) {
    const int begin = seq_begin(p.seq, s), n = max(0, seq_begin(p.seq, s + 1) - begin);
    for (int j = threadIdx.x >> 5; j < K - 1; j += kConvWarps) {
        const int place = n - (K - 1) + j;
        float f[V];
        if (place >= 0) load<T, V, kVec>(f, static_cast<const T *>(p.x) + static_cast<size_t>(begin + place) * p.ldx, ch);
        else load_state<T, K, V, kVec>(f, p.state, s, -place, ch);
        store<T, V, kVec>(static_cast<T *>(p.final_state) + (static_cast<size_t>(s) * (K - 1) + j) * p.C, f, ch);
    }
}

template <typename T, int K, int V, bool kVec>
__global__ void __launch_bounds__(kConvWarps * 32) conv1d_forward_kernel(Conv1dParams p) {
    constexpr int U = 8;
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
    float w[K][V], b[V], win[K - 1][V];
    load_weights<T, K, V, kVec>(w, b, p.w, p.bias, ch);
    Cursor cur;
    cur.place(p.seq, row0);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {  // win[j]: row row0 - (K-1) + j
        const int back = K - 1 - j;
#pragma unroll
        for (int v = 0; v < V; ++v) win[j][v] = 0.f;
        if (cur.inside(p.seq)) {
            if (row0 - back >= cur.begin) load<T, V, kVec>(win[j], x + static_cast<size_t>(row0 - back) * p.ldx, ch);
            else load_state<T, K, V, kVec>(win[j], p.state, cur.s, back - (row0 - cur.begin), ch);
        }
    }
    for (int row = row0; row < row1; row += U) {
        Raw<T, V> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (row + u < row1) raw[u] = load_raw<T, V, kVec>(x + static_cast<size_t>(row + u) * p.ldx, ch);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row + u >= row1) break;
            if (row + u >= cur.end) {
                cur.next(p.seq, row + u);
                if (cur.inside(p.seq)) {
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) load_state<T, K, V, kVec>(win[j], p.state, cur.s, K - 1 - j, ch);
                }
            }
            float z[V], xv[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                xv[v] = to_float(raw[u].v[v]);
                z[v] = b[v];
            }
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) z[v] = fmaf(w[k][v], win[k][v], z[v]);
#pragma unroll
            for (int v = 0; v < V; ++v) z[v] = fmaf(w[K - 1][v], xv[v], z[v]);
            if (p.silu) {
#pragma unroll
                for (int v = 0; v < V; ++v) z[v] *= sigmoid(z[v]);
            }
            if (cur.inside(p.seq)) store<T, V, kVec>(y + static_cast<size_t>(row + u) * p.ldy, z, ch);
#pragma unroll
            for (int j = 0; j + 1 < K - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) win[j][v] = win[j + 1][v];
#pragma unroll
            for (int v = 0; v < V; ++v) win[K - 2][v] = xv[v];
        }
    }
}

// Backward.  Going down the rows, row t's dz completes the gradient of row t-(K-1), so the last
// K-1 dz's wait in registers as partly summed gradients: dxp[j] is the sum so far for the row
// K-1-j rows back (a row ahead of the sequence is a row of the carried window).  K-1 rows behind
// the strip are read for the dz's that its last rows still need.
template <typename T, int K, int V, bool kVec>
__global__ void __launch_bounds__(kConvWarps * 32) conv1d_backward_kernel(Conv1dParams p) {
    constexpr int U = 4;
    __shared__ float s_sum[kConvWarps][32 * V];
    const int tile = blockIdx.x % p.tiles, block = blockIdx.x / p.tiles;  // neighbours share rows
    const Chan<T, V, kVec> ch(tile, p.C);
    if (blockIdx.x == 0) check_offsets(p.seq, p.status);
    const int warp = threadIdx.x >> 5;
    if (block >= p.row_blocks) {  // d_state of an empty sequence: d_final itself
        const int s = block - p.row_blocks;
        if (seq_begin(p.seq, s + 1) > seq_begin(p.seq, s)) return;
        for (int j = warp; j < K - 1; j += kConvWarps) {
            float f[V];
            load_state<T, K, V, kVec>(f, p.d_final, s, K - 1 - j, ch);
            store<T, V, kVec>(static_cast<T *>(p.d_state) + (static_cast<size_t>(s) * (K - 1) + j) * p.C, f, ch);
        }
        return;
    }
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    T *dx = static_cast<T *>(p.y);
    float w[K][V], b[V], dw[K][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][v] = 0.f;
    }
    const long long first = (static_cast<long long>(block) * kConvWarps + warp) * p.strip;
    if (first < p.seq.rows) {
        const int row0 = static_cast<int>(first), row1 = min(p.seq.rows - row0, p.strip) + row0;
        const int last = min(p.seq.rows - row1, K - 1) + row1;  // rows read
        load_weights<T, K, V, kVec>(w, b, p.w, p.bias, ch);
        float win[K - 1][V], dxp[K][V];
        Cursor cur;
        cur.place(p.seq, row0);
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) dxp[j][v] = 0.f;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int back = K - 1 - j;
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = 0.f;
            if (cur.inside(p.seq)) {
                if (row0 - back >= cur.begin) load<T, V, kVec>(win[j], x + static_cast<size_t>(row0 - back) * p.ldx, ch);
                else load_state<T, K, V, kVec>(win[j], p.state, cur.s, back - (row0 - cur.begin), ch);
            }
        }
        // Writes the finished gradient of the row K-1 rows ahead of `t` of sequence `cur`.
        auto emit = [&](int t) {
            const int target = t - (K - 1);
            if (target >= cur.begin) {
                if (target >= row0 && target < row1) store<T, V, kVec>(dx + static_cast<size_t>(target) * p.ldy, dxp[0], ch);
            } else if (p.d_state && cur.begin >= row0 && cur.begin < row1) {
                store<T, V, kVec>(static_cast<T *>(p.d_state) +
                                      (static_cast<size_t>(cur.s) * (K - 1) + (target - cur.begin + K - 1)) * p.C,
                                  dxp[0], ch);
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) dxp[j][v] = dxp[j + 1][v];
#pragma unroll
            for (int v = 0; v < V; ++v) dxp[K - 1][v] = 0.f;
        };
        // Behind a sequence's last row: its last K-1 rows (and d_final) are finished.
        auto flush = [&](int end) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                if (p.d_final) {
                    float f[V];
                    load_state<T, K, V, kVec>(f, p.d_final, cur.s, K - 1 - j, ch);
#pragma unroll
                    for (int v = 0; v < V; ++v) dxp[0][v] += f[v];
                }
                emit(end + j);
            }
        };
        bool done = false;
        for (int row = row0; row < last && !done; row += U) {
            Raw<T, V> rx[U], rd[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (row + u < last) {
                    rx[u] = load_raw<T, V, kVec>(x + static_cast<size_t>(row + u) * p.ldx, ch);
                    rd[u] = load_raw<T, V, kVec>(dy + static_cast<size_t>(row + u) * p.lddy, ch);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = row + u;
                if (t >= last || done) break;
                if (t >= cur.end) {
                    if (cur.inside(p.seq)) flush(cur.end);
                    if (t >= row1) {  // what follows the strip's last sequence is none of the strip's
                        done = true;
                        break;
                    }
                    cur.next(p.seq, t);
                    if (cur.inside(p.seq)) {
#pragma unroll
                        for (int j = 0; j < K - 1; ++j) load_state<T, K, V, kVec>(win[j], p.state, cur.s, K - 1 - j, ch);
                    }
                }
                if (!cur.inside(p.seq)) {
                    if (t >= row1) done = true;
                    continue;
                }
                float xv[V], dz[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    xv[v] = to_float(rx[u].v[v]);
                    dz[v] = to_float(rd[u].v[v]);
                }
                if (p.silu) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float z = b[v];
#pragma unroll
                        for (int k = 0; k < K - 1; ++k) z = fmaf(w[k][v], win[k][v], z);
                        z = fmaf(w[K - 1][v], xv[v], z);
                        const float sg = sigmoid(z);
                        dz[v] *= sg * fmaf(z, 1.f - sg, 1.f);
                    }
                }
                if (t < row1) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        db[v] += dz[v];
#pragma unroll
                        for (int k = 0; k < K - 1; ++k) dw[k][v] = fmaf(dz[v], win[k][v], dw[k][v]);
                        dw[K - 1][v] = fmaf(dz[v], xv[v], dw[K - 1][v]);
                    }
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int k = 0; k < K; ++k) dxp[k][v] = fmaf(w[k][v], dz[v], dxp[k][v]);
#pragma unroll
                    for (int j = 0; j + 1 < K - 1; ++j) win[j][v] = win[j + 1][v];
                    win[K - 2][v] = xv[v];
                }
                emit(t);
            }
        }
        // the rows ended with this sequence
        if (!done && cur.inside(p.seq) && last >= cur.end) flush(cur.end);
    }
    // The block's sums of dw and db: its warps' in order, so that equal inputs give equal bits.
#pragma unroll
    for (int k = 0; k < K + 1; ++k) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) s_sum[warp][v * 32 + (threadIdx.x & 31)] = k < K ? dw[k < K ? k : 0][v] : db[v];
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * V; i += kConvWarps * 32) {
            const int v = i >> 5, lane = i & 31;
            const int c = tile * 32 * V + (kVec ? lane * V + v : lane + 32 * v);
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < kConvWarps; ++q) sum += s_sum[q][i];
            if (c < p.C) p.partial[(static_cast<size_t>(block) * (K + 1) + k) * p.C + c] = sum;
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

template <typename T, int K, int V, bool kVec>
__global__ void __launch_bounds__(128) conv1d_step_kernel(Conv1dStepParams p) {
    const Chan<T, V, kVec> ch(blockIdx.x % p.tiles * 4 + (threadIdx.x >> 5), p.C);
    const int b = blockIdx.x / p.tiles;
    const int slot = p.slots ? p.slots[b] : b;
    float w[K][V], bias[V], xv[V];
    load<T, V, kVec>(xv, static_cast<const T *>(p.x) + static_cast<size_t>(b) * p.ldx, ch);
    load_weights<T, K, V, kVec>(w, bias, p.w, p.bias, ch);
    if (slot < 0 || slot >= p.pool) return;  // the whole block: b names no window
    T *state = static_cast<T *>(p.state) + static_cast<size_t>(slot) * (K - 1) * p.C;
    float win[K - 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load<T, V, kVec>(win[j], state + static_cast<size_t>(j) * p.C, ch);
    if (p.slots && slot_named_before(p.slots, b, slot)) {
        if (threadIdx.x == 0) atomicExch(p.status, kDevBadSlot);
        return;
    }
    float z[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        z[v] = bias[v];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) z[v] = fmaf(w[k][v], win[k][v], z[v]);
        z[v] = fmaf(w[K - 1][v], xv[v], z[v]);
        if (p.silu) z[v] *= sigmoid(z[v]);
    }
    store<T, V, kVec>(static_cast<T *>(p.y) + static_cast<size_t>(b) * p.ldy, z, ch);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        if (j + 1 < K - 1) store<T, V, kVec>(state + static_cast<size_t>(j) * p.C, win[j + 1 < K - 1 ? j + 1 : 0], ch);
        else store<T, V, kVec>(state + static_cast<size_t>(j) * p.C, xv, ch);
    }
}

// Channels of one lane: few enough that weights, window and gradient sums stay in registers.
constexpr int lane_channels(int K) { return K <= 4 ? 4 : 2; }

template <typename T, bool kVec, int K>
cudaError_t forward_k(const Conv1dParams &p, cudaStream_t s) {
    constexpr int V = lane_channels(K);
    conv1d_forward_kernel<T, K, V, kVec>
        <<<p.tiles * (p.row_blocks + (p.final_state ? p.seq.nseq : 0)), kConvWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, bool kVec, int K>
cudaError_t backward_k(const Conv1dParams &p, cudaStream_t s) {
    constexpr int V = lane_channels(K);
    conv1d_backward_kernel<T, K, V, kVec>
        <<<p.tiles * (p.row_blocks + (p.d_state ? p.seq.nseq : 0)), kConvWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, bool kVec, int K>
cudaError_t step_k(const Conv1dStepParams &p, cudaStream_t s) {
    constexpr int V = lane_channels(K);
    conv1d_step_kernel<T, K, V, kVec><<<p.tiles * p.B, 128, 0, s>>>(p);
    return cudaGetLastError();
}

#define CONV1D_BY_K(fn, p, s)                   \
    switch ((p).K) {                            \
        case 2: return fn<T, kVec, 2>(p, s);    \
        case 3: return fn<T, kVec, 3>(p, s);    \
        case 4: return fn<T, kVec, 4>(p, s);    \
        case 5: return fn<T, kVec, 5>(p, s);    \
        case 6: return fn<T, kVec, 6>(p, s);    \
        case 7: return fn<T, kVec, 7>(p, s);    \
        case 8: return fn<T, kVec, 8>(p, s);    \
        default: return cudaErrorInvalidValue;  \
    }

template <typename T, bool kVec> cudaError_t forward_t(const Conv1dParams &p, cudaStream_t s) { CONV1D_BY_K(forward_k, p, s) }
template <typename T, bool kVec> cudaError_t backward_t(const Conv1dParams &p, cudaStream_t s) { CONV1D_BY_K(backward_k, p, s) }
template <typename T, bool kVec> cudaError_t step_t(const Conv1dStepParams &p, cudaStream_t s) { CONV1D_BY_K(step_k, p, s) }

}  // namespace

int conv1d_channels_per_block(int K) { return 32 * lane_channels(K); }

// Rows of a warp's strip: 64, fewer where that leaves SMs without a block.
int conv1d_strip(int rows, int C, int K, int sms) {
    const long long tiles = (C + conv1d_channels_per_block(K) - 1) / conv1d_channels_per_block(K);
    int strip = 64;
    while (strip > 8 && tiles * ((rows + kConvWarps * strip - 1) / (kConvWarps * strip)) < 4LL * sms) strip >>= 1;
    return strip;
}

cudaError_t launch_conv1d_forward(const Conv1dParams &p, bool f32, bool vec, cudaStream_t s) {
    if (f32) return vec ? forward_t<float, true>(p, s) : forward_t<float, false>(p, s);
    return vec ? forward_t<__nv_bfloat16, true>(p, s) : forward_t<__nv_bfloat16, false>(p, s);
}

cudaError_t launch_conv1d_backward(const Conv1dParams &p, bool f32, bool vec, cudaStream_t s) {
    if (f32) return vec ? backward_t<float, true>(p, s) : backward_t<float, false>(p, s);
    return vec ? backward_t<__nv_bfloat16, true>(p, s) : backward_t<__nv_bfloat16, false>(p, s);
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
