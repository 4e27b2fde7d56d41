// sequence.cuh -- what the kernels over sequences (conv1d.cu, recurrence.cu) share: the
// description of the rows of a batch, element access, and the launchers' parameters.
//
// A tensor over sequences is a matrix of `rows` rows of C channels (channels-last, the last
// dimension contiguous, rows a fixed stride apart).  Either the rows are nseq sequences of
// T rows each, or `offsets` (nseq + 1 device ints) packs sequences of their own lengths one
// behind the other: sequence s has rows offsets[s] .. offsets[s+1]-1.  Rows from
// offsets[nseq] on belong to none; nothing is written there.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace conv2d_b200 {

struct Sequences {
    const int *offsets;  // NULL: nseq sequences of T rows
    int nseq;
    int T;
    int rows;
};

struct Conv1dParams {
    const void *x, *w, *bias, *dy;
    void *y;               // forward: y; backward: dx
    const void *state;     // (nseq, K-1, C) rows before each sequence, or NULL (zeros)
    void *final_state;     // forward: (nseq, K-1, C) or NULL
    const void *d_final;   // backward: gradient of final_state, or NULL
    void *d_state;         // backward: gradient of state, or NULL
    float *partial;        // backward: [row blocks][K+1][C] sums of dw (taps 0..K-1) and db
    long long ldx, ldy, lddy;  // row strides in elements: x, the output, dy
    Sequences seq;
    int C, K, silu;
    int strip;             // rows of one warp
    int tiles;             // channel tiles
    int row_blocks;        // blocks of kConvWarps strips; blocks behind them copy states
    int *status;
    long long timeout_ns;
};

// The convolution with rows that travel by TMA, in boxes of a warp's channels x kConvBatch / sizeof(element) rows.
struct Conv1dTiles {
    CUtensorMap in[2];     // x, dy
    CUtensorMap out;       // y or dx
    Conv1dParams p;
};

struct Conv1dStepParams {
    const void *x, *w, *bias;
    void *y, *state;
    const int *slots;      // row b's window is state[slots[b]]; NULL: state[b]
    long long ldx, ldy;
    int B, C, K, silu, pool, tiles;
    int *status;
};

struct RecParams {
    const void *x, *ga, *gx, *dy;
    const float *decay;    // (C,)
    float kappa;
    void *y;               // forward: h; backward: dx
    void *dga, *dgx;       // backward
    const float *state;    // (nseq, C) or NULL
    float *final_state;    // forward: (nseq, C) or NULL
    const float *d_final;  // backward: gradient of final_state, or NULL
    float *d_state;        // backward: gradient of state, or NULL
    float *decay_partial;  // backward: [chunks][Cpad] sums
    float *saved;          // [runs][Cpad] the state that enters each run of kRecRun rows: written by the forward pass (or
                           // NULL), read by the backward pass
    const float *rates;    // (C,) decay rates from the start of the call, or NULL (computed on the spot)
    float *carry;          // [chunks][Cpad] carries behind each chunk (against the order of time: in front)
    float2 *aggregate;     // [chunks][Cpad] (product of decays, state of a zero start)
    unsigned *ticket;      // starts at 0xffffffff
    long long ldx, lda, ldg, ldy, lddy, ld_da, ld_dg;
    Sequences seq;
    int C, Cpad, tiles, chunks;
    int per_seq;           // chunks of each sequence; 0: the chunks follow one another over all rows
    int *status;
    long long timeout_ns;
    int starve;
};

// The recurrence in tiles that travel by TMA.
struct RecTiles {
    CUtensorMap in[4];     // x, gate_a, gate_x, dy as {C, rows}: boxes of kRecTile x a chunk's rows
    CUtensorMap out[3];    // y, or dx, d_gate_a, d_gate_x: boxes of kRecTile x the rows of a warp's two runs
    RecParams p;
};

struct RecStepParams {
    const void *x, *ga, *gx;
    const float *decay;
    float kappa;
    void *y;
    float *state;
    const int *slots;
    long long ldx, lda, ldg, ldy;
    int B, C, pool, tiles;
    int *status;
};

constexpr int kConvWarps = 4;     // warps of a conv1d block, one strip of rows each
constexpr int kConvBlocks = 6, kConvBlocksBack = 4;  // blocks an SM
constexpr int kConvBatch = 16;    // bytes of one channel's rows in a batch: 8 rows in bf16, 4 in fp32
constexpr int kRecTile = 32;      // channels of a work item of the recurrence
constexpr int kRecStepTile = 256; // channels of a block of its step
constexpr int kRecRun = 8;        // rows of one saved state

// How a kernel of the recurrence is laid out: working warps, rows that half of one scans, stages of shared memory,
// blocks an SM.  With 8 warps (and the joining one) a thread has 96 registers, with 6 or 7 it has 128: bf16 backward 281 us
// with 8 against 303 us with 7 (16384 x 4096), forward 143 against 164 us; fp32 backward 194 us with 6 against
// 283 us with 7 (16384 x 2048; shared memory then holds one block an SM).
struct RecShape {
    int warps, run, stages, blocks;
    constexpr int rows() const { return 2 * warps * run; }
};
constexpr RecShape rec_shape(int elt, bool back) {
    if (back) return elt == 2 ? RecShape{8, 8, 2, 2} : RecShape{6, 8, 2, 2};
    return elt == 2 ? RecShape{8, 16, 2, 2} : RecShape{8, 8, 2, 2};
}

cudaError_t launch_conv1d_forward(const Conv1dTiles &q, bool f32, bool tma, cudaStream_t s);
cudaError_t launch_conv1d_backward(const Conv1dTiles &q, bool f32, bool tma, cudaStream_t s);
cudaError_t launch_conv1d_reduce(const float *partial, void *dw, void *db, int row_blocks, int C, int K, bool f32,
                                 cudaStream_t s);
cudaError_t launch_conv1d_step(const Conv1dStepParams &p, bool f32, bool vec, cudaStream_t s);
int conv1d_strip(int rows, int C, int K, int sms, bool back);
int conv1d_channels_per_block(int K);

cudaError_t launch_rec_init(const RecParams &p, size_t words, float *rates, cudaStream_t s);
cudaError_t launch_rec_plain(const RecParams &p, bool f32, bool back, cudaStream_t s);
cudaError_t launch_rec_tiles(const RecTiles &q, bool f32, bool back, cudaStream_t s);
cudaError_t launch_rec_decay(const float *partial, const float *decay, float kappa, float *d_decay, int chunks, int C,
                             int Cpad, cudaStream_t s);
cudaError_t launch_rec_step(const RecStepParams &p, bool f32, cudaStream_t s);

#ifdef __CUDACC__

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// First row of sequence s, kept inside [0, rows] whatever the offsets hold.
__device__ __forceinline__ int seq_begin(const Sequences &q, int s) {
    if (!q.offsets) return s * q.T;
    return min(max(q.offsets[s], 0), q.rows);
}

// The last sequence that begins at or before `row` (-1: none): with empty sequences at that
// row, the one that holds it.
__device__ __forceinline__ int seq_of(const Sequences &q, int row, int lo, int hi) {  // known to lie in lo .. hi
    if (!q.offsets) return q.T > 0 ? min(row / q.T, q.nseq - 1) : -1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (q.offsets[mid] <= row) lo = mid; else hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ int seq_of(const Sequences &q, int row) { return seq_of(q, row, -1, q.nseq - 1); }

// Whether the offsets begin at 0, never fall and end inside the rows: looked at by `count` threads,
// of which this is number `i`.  A violation is reported through the status word.
__device__ __forceinline__ void check_offsets(const Sequences &q, int *status, int i, int count) {
    if (!q.offsets) return;
    for (int s = i; s <= q.nseq; s += count) {
        const int v = q.offsets[s], before = s ? q.offsets[s - 1] : 0;
        if (v < before || v > q.rows || (s == 0 && v != 0)) atomicExch(status, kDevBadOffsets);
    }
}

__device__ __forceinline__ void check_offsets(const Sequences &q, int *status) {
    check_offsets(q, status, threadIdx.x, blockDim.x);
}

// Whether an earlier row of the batch names the same slot.  Called by all threads of a block.
__device__ __forceinline__ bool slot_named_before(const int *slots, int b, int slot) {
    int dup = 0;
    for (int j = threadIdx.x; j < b; j += blockDim.x) dup |= slots[j] == slot;
    return __syncthreads_or(dup) != 0;
}

// Copies 4 bytes, aligned to that, to shared memory; a thread waits for its own copies.
__device__ __forceinline__ void cp_async_4(void *to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most kPending of the thread's committed groups are outstanding.
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Arrives at a named barrier of `count` threads without waiting for it.
__device__ __forceinline__ void named_barrier_arrive(int id, int count) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

#endif  // __CUDACC__

}  // namespace conv2d_b200
