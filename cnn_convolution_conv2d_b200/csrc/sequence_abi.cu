// sequence_abi.cu -- the C ABI declared in include/sequence_b200.h: argument validation, the
// scratch layout and kernel dispatch.  Host code only.
#include <algorithm>
#include <cmath>

#include "host.cuh"
#include "sequence.cuh"
#include "sequence_b200.h"

namespace conv2d_b200 {
namespace {

constexpr long long kMaxRows = 1LL << 30;
constexpr int kMaxChannels = 1 << 30;  // a tile's last channel stays an int
constexpr long long kMaxBlocks = 0x7fffffffLL;
constexpr int kSms = 148;  // a B200's: the layout of what a forward pass saves depends on the arguments alone

int elt_bytes(conv_dtype_t dtype) { return dtype == CONV_F32 ? 4 : dtype == CONV_BF16 ? 2 : 0; }

bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// A tensor over rows, as an argument.
struct RowsArg {
    const char *name;
    const void *p;
    long long stride;
    bool written;
};

int check_sequences(const int *offsets, int nseq, int T, long long rows, int C, conv_dtype_t dtype) {
    if (elt_bytes(dtype) == 0) return abi_fail(CONV_ERR_INVALID_ARG, "dtype must be CONV_F32 or CONV_BF16");
    if (nseq < 1 || rows < 0 || C < 1)
        return abi_fail(CONV_ERR_INVALID_ARG, "nseq and C must be at least 1 and rows at least 0");
    if (!offsets && (T < 0 || rows != static_cast<long long>(nseq) * T))
        return abi_fail(CONV_ERR_INVALID_ARG, "without offsets, rows must be nseq * T");
    if (!aligned(offsets, 4)) return abi_fail(CONV_ERR_UNSUPPORTED, "offsets must be aligned to 4 bytes");
    if (rows > kMaxRows || C > kMaxChannels) return abi_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 rows or channels");
    return CONV_OK;
}

// Checks the tensors over rows; *wide: whether all of them take `lanes` channels at a time.
template <int N>
int check_rows(const RowsArg (&args)[N], long long rows, int C, int elt, int lanes, bool *wide) {
    *wide = C % lanes == 0;
    for (const RowsArg &a : args) {
        if (rows > 0 && !a.p) return abi_fail(CONV_ERR_INVALID_ARG, "%s must not be NULL", a.name);
        if (a.stride < (a.written ? C : 0))
            return abi_fail(CONV_ERR_INVALID_ARG, "row stride %lld of %s: at least %d is wanted", a.stride, a.name,
                            a.written ? C : 0);
        if (!aligned(a.p, elt)) return abi_fail(CONV_ERR_UNSUPPORTED, "%s is not aligned to its elements", a.name);
        *wide = *wide && a.stride % lanes == 0 && aligned(a.p, lanes * elt);
    }
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j)
            if (i != j && args[i].written && args[i].p && args[i].p == args[j].p)
                return abi_fail(CONV_ERR_INVALID_ARG, "%s and %s are the same buffer", args[i].name, args[j].name);
    return CONV_OK;
}

int check_state(const char *name, const void *state, const char *other_name, const void *other, int elt) {
    if (state && state == other)
        return abi_fail(CONV_ERR_INVALID_ARG, "%s must not be %s itself", name, other_name);
    if (!aligned(state, elt)) return abi_fail(CONV_ERR_UNSUPPORTED, "%s is not aligned to its elements", name);
    return CONV_OK;
}

// States are read in the rows' way; their own alignment can make the call a narrow one.
bool wide_state(const void *p, int bytes) { return !p || aligned(p, bytes); }

int check_conv(int K, conv_activation_t act) {
    if (K < 2 || K > 8) return abi_fail(CONV_ERR_INVALID_ARG, "K must lie in 2 .. 8");
    if (act != CONV_ACT_NONE && act != CONV_ACT_SILU) return abi_fail(CONV_ERR_INVALID_ARG, "unknown activation");
    return CONV_OK;
}

int check_workspace(const void *workspace, size_t have, size_t need) {
    if (need && (!workspace || have < need))
        return abi_fail(CONV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                        workspace ? have : static_cast<size_t>(0));
    if (!aligned(workspace, 16)) return abi_fail(CONV_ERR_UNSUPPORTED, "the workspace must be 16-byte aligned");
    return CONV_OK;
}

int sms_or_zero() {
    AbiDevice dev;
    int n = 0;
    if (cudaGetDeviceCount(&n) != cudaSuccess || n == 0) {
        cudaGetLastError();
        return 0;
    }
    return abi_device(&dev) == CONV_OK ? dev.sms : 0;
}

// Blocks of kConvWarps strips over the rows, and the strip.
long long conv_row_blocks(long long rows, int C, int K, int sms, bool back, int *strip) {
    *strip = conv1d_strip(static_cast<int>(rows), C, K, sms, back);
    return ceil_div(rows, static_cast<long long>(*strip) * kConvWarps);
}

// A tensor over rows as a tensor map of {C, rows}; false where TMA does not take it.
bool tile_map(const void *ptr, long long stride, long long rows, int C, int elt, int box_cols, int box_rows, CUtensorMap *map) {
    const long long bytes = stride * elt;
    if (rows < 1 || stride < C || bytes % 16 || bytes >= 1LL << 40 || !aligned(ptr, 16)) return false;
    return abi_tensor_map_2d(map, ptr, elt, C, rows, bytes, box_cols, box_rows) == CONV_OK;
}

// The recurrence's scratch: [counter][aggregates][carries][decay rates][decay sums], each at a multiple of 128 bytes.
struct RecLayout {
    int chunks, per_seq, tiles, Cpad, chunk_rows;
    size_t aggregate, carry, rates, decay, forward_total, backward_total;
};

// Whether each of nseq sequences of T rows has chunks of its own, in both directions (they share the saved states):
// then a chunk hardly ever waits for the one in front of it, and sequences begin and end with their chunks, but the last
// chunk of each is not full.  Taken where that costs a third at most (bf16, rows of 2048 channels, forward and backward,
// without and with: 4 x 1100 rows 51 -> 44 and 70 -> 59 us, 4 x 1030 49 -> 43 and 66 -> 61 us, 8 x 600 55 -> 57 and
// 88 -> 70 us; fp32, 8 x 420 rows 45 -> 45 and 74 -> 64 us; where it costs more, 16 x 350 rows in bf16: 66 -> 80 and
// 98 -> 84 us, a loss for a forward pass alone), and up to half where all items still run at once (fp32, 8 x 100 rows of 512
// channels: 20.4 -> 16.4 and 24.6 -> 22.5 us; where they do not, 16 x 150 rows of 2048 in bf16: 47 -> 59 and 51 -> 64 us).
bool own_chunks(int nseq, int T, long long tiles, int elt) {
    if (T < 1) return false;
    bool full = true, few = true;
    for (const bool back : {false, true}) {
        const RecShape shape = rec_shape(elt, back);
        const long long chunk_rows = shape.rows(), per_seq = ceil_div(T, chunk_rows);
        full = full && 3 * per_seq * chunk_rows <= 4LL * T;
        few = few && per_seq * chunk_rows <= 2LL * T && per_seq * nseq * tiles <= shape.blocks * kSms;
    }
    return full || few;
}

// T = 0: packed sequences.
int rec_layout(int nseq, int T, long long rows, int C, conv_dtype_t dtype, bool back, RecLayout *r) {
    const int elt = elt_bytes(dtype);
    if (elt == 0) return abi_fail(CONV_ERR_INVALID_ARG, "dtype must be CONV_F32 or CONV_BF16");
    if (nseq < 1 || T < 0 || rows < 0 || C < 1)
        return abi_fail(CONV_ERR_INVALID_ARG, "nseq and C must be at least 1, T and rows at least 0");
    if (T > 0 && rows != static_cast<long long>(nseq) * T) return abi_fail(CONV_ERR_INVALID_ARG, "rows must be nseq * T");
    if (rows > kMaxRows || C > kMaxChannels) return abi_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 rows or channels");
    const long long chunk_rows = rec_shape(elt, back).rows(), tiles = ceil_div(C, kRecTile);
    const bool own = nseq > 1 && own_chunks(nseq, T, tiles, elt);
    r->per_seq = own ? static_cast<int>(ceil_div(T, chunk_rows)) : 0;
    long long chunks = rows ? ceil_div(rows, chunk_rows) : 1;
    if (own) chunks = static_cast<long long>(r->per_seq) * nseq;
    if (chunks * tiles > kMaxBlocks) return abi_fail(CONV_ERR_UNSUPPORTED, "too many rows and channels for one launch");
    r->chunks = static_cast<int>(chunks);
    r->tiles = static_cast<int>(tiles);
    r->chunk_rows = static_cast<int>(chunk_rows);
    r->Cpad = r->tiles * kRecTile;
    const size_t each = static_cast<size_t>(chunks) * r->Cpad * 4;  // a multiple of 128
    const bool joins = chunks > 1;
    r->aggregate = joins ? 256 : 0;
    r->carry = r->aggregate + (joins ? 2 * each : 0);
    r->rates = r->carry + (joins ? each : 0);
    r->forward_total = r->rates + (joins ? static_cast<size_t>(r->Cpad) * 4 : 0);
    r->decay = r->forward_total;
    r->backward_total = r->decay + each;
    return CONV_OK;
}

// Points p into the scratch and fills the words that are their own flags.
int rec_begin(RecParams *p, const RecLayout &r, void *workspace, cudaStream_t stream) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p->chunks = r.chunks;
    p->per_seq = r.per_seq;
    p->tiles = r.tiles;
    p->Cpad = r.Cpad;
    if (r.chunks == 1) return CONV_OK;
    p->ticket = reinterpret_cast<unsigned *>(ws);
    p->aggregate = reinterpret_cast<float2 *>(ws + r.aggregate);
    p->carry = reinterpret_cast<float *>(ws + r.carry);
    float *rates = reinterpret_cast<float *>(ws + r.rates);
    p->rates = rates;
    return abi_launch(launch_rec_init(*p, r.rates / 4, rates, stream), "recurrence scratch");
}

// Runs the recurrence: in tiles where TMA takes every tensor, element by element otherwise.
int run_rec(const RecParams &p, const RecLayout &r, int elt, bool back, cudaStream_t s) {
    RecTiles q{};
    const long long rows = p.seq.rows;
    const int runs = 2 * rec_shape(elt, back).run, chunk = r.chunk_rows;
    bool tiles = tile_map(p.x, p.ldx, rows, p.C, elt, kRecTile, chunk, &q.in[0]) &&
                 tile_map(p.ga, p.lda, rows, p.C, elt, kRecTile, chunk, &q.in[1]) &&
                 tile_map(p.gx, p.ldg, rows, p.C, elt, kRecTile, chunk, &q.in[2]) &&
                 tile_map(p.y, p.ldy, rows, p.C, elt, kRecTile, runs, &q.out[0]);
    if (back)
        tiles = tiles && tile_map(p.dy, p.lddy, rows, p.C, elt, kRecTile, chunk, &q.in[3]) &&
                tile_map(p.dga, p.ld_da, rows, p.C, elt, kRecTile, runs, &q.out[1]) &&
                tile_map(p.dgx, p.ld_dg, rows, p.C, elt, kRecTile, runs, &q.out[2]);
    const char *what = back ? "recurrence gradient" : "recurrence";
    if (!tiles) return abi_launch(launch_rec_plain(p, elt == 4, back, s), what);
    q.p = p;
    return abi_launch(launch_rec_tiles(q, elt == 4, back, s), what);
}

int check_rec(const float *decay, float kappa) {
    if (!decay) return abi_fail(CONV_ERR_INVALID_ARG, "decay must not be NULL");
    if (!aligned(decay, 4)) return abi_fail(CONV_ERR_UNSUPPORTED, "decay is not aligned to its elements");
    if (!(kappa > 0.f) || std::isinf(kappa)) return abi_fail(CONV_ERR_INVALID_ARG, "kappa must be finite and above 0");
    return CONV_OK;
}

}  // namespace
}  // namespace conv2d_b200

using namespace conv2d_b200;

#define RETURN_IF(expr)                             \
    do {                                            \
        const int st_ = (expr);                     \
        if (st_ != CONV_OK) return st_;             \
    } while (0)

#pragma GCC visibility push(default)
extern "C" {

int conv1d_causal_forward(const void *x, const void *w, const void *bias, void *y, const void *state,
                          void *final_state, const int *offsets, int nseq, int T, long long rows, int C, int K,
                          conv_activation_t activation, long long x_stride, long long y_stride, conv_dtype_t dtype,
                          conv_stream_t stream) {
    RETURN_IF(check_sequences(offsets, nseq, T, rows, C, dtype));
    RETURN_IF(check_conv(K, activation));
    const int elt = elt_bytes(dtype), lanes = conv1d_channels_per_block(K) / 32;
    bool wide = false;
    RETURN_IF(check_rows({{"x", x, x_stride, false}, {"y", y, y_stride, true}}, rows, C, elt, lanes, &wide));
    if (!w) return abi_fail(CONV_ERR_INVALID_ARG, "w must not be NULL");
    if (!aligned(w, elt) || !aligned(bias, elt))
        return abi_fail(CONV_ERR_UNSUPPORTED, "w or bias is not aligned to its elements");
    RETURN_IF(check_state("final_state", final_state, "state", state, elt));
    RETURN_IF(check_state("state", state, "y", y, elt));
    wide = wide && wide_state(state, lanes * elt) && wide_state(final_state, lanes * elt);
    AbiDevice dev;
    RETURN_IF(abi_device(&dev));
    Conv1dTiles q{};
    Conv1dParams &p = q.p;
    p.timeout_ns = dev.timeout_ns;
    p.x = x; p.w = w; p.bias = bias; p.y = y; p.state = state; p.final_state = final_state;
    p.ldx = x_stride; p.ldy = y_stride;
    p.seq = Sequences{offsets, nseq, T, static_cast<int>(rows)};
    p.C = C; p.K = K; p.silu = activation == CONV_ACT_SILU; p.status = dev.status;
    p.tiles = static_cast<int>(ceil_div(C, conv1d_channels_per_block(K)));
    const long long blocks = conv_row_blocks(rows, C, K, dev.sms, false, &p.strip);
    const long long all = (blocks + (final_state ? nseq : 0)) * p.tiles;
    if (all > kMaxBlocks) return abi_fail(CONV_ERR_UNSUPPORTED, "too many rows and channels for one launch");
    p.row_blocks = static_cast<int>(blocks);
    const int box = conv1d_channels_per_block(K), batch = kConvBatch / elt;
    const bool tma = wide && tile_map(x, x_stride, rows, C, elt, box, batch, &q.in[0]) &&
                     tile_map(y, y_stride, rows, C, elt, box, batch, &q.out);
    if (all > 0)
        RETURN_IF(abi_launch(launch_conv1d_forward(q, elt == 4, tma, reinterpret_cast<cudaStream_t>(stream)),
                             "causal convolution"));
    return abi_ok();
}

int conv1d_causal_backward_workspace_size(long long rows, int C, int K, size_t *bytes) {
    if (!bytes || rows < 0 || C < 1) return abi_fail(CONV_ERR_INVALID_ARG, "workspace size: invalid argument");
    RETURN_IF(check_conv(K, CONV_ACT_NONE));
    if (rows > kMaxRows || C > kMaxChannels) return abi_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 rows or channels");
    int strip = 0;
    *bytes = static_cast<size_t>(conv_row_blocks(rows, C, K, sms_or_zero(), true, &strip)) * (K + 1) * C * sizeof(float);
    return abi_ok();
}

int conv1d_causal_backward(const void *x, const void *w, const void *bias, const void *dy, const void *state,
                           const void *d_final_state, void *dx, void *dw, void *db, void *d_state,
                           const int *offsets, int nseq, int T, long long rows, int C, int K,
                           conv_activation_t activation, long long x_stride, long long dy_stride,
                           long long dx_stride, conv_dtype_t dtype, void *workspace, size_t workspace_bytes,
                           conv_stream_t stream) {
    RETURN_IF(check_sequences(offsets, nseq, T, rows, C, dtype));
    RETURN_IF(check_conv(K, activation));
    const int elt = elt_bytes(dtype), lanes = conv1d_channels_per_block(K) / 32;
    bool wide = false;
    RETURN_IF(check_rows({{"x", x, x_stride, false}, {"dy", dy, dy_stride, false}, {"dx", dx, dx_stride, true}}, rows, C,
                         elt, lanes, &wide));
    if (!w || !dw) return abi_fail(CONV_ERR_INVALID_ARG, "w and dw must not be NULL");
    if (!aligned(w, elt) || !aligned(bias, elt) || !aligned(dw, elt) || !aligned(db, elt))
        return abi_fail(CONV_ERR_UNSUPPORTED, "w, bias, dw or db is not aligned to its elements");
    RETURN_IF(check_state("d_state", d_state, "d_final_state", d_final_state, elt));
    RETURN_IF(check_state("state", state, "d_state", d_state, elt));
    RETURN_IF(check_state("d_final_state", d_final_state, "dx", dx, elt));
    wide = wide && wide_state(state, lanes * elt) && wide_state(d_final_state, lanes * elt) &&
           wide_state(d_state, lanes * elt);
    AbiDevice dev;
    RETURN_IF(abi_device(&dev));
    Conv1dTiles q{};
    Conv1dParams &p = q.p;
    p.timeout_ns = dev.timeout_ns;
    p.x = x; p.w = w; p.bias = bias; p.dy = dy; p.y = dx; p.state = state; p.d_final = d_final_state;
    p.d_state = d_state;
    p.ldx = x_stride; p.ldy = dx_stride; p.lddy = dy_stride;
    p.seq = Sequences{offsets, nseq, T, static_cast<int>(rows)};
    p.C = C; p.K = K; p.silu = activation == CONV_ACT_SILU; p.status = dev.status;
    p.tiles = static_cast<int>(ceil_div(C, conv1d_channels_per_block(K)));
    const long long blocks = conv_row_blocks(rows, C, K, dev.sms, true, &p.strip);
    const long long all = (blocks + (d_state ? nseq : 0)) * p.tiles;
    if (all > kMaxBlocks) return abi_fail(CONV_ERR_UNSUPPORTED, "too many rows and channels for one launch");
    p.row_blocks = static_cast<int>(blocks);
    RETURN_IF(check_workspace(workspace, workspace_bytes, static_cast<size_t>(blocks) * (K + 1) * C * sizeof(float)));
    p.partial = static_cast<float *>(workspace);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int box = conv1d_channels_per_block(K), batch = kConvBatch / elt;
    const bool tma = wide && tile_map(x, x_stride, rows, C, elt, box, batch, &q.in[0]) &&
                     tile_map(dy, dy_stride, rows, C, elt, box, batch, &q.in[1]) &&
                     tile_map(dx, dx_stride, rows, C, elt, box, batch, &q.out);
    if (all > 0) RETURN_IF(abi_launch(launch_conv1d_backward(q, elt == 4, tma, s), "causal convolution gradient"));
    RETURN_IF(abi_launch(launch_conv1d_reduce(p.partial, dw, db, p.row_blocks, C, K, elt == 4, s), "weight gradient sum"));
    return abi_ok();
}

int conv1d_causal_step(const void *x, const void *w, const void *bias, void *y, void *state, const int *slots, int B,
                       int pool, int C, int K, conv_activation_t activation, long long x_stride, long long y_stride,
                       conv_dtype_t dtype, conv_stream_t stream) {
    const int elt = elt_bytes(dtype);
    if (elt == 0) return abi_fail(CONV_ERR_INVALID_ARG, "dtype must be CONV_F32 or CONV_BF16");
    if (B < 1 || C < 1 || pool < 1) return abi_fail(CONV_ERR_INVALID_ARG, "B, pool and C must be at least 1");
    if (C > kMaxChannels) return abi_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 channels");
    if (!slots && pool < B) return abi_fail(CONV_ERR_INVALID_ARG, "without slots, pool must be at least B");
    RETURN_IF(check_conv(K, activation));
    const int lanes = conv1d_channels_per_block(K) / 32;
    bool wide = false;
    RETURN_IF(check_rows({{"x", x, x_stride, false}, {"y", y, y_stride, true}}, B, C, elt, lanes, &wide));
    if (!w || !state) return abi_fail(CONV_ERR_INVALID_ARG, "w and state must not be NULL");
    if (!aligned(w, elt) || !aligned(bias, elt) || !aligned(slots, 4))
        return abi_fail(CONV_ERR_UNSUPPORTED, "w, bias or slots is not aligned to its elements");
    RETURN_IF(check_state("state", state, "x", x, elt));
    RETURN_IF(check_state("state", state, "y", y, elt));
    wide = wide && wide_state(state, lanes * elt);
    AbiDevice dev;
    RETURN_IF(abi_device(&dev));
    Conv1dStepParams p{};
    p.x = x; p.w = w; p.bias = bias; p.y = y; p.state = state; p.slots = slots;
    p.ldx = x_stride; p.ldy = y_stride;
    p.B = B; p.C = C; p.K = K; p.silu = activation == CONV_ACT_SILU; p.pool = pool; p.status = dev.status;
    p.tiles = static_cast<int>(ceil_div(C, 4 * conv1d_channels_per_block(K)));
    if (static_cast<long long>(p.tiles) * B > kMaxBlocks)
        return abi_fail(CONV_ERR_UNSUPPORTED, "too many rows and channels for one launch");
    RETURN_IF(abi_launch(launch_conv1d_step(p, elt == 4, wide, reinterpret_cast<cudaStream_t>(stream)),
                         "causal convolution step"));
    return abi_ok();
}

int gated_recurrence_saved_size(int nseq, int T, long long rows, int C, conv_dtype_t dtype, size_t *bytes) {
    RecLayout r;
    if (!bytes) return abi_fail(CONV_ERR_INVALID_ARG, "bytes must not be NULL");
    RETURN_IF(rec_layout(nseq, T, rows, C, dtype, true, &r));
    // one for every kRecRun rows that have begun -- of each sequence, where each has chunks of its own
    const size_t states = r.per_seq ? static_cast<size_t>(nseq) * ceil_div(T, kRecRun) : ceil_div(rows, kRecRun);
    *bytes = std::max<size_t>(states, 1) * r.Cpad * sizeof(float);
    return abi_ok();
}

int gated_recurrence_workspace_size(int nseq, int T, long long rows, int C, conv_dtype_t dtype, size_t *bytes) {
    RecLayout r;
    if (!bytes) return abi_fail(CONV_ERR_INVALID_ARG, "bytes must not be NULL");
    RETURN_IF(rec_layout(nseq, T, rows, C, dtype, false, &r));
    *bytes = r.forward_total;
    return abi_ok();
}

int gated_recurrence_backward_workspace_size(int nseq, int T, long long rows, int C, conv_dtype_t dtype, size_t *bytes) {
    RecLayout r;
    if (!bytes) return abi_fail(CONV_ERR_INVALID_ARG, "bytes must not be NULL");
    RETURN_IF(rec_layout(nseq, T, rows, C, dtype, true, &r));
    *bytes = r.backward_total;
    return abi_ok();
}

int gated_recurrence_forward(const void *x, const void *gate_a, const void *gate_x, const float *decay, float kappa,
                             void *y, const float *state, float *final_state, void *saved, const int *offsets,
                             int nseq, int T, long long rows, int C, long long x_stride, long long gate_a_stride,
                             long long gate_x_stride, long long y_stride, conv_dtype_t dtype, void *workspace,
                             size_t workspace_bytes, conv_stream_t stream) {
    RETURN_IF(check_sequences(offsets, nseq, T, rows, C, dtype));
    RETURN_IF(check_rec(decay, kappa));
    const int elt = elt_bytes(dtype);
    bool wide = false;
    RETURN_IF(check_rows({{"x", x, x_stride, false}, {"gate_a", gate_a, gate_a_stride, false},
                          {"gate_x", gate_x, gate_x_stride, false}, {"y", y, y_stride, true}},
                         rows, C, elt, 2, &wide));
    RETURN_IF(check_state("final_state", final_state, "state", state, 4));
    RETURN_IF(check_state("state", state, "y", y, 4));
    RETURN_IF(check_state("saved", saved, "final_state", final_state, 16));
    RecLayout r;
    RETURN_IF(rec_layout(nseq, offsets ? 0 : T, rows, C, dtype, false, &r));
    RETURN_IF(check_workspace(workspace, workspace_bytes, r.forward_total));
    AbiDevice dev;
    RETURN_IF(abi_device(&dev));
    RecParams p{};
    p.x = x; p.ga = gate_a; p.gx = gate_x; p.decay = decay; p.kappa = kappa; p.y = y;
    p.state = state; p.final_state = final_state; p.saved = static_cast<float *>(saved);
    p.ldx = x_stride; p.lda = gate_a_stride; p.ldg = gate_x_stride; p.ldy = y_stride;
    p.seq = Sequences{offsets, nseq, T, static_cast<int>(rows)};
    p.C = C; p.status = dev.status; p.timeout_ns = dev.timeout_ns; p.starve = dev.starve;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    RETURN_IF(rec_begin(&p, r, workspace, s));
    RETURN_IF(run_rec(p, r, elt, false, s));
    return abi_ok();
}

int gated_recurrence_backward(const void *x, const void *gate_a, const void *gate_x, const float *decay, float kappa,
                              const void *dy, const void *saved, const float *state, const float *d_final_state,
                              void *dx, void *d_gate_a, void *d_gate_x, float *d_decay, float *d_state,
                              const int *offsets, int nseq, int T, long long rows, int C, long long x_stride,
                              long long gate_a_stride, long long gate_x_stride, long long dy_stride,
                              long long dx_stride, long long d_gate_a_stride, long long d_gate_x_stride,
                              conv_dtype_t dtype, void *workspace, size_t workspace_bytes, conv_stream_t stream) {
    RETURN_IF(check_sequences(offsets, nseq, T, rows, C, dtype));
    RETURN_IF(check_rec(decay, kappa));
    const int elt = elt_bytes(dtype);
    bool wide = false;
    RETURN_IF(check_rows({{"x", x, x_stride, false}, {"gate_a", gate_a, gate_a_stride, false},
                          {"gate_x", gate_x, gate_x_stride, false}, {"dy", dy, dy_stride, false},
                          {"dx", dx, dx_stride, true}, {"d_gate_a", d_gate_a, d_gate_a_stride, true},
                          {"d_gate_x", d_gate_x, d_gate_x_stride, true}},
                         rows, C, elt, 2, &wide));
    if (!d_decay || !saved) return abi_fail(CONV_ERR_INVALID_ARG, "saved and d_decay must not be NULL");
    RETURN_IF(check_state("d_state", d_state, "d_final_state", d_final_state, 4));
    RETURN_IF(check_state("d_state", d_state, "state", state, 4));
    RETURN_IF(check_state("saved", saved, "d_state", d_state, 16));
    RETURN_IF(check_state("d_decay", d_decay, "decay", decay, 4));
    RecLayout r;
    RETURN_IF(rec_layout(nseq, offsets ? 0 : T, rows, C, dtype, true, &r));
    RETURN_IF(check_workspace(workspace, workspace_bytes, r.backward_total));
    AbiDevice dev;
    RETURN_IF(abi_device(&dev));
    RecParams p{};
    p.x = x; p.ga = gate_a; p.gx = gate_x; p.dy = dy; p.decay = decay; p.kappa = kappa;
    p.y = dx; p.dga = d_gate_a; p.dgx = d_gate_x;
    p.state = state; p.d_final = d_final_state; p.d_state = d_state;
    p.saved = static_cast<float *>(const_cast<void *>(saved));  // only read
    p.decay_partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + r.decay);
    p.ldx = x_stride; p.lda = gate_a_stride; p.ldg = gate_x_stride; p.lddy = dy_stride;
    p.ldy = dx_stride; p.ld_da = d_gate_a_stride; p.ld_dg = d_gate_x_stride;
    p.seq = Sequences{offsets, nseq, T, static_cast<int>(rows)};
    p.C = C; p.status = dev.status; p.timeout_ns = dev.timeout_ns; p.starve = dev.starve;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    RETURN_IF(rec_begin(&p, r, workspace, s));
    RETURN_IF(run_rec(p, r, elt, true, s));
    RETURN_IF(abi_launch(launch_rec_decay(p.decay_partial, decay, kappa, d_decay, p.chunks, C, p.Cpad, s),
                         "decay gradient sum"));
    return abi_ok();
}

int gated_recurrence_step(const void *x, const void *gate_a, const void *gate_x, const float *decay, float kappa,
                          void *y, float *state, const int *slots, int B, int pool, int C, long long x_stride,
                          long long gate_a_stride, long long gate_x_stride, long long y_stride, conv_dtype_t dtype,
                          conv_stream_t stream) {
    const int elt = elt_bytes(dtype);
    if (elt == 0) return abi_fail(CONV_ERR_INVALID_ARG, "dtype must be CONV_F32 or CONV_BF16");
    if (B < 1 || C < 1 || pool < 1) return abi_fail(CONV_ERR_INVALID_ARG, "B, pool and C must be at least 1");
    if (C > kMaxChannels) return abi_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 channels");
    if (!slots && pool < B) return abi_fail(CONV_ERR_INVALID_ARG, "without slots, pool must be at least B");
    RETURN_IF(check_rec(decay, kappa));
    bool wide = false;
    RETURN_IF(check_rows({{"x", x, x_stride, false}, {"gate_a", gate_a, gate_a_stride, false},
                          {"gate_x", gate_x, gate_x_stride, false}, {"y", y, y_stride, true}},
                         B, C, elt, 2, &wide));
    if (!state) return abi_fail(CONV_ERR_INVALID_ARG, "state must not be NULL");
    if (!aligned(slots, 4)) return abi_fail(CONV_ERR_UNSUPPORTED, "slots is not aligned to its elements");
    RETURN_IF(check_state("state", state, "x", x, 4));
    RETURN_IF(check_state("state", state, "y", y, 4));
    AbiDevice dev;
    RETURN_IF(abi_device(&dev));
    RecStepParams p{};
    p.x = x; p.ga = gate_a; p.gx = gate_x; p.decay = decay; p.kappa = kappa; p.y = y; p.state = state;
    p.slots = slots;
    p.ldx = x_stride; p.lda = gate_a_stride; p.ldg = gate_x_stride; p.ldy = y_stride;
    p.B = B; p.C = C; p.pool = pool; p.status = dev.status;
    p.tiles = static_cast<int>(ceil_div(C, kRecStepTile));
    if (static_cast<long long>(p.tiles) * B > kMaxBlocks)
        return abi_fail(CONV_ERR_UNSUPPORTED, "too many rows and channels for one launch");
    RETURN_IF(abi_launch(launch_rec_step(p, elt == 4, reinterpret_cast<cudaStream_t>(stream)), "recurrence step"));
    return abi_ok();
}

}  // extern "C"
#pragma GCC visibility pop
