// optimizer_abi.cu -- the C ABI declared in include/optimizer_b200.h: argument validation and
// the launches of the AdamW kernel, kAdamTensors tensors each.  Host code only.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <new>
#include <utility>
#include <vector>

#include "adamw.cuh"
#include "host.cuh"
#include "optimizer_b200.h"

namespace conv2d_b200 {
namespace {

constexpr long long kMaxElements = 0x7fffffffLL * kAdamBatch;  // one tensor needs at most the blocks that a launch takes

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// *master: whether the tensors that have elements have master weights (those without are passed over, whatever they hold).
int check_tensors(const adamw_tensor_t *t, int count, int elt, int state_bits, bool *master) {
    std::vector<std::pair<uintptr_t, uintptr_t>> weights;
    weights.reserve(count);
    bool none = false;
    *master = false;
    for (int i = 0; i < count; ++i) {
        const adamw_tensor_t &a = t[i];
        if (a.numel < 0) return abi_fail(CONV_ERR_INVALID_ARG, "tensor %d: numel is negative", i);
        if (a.numel == 0) continue;
        if (a.numel > kMaxElements) return abi_fail(CONV_ERR_UNSUPPORTED, "tensor %d: more than (2^31 - 1) * 1024 elements", i);
        if (!a.param || !a.grad || !a.exp_avg || !a.exp_avg_sq)
            return abi_fail(CONV_ERR_INVALID_ARG, "tensor %d: param, grad, exp_avg and exp_avg_sq must not be NULL", i);
        if (state_bits == 8 && (!a.exp_avg_scale || !a.exp_avg_sq_scale))
            return abi_fail(CONV_ERR_INVALID_ARG, "tensor %d: 8-bit states need their scales", i);
        if (!aligned16(a.param) || !aligned16(a.master) || !aligned16(a.grad) || !aligned16(a.exp_avg) ||
            !aligned16(a.exp_avg_sq) || ((reinterpret_cast<uintptr_t>(a.exp_avg_scale) |
                                          reinterpret_cast<uintptr_t>(a.exp_avg_sq_scale)) & 3u))
            return abi_fail(CONV_ERR_UNSUPPORTED, "tensor %d: device pointers must be 16-byte aligned", i);
        if (a.master) *master = true; else none = true;
        if (a.master && elt == 4)
            return abi_fail(CONV_ERR_INVALID_ARG, "tensor %d: fp32 weights are their own master weights", i);
        const uintptr_t p = reinterpret_cast<uintptr_t>(a.param);
        weights.emplace_back(p, p + static_cast<uintptr_t>(a.numel) * elt);
    }
    if (*master && none) return abi_fail(CONV_ERR_INVALID_ARG, "either all or no tensors have master weights");
    std::sort(weights.begin(), weights.end());
    for (size_t i = 1; i < weights.size(); ++i)
        if (weights[i].first < weights[i - 1].second)
            return abi_fail(CONV_ERR_INVALID_ARG, "two weight tensors overlap");
    return CONV_OK;
}

bool at_least_zero(double v) { return v >= 0.0 && std::isfinite(v); }

int check_types(int count, const adamw_tensor_t *tensors, conv_dtype_t param_dtype, int state_bits) {
    if (count < 0 || (count > 0 && !tensors))
        return abi_fail(CONV_ERR_INVALID_ARG, "count must be at least 0 and tensors not NULL");
    if (param_dtype != CONV_F32 && param_dtype != CONV_BF16)
        return abi_fail(CONV_ERR_INVALID_ARG, "dtypes must be CONV_F32 or CONV_BF16");
    if (state_bits != 8 && state_bits != 32) return abi_fail(CONV_ERR_INVALID_ARG, "state_bits must be 8 or 32");
    return CONV_OK;
}

int checked_tensors(const adamw_tensor_t *tensors, int count, int elt, int state_bits, bool *master) {
    try {
        return check_tensors(tensors, count, elt, state_bits, master);
    } catch (const std::bad_alloc &) {
        return abi_fail(CONV_ERR_INVALID_ARG, "out of host memory");
    }
}

// Batches of a block.  With 8-bit states a block takes more batches, and finds its tensor once for them, where that leaves
// 8 blocks an SM (100 M elements: 313 -> 258 us); with 32-bit states, which wait for memory alone, that costs (422 -> 438 us).
int batches_of(const adamw_tensor_t *tensors, int count, int state_bits, int sms) {
    if (state_bits == 32) return 1;
    long long elements = 0;
    for (int k = 0; k < count; ++k) elements += std::min(tensors[k].numel, kMaxElements);
    return static_cast<int>(std::min<long long>(std::max<long long>(elements / kAdamBatch / (8LL * std::max(sms, 1)), 1),
                                                kAdamBatches));
}

// The next launch: the tensors from *i on, as many as one launch takes; *i moves behind them.  Its table, first blocks and
// first place are p's; returns its blocks.
unsigned long long next_launch(const adamw_tensor_t *tensors, int count, int state_bits, int *i, AdamParams *p) {
    const unsigned long long per_block = static_cast<unsigned long long>(p->batches) * kAdamBatch;
    unsigned long long blocks = 0;
    p->count = 0;
    p->index0 = static_cast<unsigned>(*i);
    for (; *i < count && p->count < kAdamTensors; ++*i) {
        const adamw_tensor_t &a = tensors[*i];
        const unsigned long long need = (static_cast<unsigned long long>(a.numel) + per_block - 1) / per_block;
        if (blocks + need > 0x7fffffffULL) break;
        p->t[p->count] = AdamTensor{a.param, a.master, a.grad, a.exp_avg, a.exp_avg_sq,
                                    state_bits == 8 ? a.exp_avg_scale : nullptr,
                                    state_bits == 8 ? a.exp_avg_sq_scale : nullptr, a.numel};
        p->first[p->count++] = static_cast<unsigned>(blocks);
        blocks += need;
    }
    p->first[p->count] = static_cast<unsigned>(blocks);
    return blocks;
}

}  // namespace
}  // namespace conv2d_b200

using namespace conv2d_b200;

#pragma GCC visibility push(default)
extern "C" {

int adamw_step(const adamw_tensor_t *tensors, int count, conv_dtype_t param_dtype, conv_dtype_t grad_dtype,
               int state_bits, double lr, double beta1, double beta2, double eps, double weight_decay, long long step,
               const long long *step_device, const float *grad_scale, unsigned seed, conv_stream_t stream) {
    int st = check_types(count, tensors, param_dtype, state_bits);
    if (st != CONV_OK) return st;
    if (grad_dtype != CONV_F32 && grad_dtype != CONV_BF16)
        return abi_fail(CONV_ERR_INVALID_ARG, "dtypes must be CONV_F32 or CONV_BF16");
    if (!at_least_zero(lr) || !at_least_zero(eps) || !at_least_zero(weight_decay))
        return abi_fail(CONV_ERR_INVALID_ARG, "lr, eps and weight_decay must be finite and at least 0");
    if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0))
        return abi_fail(CONV_ERR_INVALID_ARG, "betas must lie in [0, 1)");
    if (!step_device && step < 1) return abi_fail(CONV_ERR_INVALID_ARG, "step must be at least 1");
    if ((reinterpret_cast<uintptr_t>(step_device) & 7u) || (reinterpret_cast<uintptr_t>(grad_scale) & 3u))
        return abi_fail(CONV_ERR_UNSUPPORTED, "step_device or grad_scale is not aligned to its element");
    const int elt = param_dtype == CONV_F32 ? 4 : 2;
    bool master = false;
    st = checked_tensors(tensors, count, elt, state_bits, &master);
    if (st != CONV_OK) return st;
    AbiDevice dev;
    st = abi_device(&dev);
    if (st != CONV_OK) return st;
    AdamParams p{};
    p.beta1 = static_cast<float>(beta1);
    p.beta1c = static_cast<float>(1.0 - beta1);
    p.beta2 = static_cast<float>(beta2);
    p.beta2c = static_cast<float>(1.0 - beta2);
    p.keep = static_cast<float>(1.0 - lr * weight_decay);
    p.eps = static_cast<float>(eps);
    p.lr = lr;
    p.ln_beta1 = std::log(beta1);
    p.ln_beta2 = std::log(beta2);
    if (!step_device) {
        p.rate = static_cast<float>(lr / -std::expm1(static_cast<double>(step) * p.ln_beta1));
        p.root = static_cast<float>(1.0 / std::sqrt(-std::expm1(static_cast<double>(step) * p.ln_beta2)));
    }
    p.step = step;
    p.step_device = step_device;
    p.grad_scale = grad_scale;
    p.seed = seed;
    p.status = dev.status;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    p.batches = batches_of(tensors, count, state_bits, dev.sms);
    for (int i = 0; i < count;) {
        if (next_launch(tensors, count, state_bits, &i, &p) == 0) continue;
        st = abi_launch(launch_adamw(p, elt == 4, grad_dtype == CONV_F32, master, state_bits == 8, s), "AdamW");
        if (st != CONV_OK) return st;
    }
    return abi_ok();
}

int adamw_describe_plan(const adamw_tensor_t *tensors, int count, conv_dtype_t param_dtype, int state_bits, int sms, char *buf,
                        size_t buflen) {
    int st = check_types(count, tensors, param_dtype, state_bits);
    if (st != CONV_OK) return st;
    if (!buf) return abi_fail(CONV_ERR_INVALID_ARG, "buf must not be NULL");
    bool master = false;
    st = checked_tensors(tensors, count, param_dtype == CONV_F32 ? 4 : 2, state_bits, &master);
    if (st != CONV_OK) return st;
    AdamParams p{};
    p.batches = batches_of(tensors, count, state_bits, sms);
    size_t at = 0;
    const auto put = [&](const char *fmt, auto... v) {
        const int n = at < buflen ? std::snprintf(buf + at, buflen - at, fmt, v...) : -1;
        at = n < 0 ? buflen : at + static_cast<size_t>(n);
    };
    put("{\"master\": %d, \"batches\": %d, \"launches\": [", master ? 1 : 0, p.batches);
    const char *comma = "";
    for (int i = 0; i < count;) {
        const unsigned long long blocks = next_launch(tensors, count, state_bits, &i, &p);
        if (blocks == 0) continue;
        put("%s{\"first\": %u, \"count\": %d, \"blocks\": %llu}", comma, p.index0, p.count, blocks);
        comma = ", ";
    }
    put("]%s", "}");
    if (at >= buflen) return abi_fail(CONV_ERR_INVALID_ARG, "the buffer is too small for the plan");
    return abi_ok();
}

}  // extern "C"
#pragma GCC visibility pop
