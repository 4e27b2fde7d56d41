// optimizer_abi.cu -- the C ABI declared in include/optimizer_b200.h: argument validation and
// the launches of the AdamW kernel, kAdamTensors tensors each.  Host code only.
#include <algorithm>
#include <cmath>
#include <new>
#include <utility>
#include <vector>

#include "adamw.cuh"
#include "host.cuh"
#include "optimizer_b200.h"

namespace conv2d_b200 {
namespace {

constexpr long long kMaxElements = 1LL << 41;  // the blocks of one tensor stay below 2^31

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_tensors(const adamw_tensor_t *t, int count, int elt, int state_bits) {
    std::vector<std::pair<uintptr_t, uintptr_t>> weights;
    weights.reserve(count);
    bool master = false, none = false;
    for (int i = 0; i < count; ++i) {
        const adamw_tensor_t &a = t[i];
        if (a.numel < 0) return abi_fail(CONV_ERR_INVALID_ARG, "tensor %d: numel is negative", i);
        if (a.numel == 0) continue;
        if (a.numel > kMaxElements) return abi_fail(CONV_ERR_UNSUPPORTED, "tensor %d: more than 2^41 elements", i);
        if (!a.param || !a.grad || !a.exp_avg || !a.exp_avg_sq)
            return abi_fail(CONV_ERR_INVALID_ARG, "tensor %d: param, grad, exp_avg and exp_avg_sq must not be NULL", i);
        if (state_bits == 8 && (!a.exp_avg_scale || !a.exp_avg_sq_scale))
            return abi_fail(CONV_ERR_INVALID_ARG, "tensor %d: 8-bit states need their scales", i);
        if (!aligned16(a.param) || !aligned16(a.master) || !aligned16(a.grad) || !aligned16(a.exp_avg) ||
            !aligned16(a.exp_avg_sq) || ((reinterpret_cast<uintptr_t>(a.exp_avg_scale) |
                                          reinterpret_cast<uintptr_t>(a.exp_avg_sq_scale)) & 3u))
            return abi_fail(CONV_ERR_UNSUPPORTED, "tensor %d: device pointers must be 16-byte aligned", i);
        if (a.master) master = true; else none = true;
        if (a.master && elt == 4)
            return abi_fail(CONV_ERR_INVALID_ARG, "tensor %d: fp32 weights are their own master weights", i);
        const uintptr_t p = reinterpret_cast<uintptr_t>(a.param);
        weights.emplace_back(p, p + static_cast<uintptr_t>(a.numel) * elt);
    }
    if (master && none) return abi_fail(CONV_ERR_INVALID_ARG, "either all or no tensors have master weights");
    std::sort(weights.begin(), weights.end());
    for (size_t i = 1; i < weights.size(); ++i)
        if (weights[i].first < weights[i - 1].second)
            return abi_fail(CONV_ERR_INVALID_ARG, "two weight tensors overlap");
    return CONV_OK;
}

bool at_least_zero(double v) { return v >= 0.0 && std::isfinite(v); }

}  // namespace
}  // namespace conv2d_b200

using namespace conv2d_b200;

#pragma GCC visibility push(default)
extern "C" {

int adamw_step(const adamw_tensor_t *tensors, int count, conv_dtype_t param_dtype, conv_dtype_t grad_dtype,
               int state_bits, double lr, double beta1, double beta2, double eps, double weight_decay, long long step,
               const long long *step_device, const float *grad_scale, unsigned seed, conv_stream_t stream) {
    if (count < 0 || (count > 0 && !tensors))
        return abi_fail(CONV_ERR_INVALID_ARG, "count must be at least 0 and tensors not NULL");
    if ((param_dtype != CONV_F32 && param_dtype != CONV_BF16) || (grad_dtype != CONV_F32 && grad_dtype != CONV_BF16))
        return abi_fail(CONV_ERR_INVALID_ARG, "dtypes must be CONV_F32 or CONV_BF16");
    if (state_bits != 8 && state_bits != 32) return abi_fail(CONV_ERR_INVALID_ARG, "state_bits must be 8 or 32");
    if (!at_least_zero(lr) || !at_least_zero(eps) || !at_least_zero(weight_decay))
        return abi_fail(CONV_ERR_INVALID_ARG, "lr, eps and weight_decay must be finite and at least 0");
    if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0))
        return abi_fail(CONV_ERR_INVALID_ARG, "betas must lie in [0, 1)");
    if (!step_device && step < 1) return abi_fail(CONV_ERR_INVALID_ARG, "step must be at least 1");
    if ((reinterpret_cast<uintptr_t>(step_device) & 7u) || (reinterpret_cast<uintptr_t>(grad_scale) & 3u))
        return abi_fail(CONV_ERR_UNSUPPORTED, "step_device or grad_scale is not aligned to its element");
    const int elt = param_dtype == CONV_F32 ? 4 : 2;
    try {
        const int st = check_tensors(tensors, count, elt, state_bits);
        if (st != CONV_OK) return st;
    } catch (const std::bad_alloc &) {
        return abi_fail(CONV_ERR_INVALID_ARG, "out of host memory");
    }
    AbiDevice dev;
    int st = abi_device(&dev);
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
    // With 8-bit states a block takes more batches, and finds its tensor once for them, where that leaves 8 blocks an SM
    // (100 M elements: 313 -> 258 us); with 32-bit states, which wait for memory alone, that costs (422 -> 438 us).
    long long elements = 0;
    for (int k = 0; k < count; ++k) elements += std::min(tensors[k].numel, kMaxElements);
    p.batches = state_bits == 32 ? 1
                                 : static_cast<int>(std::min<long long>(std::max<long long>(elements / kAdamBatch / (8LL * dev.sms), 1),
                                                                        kAdamBatches));
    const unsigned long long per_block = static_cast<unsigned long long>(p.batches) * kAdamBatch;
    int i = 0;
    while (i < count) {
        // the next tensors that have elements, as many as one launch takes
        p.count = 0;
        unsigned long long blocks = 0;
        bool master = false;
        p.index0 = static_cast<unsigned>(i);
        for (; i < count && p.count < kAdamTensors; ++i) {
            const adamw_tensor_t &a = tensors[i];
            const unsigned long long need = (static_cast<unsigned long long>(a.numel) + per_block - 1) / per_block;
            if (blocks + need > 0x7fffffffULL) break;
            p.t[p.count] = AdamTensor{a.param, a.master, a.grad, a.exp_avg, a.exp_avg_sq,
                                      state_bits == 8 ? a.exp_avg_scale : nullptr,
                                      state_bits == 8 ? a.exp_avg_sq_scale : nullptr, a.numel};
            p.first[p.count++] = static_cast<unsigned>(blocks);
            master = master || a.master;
            blocks += need;
        }
        p.first[p.count] = static_cast<unsigned>(blocks);
        if (blocks == 0) continue;
        st = abi_launch(launch_adamw(p, elt == 4, grad_dtype == CONV_F32, master, state_bits == 8, s), "AdamW");
        if (st != CONV_OK) return st;
    }
    return abi_ok();
}

}  // extern "C"
#pragma GCC visibility pop
