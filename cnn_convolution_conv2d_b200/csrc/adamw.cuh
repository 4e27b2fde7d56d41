// adamw.cuh -- one launch of the AdamW kernel.
#pragma once

#include "common.cuh"

namespace conv2d_b200 {

constexpr int kAdamTensors = 48;     // tensors of one launch: their table travels as a kernel argument
constexpr int kAdamThreads = 128;
constexpr int kAdamPerThread = 8;
constexpr int kAdamQuant = 256;      // elements of one scale of an 8-bit state: a warp's
constexpr int kAdamBatch = kAdamThreads * kAdamPerThread;  // elements that a block takes at a time
constexpr int kAdamBatches = 8;      // batches of a block where there are enough elements

struct AdamTensor {
    void *p;
    float *master;
    const void *g;
    void *m, *v;
    float *m_scale, *v_scale;
    long long n;
};

struct AdamParams {
    AdamTensor t[kAdamTensors];
    unsigned first[kAdamTensors + 1];  // the first block of each tensor; [count]: all blocks
    int count;
    int batches;                       // batches of a block
    unsigned index0;                   // the first tensor's place in the whole list
    float beta1, beta1c, beta2, beta2c;  // c: 1 - beta
    float keep;                        // 1 - lr * weight_decay
    float rate, root;                  // lr / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
    float eps;
    double lr, ln_beta1, ln_beta2;     // for a step read on the device
    long long step;
    const long long *step_device;
    const float *grad_scale;
    unsigned seed;
    int *status;
};

cudaError_t launch_adamw(const AdamParams &p, bool p32, bool g32, bool master, bool eight, cudaStream_t s);

}  // namespace conv2d_b200
