// adamw.cu -- one AdamW step over many tensors in one launch.
//
//   g = grad scale, m = b1 m + (1-b1) g, v = b2 v + (1-b2) g^2,
//   p = p (1 - lr wd) - lr m / (1-b1^t) / (sqrt(v / (1-b2^t)) + eps)
//
// With 32-bit states bound by HBM (28 bytes an element, 6.7 TB/s); with 8-bit states by the issue of
// instructions, about 75 for an element's 10 bytes: a third of them the random bits and the rounding, most of the others the update
// itself, one element to an instruction.  So there a thread
// keeps to 40 registers, for 48 warps an SM, and a block takes several batches of 1024 elements of one tensor, which it
// finds by a search in the table of tensors.  The table is a kernel argument: nothing is uploaded, and a captured
// launch keeps its own copy.  Every element is read and written once.
// 100 M elements: fp32 414 us (6.8 TB/s); bf16 with fp32 master weights 420 us, with 8-bit states 268 us (3.7 TB/s),
// with both 303 us (5.3 TB/s).  With the step's number on the device, for captured steps, every block works out the rates in 64
// bits: fp32 414 us, 8-bit states 274 us, 100 000 elements 8.2 us, as without.
//
// 8-bit states hold 256 elements (a warp's) to one scale, a power of two, so that scaling is
// exact: m in e4m3 (largest element in [2^7, 2^8)), v in e5m2 ([2^14, 2^15): v spans twice the
// binades of m).  They are rounded up or down by chance, in proportion to the distance: v moves
// by about (1-b2) of itself a step, a hundredth of the distance between two codes, and rounding
// to the nearest would leave it where it is for good.  The chance comes from a hash of (seed,
// step, tensor, element), so a step repeated on the same data gives the same bits.  A v above
// zero is held at least at the smallest code: at zero, its element would step by m / eps.
// Elements that are not finite are held as NaN and leave the scale to the others.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "adamw.cuh"

namespace conv2d_b200 {
namespace {

constexpr int E = kAdamPerThread;

// (With numbers below 2^-126: where eps is 0 or near it, such a v counts.  8 of the 268 us above.)
__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ void load8(float (&f)[E], const T *p, int valid) {
    if (valid == E) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        } else {
            const uint4 r = __ldcs(reinterpret_cast<const uint4 *>(p));
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = i < valid ? static_cast<float>(p[i]) : 0.f;
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[E], int valid) {
    if (valid == E) {
        if constexpr (sizeof(T) == 4) {
            __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
            __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
        } else {
            __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                            pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < valid) p[i] = static_cast<T>(f[i]);
    }
}

// 8 codes of an 8-bit state and their scale.
template <__nv_fp8_interpretation_t kKind>
__device__ __forceinline__ void load_codes(float (&f)[E], const uint8_t *p, float scale, int valid) {
    uint32_t w[2] = {0, 0};
    if (valid == E) {
        const uint2 r = __ldcs(reinterpret_cast<const uint2 *>(p));
        w[0] = r.x;
        w[1] = r.y;
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < valid) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
    }
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 2] >> (8 * (i & 3))), kKind);
        const float2 v = __half22float2(__half2(h));
        f[i] = v.x * scale;
        f[i + 1] = v.y * scale;
    }
}

// Appleby's public-domain finaliser of a 32-bit hash.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
    h = (h ^ (h >> 13)) * 0xC2B2AE35u;
    return h ^ (h >> 16);
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7fffffffu) < 0x7f800000u; }

__device__ __forceinline__ uint32_t size_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale of a warp's values from the bits of the largest size: a power of two that brings it into
// [2^kTop, 2^(kTop+1)).
template <int kTop>
__device__ __forceinline__ float scale_of(uint32_t big, float &inverse) {
    const uint32_t e = max(big >> 23, static_cast<uint32_t>(kTop + 1)) - kTop;
    inverse = big ? __uint_as_float((254u - e) << 23) : 1.f;
    return big ? __uint_as_float(e << 23) : 1.f;
}

// Rounds v (already scaled) to kKeep fraction bits, up where the random bits carry: the lowest of them weighs
// 2^-16 of a step.  Below 2^kSmall, the smallest normal number, the steps stay equal: there v is rounded one binade higher
// and brought back.  (The bits of a float grow with its size whatever its sign.)
template <int kSmall, int kKeep, bool kSigned>
__device__ __forceinline__ float round_by_chance(float v, uint32_t bits16) {
    constexpr float kLift = kSmall == -6 ? 0x1p-6f : 0x1p-14f;
    constexpr int kLow = 23 - kKeep;
    const float lift = fabsf(v) < kLift ? (kSigned ? copysignf(kLift, v) : kLift) : 0.f;
    const uint32_t whole = __float_as_uint(__fadd_rn(v, lift)) + bits16 * (1u << (kLow - 16));
    return __uint_as_float(whole & ~((1u << kLow) - 1u)) - lift;
}

template <__nv_fp8_interpretation_t kKind>
__device__ __forceinline__ void store_codes(uint8_t *p, const float (&f)[E], int valid) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(f[i], f[i + 1]), __NV_SATFINITE, kKind);
        w[i >> 2] |= c << (8 * (i & 3));
    }
    if (valid == E) {
        __stcs(reinterpret_cast<uint2 *>(p), make_uint2(w[0], w[1]));
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < valid) p[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
    }
}

template <typename P, typename G, bool kMaster, bool kEight>
__global__ void __launch_bounds__(kAdamThreads, kEight ? 12 : 1) adamw_kernel(const __grid_constant__ AdamParams q) {
    __shared__ float s_rate[2];
    float rate = q.rate, root = q.root;
    long long step = q.step;
    if (q.step_device) {  // 1 - beta^step in 64 bits: it is small for the first steps
        step = *q.step_device;
        if (step < 1) {
            if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(q.status, kDevBadStep);
            return;
        }
        if (threadIdx.x == 0) {
            s_rate[0] = static_cast<float>(q.lr / -expm1(static_cast<double>(step) * q.ln_beta1));
            s_rate[1] = static_cast<float>(1.0 / sqrt(-expm1(static_cast<double>(step) * q.ln_beta2)));
        }
        __syncthreads();
        rate = s_rate[0];
        root = s_rate[1];
    }
    const float scale = q.grad_scale ? *q.grad_scale : 1.f;
    if (!(scale > 0.f && finite(scale))) return;
    int lo = 0, hi = q.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (q.first[mid] <= blockIdx.x) lo = mid; else hi = mid - 1;
    }
    const AdamTensor &t = q.t[lo];
    const uint32_t key = kEight ? mix(mix(q.seed + 0x9E3779B9u * static_cast<uint32_t>(step)) + 0x85EBCA77u * (q.index0 + lo + 1)) : 0u;
    const float minus_rate = -rate;
    long long at = static_cast<long long>(blockIdx.x - q.first[lo]) * q.batches * kAdamBatch + threadIdx.x * E;
    for (int batch = 0; batch < q.batches; ++batch, at += kAdamBatch) {
        const long long quant = at / kAdamQuant;   // the same for the lanes of a warp
        if (quant * kAdamQuant >= t.n) return;
        const int valid = at >= t.n ? 0 : t.n - at < E ? static_cast<int>(t.n - at) : E;
        float g[E], m[E], v[E], w[E];
        load8(g, static_cast<const G *>(t.g) + at, valid);
        if constexpr (kMaster) load8(w, t.master + at, valid);
        else load8(w, static_cast<const P *>(t.p) + at, valid);
        if constexpr (kEight) {
            load_codes<__NV_E4M3>(m, static_cast<const uint8_t *>(t.m) + at, t.m_scale[quant], valid);
            load_codes<__NV_E5M2>(v, static_cast<const uint8_t *>(t.v) + at, t.v_scale[quant], valid);
        } else {
            load8(m, static_cast<const float *>(t.m) + at, valid);
            load8(v, static_cast<const float *>(t.v) + at, valid);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float gs = g[i] * scale;
            // each product rounded by itself: the 8-bit codes below are a fixed function of the inputs
            m[i] = __fadd_rn(__fmul_rn(m[i], q.beta1), __fmul_rn(gs, q.beta1c));
            v[i] = __fadd_rn(__fmul_rn(v[i], q.beta2), __fmul_rn(__fmul_rn(gs, gs), q.beta2c));
            // (the root and the quotient are off by a few units of an update that is a thousandth of the weight or less)
            w[i] = fmaf(w[i], q.keep, minus_rate * (m[i] * rcp_approx(fmaf(sqrt_approx(v[i]), root, q.eps))));
        }
        if constexpr (kMaster) store8(t.master + at, w, valid);
        store8(static_cast<P *>(t.p) + at, w, valid);
        if constexpr (kEight) {
            uint32_t big_m = 0, big_v = 0;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                big_m = max(big_m, size_bits(m[i]));
                big_v = max(big_v, __float_as_uint(v[i]));  // v has no sign
            }
            big_m = __reduce_max_sync(0xffffffffu, big_m);
            big_v = __reduce_max_sync(0xffffffffu, big_v);
            // Elements that are not finite: they are held as NaN and leave the scale to the others.  Rare, and the warp's own.
            uint32_t lost_m = 0, lost_v = 0;
            if (big_m >= 0x7f800000u || big_v >= 0x7f800000u) {
                big_m = big_v = 0;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (finite(m[i])) big_m = max(big_m, size_bits(m[i])); else lost_m |= 1u << i;
                    if (finite(v[i])) big_v = max(big_v, size_bits(v[i])); else lost_v |= 1u << i;
                }
                big_m = __reduce_max_sync(0xffffffffu, big_m);
                big_v = __reduce_max_sync(0xffffffffu, big_v);
            }
            float im, iv;
            const float scale_m = scale_of<7>(big_m, im), scale_v = scale_of<14>(big_v, iv);
            const uint32_t first = static_cast<uint32_t>(at) * 0x9E3779B1u + key;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const uint32_t h = mix(first + i * 0x9E3779B1u);
                m[i] = round_by_chance<-6, 3, true>(m[i] * im, h & 0xffffu);
                const float sv = v[i] * iv;
                // the smallest code where v is above zero (and not 2^-142 of the largest), else 0
                v[i] = fmaxf(round_by_chance<-14, 2, false>(sv, h >> 16), fminf(sv * 0x1p126f, 0x1p-16f));
            }
            if (lost_m | lost_v) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (lost_m >> i & 1u) m[i] = __int_as_float(0x7fc00000);
                    if (lost_v >> i & 1u) v[i] = __int_as_float(0x7fc00000);
                }
            }
            store_codes<__NV_E4M3>(static_cast<uint8_t *>(t.m) + at, m, valid);
            store_codes<__NV_E5M2>(static_cast<uint8_t *>(t.v) + at, v, valid);
            if ((threadIdx.x & 31) == 0) {
                t.m_scale[quant] = scale_m;
                t.v_scale[quant] = scale_v;
            }
        } else {
            store8(static_cast<float *>(t.m) + at, m, valid);
            store8(static_cast<float *>(t.v) + at, v, valid);
        }
    }
}

template <typename P, typename G, bool kMaster>
cudaError_t launch_bits(const AdamParams &p, bool eight, cudaStream_t s) {
    if (eight) adamw_kernel<P, G, kMaster, true><<<p.first[p.count], kAdamThreads, 0, s>>>(p);
    else adamw_kernel<P, G, kMaster, false><<<p.first[p.count], kAdamThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamParams &p, bool p32, bool g32, bool master, bool eight, cudaStream_t s) {
    if (p32) return g32 ? launch_bits<float, float, false>(p, eight, s) : launch_bits<float, __nv_bfloat16, false>(p, eight, s);
    if (master)
        return g32 ? launch_bits<__nv_bfloat16, float, true>(p, eight, s)
                   : launch_bits<__nv_bfloat16, __nv_bfloat16, true>(p, eight, s);
    return g32 ? launch_bits<__nv_bfloat16, float, false>(p, eight, s)
               : launch_bits<__nv_bfloat16, __nv_bfloat16, false>(p, eight, s);
}

}  // namespace conv2d_b200
