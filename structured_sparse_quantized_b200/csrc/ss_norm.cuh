// ss_norm.cuh -- RMS norm fused into the per-token quantisation and lift of
// the next product's activation:
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   s_x = max|y| / Q,   codes RNE(y (Q / max|y|))
//
// in fp32 (the bf16 tier stores y rounded to bf16), with the window map of
// ss_quant.cuh.  The normalised row is never written: X is read and the codes
// are written, which is all the memory traffic there is.
#pragma once

#include "ss_quant.cuh"

namespace ss {

constexpr float kNormTiny = 1e-35f;

__device__ __forceinline__ float norm_weight(const void* w, int wf32, int k) {
    return wf32 ? __ldg(static_cast<const float*>(w) + k)
                : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[k]);
}

// One block per token row, any K, any element type.  The output is walked in
// lifted order, each code recomputed from its source element.
template <typename T, int kQ>
__global__ void __launch_bounds__(kWarpRowThreads) norm_quant_lift_kernel(
    const T* __restrict__ X, const void* __restrict__ w, int wf32, float eps, int64_t M, int K,
    int Nh, int K_lift, int K_lp, uint8_t* __restrict__ Xq, float* __restrict__ s_x) {
    __shared__ float part[kWarpRowThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int64_t m = blockIdx.x;
    const T* x = X + m * K;
    auto reduce = [&](float v, bool sum) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float u = __shfl_xor_sync(0xffffffffu, v, o);
            v = sum ? v + u : fmaxf(v, u);
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int i = 1; i < kWarpRowThreads / 32; ++i) v = sum ? v + part[i] : fmaxf(v, part[i]);
        return v;
    };
    float ss = 0.0f;
    for (int k = threadIdx.x; k < K; k += kWarpRowThreads) {
        const float f = to_f32<T>(x[k]);
        ss = fmaf(f, f, ss);
    }
    const float r = 1.0f / sqrtf(reduce(ss, true) / static_cast<float>(K) + eps);
    auto value = [&](int k) { return to_f32<T>(x[k]) * r * norm_weight(w, wf32, k); };
    float inv = 0.0f, s = 0.0f;
    if constexpr (kQ != kQBf16) {
        float a = 0.0f;
        for (int k = threadIdx.x; k < K; k += kWarpRowThreads) a = fmaxf(a, fabsf(value(k)));
        a = reduce(a, false);
        // a row too small for Q / a in fp32 has codes 0
        scale_from_absmax<kQ == kQInt8>(a < kNormTiny ? 0.0f : a, inv, s);
        if (threadIdx.x == 0) s_x[m] = s;
    }
    for (int o = threadIdx.x; o < K_lp; o += kWarpRowThreads) {
        int k = o;
        if (Nh > 2) {
            const int win = o >> 2, g = win / (Nh - 1);
            k = o < K_lift ? 2 * Nh * g + 2 * (win - g * (Nh - 1)) + (o & 3) : K;
        }
        const float y = k < K ? value(k) : 0.0f;
        if constexpr (kQ == kQBf16)
            reinterpret_cast<uint16_t*>(Xq)[m * K_lp + o] = static_cast<uint16_t>(bf16_bits(y));
        else
            Xq[m * K_lp + o] = static_cast<uint8_t>(quantize<kQ == kQInt8>(y, inv));
    }
}

}  // namespace ss
