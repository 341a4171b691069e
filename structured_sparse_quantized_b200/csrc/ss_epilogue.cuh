// ss_epilogue.cuh -- what the fused GEMM entry points do to an accumulator
// between the dequantisation and the one rounding to Y's type:
//
//   v[m, n] = ((float)acc[m, n] * s_x[m]) * s_w[n] + bias[n]
//   plain:  Y[m, n]         = act(v[m, n]) + residual[m, n]
//   gated:  Y[m, 8 g + i]   = act(v[m, 16 g + i]) * v[m, 16 g + 8 + i],  i < 8
//
// all in fp32.  A gated weight holds its rows in groups of 16, eight gates
// and then their eight partners: the two factors of an output then sit 8 rows
// apart inside one 16-row group, which no kernel shape splits (tiles, K-split
// reduction slices and tensor-memory lane quarters are multiples of 16), and
// the 16x256b tensor-memory fragments hold both in one thread.
#pragma once

#include "ss_common.cuh"

namespace ss {

constexpr int kActNone = 0;
constexpr int kActRelu = 1;
constexpr int kActSilu = 2;
constexpr int kActGelu = 3;     // the tanh form
constexpr int kActGeluErf = 4;  // v Phi(v)

struct EpiArgs {
    const void* bias;      // [N], or null
    const void* residual;  // [M, N], or null
    int bias_f32;          // 1: fp32 bias, 0: bf16
    int res_f32;           // 1: fp32 residual, 0: bf16
    int act;               // kAct*
    int gated;
};

// silu(v) = v / (1 + e^-v).  The tanh form of GELU is v / (1 + e^-2u) with
// u = sqrt(2/pi) (v + 0.044715 v^3), because (1 + tanh u) / 2 = 1 / (1 + e^-2u):
// unlike 1 + tanh u it does not cancel for negative v.  For the same reason
// the exact form is v erfc(-v / sqrt 2) / 2.  The fast exponential and divide
// are within a few units of 2^-23, far below the rounding to bf16 and within
// what fp32 products of this length carry; e^-v = inf gives -0.
template <int kAct>
__device__ __forceinline__ float activate(float v) {
    if constexpr (kAct == kActRelu) {
        return v < 0.0f ? 0.0f : v;  // NaN stays
    } else if constexpr (kAct == kActSilu) {
        return __fdividef(v, 1.0f + __expf(-v));
    } else if constexpr (kAct == kActGelu) {
        const float u2 = v * fmaf(0.0713548162726f, v * v, 1.5957691216057f);  // 2 u
        return __fdividef(v, 1.0f + __expf(-u2));
    } else if constexpr (kAct == kActGeluErf) {
        return 0.5f * v * erfcf(v * -0.70710678118655f);
    } else {
        return v;
    }
}

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case kActRelu: return activate<kActRelu>(v);
        case kActSilu: return activate<kActSilu>(v);
        case kActGelu: return activate<kActGelu>(v);
        case kActGeluErf: return activate<kActGeluErf>(v);
        default: return v;
    }
}

__device__ __forceinline__ float load_f32_or_bf16(const void* p, int64_t i, int is_f32) {
    return is_f32 ? __ldg(static_cast<const float*>(p) + i)
                  : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ float epi_bias(const EpiArgs& e, int ch, bool in_range) {
    return e.bias && in_range ? load_f32_or_bf16(e.bias, ch, e.bias_f32) : 0.0f;
}

// The residual may be Y itself (same elements, read before they are written
// by the same thread), so it is not read through the non-coherent path.
__device__ __forceinline__ float epi_residual(const EpiArgs& e, int64_t off) {
    return e.res_f32 ? static_cast<const float*>(e.residual)[off]
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[off]);
}

// Output column of weight row ch of a gated product (its gate rows).
__device__ __forceinline__ int gated_col(int ch) { return ((ch >> 4) << 3) | (ch & 7); }

// act on the fragment y[2][16] of a thread (see epi_tile_channels): every
// value, or the gates (values 4 r + k).
template <int kAct, bool kGates>
__device__ __forceinline__ void activate_fragment(float (&y)[2][16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (!kGates || (j & 2) == 0) y[h][j] = activate<kAct>(y[h][j]);
}

template <bool kGates>
__device__ __forceinline__ void epi_activate(float (&y)[2][16], int act) {
    switch (act) {
        case kActRelu: activate_fragment<kActRelu, kGates>(y); break;
        case kActSilu: activate_fragment<kActSilu, kGates>(y); break;
        case kActGelu: activate_fragment<kActGelu, kGates>(y); break;
        case kActGeluErf: activate_fragment<kActGeluErf, kGates>(y); break;
        default: break;
    }
}
__device__ __forceinline__ void epi_activate_all(float (&y)[2][16], int act) {
    epi_activate<false>(y, act);
}
__device__ __forceinline__ void epi_activate_gates(float (&y)[2][16], int act) {
    epi_activate<true>(y, act);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Address of this thread's row of the four 8x8 blocks (r = 2 rp, 2 rp + 1) x
// (channel blocks e = 0, 1) in a staged [2 halves][32 tokens][64 channels]
// chunk with 128B swizzle.
__device__ __forceinline__ uint32_t epi_block_addr(uint32_t base, int rp, int q, int h, int mi,
                                                   int mj) {
    const int tok = 8 * (2 * rp + (mi >> 1)) + mj;
    const int ch = q * 32 + 16 * h + 8 * (mi & 1);
    return base + (ch >> 6) * (32 * 128) + tok * 128 + ((((ch & 63) >> 3) ^ (tok & 7)) << 4);
}

template <bool kOutBf16>
__device__ __forceinline__ void store_y(void* y, int64_t off, float v) {
    if constexpr (kOutBf16)
        static_cast<__nv_bfloat16*>(y)[off] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(y)[off] = v;
}

}  // namespace ss
