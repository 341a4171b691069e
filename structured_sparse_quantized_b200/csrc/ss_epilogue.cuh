// ss_epilogue.cuh -- what the fused GEMM entry points do to an accumulator
// between the dequantisation and the one rounding to Y's type:
//
//   v[m, n] = fma((float)acc[m, n] * s_x[m], s_w[n], bias[n])
//   plain:  Y[m, n]         = act(v[m, n]) + residual[m, n]
//   gated:  Y[m, 8 g + i]   = act(v[m, 16 g + i]) * v[m, 16 g + 8 + i],  i < 8
//
// all in fp32; without a bias v is the plain product's fp32 value.  A gated
// weight holds its rows in groups of 16, eight gates and then their eight
// partners: the two factors of an output then sit 8 rows apart inside one
// 16-row group, which no kernel shape splits (tiles, K-split reduction slices
// and tensor-memory lane quarters are multiples of 16), and the 16x256b
// tensor-memory fragments hold both in one thread.
#pragma once

#include "ss_common.cuh"

namespace ss {

constexpr int kActNone = 0;
constexpr int kActRelu = 1;
constexpr int kActSilu = 2;
constexpr int kActGelu = 3;     // the tanh form
constexpr int kActGeluErf = 4;  // v Phi(v)

// How a kernel's fused epilogue writes Y: by TMA with A rows = channels or
// tokens (bf16 Y), or straight from registers (fp32 Y or residual, rows that
// are not 16-byte aligned).  Kernels of their own: in one kernel the ways share
// the registers of the widest, and the TMA ways spill (8192 x 4096 x 4096 with
// a bias 67 us instead of 64.5).
constexpr int kEpiNone = 0, kEpiChannels = 1, kEpiTokens = 2, kEpiDirect = 3;
// The TMA ways with tiles of at most kFewRows B rows: such a product streams its
// A rows, and small B tiles leave room for rings of 5 to 8 stages instead of 2
// to 6 (16 tokens, 28672 x 4096 6:8 FP8 gated: 26 -> 22.4 us; weight and
// selectors 110 MB).
constexpr int kEpiChannelsFew = 4, kEpiTokensFew = 5;
constexpr int kFewRows = 64;
constexpr bool epi_is_few(int epi) { return epi == kEpiChannelsFew || epi == kEpiTokensFew; }

struct EpiArgs {
    const void* bias;      // [N], or null
    const void* residual;  // [M, N], or null
    int bias_f32;          // 1: fp32 bias, 0: bf16
    int res_f32;           // 1: fp32 residual, 0: bf16
    int act;               // kAct*
    int gated;
};

// Activations, two values at a time (packed fp32 arithmetic).
//
// silu(v) = v / (1 + e^-v).  The tanh form of GELU is v / (1 + e^-2u) with
// u = sqrt(2/pi) (v + 0.044715 v^3), because (1 + tanh u) / 2 = 1 / (1 + e^-2u):
// unlike 1 + tanh u it does not cancel for negative v.
//
// The exact GELU is v Phi(v) = max(v, 0) - |v| Phi(-|v|), and Phi(-u) =
// e^(-u^2 / 2) G(u) with G(u) = erfcx(u / sqrt 2) / 2 smooth and slowly falling:
// G = t Q(t) with t = 1 / (1 + 0.34 u) and a polynomial Q of degree 8 fitted to
// a small relative error over u in [0, 16]: 6.8e-8 with the constants as fp32
// holds them, 2.8 units of 2^-23 evaluated in fp32 from a rounded t, 4.2 from a t
// that is one unit off.  Unlike v (1 + erf) / 2 it keeps its digits for
// negative v, at two special-function operations a value; CUDA's erfcf in this
// place took the epilogue of a 256 x 224 tile past its MMAs (8192 x 4096 x
// 4096 2:4 INT8: 149 us against 63 for the plain product).
//
// Each result is within a few units of 2^-23 (plus those of the exponent, which
// grow with it), far below the rounding to bf16.  e^-v = inf gives -0 for finite
// v; at v = -inf it is 0 * inf, and SiLU and the tanh GELU are NaN, as their
// formulas are (the exact GELU is 0).
template <int kAct>
__device__ __forceinline__ void activate2(float& v0, float& v1) {
    if constexpr (kAct == kActRelu) {
        v0 = relu_nan(v0);
        v1 = relu_nan(v1);
    } else if constexpr (kAct == kActSilu || kAct == kActGelu) {
        float x0, x1;  // -(exponent of e) log2(e)
        if constexpr (kAct == kActSilu) {
            mul_rn_f32x2(v0, v1, -1.4426950409f, -1.4426950409f, x0, x1);
        } else {
            constexpr float c1 = -2.3022081986f;  // -2 sqrt(2 / pi) log2 e
            constexpr float c3 = -0.10294323960f;  // 0.044715 c1
            mul_rn_f32x2(v0, v1, v0, v1, x0, x1);
            fma_rn_f32x2(x0, x1, c3, c3, c1, c1, x0, x1);
            mul_rn_f32x2(x0, x1, v0, v1, x0, x1);
        }
        x0 = ex2_fast(x0);
        x1 = ex2_fast(x1);
        add_rn_f32x2(x0, x1, 1.0f, 1.0f, x0, x1);
        mul_rn_f32x2(v0, v1, rcp_fast(x0), rcp_fast(x1), v0, v1);
    } else if constexpr (kAct == kActGeluErf) {
        // |v| is cut at 16, where Phi(-u) is 0 in fp32, so that infinities pass
        const float u0 = fminf(fabsf(v0), 16.0f), u1 = fminf(fabsf(v1), 16.0f);
        float t0, t1, e0, e1, q0, q1;
        fma_rn_f32x2(u0, u1, 0.34f, 0.34f, 1.0f, 1.0f, t0, t1);
        t0 = rcp_fast(t0);
        t1 = rcp_fast(t1);
        mul_rn_f32x2(u0, u1, u0, u1, e0, e1);
        mul_rn_f32x2(e0, e1, -0.72134752044f, -0.72134752044f, e0, e1);  // log2(e) / 2
        e0 = ex2_fast(e0);
        e1 = ex2_fast(e1);
        constexpr float kQ[9] = {-0.025177352130f, 0.13510350883f,   -0.26447525620f,
                                 0.19280642271f,   -0.038633506745f, 0.11294532567f,
                                 0.11576713622f,   0.13603937626f,   0.13562436402f};
        q0 = q1 = kQ[0];
#pragma unroll
        for (int i = 1; i < 9; ++i) fma_rn_f32x2(q0, q1, t0, t1, kQ[i], kQ[i], q0, q1);
        mul_rn_f32x2(q0, q1, t0, t1, q0, q1);
        mul_rn_f32x2(q0, q1, e0, e1, q0, q1);  // Phi(-u)
        fma_rn_f32x2(-u0, -u1, q0, q1, relu_nan(v0), relu_nan(v1), v0, v1);
    }
}

// act on y[0..N), or, with kGates, on the values whose index has bit 1 clear
// (the gates of a fragment, see epi_tile_tma).
template <int kAct, bool kGates, int N>
__device__ __forceinline__ void activate_values(float (&y)[N]) {
#pragma unroll
    for (int j = 0; j < N; j += 2)
        if (!kGates || (j & 2) == 0) activate2<kAct>(y[j], y[j + 1]);
}

template <bool kGates, int N>
__device__ __forceinline__ void activate(float (&y)[N], int act) {
    switch (act) {
        case kActRelu: activate_values<kActRelu, kGates>(y); break;
        case kActSilu: activate_values<kActSilu, kGates>(y); break;
        case kActGelu: activate_values<kActGelu, kGates>(y); break;
        case kActGeluErf: activate_values<kActGeluErf, kGates>(y); break;
        default: break;
    }
}

__device__ __forceinline__ float activate(float v, int act) {
    float y[2] = {v, 0.0f};
    activate<false>(y, act);
    return y[0];
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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool kOutBf16>
__device__ __forceinline__ void store_y(void* y, int64_t off, float v) {
    if constexpr (kOutBf16)
        static_cast<__nv_bfloat16*>(y)[off] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(y)[off] = v;
}

}  // namespace ss
