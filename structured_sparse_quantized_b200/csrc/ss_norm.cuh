// ss_norm.cuh -- RMS norm fused into the per-token quantisation and lift of
// the next product's activation:
//
//   y = x * r * w,  r = rsqrt(mean(x^2) + eps);   s_x = max|y| / Q,   codes RNE(Q y / max|y|)
//
// with the window map of ss_quant.cuh (the bf16 tier stores y rounded).
//
// The row's factor r cancels in Q y / max|y|: the codes come from z = x w
// alone, and r enters s_x = r max|z| / Q.  For bf16 x and w the product z is
// exact, and so is Q z; the quotient Q z / max|z| is rounded correctly (one
// Newton correction of the product with 1 / max|z|).  Ratios of 16-bit
// products fall on the border between two codes often (1200 of 16M elements
// at FP8), and the correctly rounded quotient then goes to the even code, as
// the definition says, instead of either way.
//
// The normalised row is never written: X is read and the codes are written,
// which is all the memory traffic there is.
#pragma once

#include "ss_quant.cuh"

namespace ss {

constexpr float kNormTiny = 1e-35f;  // max|z| below this: codes 0 (1 / max|z| stays finite)

__device__ __forceinline__ float norm_weight(const void* w, int wf32, int k) {
    return wf32 ? __ldg(static_cast<const float*>(w) + k)
                : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[k]);
}

// Sixteen weights at k0 (zero past K).
__device__ __forceinline__ void norm_weight16(const void* w, int wf32, int k0, int K,
                                              float (&f)[16]) {
    if (wf32)
        gload16<float>(static_cast<const float*>(w), k0, K, true, f);
    else
        gload16<__nv_bfloat16>(static_cast<const __nv_bfloat16*>(w), k0, K, true, f);
}

// Scale factors of a row with the largest |z| = a: z -> RN(Q z / a).
template <int kQ>
struct NormQuant {
    float a, inv;
    __device__ __forceinline__ NormQuant(float amax) {
        a = amax;
        inv = amax < kNormTiny ? 0.0f : __frcp_rn(amax);
    }
    __device__ __forceinline__ float scaled(float z) const {
        const float zq = z * q_max<kQ == kQInt8>();
        const float p = zq * inv;
        return fmaf(fmaf(-p, a, zq), inv, p);
    }
    // s_x of the row
    __device__ __forceinline__ float scale(float r) const {
        return inv == 0.0f ? 0.0f : __fdiv_rn(a * r, q_max<kQ == kQInt8>());
    }
};

// Four scaled values as four code bytes.
template <int kQ>
__device__ __forceinline__ uint32_t norm_codes4(float p0, float p1, float p2, float p3) {
    if constexpr (kQ == kQInt8) {  // |p| <= 127: the integer in the low mantissa bits
        const uint32_t b0 = __float_as_uint(p0 + 12582912.0f), b1 = __float_as_uint(p1 + 12582912.0f);
        const uint32_t b2 = __float_as_uint(p2 + 12582912.0f), b3 = __float_as_uint(p3 + 12582912.0f);
        return __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410);
    } else {
        const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(p0, p1), __NV_SATFINITE, __NV_E4M3);
        const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(p2, p3), __NV_SATFINITE, __NV_E4M3);
        return (l & 0xFFFFu) | (h << 16);
    }
}

// Rows of up to 512 kChunks kWpr elements, read once: kWpr warps hold a row's
// z in fp32 registers, 16 kChunks per lane; 8 / kWpr rows per CTA.  One
// exchange gives the row's sum of squares and largest |z|.  Bound by HBM; with
// z in registers each weight is read once per row, from L1.
// q_stride: bytes of one row of codes in shared memory (4:6 and 8:10 only,
// whose windows take codes of neighbouring lanes).
template <typename T, int kQ, int kChunks, int kWpr>
__global__ void __launch_bounds__(kWarpRowThreads) norm_quant_lift_reg_kernel(
    const T* __restrict__ X, const void* __restrict__ w, int wf32, float eps, int64_t M, int K,
    int Nh, int K_lift, int K_lp, int q_stride, uint8_t* __restrict__ Xq,
    float* __restrict__ s_x) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int kRowsPerCta = kWarpRowThreads / (32 * kWpr);
    constexpr int kRowThreads = 32 * kWpr;
    constexpr bool kBf16 = kQ == kQBf16;
    constexpr int kWords = kBf16 ? 8 : 4;  // 32-bit words of a chunk's codes
    __shared__ float2 part[kRowsPerCta][kWpr];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slot = warp / kWpr, sub = warp % kWpr;
    const int rt = sub * 32 + lane;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * kRowsPerCta + slot;
    if (m >= M) return;  // a row's warps leave (or stay) together
    const T* x = X + m * K;
    const bool vec = K * static_cast<int>(sizeof(T)) % 16 == 0;
    const int n16 = (K + 15) / 16;
    const int c0 = sub * 32 * kChunks + lane;  // chunks c0 + 32 i, i < kChunks
    float z[kChunks][16];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) gload16<T>(x, (c0 + 32 * i) * 16, K, vec, z[i]);
    float ss = 0.0f, a = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        float f[16];
        norm_weight16(w, wf32, (c0 + 32 * i) * 16, K, f);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            ss = fmaf(z[i][j], z[i][j], ss);
            z[i][j] *= f[j];
            a = fmaxf(a, fabsf(z[i][j]));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    }
    if constexpr (kWpr > 1) {
        if (lane == 0) part[slot][sub] = make_float2(ss, a);
        named_bar_sync(1 + slot, kRowThreads);
        ss = a = 0.0f;
#pragma unroll
        for (int v = 0; v < kWpr; ++v) {
            ss += part[slot][v].x;
            a = fmaxf(a, part[slot][v].y);
        }
    }
    const float r = 1.0f / sqrtf(ss / static_cast<float>(K) + eps);
    const NormQuant<kQ> nq(a);
    if constexpr (!kBf16) {
        if (rt == 0) s_x[m] = nq.scale(r);
    }
    const int64_t row_bytes = static_cast<int64_t>(K_lp) * (kBf16 ? 2 : 1);
    uint8_t* out = Xq + m * row_bytes;
    uint4* qrow = reinterpret_cast<uint4*>(smem_raw + slot * q_stride);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = c0 + 32 * i;
        if (c >= n16) break;
        uint32_t u[kWords];
        if constexpr (kBf16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(z[i][2 * j] * r, z[i][2 * j + 1] * r);
                u[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                u[j] = norm_codes4<kQ>(nq.scaled(z[i][4 * j]), nq.scaled(z[i][4 * j + 1]),
                                       nq.scaled(z[i][4 * j + 2]), nq.scaled(z[i][4 * j + 3]));
        }
        if (Nh <= 2 || Nh == 3 || Nh == 5) {  // in order: to the output, or to the code row
            uint4* o = Nh <= 2 ? reinterpret_cast<uint4*>(out) : qrow;
#pragma unroll
            for (int j = 0; j < kWords / 4; ++j) {
                const uint4 v = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
                if (Nh <= 2) __stcs(o + c * (kWords / 4) + j, v);
                else o[c * (kWords / 4) + j] = v;
            }
        } else if constexpr (kBf16) {
            // 6:8: two groups of four words u0..u3, windows (u0 u1) (u1 u2) (u2 u3)
            uint2* o = reinterpret_cast<uint2*>(out) + 6 * c;
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if ((6 * c + 3 * g + j) * 8 < row_bytes)
                        __stcs(o + 3 * g + j, make_uint2(u[4 * g + j], u[4 * g + j + 1]));
        } else {
            // 6:8: two groups of eight codes, windows at 0, 2, 4 of each
            uint2* o = reinterpret_cast<uint2*>(out) + 3 * c;
            const uint2 v[3] = {make_uint2(u[0], __byte_perm(u[0], u[1], 0x5432)),
                                make_uint2(u[1], u[2]),
                                make_uint2(__byte_perm(u[2], u[3], 0x5432), u[3])};
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if ((3 * c + j) * 8 < row_bytes) __stcs(o + j, v[j]);
        }
    }
    const int eb = kBf16 ? 2 : 1;
    if (Nh <= 2 || Nh == 4) {  // zeros past the last chunk's windows
        const int from = Nh <= 2 ? n16 * 16 * eb : n16 * 24 * eb;
        for (int o = from / 8 + rt; o < row_bytes / 8; o += kRowThreads)
            __stcs(reinterpret_cast<uint2*>(out) + o, make_uint2(0, 0));
        return;
    }
    // 4:6, 8:10: zero codes from the last chunk to one chunk past the last group
    // (the reads below run at most one chunk past it), then the windows
    const int q_chunks = ((K_lift / (4 * (Nh - 1))) * 2 * Nh * eb + 15) / 16;
    for (int c = n16 * eb + rt; c <= q_chunks; c += kRowThreads) qrow[c] = make_uint4(0, 0, 0, 0);
    if constexpr (kWpr > 1) named_bar_sync(1 + slot, kRowThreads);
    else __syncwarp();
    // units: the 2-element words of the code row (uint16 of 8-bit codes, uint32
    // of bf16); window i of group g is words Nh g + i, Nh g + i + 1
    const int n_win = K_lift / 4, per = Nh - 1;
    constexpr int kWin = kBf16 ? 2 : 4;  // windows per 16-byte store
    for (int c = rt; c < row_bytes / 16; c += kRowThreads) {
        int win = c * kWin, g = win / per, j = win - g * per;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < kWin; ++i) {
            const int at = Nh * g + j;
            const bool in = win + i < n_win;
            if constexpr (kBf16) {
                const uint32_t* q32 = reinterpret_cast<const uint32_t*>(qrow);
                o[2 * i] = in ? q32[at] : 0u;
                o[2 * i + 1] = in ? q32[at + 1] : 0u;
            } else {
                const uint16_t* q16 = reinterpret_cast<const uint16_t*>(qrow);
                o[i] = in ? q16[at] | (static_cast<uint32_t>(q16[at + 1]) << 16) : 0u;
            }
            if (++j == per) {
                j = 0;
                ++g;
            }
        }
        __stcs(reinterpret_cast<uint4*>(out) + c, make_uint4(o[0], o[1], o[2], o[3]));
    }
}

// One block per token row, any K.  The output is walked in lifted order, each
// code recomputed from its source element (rows longer than the registers of
// a block).
template <typename T, int kQ>
__global__ void __launch_bounds__(kWarpRowThreads) norm_quant_lift_kernel(
    const T* __restrict__ X, const void* __restrict__ w, int wf32, float eps, int64_t M, int K,
    int Nh, int K_lift, int K_lp, uint8_t* __restrict__ Xq, float* __restrict__ s_x) {
    __shared__ float2 part[kWarpRowThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int64_t m = blockIdx.x;
    const T* x = X + m * K;
    auto z_at = [&](int k) { return to_f32<T>(x[k]) * norm_weight(w, wf32, k); };
    float ss = 0.0f, a = 0.0f;
    for (int k = threadIdx.x; k < K; k += kWarpRowThreads) {
        const float f = to_f32<T>(x[k]);
        ss = fmaf(f, f, ss);
        a = fmaxf(a, fabsf(z_at(k)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    }
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(ss, a);
    __syncthreads();
    ss = a = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarpRowThreads / 32; ++i) {
        ss += part[i].x;
        a = fmaxf(a, part[i].y);
    }
    const float r = 1.0f / sqrtf(ss / static_cast<float>(K) + eps);
    const NormQuant<kQ> nq(a);
    if constexpr (kQ != kQBf16) {
        if (threadIdx.x == 0) s_x[m] = nq.scale(r);
    }
    for (int o = threadIdx.x; o < K_lp; o += kWarpRowThreads) {
        int k = o;
        if (Nh > 2) {
            const int win = o >> 2, g = win / (Nh - 1);
            k = o < K_lift ? 2 * Nh * g + 2 * (win - g * (Nh - 1)) + (o & 3) : K;
        }
        const float z = k < K ? z_at(k) : 0.0f;
        const int64_t at = m * K_lp + o;
        if constexpr (kQ == kQBf16)
            reinterpret_cast<uint16_t*>(Xq)[at] = static_cast<uint16_t>(bf16_bits(z * r));
        else
            Xq[at] = static_cast<uint8_t>(norm_codes4<kQ>(nq.scaled(z), 0.0f, 0.0f, 0.0f));
    }
}

}  // namespace ss
