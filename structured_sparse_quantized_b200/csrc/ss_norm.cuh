// ss_norm.cuh -- RMS norm fused into the per-token quantisation and lift of
// the next product's activation:
//
//   y = x * r * w,  r = rsqrt(mean(x^2) + eps);   s_x = max|y| / Q,   codes RNE(Q y / max|y|)
//
// with the window map of ss_quant.cuh (the bf16 tier stores y rounded).
//
// The row's factor r cancels in Q y / max|y|: the codes come from z = x w
// alone, and r enters s_x = r max|z| / Q.  For bf16 x and w the product z is
// exact, and the quotient Q z / max|z| is formed with Q / max|z| in two parts
// and rounded once.  Ratios of 16-bit products fall on the border between two
// codes often (1200 of 16M elements at FP8), and they then go to the even code,
// as the definition says, instead of either way.
//
// A row without a finite norm (NaN or infinity in x or in x w, or a sum of squares
// past the fp32 range) has NaN in s_x, so that all of its product is NaN, as
// the definition's is for NaN and infinity: the codes alone could not say so in
// INT8.  In the bf16 tier all of its elements are NaN.  The largest |z| is taken by
// maxima that keep NaN (16384 rows of 4096 to 6:8 FP8: 45.9 us, with maxima that
// pass over it 45.6).
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

// Scale factors of a row with the largest |z| = a: z -> Q z / a, with Q / a
// held as hi + lo to 2^-48, so that the sum of the two products is the
// quotient rounded once (but for values within 2^-24 of halfway between two
// fp32 numbers, which no code border is).
template <int kQ>
struct NormQuant {
    float a, hi, lo;
    __device__ __forceinline__ NormQuant(float amax) {
        const float Q = q_max<kQ == kQInt8>();
        const float inv = amax < kNormTiny ? 0.0f : __frcp_rn(amax);
        a = amax;
        hi = Q * inv;
        lo = fmaf(-hi, amax, Q) * inv;
    }
    __device__ __forceinline__ float scaled(float z) const { return fmaf(z, hi, z * lo); }
    __device__ __forceinline__ void scaled2(float z0, float z1, float& p0, float& p1) const {
        mul_rn_f32x2(z0, z1, lo, lo, p0, p1);
        fma_rn_f32x2(z0, z1, hi, hi, p0, p1, p0, p1);
    }
    // s_x of the row with factor r
    __device__ __forceinline__ float scale(float r) const {
        return a < kNormTiny ? 0.0f : __fdiv_rn(a * r, q_max<kQ == kQInt8>());
    }
};

// The row's factor, from its sum of squares and largest |z|: NaN unless both are
// finite.
__device__ __forceinline__ float norm_factor(float sum, float amax, int K, float eps) {
    const float top = __int_as_float(0x7F7FFFFF);
    return sum <= top && amax <= top ? 1.0f / sqrtf(sum / static_cast<float>(K) + eps)
                                     : __int_as_float(0x7FFFFFFF);
}

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
        return __byte_perm(l, h, 0x5410);
    }
}

// What a set of kWpr warps knows of the rows it works on.
struct NormShape {
    int K, Nh, K_lift, K_lp, n16;  // n16: 16-element chunks of a row, the last perhaps partial
};

// z = x w of this thread's chunks (in place of x), the row's sum of squares
// and largest |z| over the warp.
template <int kChunks, typename Weight>
__device__ __forceinline__ float2 norm_products(float (&z)[kChunks][16], Weight weight) {
    float s0 = 0.0f, s1 = 0.0f, a = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        float f[16];
        weight(i, f);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            float &z0 = z[i][j], &z1 = z[i][j + 1];
            fma_rn_f32x2(z0, z1, z0, z1, s0, s1, s0, s1);
            mul_rn_f32x2(z0, z1, f[j], f[j + 1], z0, z1);
            a = max_abs3_nan(a, z0, z1);
        }
    }
    float s = s0 + s1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return make_float2(s, warp_max_abs_nan(a));
}

// The set's warps' parts together.
template <int kWpr>
__device__ __forceinline__ float2 norm_combine(const float2 (&part)[kWpr]) {
    float2 v = part[0];
#pragma unroll
    for (int i = 1; i < kWpr; ++i) {
        v.x += part[i].x;
        v.y = max_nan(v.y, part[i].y);
    }
    return v;
}

// Writes one row's codes and scale from z; c0: this thread's first chunk (then
// every 32nd), rt: its index in the set.  The windows of 4:6 and 8:10 take
// codes of neighbouring threads, through the set's row of codes qrow.
template <int kQ, int kChunks, int kWpr>
__device__ __forceinline__ void norm_write_row(const float (&z)[kChunks][16], float2 sums,
                                               float eps, const NormShape& s, int c0, int rt,
                                               int bar, uint4* qrow, uint8_t* out, float* s_x) {
    constexpr bool kBf16 = kQ == kQBf16;
    constexpr int kWords = kBf16 ? 8 : 4;  // 32-bit words of a chunk's codes
    constexpr int eb = kBf16 ? 2 : 1;
    constexpr int kSetThreads = 32 * kWpr;
    const int Nh = s.Nh, row_bytes = s.K_lp * eb;
    const NormQuant<kQ> nq(sums.y);
    float rn = 0.0f;
    if (kBf16 || rt == 0) rn = norm_factor(sums.x, sums.y, s.K, eps);
    if (!kBf16 && rt == 0) *s_x = nq.scale(rn);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = c0 + 32 * i;
        if (c >= s.n16) break;
        uint32_t u[kWords];
        if constexpr (kBf16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 h =
                    __floats2bfloat162_rn(z[i][2 * j] * rn, z[i][2 * j + 1] * rn);
                u[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float p[4];
                nq.scaled2(z[i][4 * j], z[i][4 * j + 1], p[0], p[1]);
                nq.scaled2(z[i][4 * j + 2], z[i][4 * j + 3], p[2], p[3]);
                u[j] = norm_codes4<kQ>(p[0], p[1], p[2], p[3]);
            }
        }
        if (Nh <= 2 || Nh == 3 || Nh == 5) {  // in order: to the output, or the code row
            uint4* o = Nh <= 2 ? reinterpret_cast<uint4*>(out) : qrow;
#pragma unroll
            for (int j = 0; j < kWords / 4; ++j) {
                const uint4 v = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
                if (Nh <= 2) __stcs(o + c * (kWords / 4) + j, v);
                else o[c * (kWords / 4) + j] = v;
            }
        } else if constexpr (kBf16) {
            // 6:8: two groups of four words u0..u3, windows (u0 u1) (u1 u2) (u2 u3)
            uint4* o = reinterpret_cast<uint4*>(out) + 3 * c;
            const uint4 v[3] = {make_uint4(u[0], u[1], u[1], u[2]),
                                make_uint4(u[2], u[3], u[4], u[5]),
                                make_uint4(u[5], u[6], u[6], u[7])};
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if ((3 * c + j) * 16 < row_bytes) __stcs(o + j, v[j]);
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
    if (Nh <= 2 || Nh == 4) {  // zeros past the last chunk's windows
        const int from = Nh <= 2 ? s.n16 * 16 * eb : s.n16 * 24 * eb;
        for (int o = from / 8 + rt; o < row_bytes / 8; o += kSetThreads)
            __stcs(reinterpret_cast<uint2*>(out) + o, make_uint2(0, 0));
        return;
    }
    // zero codes from the last chunk to one chunk past the last group: the
    // reads below run at most that far
    const int q_chunks = ((s.K_lift / (4 * (Nh - 1))) * 2 * Nh * eb + 15) / 16;
    for (int c = s.n16 * eb + rt; c <= q_chunks; c += kSetThreads) qrow[c] = make_uint4(0, 0, 0, 0);
    if constexpr (kWpr > 1) named_bar_sync(bar, kSetThreads);
    else __syncwarp();
    // 16 output bytes of 8-bit codes are two 6-code groups or one 10-code
    // group, of bf16 half of that
    const int n_words = (s.K_lift * eb + 15) / 16;  // with windows (the rest are zero)
    const uint32_t* q32 = reinterpret_cast<const uint32_t*>(qrow);
    for (int c = rt; c < row_bytes / 16; c += kSetThreads) {
        uint4 o = make_uint4(0, 0, 0, 0);
        if (c < n_words) {
            if constexpr (kBf16) {
                // words of two codes; windows 2 c, 2 c + 1 of the row
                const int at = Nh == 3 ? 3 * c : 5 * (c >> 1) + 2 * (c & 1);
                o = make_uint4(q32[at], q32[at + 1], q32[at + 1], q32[at + 2]);
            } else if (Nh == 3) {
                // groups 2c, 2c + 1: code bytes 12c .. 12c + 11; windows at 0, 2, 6, 8
                const uint32_t u0 = q32[3 * c], u1 = q32[3 * c + 1], u2 = q32[3 * c + 2];
                o = make_uint4(u0, __byte_perm(u0, u1, 0x5432), __byte_perm(u1, u2, 0x5432), u2);
            } else {
                // group c: code bytes 10c .. 10c + 9; windows at 0, 2, 4, 6
                const int at = (10 * c) >> 2;
                const uint32_t u0 = q32[at], u1 = q32[at + 1], u2 = q32[at + 2];
                if ((c & 1) == 0)
                    o = make_uint4(u0, __byte_perm(u0, u1, 0x5432), u1,
                                   __byte_perm(u1, u2, 0x5432));
                else
                    o = make_uint4(__byte_perm(u0, u1, 0x5432), u1, __byte_perm(u1, u2, 0x5432),
                                   u2);
            }
        }
        __stcs(reinterpret_cast<uint4*>(out) + c, o);
    }
}

// Elements at, at + 1, ... at + 15 of X (`all` elements, 16-byte aligned), of
// which the first n are wanted (zero for the rest): from the 16-byte words that
// hold them, shifted into place.  (16 loads of an element each made 16384 rows of
// 4095 take 105 us.)
template <typename T>
__device__ __forceinline__ void gload16_shifted(const T* __restrict__ X, int64_t at, int n,
                                                int64_t all, float (&f)[16]) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));  // elements of a word
    constexpr int kW = 16 / V + 1;                       // words that may hold 16 elements
    if (n <= 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = 0.0f;
        return;
    }
    const int64_t w0 = at / V;
    const int s = static_cast<int>(at - w0 * V);  // elements before ours in the first word
    uint32_t x[4 * kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        const int64_t first = (w0 + i) * V;
        if (i * V < s + n) {  // holds an element of ours
            if (first + V <= all) {
                v = __ldg(reinterpret_cast<const uint4*>(X) + w0 + i);
            } else {  // the last word of X, not whole
                uint32_t p[4] = {0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (first + j < all) {
                        if constexpr (sizeof(T) == 2)
                            p[j / 2] |= bf16_bits(to_f32<T>(X[first + j])) << (16 * (j & 1));
                        else
                            p[j] = __float_as_uint(to_f32<T>(X[first + j]));
                    }
                v = make_uint4(p[0], p[1], p[2], p[3]);
            }
        }
        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
    // move down by s elements: by whole 32-bit words, then by half a word
    const int words = sizeof(T) == 2 ? s >> 1 : s;
#pragma unroll
    for (int i = 0; i < 4 * kW - 2; ++i) x[i] = (words & 2) ? x[i + 2] : x[i];
#pragma unroll
    for (int i = 0; i < 4 * kW - 3; ++i) x[i] = (words & 1) ? x[i + 1] : x[i];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        if constexpr (sizeof(T) == 2) {
            // element j: half s + j of the words, i.e. (j + (s & 1)) of the moved ones
            const uint32_t a = x[j / 2], b = x[j / 2 + 1];
            const uint32_t even = (j & 1) ? a & 0xFFFF0000u : a << 16;
            const uint32_t odd = (j & 1) ? b << 16 : a & 0xFFFF0000u;
            f[j] = __uint_as_float((s & 1) ? odd : even);
        } else {
            f[j] = __uint_as_float(x[j]);
        }
        if (j >= n) f[j] = 0.0f;
    }
}

// Rows of up to 512 kChunks kWpr elements, read once: kWpr warps hold a row's
// z in fp32 registers, 16 kChunks per lane; 8 / kWpr rows per CTA.  For few
// rows, and for rows that are not whole 16-byte words.
template <typename T, int kQ, int kChunks, int kWpr>
__global__ void __launch_bounds__(kWarpRowThreads) norm_quant_lift_reg_kernel(
    const T* __restrict__ X, const void* __restrict__ w, int wf32, float eps, int64_t M,
    const NormShape s, int q_stride, uint8_t* __restrict__ Xq, float* __restrict__ s_x) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int kSets = kWarpRowThreads / (32 * kWpr);
    __shared__ float2 part[kSets][kWpr];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int set = warp / kWpr, sub = warp % kWpr;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * kSets + set;
    if (m >= M) return;  // a set's warps leave (or stay) together
    const bool vec = s.K * static_cast<int>(sizeof(T)) % 16 == 0;
    const int c0 = sub * 32 * kChunks + lane;  // chunks c0 + 32 i, i < kChunks
    float z[kChunks][16];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int k = (c0 + 32 * i) * 16;
        if (vec)
            gload16<T>(X + m * s.K, k, s.K, true, z[i]);
        else
            gload16_shifted<T>(X, m * s.K + k, s.K - k, M * s.K, z[i]);
    }
    float2 sums = norm_products<kChunks>(z, [&](int i, float (&f)[16]) {
        norm_weight16(w, wf32, (c0 + 32 * i) * 16, s.K, f);
    });
    if constexpr (kWpr > 1) {
        if (lane == 0) part[set][sub] = sums;
        named_bar_sync(1 + set, 32 * kWpr);
        sums = norm_combine<kWpr>(part[set]);
    }
    norm_write_row<kQ, kChunks, kWpr>(
        z, sums, eps, s, c0, sub * 32 + lane, 1 + set,
        reinterpret_cast<uint4*>(smem_raw + set * q_stride),
        Xq + m * static_cast<int64_t>(s.K_lp) * (kQ == kQBf16 ? 2 : 1), s_x + m);
}

// Many rows of whole 16-byte words: CTAs stay, each set of kWpr warps keeps
// the weights of its chunks in registers and kNormSlots rows in flight from
// HBM into shared memory (1-D bulk copies), so that the copies of the next
// rows go on while a row is reduced, quantised and stored.  Bound by HBM: 16384
// rows of 4096 bf16 to 6:8 FP8 in 44-47 us, 78-83% of the measured copy rate.
// Without the copies in flight (rows straight to registers, 2 to 8 warps per
// row) 16384 rows of 4096 took 50-89 us: the loads pause in every row's
// reduction, and a weight read per row costs as much L1 time as the row.
constexpr int kNormSlots = 4;  // at most: as many as fit shared memory

// As many sets as eight warps hold, or one larger set (rows past 8192: eight warps
// would hold too much of a row each to keep its weights too; 5041 x 13312 78 -> 51 us).
constexpr int norm_stream_threads(int wpr) { return 32 * wpr * (wpr > 8 ? 1 : 8 / wpr); }

template <typename T, int kQ, int kChunks, int kWpr>
__global__ void __launch_bounds__(norm_stream_threads(kWpr)) norm_quant_lift_stream_kernel(
    const T* __restrict__ X, const void* __restrict__ w, int wf32, float eps, int64_t M,
    const NormShape s, int n_slots, int slot_stride, int q_stride, uint8_t* __restrict__ Xq,
    float* __restrict__ s_x) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int kSets = norm_stream_threads(kWpr) / (32 * kWpr);
    __shared__ uint64_t full[kSets][kNormSlots];
    __shared__ float2 part[2][kSets][kWpr];
    __shared__ int abort_flag_storage;
    volatile int* abort_flag = &abort_flag_storage;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int set = warp / kWpr, sub = warp % kWpr;
    const int rt = sub * 32 + lane;
    const int c0 = sub * 32 * kChunks + lane;
    if (threadIdx.x == 0) *abort_flag = 0;
    if (rt == 0) {
        for (int b = 0; b < n_slots; ++b) mbar_init(&full[set][b], 1);
        fence_barrier_init();
    }
    __syncthreads();
    pdl_trigger();
    pdl_wait();
    uint8_t* slots = smem_raw + set * (n_slots * slot_stride);
    uint4* qrow = reinterpret_cast<uint4*>(smem_raw + kSets * n_slots * slot_stride +
                                           set * q_stride);
    const uint32_t bytes = static_cast<uint32_t>(s.K) * static_cast<uint32_t>(sizeof(T));
    const int64_t step = static_cast<int64_t>(gridDim.x) * kSets;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kSets + set;
    uint32_t pending = 0;  // slots with a copy in flight (thread 0 of the set)
    auto issue = [&](int64_t m, int b) {
        if (m >= M) return;
        pending |= 1u << b;
        mbar_arrive_expect_tx(&full[set][b], bytes);
        bulk_load_1d(slots + b * slot_stride, X + m * s.K, bytes, &full[set][b]);
    };
    if (rt == 0)
        for (int b = 0; b < n_slots; ++b) issue(m0 + b * step, b);
    float f[kChunks][16];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) norm_weight16(w, wf32, (c0 + 32 * i) * 16, s.K, f[i]);
    const bool whole = s.K == 512 * kChunks * kWpr;  // every thread's chunks are whole
    int b = 0;             // slot of this row
    uint32_t phase = 0, odd = 0;  // parity of the slot's copies, and of the rows
    for (int64_t m = m0; m < M; m += step, odd ^= 1u) {
        const bool got = mbar_wait(&full[set][b], phase, abort_flag);
        const T* x = reinterpret_cast<const T*>(slots + b * slot_stride);
        float z[kChunks][16];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = c0 + 32 * i;
            const uint4* v = reinterpret_cast<const uint4*>(x + c * 16);
            constexpr int kVec = 16 / static_cast<int>(sizeof(T));
#pragma unroll
            for (int j = 0; j < 16 / kVec; ++j) {  // K is whole 16-byte words
                const uint4 u = whole || c * 16 + (j + 1) * kVec <= s.K ? v[j] : make_uint4(0, 0, 0, 0);
                const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (sizeof(T) == 2) {
                        z[i][8 * j + 2 * k] = __uint_as_float(uw[k] << 16);
                        z[i][8 * j + 2 * k + 1] = __uint_as_float(uw[k] & 0xFFFF0000u);
                    } else {
                        z[i][4 * j + k] = __uint_as_float(uw[k]);
                    }
                }
            }
        }
        float2 sums = norm_products<kChunks>(z, [&](int i, float (&g)[16]) {
#pragma unroll
            for (int j = 0; j < 16; ++j) g[j] = f[i][j];
        });
        bool all = got;
        if constexpr (kWpr > 1) {
            if (lane == 0) part[odd][set][sub] = sums;
            // also: every warp of the set has read the slot, and is done with
            // the code row and the parts of two rows ago
            all = named_bar_and(1 + set, 32 * kWpr, got);
            sums = norm_combine<kWpr>(part[odd][set]);
        } else {
            all = __all_sync(0xffffffffu, got);
        }
        if (!all) break;
        if (rt == 0) {
            pending &= ~(1u << b);
            fence_async_shared();
            issue(m + n_slots * step, b);
        }
        if (++b == n_slots) {
            b = 0;
            phase ^= 1u;
        }
        norm_write_row<kQ, kChunks, kWpr>(
            z, sums, eps, s, c0, rt, 1 + set, qrow,
            Xq + m * static_cast<int64_t>(s.K_lp) * (kQ == kQBf16 ? 2 : 1), s_x + m);
    }
    // after a wait that ran out: copies in flight land before exit (a slot from b
    // on waits for this phase, one before b for the next)
    if (rt == 0 && pending)
        for (int i = 0; i < n_slots; ++i)
            if ((pending >> i) & 1u) mbar_drain(&full[set][i], i >= b ? phase : phase ^ 1u);
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
        a = max_nan(a, fabsf(z_at(k)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    }
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(ss, a);
    __syncthreads();
    ss = a = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarpRowThreads / 32; ++i) {
        ss += part[i].x;
        a = max_nan(a, part[i].y);
    }
    const float r = norm_factor(ss, a, K, eps);
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
