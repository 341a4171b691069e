// ss_rope.cuh -- rotary positions of the query and key heads that a projection
// leaves.  Of each head's D elements the first `rot` are turned in pairs
// (a, b) -- elements (i, i + rot/2) in the half layout, (2i, 2i + 1) in the
// interleaved one -- by the angle position * freq[i]:
//
//   a' = scale (a cos - b sin),   b' = scale (b cos + a sin)
//
// in fp32, rounded once; the elements from `rot` on are copied.
//
// The angle of a far position needs more than fp32: position * freq is up to
// 1e6 radians and beyond, where fp32 steps by 0.06.  It is formed in 64 bits
// in units of turns, t = position * (freq / 2 pi), and only its fractional
// part goes on in fp32 (sincospi), which costs one 64-bit product and one
// 64-bit rounding per pair and token, shared by all heads.
//
// Bound by memory: 2 * (Hq + Hk) * D elements per token against 3 flops each.
// A block takes a few tokens, computes their cos / sin into shared memory, and
// its threads sweep the tokens' heads 32 bytes at a time, in address order.
// Holding a unit's cos / sin in registers across heads takes fewer instructions
// but so many registers that too few loads are in flight (16384 tokens of 28 + 4
// heads of 128: 54-58 us; this way 45-48, the measured copy rate allows 41.8).
#pragma once

#include <type_traits>

#include "ss_common.cuh"

namespace ss {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 1024;        // elements per head, at most
constexpr int kRopeMaxTokens = 8;        // tokens per block, at most

struct RopeTensor {
    const void* in;
    void* out;
    int heads;                           // 0: none
    int64_t in_token, in_head;           // strides in elements
    int64_t out_token, out_head;
};

struct RopeArgs {
    RopeTensor t[2];                     // query, key heads
    const void* pos;
    const double* freq;                  // [rot / 2], radians per position
    float scale;
    int pos64;                           // 1: int64 positions, 0: int32
    int T, D, rot;
    int tokens;                          // per block
    int rows;                            // (token, head) rows per blockIdx.y
    int units;                           // work units per head
    int rot_units;                       // of them, units that rotate
    int rest;                            // elements of a unit past rot
};

template <typename T>
__device__ __forceinline__ T from_f32(float f);
template <>
__device__ __forceinline__ float from_f32<float>(float f) {
    return f;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float f) {
    return __float2bfloat16_rn(f);
}

// N consecutive elements at p, in words of V elements (16, 8 or 4 bytes, or one
// element); p is on a boundary of V elements.
template <int kBytes>
using RopeWord = std::conditional_t<
    kBytes == 16, uint4,
    std::conditional_t<kBytes == 8, uint2, std::conditional_t<kBytes == 4, uint32_t, uint16_t>>>;

template <typename T, int V, int N>
__device__ __forceinline__ void rope_load(const T* p, T (&v)[N]) {
    using W = RopeWord<V * static_cast<int>(sizeof(T))>;
    static_assert(sizeof(W) == V * sizeof(T) && N % V == 0, "whole words");
#pragma unroll
    for (int i = 0; i < N / V; ++i)
        reinterpret_cast<W*>(v)[i] = reinterpret_cast<const W*>(p)[i];
}
template <typename T, int V, int N>
__device__ __forceinline__ void rope_store(T* p, const T (&v)[N]) {
    using W = RopeWord<V * static_cast<int>(sizeof(T))>;
    static_assert(sizeof(W) == V * sizeof(T) && N % V == 0, "whole words");
#pragma unroll
    for (int i = 0; i < N / V; ++i)
        reinterpret_cast<W*>(p)[i] = reinterpret_cast<const W*>(v)[i];
}

// Work units of a head, kX elements each per load: half layout, kX elements of
// each half (kX pairs); interleaved, kX elements (kX / 2 pairs); then, unless in
// and out are the same memory, units of a.rest elements past rot (V or 2 V).
// Elements of a unit as two lists of pair members (p, q), and back.
template <typename T, int kX, int kPairs, bool kHalf>
__device__ __forceinline__ void rope_turn(T (&x)[kX], T (&y)[kX], const float (&c)[kPairs],
                                          const float (&s)[kPairs]) {
    auto p_at = [&](int i) -> T& { return kHalf ? x[i] : x[2 * i]; };
    auto q_at = [&](int i) -> T& { return kHalf ? y[i] : x[2 * i + 1]; };
    if constexpr (kPairs == 1) {
        const float p = to_f32<T>(p_at(0)), q = to_f32<T>(q_at(0));
        p_at(0) = from_f32<T>(p * c[0] - q * s[0]);
        q_at(0) = from_f32<T>(q * c[0] + p * s[0]);
    } else {
#pragma unroll
        for (int i = 0; i < kPairs; i += 2) {
            const float p0 = to_f32<T>(p_at(i)), p1 = to_f32<T>(p_at(i + 1));
            const float q0 = to_f32<T>(q_at(i)), q1 = to_f32<T>(q_at(i + 1));
            float a0, a1, b0, b1;
            mul_rn_f32x2(q0, q1, -s[i], -s[i + 1], a0, a1);
            fma_rn_f32x2(p0, p1, c[i], c[i + 1], a0, a1, a0, a1);
            mul_rn_f32x2(p0, p1, s[i], s[i + 1], b0, b1);
            fma_rn_f32x2(q0, q1, c[i], c[i + 1], b0, b1, b0, b1);
            p_at(i) = from_f32<T>(a0);
            p_at(i + 1) = from_f32<T>(a1);
            q_at(i) = from_f32<T>(b0);
            q_at(i + 1) = from_f32<T>(b1);
        }
    }
}

// V: elements of a word of 16, 8 or 4 bytes (1: element by element).
template <typename T, int V, int kX, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
    extern __shared__ __align__(16) float cs[];  // [tokens][rot / 2] cos, then sin, * scale
    pdl_trigger();
    pdl_wait();
    constexpr int kPairs = kHalf ? kX : kX / 2;
    const int half = a.rot / 2;
    const int tok0 = static_cast<int>(blockIdx.x) * a.tokens;
    const int n_tok = min(a.tokens, a.T - tok0);
    float* sn = cs + a.tokens * half;
    for (int i = threadIdx.x; i < n_tok * half; i += blockDim.x) {
        const int tk = i / half, p = i - tk * half;
        const int64_t pos = a.pos64 ? static_cast<const int64_t*>(a.pos)[tok0 + tk]
                                    : static_cast<const int32_t*>(a.pos)[tok0 + tk];
        const double turns = static_cast<double>(pos) * (a.freq[p] * 0.15915494309189533577);
        float s, c;
        sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
        cs[i] = c * a.scale;
        sn[i] = s * a.scale;
    }
    __syncthreads();
    const int heads = a.t[0].heads + a.t[1].heads;
    const int row0 = static_cast<int>(blockIdx.y) * a.rows;
    const int n_rows = min(row0 + a.rows, n_tok * heads);
    const int units = a.units, du = kRopeThreads % units, dr = kRopeThreads / units;
    int row = static_cast<int>(threadIdx.x) / units, u = static_cast<int>(threadIdx.x) - row * units;
    row += row0;
    int tk = row / heads, h = row - tk * heads;
    while (row < n_rows) {
        const int k = h < a.t[0].heads ? 0 : 1;
        const int64_t hh = h - (k ? a.t[0].heads : 0), token = tok0 + tk;
        const T* in = static_cast<const T*>(a.t[k].in) + token * a.t[k].in_token + hh * a.t[k].in_head;
        T* out = static_cast<T*>(a.t[k].out) + token * a.t[k].out_token + hh * a.t[k].out_head;
        if (u < a.rot_units) {
            alignas(16) T x[kX];
            alignas(16) T y[kX];
            rope_load<T, V, kX>(in + u * kX, x);
            if constexpr (kHalf) rope_load<T, V, kX>(in + half + u * kX, y);
            alignas(16) float c[kPairs];
            alignas(16) float s[kPairs];
            const int at = tk * half + u * kPairs;
            if constexpr (kPairs % 4 == 0) {
#pragma unroll
                for (int i = 0; i < kPairs; i += 4) {
                    *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + at + i);
                    *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(sn + at + i);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kPairs; ++i) c[i] = cs[at + i], s[i] = sn[at + i];
            }
            rope_turn<T, kX, kPairs, kHalf>(x, y, c, s);
            rope_store<T, V, kX>(out + u * kX, x);
            if constexpr (kHalf) rope_store<T, V, kX>(out + half + u * kX, y);
        } else {
            const int e = a.rot + (u - a.rot_units) * a.rest;
            alignas(16) T x[V];
            alignas(16) T y[V];
            rope_load<T, V, V>(in + e, x);
            if (a.rest > V) rope_load<T, V, V>(in + e + V, y);
            rope_store<T, V, V>(out + e, x);
            if (a.rest > V) rope_store<T, V, V>(out + e + V, y);
        }
        u += du;
        int d = dr;
        if (u >= units) {
            u -= units;
            ++d;
        }
        row += d;
        h += d;
        if (h >= heads) {
            const int q = h < 2 * heads ? 1 : h / heads;
            h -= q * heads;
            tk += q;
        }
    }
}

}  // namespace ss
