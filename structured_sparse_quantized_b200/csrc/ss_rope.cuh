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
// A block takes a few tokens; its threads first compute the tokens' cos / sin
// into shared memory, then walk the tokens' heads with 16-byte accesses.
#pragma once

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
    int units;                           // work units per head
    int rot_units;                       // of them, units that rotate
};

template <typename T, int V>
struct RopeVec {
    T v[V];
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

// V consecutive elements at p (aligned to V elements).
template <typename T, int V>
__device__ __forceinline__ void rope_load(const T* p, T (&v)[V]) {
    if constexpr (V * sizeof(T) == 16)
        *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    else
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = p[i];
}
template <typename T, int V>
__device__ __forceinline__ void rope_store(T* p, const T (&v)[V]) {
    if constexpr (V * sizeof(T) == 16)
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    else
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = v[i];
}

// Work units of a head: half layout, V elements of each half (V pairs);
// interleaved, V elements (V / 2 pairs; two elements when V = 1); then, unless
// in and out are the same memory, V elements of the rest.
template <typename T, int V, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
    extern __shared__ __align__(16) float2 cs[];  // [tokens][rot / 2] (cos, sin) * scale
    pdl_trigger();
    pdl_wait();
    constexpr int kPairs = kHalf ? V : (V > 1 ? V / 2 : 1);
    constexpr int kIv = V > 1 ? V : 2;  // elements of an interleaved unit
    const int half = a.rot / 2;
    const int tok0 = static_cast<int>(blockIdx.x) * a.tokens;
    const int n_tok = min(a.tokens, a.T - tok0);
    for (int i = threadIdx.x; i < n_tok * half; i += kRopeThreads) {
        const int t = i / half, p = i - t * half;
        const int64_t pos = a.pos64 ? static_cast<const int64_t*>(a.pos)[tok0 + t]
                                    : static_cast<const int32_t*>(a.pos)[tok0 + t];
        const double turns = static_cast<double>(pos) * (a.freq[p] * 0.15915494309189533577);
        float s, c;
        sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
        cs[i] = make_float2(c * a.scale, s * a.scale);
    }
    __syncthreads();
    const int heads = a.t[0].heads + a.t[1].heads;
    const int n = n_tok * heads * a.units;
    for (int w = threadIdx.x; w < n; w += kRopeThreads) {
        const int row = w / a.units, u = w - row * a.units;
        const int t = row / heads;
        int h = row - t * heads;
        const int k = h < a.t[0].heads ? 0 : 1;
        h -= k ? a.t[0].heads : 0;
        const int64_t token = tok0 + t;
        const T* in = static_cast<const T*>(a.t[k].in) + token * a.t[k].in_token +
                      h * a.t[k].in_head;
        T* out = static_cast<T*>(a.t[k].out) + token * a.t[k].out_token + h * a.t[k].out_head;
        if (u < a.rot_units) {
            const float2* c = cs + t * half + u * kPairs;
            if constexpr (kHalf) {
                T x[V], y[V];
                rope_load<T, V>(in + u * V, x);
                rope_load<T, V>(in + half + u * V, y);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float p = to_f32<T>(x[i]), q = to_f32<T>(y[i]);
                    x[i] = from_f32<T>(p * c[i].x - q * c[i].y);
                    y[i] = from_f32<T>(q * c[i].x + p * c[i].y);
                }
                rope_store<T, V>(out + u * V, x);
                rope_store<T, V>(out + half + u * V, y);
            } else {
                T x[kIv];
                rope_load<T, kIv>(in + u * kIv, x);
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    const float p = to_f32<T>(x[2 * i]), q = to_f32<T>(x[2 * i + 1]);
                    x[2 * i] = from_f32<T>(p * c[i].x - q * c[i].y);
                    x[2 * i + 1] = from_f32<T>(q * c[i].x + p * c[i].y);
                }
                rope_store<T, kIv>(out + u * kIv, x);
            }
        } else {
            const int e = a.rot + (u - a.rot_units) * V;
            T x[V];
            rope_load<T, V>(in + e, x);
            rope_store<T, V>(out + e, x);
        }
    }
}

}  // namespace ss
