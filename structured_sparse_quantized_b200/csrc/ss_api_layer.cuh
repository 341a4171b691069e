// ss_api_layer.cuh -- the C entry points of libss (declared in include/ss.h)
// for what a transformer layer does around its products: rotary positions
// (ss_rope, ss_rope_frequencies) and the RMS norm fused into the activation's
// quantisation (ss_norm_quant_lift_act).  Included once, at the end of
// ss_api.cu, whose host helpers (device checks, launches) it uses.
#pragma once

namespace {

template <typename T, int V, int kX, bool kHalf>
ss_status launch_rope(int dev, ss::RopeArgs a, cudaStream_t s) {
    const int64_t heads = static_cast<int64_t>(a.t[0].heads) + a.t[1].heads;
    a.rot_units = a.rot / 2 / (kHalf ? kX : kX / 2);
    a.rest = V > 1 && (a.D - a.rot) % (2 * V) == 0 ? 2 * V : V;
    bool in_place = true;
    for (const ss::RopeTensor& t : a.t)
        in_place = in_place && (t.heads == 0 || (t.in == t.out && t.in_token == t.out_token &&
                                                 t.in_head == t.out_head));
    a.units = a.rot_units + (in_place ? 0 : (a.D - a.rot) / a.rest);
    // about four units per thread, but at least two blocks per SM
    const int64_t per_token = heads * a.units;
    a.tokens = static_cast<int>(std::min<int64_t>(
        {std::max<int64_t>(4 * ss::kRopeThreads / per_token, 1), ss::kRopeMaxTokens,
         std::max<int64_t>(a.T / (2 * g_num_sms[dev]), 1)}));
    const size_t smem = static_cast<size_t>(a.tokens) * a.rot * sizeof(float);
    const int64_t blocks = (a.T + a.tokens - 1) / a.tokens;
    // with too few tokens for that, a token's heads go to several blocks, as long
    // as each keeps a unit for every thread (every block forms its own cos and sin)
    const int64_t rows = a.tokens * heads, passes = a.tokens * per_token / ss::kRopeThreads;
    const int64_t parts = std::max<int64_t>(std::min(passes, 2 * g_num_sms[dev] / blocks), 1);
    a.rows = static_cast<int>((rows + parts - 1) / parts);
    return launch_ex(ss::rope_kernel<T, V, kX, kHalf>,
                     dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(parts)),
                     dim3(ss::kRopeThreads), smem, s, 1, a);
}

// The widest word (V elements: 16, 8 or 4 bytes, or one element) on whose
// boundaries every row start and every unit lie.
template <typename T>
ss_status dispatch_rope(int dev, const ss::RopeArgs& a, bool half, cudaStream_t s) {
    int64_t all = 16 / static_cast<int64_t>(sizeof(T));  // then gcd with every offset, in elements
    auto meet = [&](int64_t n) {
        while (all > 1 && n % all != 0) all /= 2;
    };
    meet(a.D - a.rot);
    meet(half ? a.rot / 2 : a.rot);
    for (const ss::RopeTensor& t : a.t) {
        if (!t.heads) continue;
        meet(static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.in) / sizeof(T)));
        meet(static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.out) / sizeof(T)));
        if (a.T > 1) meet(t.in_token), meet(t.out_token);
        if (t.heads > 1) meet(t.in_head), meet(t.out_head);
    }
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    if (half) {
        if (all == V) return launch_rope<T, V, V, true>(dev, a, s);
        if (all == V / 2) return launch_rope<T, V / 2, V / 2, true>(dev, a, s);
        if constexpr (V == 8)
            if (all == 2) return launch_rope<T, 2, 2, true>(dev, a, s);
        return launch_rope<T, 1, 1, true>(dev, a, s);
    }
    if (all == V && a.rot % (2 * V) == 0) return launch_rope<T, V, 2 * V, false>(dev, a, s);
    if (all == V) return launch_rope<T, V, V, false>(dev, a, s);
    if (all == V / 2) return launch_rope<T, V / 2, V / 2, false>(dev, a, s);
    if constexpr (V == 8)
        if (all == 2) return launch_rope<T, 2, 2, false>(dev, a, s);
    return launch_rope<T, 1, 2, false>(dev, a, s);
}

// Bytes of a set's row of codes: 4:6 and 8:10 only, with a chunk past the last group.
int norm_code_row(const ss::NormShape& s, int eb) {
    return s.Nh == 3 || s.Nh == 5
               ? static_cast<int>(round_up((s.K + 2 * s.Nh) * eb, 16) + 16 * eb + 16)
               : 0;
}

template <typename T, int kQ, int kChunks, int kWpr>
ss_status launch_norm_reg(int dev, const void* X, const void* w, int wf32, float eps, int64_t M,
                          const ss::NormShape& shape, void* Xq, float* s_x, cudaStream_t s) {
    constexpr int kSets = ss::kWarpRowThreads / (32 * kWpr);
    const int q_stride = norm_code_row(shape, kQ == ss::kQBf16 ? 2 : 1);
    constexpr auto kern = ss::norm_quant_lift_reg_kernel<T, kQ, kChunks, kWpr>;
    const size_t smem = static_cast<size_t>(kSets) * q_stride;
    const ss_status st = set_smem<kern>(dev, smem);
    if (st != SS_OK) return st;
    return launch_ex(kern, dim3(static_cast<unsigned>((M + kSets - 1) / kSets)),
                     dim3(ss::kWarpRowThreads), smem, s, 1, static_cast<const T*>(X), w, wf32, eps,
                     M, shape, q_stride, static_cast<uint8_t*>(Xq), s_x);
}

template <typename T, int kQ, int kChunks, int kWpr>
ss_status launch_norm_stream(int dev, const void* X, const void* w, int wf32, float eps, int64_t M,
                             const ss::NormShape& shape, void* Xq, float* s_x, cudaStream_t s) {
    constexpr int kThreads = ss::norm_stream_threads(kWpr);
    constexpr int64_t kSets = kThreads / (32 * kWpr);
    const int q_stride = norm_code_row(shape, kQ == ss::kQBf16 ? 2 : 1);
    const int slot = static_cast<int>(round_up(shape.K * static_cast<int64_t>(sizeof(T)), 128));
    constexpr auto kern = ss::norm_quant_lift_stream_kernel<T, kQ, kChunks, kWpr>;
    const int n_slots = static_cast<int>(std::min<int64_t>(
        ss::kNormSlots, (static_cast<int64_t>(kMaxRowSmem) / kSets - q_stride) / slot));
    const size_t smem = static_cast<size_t>(kSets) * (n_slots * slot + q_stride);
    const ss_status st = set_smem<kern>(dev, smem);
    if (st != SS_OK) return st;
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, smem) !=
            cudaSuccess ||
        per_sm < 1)
        return SS_ERR_CUDA;
    const int64_t ctas = std::min<int64_t>((M + kSets - 1) / kSets,
                                           static_cast<int64_t>(per_sm) * g_num_sms[dev]);
    return launch_ex(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), smem, s, 1,
                     static_cast<const T*>(X), w, wf32, eps, M, shape, n_slots, slot, q_stride,
                     static_cast<uint8_t*>(Xq), s_x);
}

template <typename T, int kQ>
ss_status launch_norm(int dev, const void* X, const void* w, int wf32, float eps, int64_t M,
                      int64_t K, int Nh, int64_t K_lift, int64_t K_lp, void* Xq, float* s_x,
                      cudaStream_t s) {
    const ss::NormShape shape = {static_cast<int>(K), Nh, static_cast<int>(K_lift),
                                 static_cast<int>(K_lp), static_cast<int>((K + 15) / 16)};
#define SS_NORM_REG(C, W) \
    return launch_norm_reg<T, kQ, C, W>(dev, X, w, wf32, eps, M, shape, Xq, s_x, s)
#define SS_NORM_STREAM(C, W) \
    return launch_norm_stream<T, kQ, C, W>(dev, X, w, wf32, eps, M, shape, Xq, s_x, s)
    const bool stream = K * static_cast<int64_t>(sizeof(T)) % 16 == 0 &&
                        M >= 8 * static_cast<int64_t>(g_num_sms[dev]);
    if (stream) {
        // a warp per 1024 elements, and no warps that have nothing to do: 16384 rows
        // of 5120 FP8 6:8 in 50 us with five, 71 with eight; 8192 of 10240 in 52 with
        // ten, 75 with sixteen.  (Twelve leave no room for a second CTA on an SM and
        // run 12288 slower, 79 us, than fourteen or sixteen, 76.)
        if (K <= 512) SS_NORM_STREAM(1, 1);
        switch ((K + 1023) / 1024) {
            case 1: SS_NORM_STREAM(2, 1);
            case 2: SS_NORM_STREAM(2, 2);
            case 3: SS_NORM_STREAM(2, 3);
            case 4: SS_NORM_STREAM(2, 4);
            case 5: SS_NORM_STREAM(2, 5);
            case 6: SS_NORM_STREAM(2, 6);
            case 7: SS_NORM_STREAM(2, 7);
            case 8: SS_NORM_STREAM(2, 8);
            case 9:
            case 10: SS_NORM_STREAM(2, 10);
            case 11:
            case 12:
            case 13:
            case 14: SS_NORM_STREAM(2, 14);
            case 15:
            case 16: SS_NORM_STREAM(2, 16);
        }
    }
    if (K <= 512) SS_NORM_REG(1, 1);
    if (K <= 2048) SS_NORM_REG(1, 4);
    if (K <= 4096) SS_NORM_REG(1, 8);
    if (K <= 8192) SS_NORM_REG(2, 8);
    if (K <= 16384) SS_NORM_REG(4, 8);
#undef SS_NORM_STREAM
#undef SS_NORM_REG
    return launch_ex(ss::norm_quant_lift_kernel<T, kQ>, dim3(static_cast<unsigned>(M)),
                     dim3(ss::kWarpRowThreads), 0, s, 1, static_cast<const T*>(X), w, wf32, eps, M,
                     static_cast<int>(K), Nh, static_cast<int>(K_lift), static_cast<int>(K_lp),
                     static_cast<uint8_t*>(Xq), s_x);
}

}  // namespace

extern "C" {

ss_status ss_rope_frequencies(int64_t rot_dim, double base, const ss_rope_scaling* scaling,
                              double* freqs, double* scale) {
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > ss::kRopeMaxDim || !freqs || !scale)
        return SS_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base)) return SS_ERR_INVALID_ARG;
    const ss_rope_scaling none = {SS_ROPE_NONE, 1.0, 1.0, 1.0, 1.0};
    const ss_rope_scaling& s = scaling ? *scaling : none;
    if (s.kind < SS_ROPE_NONE || s.kind > SS_ROPE_YARN) return SS_ERR_INVALID_ARG;
    if (s.kind != SS_ROPE_NONE && (!(s.factor > 0.0) || !std::isfinite(s.factor)))
        return SS_ERR_INVALID_ARG;
    const bool banded = s.kind == SS_ROPE_LLAMA3 || s.kind == SS_ROPE_YARN;
    if (banded && (!(s.original > 0.0) || !std::isfinite(s.original) || !(s.low > 0.0) ||
                   !(s.high > s.low) || !std::isfinite(s.high)))
        return SS_ERR_INVALID_ARG;
    constexpr double kTwoPi = 6.283185307179586477;
    const double d = static_cast<double>(rot_dim);
    double b = base;
    if (s.kind == SS_ROPE_NTK && rot_dim > 2) b = base * std::pow(s.factor, d / (d - 2.0));
    double first = 0.0, last = 1.0;  // YaRN: pairs between which the two scalings mix
    if (s.kind == SS_ROPE_YARN) {
        auto pair_of = [&](double turns) {
            return d * std::log(s.original / (turns * kTwoPi)) / (2.0 * std::log(base));
        };
        first = std::max(0.0, std::floor(pair_of(s.high)));
        last = std::min(d - 1.0, std::ceil(pair_of(s.low)));
    }
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(b, -2.0 * static_cast<double>(i) / d);
        double keep = 1.0;  // share of the unscaled frequency
        if (s.kind == SS_ROPE_LINEAR) keep = 0.0;
        if (s.kind == SS_ROPE_LLAMA3) {
            const double turns = s.original * f / kTwoPi;  // over the original length
            keep = std::min(1.0, std::max(0.0, (turns - s.low) / (s.high - s.low)));
        }
        if (s.kind == SS_ROPE_YARN)
            keep = 1.0 - std::min(1.0, std::max(0.0, (static_cast<double>(i) - first) /
                                                         std::max(last - first, 0.001)));
        freqs[i] = f * (keep + (1.0 - keep) / (s.kind == SS_ROPE_NONE ? 1.0 : s.factor));
    }
    *scale = s.kind == SS_ROPE_YARN && s.factor > 1.0 ? 0.1 * std::log(s.factor) + 1.0 : 1.0;
    return SS_OK;
}

ss_status ss_rope(const ss_rope_heads* q, const ss_rope_heads* k, ss_in_dtype dtype,
                  const void* positions, int32_t positions64, const double* freqs, float scale,
                  int64_t T, int64_t head_dim, int64_t rot_dim, ss_rope_layout layout,
                  ss_stream_t stream) {
    if (!q || !positions || !freqs || (positions64 != 0 && positions64 != 1))
        return SS_ERR_INVALID_ARG;
    if (dtype != SS_IN_F32 && dtype != SS_IN_BF16) return SS_ERR_INVALID_ARG;
    if (layout != SS_ROPE_HALF && layout != SS_ROPE_INTERLEAVED) return SS_ERR_INVALID_ARG;
    if (T <= 0 || T > INT32_MAX - ss::kRopeMaxTokens || head_dim < 2 || rot_dim < 2 ||
        rot_dim % 2 != 0 || rot_dim > head_dim)
        return SS_ERR_INVALID_ARG;
    if (head_dim > ss::kRopeMaxDim) return SS_ERR_UNSUPPORTED;
    const uintptr_t esz = dtype == SS_IN_F32 ? 4 : 2;
    ss::RopeArgs a = {};
    const ss_rope_heads* hs[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
        if (!hs[i]) continue;
        const ss_rope_heads& h = *hs[i];
        if (!h.in || !h.out || h.heads <= 0 || h.heads > 65536) return SS_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(h.in) % esz || reinterpret_cast<uintptr_t>(h.out) % esz)
            return SS_ERR_ALIGNMENT;
        a.t[i] = {h.in,      h.out,      static_cast<int>(h.heads), h.in_token,
                  h.in_head, h.out_token, h.out_head};
    }
    if (reinterpret_cast<uintptr_t>(positions) % (positions64 ? 8 : 4) ||
        reinterpret_cast<uintptr_t>(freqs) % 8)
        return SS_ERR_ALIGNMENT;
    int dev;
    const ss_status st = check_device(&dev);
    if (st != SS_OK) return st;
    a.pos = positions;
    a.pos64 = positions64;
    a.freq = freqs;
    a.scale = scale;
    a.T = static_cast<int>(T);
    a.D = static_cast<int>(head_dim);
    a.rot = static_cast<int>(rot_dim);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == SS_IN_BF16 ? dispatch_rope<__nv_bfloat16>(dev, a, layout == SS_ROPE_HALF, s)
                               : dispatch_rope<float>(dev, a, layout == SS_ROPE_HALF, s);
}

ss_status ss_norm_quant_lift_act(const void* X, ss_in_dtype in_dtype, const void* weight,
                                 ss_in_dtype weight_dtype, float eps, int64_t M, int64_t K,
                                 ss_pattern p, ss_qdtype q, void* Xq_lift, float* s_x,
                                 ss_stream_t stream) {
    int64_t K_pad, K_lift, K_lp;
    ss_status st = ss_slide_shape(p, K, &K_pad, &K_lift, &K_lp);
    if (st != SS_OK) return st;
    const int kq = kernel_q(q);
    if (kq < 0) return SS_ERR_INVALID_ARG;
    const bool scaled = kq != ss::kQBf16;  // the bf16 tier has no scale (s_x unused)
    if (!X || !weight || !Xq_lift || (scaled && !s_x) || M <= 0 || M > INT32_MAX)
        return SS_ERR_INVALID_ARG;
    if ((in_dtype != SS_IN_F32 && in_dtype != SS_IN_BF16) ||
        (weight_dtype != SS_IN_F32 && weight_dtype != SS_IN_BF16))
        return SS_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return SS_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(weight) || !aligned16(Xq_lift) || (scaled && !aligned16(s_x)))
        return SS_ERR_ALIGNMENT;
    int dev;
    if ((st = check_device(&dev)) != SS_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int wf32 = weight_dtype == SS_IN_F32, Nh = p.group / 2;
#define SS_NORM(T, Q) \
    return launch_norm<T, Q>(dev, X, weight, wf32, eps, M, K, Nh, K_lift, K_lp, Xq_lift, s_x, s)
    if (in_dtype == SS_IN_BF16) {
        if (kq == ss::kQInt8) SS_NORM(__nv_bfloat16, ss::kQInt8);
        if (kq == ss::kQBf16) SS_NORM(__nv_bfloat16, ss::kQBf16);
        SS_NORM(__nv_bfloat16, ss::kQE4M3);
    }
    if (kq == ss::kQInt8) SS_NORM(float, ss::kQInt8);
    if (kq == ss::kQBf16) SS_NORM(float, ss::kQBf16);
    SS_NORM(float, ss::kQE4M3);
#undef SS_NORM
}

}  // extern "C"
