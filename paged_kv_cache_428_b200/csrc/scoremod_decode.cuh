// scoremod_decode.cuh -- single-token attention with modified scores, on decode_split.cuh.  With p the position
// of the query and t that of the key:
//
//   x = scale q . k                              the score
//   x = cap tanh(x / cap)                        softcap > 0
//   x = x - slope_h |p - t|                      alibi_slopes
//   seen:  t > p - window (window > 0)
//   out = softmax over the seen t of x, times V
//
// The logits are kept in the log2 domain (times log2 e) like all scores of this library.
#pragma once

#include "decode_split.cuh"
#include "tanh_poly.cuh"

namespace pa {

// Bound by the bytes of K and V inside the window (64 sequences of 512..4096 tokens, 613 MB: 100.1 to 103.6 us, 5.9
// to 6.1 TB/s); 4 logits a lane and 16 tokens leave room for both forms of tanh: the polynomial for small arguments,
// 1 - 2 / (e^2y + 1) for the others.
struct ScoreModExt {
    static constexpr bool kDependent = false;
    struct Args {
        const float *slopes;       // [h_q] or null
        float cap_in, cap_out;     // 2 scale log2(e) / cap and cap log2(e); cap_out = 0: no cap
    };
    template <int G>
    struct Row {
        float scale, cap_in, cap_out, slope[2];
        int last;
        __device__ __forceinline__ Row(const Args &a, const SplitParams &p, int, int kvh, int ctx, int lane)
            : scale(p.qk_scale), cap_in(a.cap_in), cap_out(a.cap_out), last(ctx - 1)
        {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = 2 * (lane & 3) + j;
                slope[j] = a.slopes != nullptr && h < G ? __ldg(a.slopes + kvh * G + h) * 1.4426950408889634f : 0.f;
            }
        }
        __device__ __forceinline__ float logit(float dot, int t, int j) const
        {
            float x = dot * scale;
            if (cap_out > 0.f) {
                const float y = dot * cap_in * 0.34657359028f, u = y * y;      // cap_in is 2 log2(e) y / dot
                const float small = y * fmaf(u, fmaf(u, PA_TANH_C2, PA_TANH_C1), PA_TANH_C0);
                const float large = 1.f - __fdividef(2.f, exp2f(dot * cap_in) + 1.f);
                x = cap_out * (fabsf(y) <= PA_TANH_RANGE ? small : large);
            }
            return fmaf(slope[j], (float)(t - last), x);
        }
        __device__ __forceinline__ void keep(const float (&)[4], int, bool, bool) const {}
    };
};

}  // namespace pa
