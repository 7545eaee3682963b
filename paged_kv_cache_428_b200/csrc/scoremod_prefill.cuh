// scoremod_prefill.cuh -- chunked-prefill attention with modified scores, on prefill_tc.cuh.  With p the position
// of the query and t that of the key:
//
//   x = scale q . k                              the score
//   x = cap tanh(x / cap)                        softcap > 0
//   x = x - slope_h |p - t|                      alibi_slopes
//   seen:  (t <= p or t < prefix)  and  t > p - window (window > 0)
//   out = softmax over the seen t of x, times V
//
// The logits are kept in the log2 domain (times log2 e) like all scores of this library.
#pragma once

#include "prefill_tc.cuh"
#include "tanh_poly.cuh"

namespace pa {

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The softmax warps bound the prefill kernel, and their registers are full: what is done to a score there
// counts, and so does every branch around it.  Hence four kernels, by whether scores are capped and biased:
//   window, prefix     only the tiles at the borders are masked; scores stay as they are.  (8 chunks of 512
//                      after 0..3584 tokens, 32 heads of 128: 166 us, 164 without either; CAP 193; BIAS 193.)
//   BIAS               one multiply-add to the raw score, slope / scale times the place in the tile; what the
//                      whole tile has in common goes into the softmax's reference.  Only tiles with tokens on
//                      both sides of a row need more.
//   CAP                tanh(y) = y q(y^2) while a warp's tile has |x| <= 0.3 cap (see tanh_poly.cuh), with cap and
//                      scale inside the coefficients, on the FMA pipe; else the exact form, an exponential and
//                      a reciprocal more for each score on the MUFU unit.
// Places of a tile's tokens, two at a time (operands of one packed multiply-add each).
__constant__ float2 kPlaces[32] = {
    {0.f, 1.f}, {2.f, 3.f}, {4.f, 5.f}, {6.f, 7.f}, {8.f, 9.f}, {10.f, 11.f}, {12.f, 13.f}, {14.f, 15.f},
    {16.f, 17.f}, {18.f, 19.f}, {20.f, 21.f}, {22.f, 23.f}, {24.f, 25.f}, {26.f, 27.f}, {28.f, 29.f}, {30.f, 31.f},
    {32.f, 33.f}, {34.f, 35.f}, {36.f, 37.f}, {38.f, 39.f}, {40.f, 41.f}, {42.f, 43.f}, {44.f, 45.f}, {46.f, 47.f},
    {48.f, 49.f}, {50.f, 51.f}, {52.f, 53.f}, {54.f, 55.f}, {56.f, 57.f}, {58.f, 59.f}, {60.f, 61.f}, {62.f, 63.f}};

template <bool CAP, bool BIAS>
struct PrefillScoreMod {
    static constexpr bool kOn = true, kCap = CAP;
    const float *slopes;           // [h_q]
    const int32_t *prefix_lens;    // [B] or null
    int window;                    // 0: no window
    float cap_in, cap_out;         // 2 scale log2(e) / cap and cap log2(e)
    float range;                   // |raw score| up to which the polynomial holds
    float c[3];                    // its coefficients, for raw scores and log2-domain logits

    __device__ __forceinline__ int prefix(int seq) const { return prefix_lens ? __ldg(prefix_lens + seq) : 0; }
    __device__ __forceinline__ int first_token(int pos) const { return window > 0 ? max(0, pos - window + 1) : 0; }
    // What logits() leaves is to be multiplied by this: uncapped scores stay raw.
    __device__ __forceinline__ float unit(float qk_scale) const { return CAP ? 1.f : qk_scale; }
    // A head's slope in those units.
    __device__ __forceinline__ float slope(int head, float qk_scale) const
    {
        return BIAS ? __ldg(slopes + head) * 1.4426950408889634f / unit(qk_scale) : 0.f;
    }

    // What the bias can still add to the largest logit of a tile whose last token lies `distance` before the row:
    // with the reference that far ahead O is rarely rescaled on the way to the row's own position (a steep
    // head gains 46 for every tile).  At most 96, so that what the reference turns out to be too far ahead
    // costs nothing: probabilities of 2^-96 are as exact as those of 1.
    __device__ __forceinline__ float ahead(float slope_log2, int distance) const
    {
        return BIAS ? fminf(96.f, fmaxf(0.f, slope_log2 * (float)distance)) : 0.f;
    }

    // Raw scores of tokens first + pos, first + pos + 1, ... of one row into logits sr + what is returned.
    // both_sides: some of the tokens may lie behind the row's position.
    __device__ __forceinline__ float logits(uint32_t (&sr)[2][32], float slope, int first, bool both_sides) const
    {
        auto at = [&](int i) -> uint32_t & { return sr[i >> 5][i & 31]; };
        auto pair = [&](int i) { return make_float2(__uint_as_float(at(i)), __uint_as_float(at(i + 1))); };
        auto put = [&](int i, float2 x) {
            at(i) = __float_as_uint(x.x);
            at(i + 1) = __float_as_uint(x.y);
        };
        if constexpr (CAP) {
            float m4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 64; i += 2)
                m4[(i >> 1) & 3] = max3f(m4[(i >> 1) & 3], fabsf(__uint_as_float(at(i))), fabsf(__uint_as_float(at(i + 1))));
            const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            // (rows of K that are no token are 0 by now: the K warp sees to it.  Leaving their columns out here took 131 to
            // 134 us for the chunk case, against 118)
            if (!__any_sync(0xffffffffu, top > range)) {
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const float2 x = pair(i), u = __fmul2_rn(x, x);
                    float2 q = __ffma2_rn(u, make_float2(c[2], c[2]), make_float2(c[1], c[1]));
                    q = __ffma2_rn(u, q, make_float2(c[0], c[0]));
                    put(i, __fmul2_rn(x, q));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const float e = ex2_approx(__uint_as_float(at(i)) * cap_in);
                    at(i) = __float_as_uint(cap_out * fmaf(-2.f, rcp_approx(e + 1.f), 1.f));
                }
            }
        }
        if constexpr (BIAS) {
            const float2 s2 = make_float2(slope, slope);
#pragma unroll
            for (int i = 0; i < 64; i += 2) put(i, __ffma2_rn(s2, kPlaces[i / 2], pair(i)));
            if (both_sides) {                          // behind the row the bias falls again
                const float d0 = (float)first;
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    at(i) = __float_as_uint(fmaf(-2.f * slope, fmaxf(d0 + (float)i, 0.f), __uint_as_float(at(i))));
            }
            return slope * (float)first;
        }
        return 0.f;
    }
};

}  // namespace pa
