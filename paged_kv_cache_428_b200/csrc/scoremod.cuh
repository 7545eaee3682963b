// scoremod.cuh -- attention with modified scores, for single tokens (on decode_split.cuh) and for chunks (on
// prefill_tc.cuh).  With p the position of the query and t that of the key:
//
//   x = scale q . k                              the score
//   x = cap tanh(x / cap)                        softcap > 0
//   x = x - slope_h |p - t|                      alibi_slopes
//   seen:  (t <= p or t < prefix)  and  t > p - window (window > 0)
//   out = softmax over the seen t of x, times V
//
// The logits are kept in the log2 domain (times log2 e) like all scores of this library.
#pragma once

#include "decode_split.cuh"
#include "prefill_tc.cuh"

namespace pa {

// ---- single tokens ----------------------------------------------------------------------------
// Bound by the bytes of K and V inside the window; 4 logits a lane and 16 tokens leave room for tanh through
// one exponential and one division: tanh(y) = 1 - 2 / (e^2y + 1), an absolute error of about 2^-23.
struct ScoreModExt {
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
            if (cap_out > 0.f) x = cap_out * (1.f - __fdividef(2.f, exp2f(dot * cap_in) + 1.f));
            return fmaf(slope[j], (float)(t - last), x);
        }
        __device__ __forceinline__ void keep(const float (&)[4], int, bool, bool) const {}
    };
};

// ---- chunks -----------------------------------------------------------------------------------------
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The softmax warps bound the prefill kernel, and their registers are full: what is done to a score there
// counts, and so does every branch around it.  Hence four kernels, by whether scores are capped and biased:
//   window, prefix     only the tiles at the borders are masked; scores stay as they are.
//   BIAS               one multiply-add to the raw score, slope / scale times the place in the tile; what the
//                      whole tile has in common goes into the softmax's reference.  Only tiles with tokens on
//                      both sides of a row need more.
//   CAP                tanh(y) = y q(y^2) while a warp's tile has |x| <= 0.3 cap, q of degree 2 interpolating
//                      tanh(y) / y at the Chebyshev nodes of [0, 0.09] in y^2 (absolute error below 4e-7), with
//                      cap and scale inside the coefficients, on the FMA pipe; else the exact form, an
//                      exponential and a reciprocal more for each score on the MUFU unit.
#define PA_TANH_RANGE 0.3f
#define PA_TANH_C0 0.99999883513f
#define PA_TANH_C1 -0.33309988804f
#define PA_TANH_C2 0.12633582392f

template <bool CAP, bool BIAS>
struct PrefillScoreMod {
    static constexpr bool kOn = true;
    const float *slopes;           // [h_q]
    const int32_t *prefix_lens;    // [B] or null
    int window;                    // 0: no window
    float cap_in, cap_out;         // as in ScoreModExt
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
#pragma unroll
            for (int i = 0; i < 64; ++i) at(i) = __float_as_uint(fmaf(slope, (float)i, __uint_as_float(at(i))));
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
