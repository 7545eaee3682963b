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

// The softmax warps of the prefill kernel are what bounds it, and their exponentials (one per score) the
// MUFU unit.  tanh through an exponential and a reciprocal would make that three.  Scores are mostly far
// below the cap, so where a warp's tile has |x| <= 0.6 cap throughout, tanh(y) = y q(y^2) with q of degree 4
// that interpolates tanh(y) / y at the five Chebyshev nodes of [0, 0.36] in y^2 (absolute error below 4e-8),
// on the FMA pipe, two scores an instruction, cap and scale inside the coefficients; else the exact form.
#define PA_TANH_RANGE 0.6f
#define PA_TANH_C0 0.99999992596f
#define PA_TANH_C1 -0.33332302040f
#define PA_TANH_C2 0.13310064426f
#define PA_TANH_C3 -0.05209665341f
#define PA_TANH_C4 0.01546875130f

struct PrefillScoreMod {
    static constexpr bool kOn = true;
    const float *slopes;           // [h_q] or null
    const int32_t *prefix_lens;    // [B] or null
    int window;                    // 0: no window
    float cap_in, cap_out;         // as in ScoreModExt
    float range;                   // |raw score| up to which the polynomial holds
    float c[5];                    // its coefficients, for raw scores and log2-domain logits

    __device__ __forceinline__ int prefix(int seq) const { return prefix_lens ? __ldg(prefix_lens + seq) : 0; }
    __device__ __forceinline__ int first_token(int pos) const { return window > 0 ? max(0, pos - window + 1) : 0; }
    __device__ __forceinline__ float slope(int head) const
    {
        return slopes ? __ldg(slopes + head) * 1.4426950408889634f : 0.f;
    }

    // Raw scores of tokens first + pos, first + pos + 1, ... of one row into log2-domain logits.
    // both_sides: some of the tokens may lie behind the row's position.
    __device__ __forceinline__ void logits(uint32_t (&sr)[2][32], float qk_scale, float slope2, int first, bool both_sides) const
    {
        auto at = [&](int i) -> uint32_t & { return sr[i >> 5][i & 31]; };
        if (cap_out > 0.f) {
            float m4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 64; i += 2)
                m4[(i >> 1) & 3] = max3f(m4[(i >> 1) & 3], fabsf(__uint_as_float(at(i))), fabsf(__uint_as_float(at(i + 1))));
            const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            if (!__any_sync(0xffffffffu, top > range)) {
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const float2 x = make_float2(__uint_as_float(at(i)), __uint_as_float(at(i + 1)));
                    const float2 u = __fmul2_rn(x, x);
                    float2 q = __ffma2_rn(u, make_float2(c[4], c[4]), make_float2(c[3], c[3]));
                    q = __ffma2_rn(u, q, make_float2(c[2], c[2]));
                    q = __ffma2_rn(u, q, make_float2(c[1], c[1]));
                    q = __ffma2_rn(u, q, make_float2(c[0], c[0]));
                    q = __fmul2_rn(x, q);
                    at(i) = __float_as_uint(q.x);
                    at(i + 1) = __float_as_uint(q.y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const float e = ex2_approx(__uint_as_float(at(i)) * cap_in);
                    at(i) = __float_as_uint(cap_out * fmaf(-2.f, rcp_approx(e + 1.f), 1.f));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
                const float2 x = __fmul2_rn(make_float2(__uint_as_float(at(i)), __uint_as_float(at(i + 1))),
                                            make_float2(qk_scale, qk_scale));
                at(i) = __float_as_uint(x.x);
                at(i + 1) = __float_as_uint(x.y);
            }
        }
        if (slopes != nullptr) {
            const float d0 = (float)first;
            if (both_sides) {
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    at(i) = __float_as_uint(fmaf(-slope2, fabsf(d0 + (float)i), __uint_as_float(at(i))));
            } else {
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const float2 d = __fadd2_rn(make_float2(d0, d0), make_float2((float)i, (float)(i + 1)));
                    const float2 x = __ffma2_rn(make_float2(slope2, slope2), d,
                                                make_float2(__uint_as_float(at(i)), __uint_as_float(at(i + 1))));
                    at(i) = __float_as_uint(x.x);
                    at(i + 1) = __float_as_uint(x.y);
                }
            }
        }
    }
};

}  // namespace pa
