// block_scales.cuh -- an 8-bit cache with one scale for each (physical block, KV head), for K and for V:
// the write that keeps the scales, and what the decode of decode_split.cuh needs to know.
//
// The scale of a block is the smallest bf16 number s with QMAX s >= max|x| over the block's rows (QMAX = 448
// for E4M3, 127 for INT8), but at least 2^-80 unless all of them are 0, kept in fp32.  A code is x / s to nearest,
// ties to even.  With 8 significant bits in x and in s, and at most 7 in a code, x / s and code * s_old / s_new
// round in fp32 exactly as in any wider type (a quotient of such numbers that is not a tie is further from one than
// 2^-17 of it): codes are what the definition says, bit for bit.  Against max|x| / QMAX itself the scale is at
// most 2^-7 larger.
//
// Bound by: latency for a decode step's rows; the rows' bytes in and codes out for prompts.
#pragma once

#include "decode_split.cuh"

namespace pa {

struct BlockScaleWriteParams {
    const __nv_bfloat16 *key;
    const __nv_bfloat16 *value;
    int64_t key_stride;            // elements between consecutive tokens
    int64_t value_stride;
    uint8_t *k_cache;
    uint8_t *v_cache;
    float *k_scales;               // [num_blocks][h_kv]
    float *v_scales;
    const int64_t *slot_mapping;
    int num_tokens;
    int h_kv;
    long long num_slots;
    int chunk;                     // tokens whose runs one CTA looks after, a power of two
};

template <int QT>
__device__ __forceinline__ constexpr float code_max() { return QT == 1 ? 448.f : 127.f; }

// The smallest bf16 value that is not below amax / QMAX (fp32 division: exact enough, see above).  Its floor keeps
// what the decode adds up, 2^15 / scale for each token, inside fp32.
template <int QT>
__device__ __forceinline__ float block_scale_of(float amax)
{
    const float s = __uint_as_float((__float_as_uint(__fdiv_rn(amax, code_max<QT>())) + 0xffffu) & 0xffff0000u);
    return s > 0.f ? fmaxf(s, kMinBlockScale) : 0.f;
}

template <int QT>
__device__ __forceinline__ uint32_t pack_codes(float x0, float x1, float x2, float x3)
{
    if constexpr (QT == 1) {
        return (uint32_t)float2_to_e4m3x2(x0, x1) | ((uint32_t)float2_to_e4m3x2(x2, x3) << 16);
    } else {
        return ((uint32_t)float_to_s8_sym(x0) & 0xffu) | (((uint32_t)float_to_s8_sym(x1) & 0xffu) << 8) |
               (((uint32_t)float_to_s8_sym(x2) & 0xffu) << 16) | ((uint32_t)float_to_s8_sym(x3) << 24);
    }
}

// Codes of four values at scale s.
template <int QT>
__device__ __forceinline__ uint32_t encode4(float x0, float x1, float x2, float x3, float s)
{
    if (s == 0.f) return 0u;
    return pack_codes<QT>(__fdiv_rn(x0, s), __fdiv_rn(x1, s), __fdiv_rn(x2, s), __fdiv_rn(x3, s));
}

// The same for finite values and a scale in [2^-100, 2^100], r = 1 / s rounded: the quotient by a product and
// one residual step (as in Markstein's division), q1 = q0 + (x - q0 s) r.  The residual is exact, so q1 is
// within a step of the quotient, and is the quotient where that is an fp32 number.  Ties between two codes are
// fp32 numbers, and every other quotient of 8-bit significands is further than that from a tie: the codes
// are those of the division, at 3 packed instructions for two values instead of about 24.  INT8: |q| <= 127 by the
// choice of the scale, and adding 1.5 * 2^23 rounds it to nearest, ties to even, into the low byte.
template <int QT>
__device__ __forceinline__ uint32_t encode4_fast(float x0, float x1, float x2, float x3, float s, float r)
{
    const float2 r2 = make_float2(r, r), s2 = make_float2(-s, -s);
    auto divide = [&](float2 x) {
        const float2 q = __fmul2_rn(x, r2);
        return __ffma2_rn(__ffma2_rn(q, s2, x), r2, q);
    };
    float2 a = divide(make_float2(x0, x1)), b = divide(make_float2(x2, x3));
    if constexpr (QT == 1) {
        return pack_codes<1>(a.x, a.y, b.x, b.y);
    } else {
        const float2 R = make_float2(12582912.f, 12582912.f);      // 1.5 * 2^23
        a = __fadd2_rn(a, R);
        b = __fadd2_rn(b, R);
        return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                           __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
    }
}

// Four codes brought from scale `was` to `now`: rne(code * was / now).
template <int QT>
__device__ __forceinline__ uint32_t requantise4(uint32_t w, float was, float now)
{
    float2 a, b;
    if constexpr (QT == 1) {
        a = e4m3x2_to_float2(w & 0xffffu);
        b = e4m3x2_to_float2(w >> 16);
    } else {
        a = make_float2((float)(int8_t)(w & 0xffu), (float)(int8_t)((w >> 8) & 0xffu));
        b = make_float2((float)(int8_t)((w >> 16) & 0xffu), (float)(int8_t)(w >> 24));
    }
    return encode4<QT>(a.x * was, a.y * was, b.x * was, b.y * was, now);
}

constexpr int kScaleWriteWarps = 4;
constexpr int kScaleWriteMaxChunk = 64;

// All warps of a team of TW (barriers by constant numbers: by a variable one, a CTA would hold all 16).
template <int TW>
__device__ __forceinline__ void team_sync(int team)
{
    static_assert(kScaleWriteWarps / TW <= 2, "one barrier a team");
    if (kScaleWriteWarps == TW || team == 0) asm volatile("bar.sync 1, %0;" ::"n"(TW * 32) : "memory");
    else asm volatile("bar.sync 2, %0;" ::"n"(TW * 32) : "memory");
}

// A run is a maximal stretch of tokens next to each other whose slots lie in one block.  A CTA looks after
// the runs that begin in its `chunk` tokens, for one KV head.  First it finds for each run which token owns
// which row of the block (the later one, if two have the same slot); then teams of warps take one (run, K or V)
// at a time: the rows into registers, maximum over them, the scale, older rows requantised if it
// grew, the rows' codes.  A team is one warp where none of the CTA's runs has more rows than its 8 loads bring, else as
// many warps as bring a whole block: 4096 one-token runs of 8 heads of 128 into blocks of 64 take 44 us by single
// warps and 138 to 218 by whole-block teams, and prompts of 32768 tokens 58 and 44.
//   37k tokens of 8 heads of 128 into INT8 blocks of 64, 229 MB: 131 us with a warp an item, rows read twice and IEEE
// divisions; 77 us with teams and the residual step; 57 us with 8 CTAs of 4 warps an SM, one head each (66 at 4
// CTAs of 8 warps and 4 heads); 54.6 us with two values an instruction; 50.7 us with rows that always stay in
// registers, against 35 us for the bytes.  Issue slots (61 %) and the latency of the lookups weigh most.  32 tokens of
// 32 heads: 4.1 us.
template <int D, int BS, int QT>
__global__ void __launch_bounds__(kScaleWriteWarps * 32, 8) write_block_scales_kernel(const BlockScaleWriteParams p)
{
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int LPR = D / 8, RPI = 32 / LPR;         // lanes per bf16 row, rows of one load
    constexpr int KEEP = 8;                            // loads kept in registers
    constexpr int WHOLE = cmax(1, BS / (KEEP * RPI));  // warps whose loads are a whole block
    static_assert(WHOLE * KEEP * RPI >= BS && kScaleWriteWarps % WHOLE == 0, "teams");
    constexpr int WINDOW = kScaleWriteMaxChunk + BS;   // tokens whose borders are looked at
    constexpr int WORDS = (WINDOW + 31) / 32;
    __shared__ uint32_t border[WORDS + 1];             // bit i: token t0 + i does not continue the run of t0 + i - 1
    __shared__ int run_first[kScaleWriteMaxChunk], run_lo[kScaleWriteMaxChunk], run_hi[kScaleWriteMaxChunk];
    __shared__ bool run_plain[kScaleWriteMaxChunk];    // row lo + i belongs to the run's token i
    __shared__ int num_runs, any_long;                 // any_long: a run has more rows than one warp's loads
    __shared__ int owner_of[kScaleWriteMaxChunk][BS];
    __shared__ uint32_t team_max[2][kScaleWriteWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long t0 = (long long)blockIdx.x * p.chunk;

    auto block_of = [&](long long t) -> long long {    // -1: not a token that is written
        if (t < 0 || t >= p.num_tokens) return -1;
        const long long slot = __ldg(reinterpret_cast<const long long *>(p.slot_mapping) + t);
        return slot >= 0 && slot < p.num_slots ? slot / BS : -1;
    };
    if (threadIdx.x == 0) num_runs = any_long = 0;
    __syncthreads();
    const int window = p.chunk + BS;
    for (int i = threadIdx.x; i < (window + 31) / 32 * 32; i += blockDim.x) {
        const long long mine = block_of(t0 + i), before = block_of(t0 + i - 1);
        const bool starts = mine != before;
        const uint32_t bits = __ballot_sync(FULL, starts);
        if (lane == 0) border[i >> 5] = bits;
        if (i < p.chunk && starts && mine >= 0) run_first[atomicAdd(&num_runs, 1)] = i;
        if (i < p.chunk && blockIdx.y == 0 && t0 + i < p.num_tokens && p.slot_mapping[t0 + i] >= p.num_slots)
            record_error(PA_DEVERR_BAD_SLOT);
    }
    __syncthreads();
    for (int run = warp; run < num_runs; run += kScaleWriteWarps) {
        const int first = run_first[run];
        const long long blk = block_of(t0 + first);
        // the run's end: the next border, or (slots given twice) further on
        int end = first + 1;
        for (;;) {
            const uint32_t w = border[end >> 5] >> (end & 31);
            if (w) {
                end += __ffs(w) - 1;
                break;
            }
            end = (end | 31) + 1;
            if (end >= window) break;
        }
        if (end >= window) {
            end = window;
            while (block_of(t0 + end) == blk) ++end;
        }
        int *owner = owner_of[run];
        for (int i = lane; i < BS; i += 32) owner[i] = -1;
        __syncwarp();
        int lo = BS, hi = -1;
        for (int i = first + lane; i < end; i += 32) {
            const int off = (int)(p.slot_mapping[t0 + i] - blk * BS);
            atomicMax(&owner[off], (int)(t0 + i));
            lo = min(lo, off);
            hi = max(hi, off);
        }
        lo = __reduce_min_sync(FULL, lo);
        hi = __reduce_max_sync(FULL, hi);
        bool plain = end - first == hi - lo + 1;
        for (int i = first + lane; i < end && plain; i += 32) plain = (int)(p.slot_mapping[t0 + i] - blk * BS) - lo == i - first;
        plain = __all_sync(FULL, plain);
        if (lane == 0) {
            run_lo[run] = lo;
            run_hi[run] = hi;
            run_plain[run] = plain;
            if (hi - lo >= KEEP * RPI) any_long = 1;
        }
    }
    __syncthreads();

    // a run's rows are in its team's registers, all at once: of one warp, or of as many as hold a whole block
    auto work = [&](auto team_warps) {
        constexpr int TW = decltype(team_warps)::value;
        const int team = warp / TW, member = warp % TW;
        const int sub = lane / LPR, col = lane % LPR;
        const int items = num_runs * 2;
        int parity = 0;
        for (int item = team; item < items; item += kScaleWriteWarps / TW, parity ^= 1) {
            const bool is_v = item & 1;
            const int run = item >> 1;
            int h = blockIdx.y;
            asm volatile("" : "+r"(h));                // what follows from it is not kept over the loop: it would spill
            const int lo = run_lo[run], hi = run_hi[run];
            const int *owner = owner_of[run];
            const long long blk = block_of(t0 + run_first[run]);
            const __nv_bfloat16 *rows = (is_v ? p.value : p.key) + (size_t)h * D;
            const int64_t stride = is_v ? p.value_stride : p.key_stride;
            uint8_t *tile = (is_v ? p.v_cache : p.k_cache) + ((size_t)blk * p.h_kv + h) * BS * D;
            float *scale = (is_v ? p.v_scales : p.k_scales) + (size_t)blk * p.h_kv + h;
            const float was = lo > 0 ? *scale : 0.f;       // a block written from its first row on has no older rows
            uint4 v[KEEP];
            const int row0 = lo + member * KEEP * RPI + sub;           // of v[0]; v[k] is row0 + k * RPI
            const bool plain = run_plain[run];
            if (plain) {
                const uint4 *from = reinterpret_cast<const uint4 *>(rows + (t0 + run_first[run] + row0 - lo) * stride) + col;
#pragma unroll
                for (int k = 0; k < KEEP; ++k, from += RPI * (stride / 8))
                    v[k] = row0 + k * RPI <= hi ? __ldg(from) : make_uint4(0, 0, 0, 0);
            } else {
#pragma unroll
                for (int k = 0; k < KEEP; ++k) {
                    const int row = row0 + k * RPI, t = row <= hi ? owner[row] : -1;
                    v[k] = t >= 0 ? __ldg(reinterpret_cast<const uint4 *>(rows + t * stride) + col) : make_uint4(0, 0, 0, 0);
                }
            }
            // maximum of |x|, two at a time; NaN stays in it
            auto max2 = [](uint32_t a, uint32_t b) {
                const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
                return *reinterpret_cast<const uint32_t *>(&m);
            };
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < KEEP; ++k) {
                top = max2(top, max2(v[k].x & 0x7fff7fffu, v[k].y & 0x7fff7fffu));
                top = max2(top, max2(v[k].z & 0x7fff7fffu, v[k].w & 0x7fff7fffu));
            }
            auto over_team = [&](uint32_t m, int slot) {   // the maximum over the team's threads
                m = __reduce_max_sync(FULL, m);
                if constexpr (TW > 1) {
                    if (lane == 0) team_max[slot][warp] = m;
                    team_sync<TW>(team);
#pragma unroll
                    for (int i = 0; i < TW; ++i) m = max(m, team_max[slot][team * TW + i]);
                }
                return m;
            };
            top = over_team(max(top & 0xffffu, top >> 16), parity);
            const bool finite = top < 0x7f80u;
            if (!finite) {                                 // infinities and NaN take no part: once more without them
                if constexpr (TW > 1) team_sync<TW>(team);
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < KEEP; ++k) {
                    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t a = (w[e >> 1] >> (16 * (e & 1))) & 0x7fffu;
                        m = a < 0x7f80u ? max(m, a) : m;
                    }
                }
                top = over_team(m, parity);
            }
            const float now = fmaxf(was, block_scale_of<QT>(__uint_as_float(top << 16)));
            __syncwarp();                                  // (the team's barrier) every lane has read the old scale
            if (lo > 0 && now > was) {
                // the scale grew: the rows before the first new one move to it (16 codes at a time)
                for (int i = member * 32 + lane; i < lo * (D / 16); i += TW * 32) {
                    uint4 c = reinterpret_cast<uint4 *>(tile)[i];
                    c.x = requantise4<QT>(c.x, was, now);
                    c.y = requantise4<QT>(c.y, was, now);
                    c.z = requantise4<QT>(c.z, was, now);
                    c.w = requantise4<QT>(c.w, was, now);
                    reinterpret_cast<uint4 *>(tile)[i] = c;
                }
            }
            if (member == 0 && lane == 0) *scale = now;
            const bool fast = finite && now >= 0x1p-100f && now <= 0x1p100f;
            const float r = __frcp_rn(now);
            uint8_t *to = tile + (size_t)row0 * D + 8 * col;
            auto store = [&](auto encode) {
#pragma unroll
                for (int k = 0; k < KEEP; ++k) {
                    const int row = row0 + k * RPI;
                    if (row <= hi && (plain || owner[row] >= 0)) {
                        const float2 a = bf16x2_to_float2(v[k].x), b = bf16x2_to_float2(v[k].y);
                        const float2 c = bf16x2_to_float2(v[k].z), d = bf16x2_to_float2(v[k].w);
                        *reinterpret_cast<uint2 *>(to + k * RPI * D) =
                            make_uint2(encode(a.x, a.y, b.x, b.y), encode(c.x, c.y, d.x, d.y));
                    }
                }
            };
            if (fast) store([&](float x, float y, float z, float w) { return encode4_fast<QT>(x, y, z, w, now, r); });
            else store([&](float x, float y, float z, float w) { return encode4<QT>(x, y, z, w, now); });
        }
    };
    if constexpr (WHOLE > 1) {
        if (any_long) return work(std::integral_constant<int, WHOLE>{});
    }
    work(std::integral_constant<int, 1>{});
}

// scales[dst][:] = scales[src][:] for every (src, dst) pair, layer, and K/V.
constexpr int kScaleCopyMaxLayers = 128;     // of one launch

struct CopyScalesParams {
    float *k[kScaleCopyMaxLayers];
    float *v[kScaleCopyMaxLayers];
    const int64_t *pairs;
    int h_kv;
    int num_blocks;
};

// grid (num_pairs, layers, 2)
__global__ void __launch_bounds__(32) copy_scales_kernel(const CopyScalesParams p)
{
    const long long src = p.pairs[2 * blockIdx.x], dst = p.pairs[2 * blockIdx.x + 1];
    if (src < 0 || dst < 0 || src >= p.num_blocks || dst >= p.num_blocks) {
        if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) record_error(PA_DEVERR_BAD_PAIR);
        return;
    }
    float *s = blockIdx.z ? p.v[blockIdx.y] : p.k[blockIdx.y];
    for (int h = threadIdx.x; h < p.h_kv; h += 32) s[dst * p.h_kv + h] = s[src * p.h_kv + h];
}

// The decode: scales per block, no change of the logits.
struct BlockScalesExt {
    static constexpr bool kDependent = false;
    struct Args {
        const float *k_scales;     // [num_blocks][h_kv]
        const float *v_scales;
    };
    template <int G>
    struct Row {
        __device__ __forceinline__ Row(const Args &, const SplitParams &, int, int, int, int) {}
    };
};

}  // namespace pa
