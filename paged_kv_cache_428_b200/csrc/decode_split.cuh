// decode_split.cuh -- single-token attention over the paged cache for the calls that need more than
// pa_decode: modified scores, a scale per block of an 8-bit cache, or the weights themselves.
//
//   out[s][h] = sum_t p_t V_t / sum_t p_t,   p_t = 2^(x_t - m),   t in [first_s, ctx_s)
// with x_t the logit in the log2 domain, m its running maximum, both sums in fp32.  What x_t is, and
// what else becomes of it, is the `Ext` of the call (see the files that include this one).
//
// Schedule.  The step's work is the list of all (sequence, KV head, block) triples in that order.  With
// C CTAs (as many as the GPU holds at once, fewer for small steps) CTA c takes the triples
// [c u, (c + 1) u), u = ceil(T / C): every CTA moves the same number of blocks, so they end together
// whatever the lengths are.  u is at least kSplitMinTokens tokens (a shorter range costs more in merging
// than it saves) and at least 1/62 of the longest sequence, so that at most kSplitMaxPieces CTAs share one
// (sequence, KV head) group.  Where the CTAs suffice for it, no range crosses the border of a group: each
// group is cut into ceil(blocks / u) even pieces, and no CTA ends two groups; with no sequence longer than
// kSplitWholeTokens each group is one piece, as its merge would take longer than its blocks.  Whole and in pieces of
// 128: 8 groups of 256 tokens of 128 dims in bf16 7.5 and 8.1 us, of 384 9.5 and 8.4, of 512 11.6 and 8.6; 256 such
// groups 11.3 and 15.4, 14.1 and 18.8, 16.5 and 20.2; 8 groups of codes of 64 dims 7.1 and 8.3, 8.2 and 8.6, 9.6 and
// 8.6; 32 groups of 1001 tokens in bf16 14.6 and 10.6.  The border stands between few groups and many.  The
// lengths are read on the device; the host's bound on them only sizes the grid.
//   A producer warp streams the blocks' K and V tiles by 2-D TMA through an mbarrier ring, without a
// pause between groups: lane j looks up triple j of the next 32 (and its scales) while the present 32
// are issued.  Consumer warps take blocks in turn (mma.sync m16n8k16, tokens or head dims on
// the 16 rows, the group's query heads on the 8 columns, as in decode_mma.cuh and decode_q8.cuh) and put
// their states together where a group or the CTA's range ends.  A group that lies in one range is
// finished there.  Otherwise each CTA leaves (m, l, o) in one of its two slots (0: the group its range
// begins in, 1: the one it ends in) and counts; the CTA that completes the count merges.  No CTA waits
// for another, and the merge adds in the order of the CTAs: results do not depend on timing.
//
// Bound by the bytes of K and V: 64 sequences of 512..4096 tokens (613 MB) 100 to 104 us, 32 x 4096 tokens of 32 heads
// in E4M3 (1076 MB) 167 to 188 us, 91 to 94 and 88 to 98 % of the copy rate.  Single short sequences are bound by
// latency: 5.8 us for 2 x 37..81 tokens, of which three dependent loads (length, table, tiles) are about 2.
//
// Masked places.  Scores of tokens outside [first, ctx) become -inf by select, V rows there are
// zeroed (in shared memory for bf16, in registers for codes): what they hold does not matter.
#pragma once

#include "decode_mma.cuh"
#include "decode_q8.cuh"

namespace pa {

constexpr int kSplitMaxSeqs = 4096;       // sequences of one launch (block prefix sums in shared memory)
constexpr int kSplitMaxCtas = 1024;       // partial slots in the workspace: two for each of this many CTAs
constexpr int kSplitMaxPieces = 64;       // CTAs that share one group
constexpr int kSplitMinTokens = 128;      // tokens of the shortest range of one CTA
constexpr int kSplitWholeTokens = 512;    // sequences up to this stay whole where there are CTAs enough
constexpr float kMinBlockScale = 0x1p-80f;    // of a block of codes, unless it is 0
constexpr int kSplitMaxGroups = 65536;    // (sequence, KV head) groups of one call: counters at the workspace's front

struct SplitParams {
    __nv_bfloat16 *out;            // [B][h_q][D]
    const __nv_bfloat16 *q;        // [B][h_q][D]
    const int32_t *block_tables;   // [B][max_blocks_per_seq]
    const int32_t *context_lens;   // [B]
    int *counters;                 // [B][h_kv] CTAs that have left their part; zero between launches
    float *part_ml;                // [num_ctas][2][G][2]  (m, l), log2 domain
    float *part_o;                 // [num_ctas][2][G][D]  unnormalised
    float *lse;                    // [B][h_q] log2 of the softmax denominator, or null
    int max_blocks_per_seq;
    int num_seqs;
    int h_q;
    int h_kv;
    int num_blocks;
    int window;                    // tokens attended, counted back from the last one; 0 = all
    float qk_scale;                // scale * log2(e)
};

// log2 of a sum that is at least 0 (0 gives -inf).
__device__ __forceinline__ float log2_sum(float m, float l) { return m + log2f(l); }

// What a stage of the ring holds besides the tiles: written by the producer before the stage is armed.
struct SplitStage {
    int bad;                       // the table entry was outside the pool
    float k_scale, v_log2, v_inv;  // QT != 0: the block's K scale, log2 and inverse of its V scale
};

template <int D, int BS, int G, int QT>
struct SplitConfig {
    // Consumer warps, ring, CTAs of an SM.  One producer warp feeds its consumers only so fast (with a lane a
    // block and one block at a time, E4M3 at 32 x 4096 tokens x 32 heads: 198 us at 5 x 2 consumers, 213 at 4 x 3, 328
    // at 2 x 7; with half the ring at a time 199, 187 and 189 at 5 x 2, 4 x 3 and 3 x 4).  bf16, 64 sequences: 102.9
    // to 107.2 us over the same range, 103.2 at 3 x 4, where single groups are also done soonest.
    static constexpr int kWarps = QT != 0 ? 3 : BS * D >= 64 * 128 ? 2 : 4;
    static constexpr int kRing = QT != 0 ? 49152 : 65536, kPerSm = QT != 0 ? 4 : 3;
    using Tile = std::conditional_t<QT == 0, MmaDecodeConfig<D, BS, G, kWarps, kRing>, MmaQ8Config<D, BS, G, kWarps, kRing>>;
    static constexpr int NW = Tile::NW;
    static constexpr int THREADS = Tile::THREADS;
    static constexpr int STAGES = Tile::STAGES;
    // blocks that the producer issues together, a lane each: half the ring (a power of two)
    static constexpr int kIssue =
        STAGES >= 64 ? 32 : STAGES >= 32 ? 16 : STAGES >= 16 ? 8 : STAGES >= 8 ? 4 : STAGES >= 4 ? 2 : 1;
    static constexpr int OFF_BARS = Tile::RING;
    static constexpr int OFF_STAGE = OFF_BARS + 2 * STAGES * 8;
    static constexpr int OFF_FLAGS = OFF_STAGE + STAGES * (int)sizeof(SplitStage);   // abort, last, longest, bad[NW]
    static constexpr int OFF_COMBINE = OFF_FLAGS + 48;
    static constexpr int OFF_MERGE = OFF_COMBINE + NW * G * (D + 2) * 4;             // [G][kSplitMaxPieces]
    static constexpr int OFF_PREFIX = OFF_MERGE + G * kSplitMaxPieces * 4;
    static constexpr int smem_bytes(int num_seqs) { return OFF_PREFIX + 2 * (num_seqs + 1) * 4 + 1024; }
    static_assert(Tile::RING % 16 == 0 && OFF_STAGE % 16 == 0 && OFF_COMBINE % 16 == 0, "alignment");
    static_assert(3 + NW <= 12, "flags");
    static_assert(kSplitMaxPieces == 64, "two pieces a lane");
};

template <int NW>
__device__ __forceinline__ void consumers_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory");
}

// What a consumer warp keeps of a group: running maximum and sum for heads 2 (lane % 4) and + 1, and
// the unnormalised output in the accumulator layout of the tile's consume function.
template <int MT>
struct SplitState {
    float m[2], l[2], o[MT][4];
    __device__ __forceinline__ void clear()
    {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    }
    // Scores x of tokens r and r + 8 (x[0], x[1] and x[2], x[3]; -inf where masked) into
    // probabilities p against m, which is the running maximum less UP: the largest p is 2^UP.  Rescales
    // o when a maximum moved.  `inv` multiplies what goes into the sum (1, or the inverse V scale of codes
    // whose scale is inside x).
    template <int UP>
    __device__ __forceinline__ void softmax(const float (&x)[4], float inv, float (&p)[4])
    {
        constexpr unsigned FULL = 0xffffffffu;
        float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(FULL, mx0, off));
            mx1 = fmaxf(mx1, __shfl_xor_sync(FULL, mx1, off));
        }
        const float mn0 = fmaxf(m[0], mx0 - UP), mn1 = fmaxf(m[1], mx1 - UP);
        const float al0 = exp2f(m[0] - mn0), al1 = exp2f(m[1] - mn1);
        m[0] = mn0;
        m[1] = mn1;
        p[0] = exp2f(x[0] - mn0);
        p[1] = exp2f(x[1] - mn1);
        p[2] = exp2f(x[2] - mn0);
        p[3] = exp2f(x[3] - mn1);
        l[0] = fmaf(p[0] + p[2], inv, l[0] * al0);
        l[1] = fmaf(p[1] + p[3], inv, l[1] * al1);
        if (__any_sync(FULL, (al0 != 1.f) | (al1 != 1.f))) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                o[mt][0] *= al0;
                o[mt][1] *= al1;
                o[mt][2] *= al0;
                o[mt][3] *= al1;
            }
        }
    }
};

// One block of bf16 rows (K tile at `ktile`, V tile behind it) into the state: rows [lo, hi) of it.
// `row.logit(dot, t, j)` gives the log2-domain logit of token t for the lane's head j, and
// `row.keep(x, t, use0, use1)` sees the four logits of tokens t and t + 8.  P is rounded to bf16 for the
// product with the bf16 V (relative error 2^-9 at most, as large as the rounding of the output).
template <class C, int BS, int G, class Row>
__device__ __forceinline__ void split_consume_bf16(uint8_t *ktile, int lo, int hi, int block_t0,
                                                   const uint32_t (&qb)[C::KS][2], const Row &row,
                                                   SplitState<C::MT> &st, int lane)
{
    uint8_t *vtile = ktile + C::TILE;
    if (lo > 0 || hi < BS) {
        const int masked = lo + BS - hi, n16 = masked * 8 * C::HALVES;
        for (int e = lane; e < n16; e += 32) {
            const int hf = e / (masked * 8), i = (e / 8) % masked;
            const int r = i < lo ? i : hi + (i - lo);
            reinterpret_cast<uint4 *>(vtile + hf * C::HALF_BYTES + r * 128)[e % 8] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
    }
    const uint32_t kbase = smem_addr(ktile), vbase = smem_addr(vtile);
    const int mrow = lane & 7, mat = lane >> 3, r = lane >> 2;
#pragma unroll 1
    for (int sub = 0; sub < C::NSUB; ++sub) {
        if (sub * 16 >= hi) break;
        if (sub * 16 + 16 <= lo) continue;
        float s[4] = {0.f, 0.f, 0.f, 0.f}, odd[4] = {0.f, 0.f, 0.f, 0.f};      // two chains of half the length
        {
            const int tok = sub * 16 + (mat & 1) * 8 + mrow;
#pragma unroll
            for (int ks = 0; ks < C::KS; ++ks) {
                uint32_t a[4];
                ldmatrix_x4(a, kbase + (ks >> 2) * C::HALF_BYTES + swz128(tok, 2 * (ks & 3) + (mat >> 1)));
                mma_bf16_16816(ks & 1 ? odd : s, a[0], a[1], a[2], a[3], qb[ks][0], qb[ks][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += odd[i];
        const int t0 = sub * 16 + r;
        const bool use0 = t0 >= lo && t0 < hi, use1 = t0 + 8 >= lo && t0 + 8 < hi;
        float x[4], p[4];
        x[0] = use0 ? row.logit(s[0], block_t0 + t0, 0) : -INFINITY;
        x[1] = use0 ? row.logit(s[1], block_t0 + t0, 1) : -INFINITY;
        x[2] = use1 ? row.logit(s[2], block_t0 + t0 + 8, 0) : -INFINITY;
        x[3] = use1 ? row.logit(s[3], block_t0 + t0 + 8, 1) : -INFINITY;
        row.keep(x, block_t0 + t0, use0, use1);
        st.template softmax<0>(x, 1.f, p);
        const uint32_t pb0 = movmatrix_trans(pack_bf16x2(p[0], p[1]));
        const uint32_t pb1 = movmatrix_trans(pack_bf16x2(p[2], p[3]));
        const int tok = sub * 16 + (mat >> 1) * 8 + mrow;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
            uint32_t a[4];
            ldmatrix_x4_trans(a, vbase + (mt >> 2) * C::HALF_BYTES + swz128(tok, ((2 * mt) & 7) + (mat & 1)));
            mma_bf16_16816(st.o[mt], a[0], a[1], a[2], a[3], pb0, pb1);
        }
    }
}

// Q^T fragments in fp16, in the order of q8_load_q: the group's q is brought by a power of two to a largest
// magnitude in [2^13, 2^14), so that neither large nor small queries leave fp16's normal range; returns what
// the logits have to be multiplied by for it.  (q8_load_q only brings large ones down: queries near 2^-14 beside
// large keys would lose digits there.)
template <class C, int G, int D>
__device__ __forceinline__ float split_load_q8(uint32_t (&qb)[C::KS][2], const __nv_bfloat16 *qg, int lane)
{
    const int gq = lane >> 2, tq = lane & 3;
    const __nv_bfloat16 *qrow = qg + (size_t)(gq < G ? gq : 0) * D;
    uint2 raw[C::KS];
    float mx = 0.f;
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
        raw[ks] = gq < G ? *reinterpret_cast<const uint2 *>(qrow + 16 * ks + 4 * tq) : make_uint2(0u, 0u);
        const float2 a = bf16x2_to_float2(raw[ks].x), b = bf16x2_to_float2(raw[ks].y);
        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))));
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    // the exponent of mx less 13, kept where both powers of two are normal numbers
    const int e = max(-100, min(114, (int)(__float_as_uint(mx) >> 23) - 127 - 13));
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
        const float2 a = bf16x2_to_float2(raw[ks].x), b = bf16x2_to_float2(raw[ks].y);
        qb[ks][0] = pack_f16x2(a.x * down, a.y * down);
        qb[ks][1] = pack_f16x2(b.x * down, b.y * down);
    }
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

// One block of codes into the state.  The block's scales enter the logit: x = dot * k_factor + log2(v),
// so that 2^(x - m) is the probability times the block's V scale v, relative to the largest such product
// seen: the products with the raw codes add up whatever the scales of different blocks are.  P goes into
// the product as fp16 (2^-11), the largest as 2^15, so that fp16's normal range reaches down to 2^-29 of
// it (a token that small still counts where the large ones have the code 0).  The sum takes 2^(x - m) / v.
template <class C, int D, int BS, int QT>
__device__ __forceinline__ void split_consume_q8(const uint8_t *ktile, int hi, const uint32_t (&qb)[C::KS][2],
                                                 const float (&kbias)[2], float k_factor, const SplitStage &sc,
                                                 SplitState<C::MT> &st, int lane)
{
    const uint32_t kbase = smem_addr(ktile), vbase = kbase + C::TILE;
    const int mrow = lane & 7, mat = lane >> 3, r = lane >> 2, tq = lane & 3;
    const float kf = k_factor * sc.k_scale, add = sc.v_log2, inv = sc.v_inv;
#pragma unroll 1
    for (int sub = 0; sub < C::NSUB; ++sub) {
        if (sub * 16 >= hi) break;
        const int tok = sub * 16 + (mat & 1) * 8 + mrow;
        float sA[4] = {0.f, 0.f, 0.f, 0.f}, sB[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < C::KS; ks += 2) {
            uint32_t w[4], a0, a1, a2, a3;
            ldmatrix_x4(w, kbase + swz_q8<D>(tok, ks + (mat >> 1)));
            q8_quad_to_f16<QT>(w[0], a0, a2);
            q8_quad_to_f16<QT>(w[1], a1, a3);
            mma_f16_16816(sA, a0, a1, a2, a3, qb[ks][0], qb[ks][1]);
            q8_quad_to_f16<QT>(w[2], a0, a2);
            q8_quad_to_f16<QT>(w[3], a1, a3);
            mma_f16_16816(sB, a0, a1, a2, a3, qb[ks + 1][0], qb[ks + 1][1]);
        }
        const int t0 = sub * 16 + r;
        float x[4], p[4];
        x[0] = t0 < hi ? fmaf(sA[0] + sB[0] - kbias[0], kf, add) : -INFINITY;
        x[1] = t0 < hi ? fmaf(sA[1] + sB[1] - kbias[1], kf, add) : -INFINITY;
        x[2] = t0 + 8 < hi ? fmaf(sA[2] + sB[2] - kbias[0], kf, add) : -INFINITY;
        x[3] = t0 + 8 < hi ? fmaf(sA[3] + sB[3] - kbias[1], kf, add) : -INFINITY;
        st.template softmax<15>(x, inv, p);
        const uint32_t pb0 = movmatrix_trans(pack_f16x2(p[0], p[1]));
        const uint32_t pb1 = movmatrix_trans(pack_f16x2(p[2], p[3]));
        if (hi < sub * 16 + 16) q8_pv<C, D, QT, true>(vbase, tok, mat, sub * 16 + 2 * tq, hi, pb0, pb1, st.o);
        else q8_pv<C, D, QT, false>(vbase, tok, mat, 0, 0, pb0, pb1, st.o);
    }
}

// Where a triple lies.
struct SplitPlace {
    int seq, kvh, block, nb;       // block: within the group's nb blocks
};

// The blocks of a sequence that its window leaves: the first one, and how many.  A context longer than
// the table row counts one block past the row, which is then reported as bad.
__host__ __device__ __forceinline__ void split_blocks(int ctx, int window, int bs, int max_blocks, int &first, int &count)
{
    first = window > 0 && ctx > window ? (ctx - window) / bs : 0;
    count = ctx > 0 ? cmin((ctx - 1) / bs + 1, cmax(max_blocks, first) + 1) - first : 0;
}

// prefix[s]: blocks (or pieces) of one KV head of the sequences before s, num_seqs + 1 entries.  x: below
// prefix[num_seqs] * h_kv.
__host__ __device__ __forceinline__ SplitPlace split_locate(const int *prefix, int num_seqs, int h_kv, long long x)
{
    int lo = 0, hi = num_seqs - 1;                     // the last sequence whose triples start at or before x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)prefix[mid] * h_kv <= x) lo = mid;
        else hi = mid - 1;
    }
    SplitPlace at;
    at.seq = lo;
    at.nb = prefix[lo + 1] - prefix[lo];
    const long long rem = x - (long long)prefix[lo] * h_kv;
    at.kvh = (int)(rem / at.nb);
    at.block = (int)(rem - (long long)at.kvh * at.nb);
    return at;
}

// Blocks of the shortest range, and of the largest piece of a whole group, when the longest sequence has
// `longest` of them.
__host__ __device__ __forceinline__ int split_shortest(int longest, int bs)
{
    return cmax(kSplitMinTokens / bs, ceil_div(longest, kSplitMaxPieces - 2));
}
__host__ __device__ __forceinline__ int split_piece(int longest, int bs)
{
    return (long long)longest * bs <= kSplitWholeTokens ? cmax(longest, 1) : split_shortest(longest, bs);
}

// The triples [x0, x1) of one CTA (none if x0 >= x1).  cuts: like prefix, in pieces of at most split_piece blocks.
struct SplitRange {
    long long x0, x1;
    long long u;                   // not aligned: triples of every CTA
    bool aligned;                  // pieces of whole groups: this CTA's group has `pieces`, from CTA `first` on
    int first, pieces;
};

__host__ __device__ __forceinline__ SplitRange split_range(const int *prefix, const int *cuts, int num_seqs, int h_kv, int bs,
                                                           int longest, int ctas, int cta)
{
    SplitRange r{0, 0, 0, (long long)cuts[num_seqs] * h_kv <= ctas, 0, 0};
    if (r.aligned) {
        if (cta < cuts[num_seqs] * h_kv) {
            const SplitPlace at = split_locate(cuts, num_seqs, h_kv, cta);          // at.nb, at.block: pieces
            const int nb = prefix[at.seq + 1] - prefix[at.seq], each = ceil_div(nb, at.nb);
            const long long group0 = (long long)prefix[at.seq] * h_kv + (long long)at.kvh * nb;
            r.first = cta - at.block;
            r.pieces = ceil_div(nb, each);
            r.x0 = group0 + cmin(nb, at.block * each);
            r.x1 = group0 + cmin(nb, (at.block + 1) * each);
        }
    } else {
        const long long total = (long long)prefix[num_seqs] * h_kv;
        r.u = (total + ctas - 1) / ctas;
        if (r.u < split_shortest(longest, bs)) r.u = split_shortest(longest, bs);
        r.x0 = cta * r.u;
        r.x1 = total < r.x0 + r.u ? total : r.x0 + r.u;
    }
    return r;
}

// The CTAs that share the group of triples [group0, group0 + nb): the first of them and how many; and which partial
// slot CTA c of them leaves its part in (of its two: 0, or 1 for a group that begins inside its range).
__host__ __device__ __forceinline__ void split_sharers(const SplitRange &r, long long group0, int nb, int &c0, int &pieces)
{
    c0 = r.aligned ? r.first : (int)(group0 / r.u);
    pieces = r.aligned ? r.pieces : (int)((group0 + nb - 1) / r.u) - c0 + 1;
}
__host__ __device__ __forceinline__ int split_slot(const SplitRange &r, long long group0, int c)
{
    return 2 * c + (!r.aligned && group0 > c * r.u ? 1 : 0);
}

// Ext: struct with `kDependent` (a programmatic dependent launch follows), `Args` (kernel argument), `Row<G>` (built
// per group; its functions for bf16 only, see split_consume_bf16) and, for codes, k_scales / v_scales
// [num_blocks][h_kv] in Args.
template <int D, int BS, int G, int QT, class Ext>
__global__ void __launch_bounds__(SplitConfig<D, BS, G, QT>::THREADS, SplitConfig<D, BS, G, QT>::kPerSm)
    paged_decode_split_kernel(const SplitParams p, const typename Ext::Args args,
                              const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v)
{
    using SC = SplitConfig<D, BS, G, QT>;
    using C = typename SC::Tile;
    constexpr int NW = SC::NW, STAGES = SC::STAGES, MT = C::MT;
    constexpr unsigned FULL = 0xffffffffu;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full_bar = reinterpret_cast<uint64_t *>(smem + SC::OFF_BARS), *empty_bar = full_bar + STAGES;
    volatile SplitStage *stage = reinterpret_cast<volatile SplitStage *>(smem + SC::OFF_STAGE);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SC::OFF_FLAGS);
    volatile int *last_flag = abort_flag + 1, *bad_flag = abort_flag + 3;       // bad_flag: one for each consumer warp
    int *longest = const_cast<int *>(abort_flag + 2);
    int *prefix = reinterpret_cast<int *>(smem + SC::OFF_PREFIX), *cuts = prefix + p.num_seqs + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // every CTA of the grid is resident at once, so a dependent grid only fills the places of CTAs that are done
    if constexpr (Ext::kDependent) pdl_launch_dependents();
    if (threadIdx.x == 32) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full_bar[i], 1);
            mbar_init(&empty_bar[i], 1);
        }
        *abort_flag = 0;
        mbar_init_fence();
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    if (warp == 0) {
        // prefix[s] = blocks of the sequences before s, and the longest one
        int carry = 0, most = 0;
        for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
            const int s = s0 + lane;
            int first = 0, n = 0;
            if (s < p.num_seqs) split_blocks(__ldg(p.context_lens + s), p.window, BS, p.max_blocks_per_seq, first, n);
            most = max(most, n);
            int sum = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(FULL, sum, off);
                if (lane >= off) sum += y;
            }
            if (s < p.num_seqs) prefix[s] = carry + sum - n;
            carry += __shfl_sync(FULL, sum, 31);
        }
        most = __reduce_max_sync(FULL, most);
        __syncwarp();
        if (lane == 0) {
            prefix[p.num_seqs] = carry;
            *longest = most;
        }
        __syncwarp();
        // cuts[s] = pieces of one KV head of the sequences before s
        const int u_cut = split_piece(most, BS);
        carry = 0;
        for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
            const int s = s0 + lane, n = s < p.num_seqs ? ceil_div(prefix[s + 1] - prefix[s], u_cut) : 0;
            int sum = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(FULL, sum, off);
                if (lane >= off) sum += y;
            }
            if (s < p.num_seqs) cuts[s] = carry + sum - n;
            carry += __shfl_sync(FULL, sum, 31);
        }
        if (lane == 0) cuts[p.num_seqs] = carry;
    }
    __syncthreads();
    // sequences without a token: zero rows
    for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x)
        if (prefix[s + 1] == prefix[s])
            for (int i = threadIdx.x; i < p.h_q * D / 8; i += SC::THREADS)
                reinterpret_cast<uint4 *>(p.out + (size_t)s * p.h_q * D)[i] = make_uint4(0, 0, 0, 0);

    const SplitRange range = split_range(prefix, cuts, p.num_seqs, p.h_kv, BS, *longest, gridDim.x, blockIdx.x);
    const long long x0 = range.x0, x1 = range.x1;
    if (x0 >= x1) return;                                      // uniform over the CTA

    if (warp == NW) {
        // ------------------------------ producer ------------------------------
        const uint64_t pol = l2_policy_evict_first();
        const int n = (int)(x1 - x0);
        // triple i of the range: its row in the tensor maps (or -1) and its scales
        auto look = [&](int i, int &row, float &ks, float &vs) {
            row = -1;
            ks = vs = 1.f;
            if (i >= n) return;
            const SplitPlace at = split_locate(prefix, p.num_seqs, p.h_kv, x0 + i);
            int first = 0, count = 0;
            split_blocks(__ldg(p.context_lens + at.seq), p.window, BS, p.max_blocks_per_seq, first, count);
            const int lb = first + at.block;
            if (lb >= p.max_blocks_per_seq) return;
            const int phys = __ldg(p.block_tables + (size_t)at.seq * p.max_blocks_per_seq + lb);
            if (phys < 0 || phys >= p.num_blocks) return;
            row = (phys * p.h_kv + at.kvh) * BS;
            if constexpr (QT != 0) {
                ks = __ldg(args.k_scales + (size_t)phys * p.h_kv + at.kvh);
                vs = __ldg(args.v_scales + (size_t)phys * p.h_kv + at.kvh);
            }
        };
        int row_n, row, issued = 0;
        float ks_n, vs_n, ks, vs;
        look(lane, row_n, ks_n, vs_n);
        bool ok = true;
        for (int i0 = 0; i0 < n && ok; i0 += 32) {
            row = row_n;
            ks = ks_n;
            vs = vs_n;
            if (i0 + 32 < n) look(i0 + 32 + lane, row_n, ks_n, vs_n);
            float v_log2 = 0.f, v_inv = 1.f;
            if constexpr (QT != 0) {
                // a block whose V codes are all 0 has scale 0; it counts as the smallest scale there is, as it must not
                // set the reference that the other blocks' probabilities are held to (see split_consume_q8)
                const float v = fmaxf(vs, kMinBlockScale);
                v_log2 = log2f(v);
                v_inv = 1.f / v;
            }
            const int cnt = min(32, n - i0);
            for (int j0 = 0; j0 < cnt && ok; j0 += SC::kIssue) {
                const bool mine = lane >= j0 && lane < min(j0 + SC::kIssue, cnt);
                const int i = i0 + lane, st = i % STAGES;
                bool free = true;
                if (mine) {
                    if (i >= STAGES) free = mbar_wait_bounded(&empty_bar[st], ((i / STAGES) - 1) & 1);
                    free = free && !*abort_flag;
                }
                ok = __all_sync(FULL, free);
                if (!ok) break;
                if (mine) {
                    stage[st].bad = row < 0;
                    if constexpr (QT != 0) {
                        stage[st].k_scale = ks;
                        stage[st].v_log2 = v_log2;
                        stage[st].v_inv = v_inv;
                    }
                    if (row >= 0) {
                        mbar_arrive_expect_tx(&full_bar[st], C::STAGE_BYTES);
                        uint8_t *dst = smem + st * C::STAGE_BYTES;
                        if constexpr (QT == 0) {
#pragma unroll
                            for (int hf = 0; hf < C::HALVES; ++hf) {
                                tma_load_2d(dst + hf * C::HALF_BYTES, &tmap_k, hf * 64, row, &full_bar[st], pol);
                                tma_load_2d(dst + C::TILE + hf * C::HALF_BYTES, &tmap_v, hf * 64, row, &full_bar[st], pol);
                            }
                        } else {
                            tma_load_2d(dst, &tmap_k, 0, row, &full_bar[st], pol);
                            tma_load_2d(dst + C::TILE, &tmap_v, 0, row, &full_bar[st], pol);
                        }
                    } else {
                        record_error(PA_DEVERR_BAD_BLOCK);
                        mbar_arrive(&full_bar[st]);
                    }
                }
                __syncwarp();
                issued = i0 + min(j0 + SC::kIssue, cnt);
            }
        }
        if (lane == 0) {
            if (!ok) {
                if (!*abort_flag) record_error(PA_DEVERR_TIMEOUT);
                *abort_flag = 1;
            }
            // no copy in flight at exit, also where nobody consumed the last tiles (bounded)
            for (int i = max(0, issued - STAGES); i < issued; ++i)
                mbar_wait_bounded(&full_bar[i % STAGES], (i / STAGES) & 1);
        }
        return;
    }

    // ------------------------------ consumers ------------------------------
    float *co = reinterpret_cast<float *>(smem + SC::OFF_COMBINE);           // [NW][G][D], read 16 bytes at a time
    float *cm = co + NW * G * D;                                             // [NW][G]
    float *cl = cm + NW * G;                                                 // [NW][G]
    float *mw = reinterpret_cast<float *>(smem + SC::OFF_MERGE);             // [G][kSplitMaxPieces]
    const int tid = threadIdx.x, tq = lane & 3, r8 = lane >> 2;
    int k0 = 0;                                                              // ring index of the group's first block
    for (long long x = x0; x < x1;) {
        const SplitPlace at = split_locate(prefix, p.num_seqs, p.h_kv, x);
        const int n = (int)min((long long)(at.nb - at.block), x1 - x);
        const int ctx = __ldg(p.context_lens + at.seq);
        int first = 0, count = 0;
        split_blocks(ctx, p.window, BS, p.max_blocks_per_seq, first, count);
        const int first_tok = p.window > 0 && ctx > p.window ? ctx - p.window : 0;
        const size_t head0 = (size_t)at.seq * p.h_q + (size_t)at.kvh * G;    // the group's first query head
        uint32_t qb[C::KS][2];
        float kbias[2] = {0.f, 0.f}, k_factor = p.qk_scale;
        if constexpr (QT == 0) {
            mma_load_q<C, G, D>(qb, p.q + head0 * D, lane);
        } else {
            k_factor *= split_load_q8<C, G, D>(qb, p.q + head0 * D, lane);
            q8_k_bias<C, QT>(qb, lane, kbias);
        }
        SplitState<MT> state;
        state.clear();
        const typename Ext::template Row<G> row(args, p, at.seq, at.kvh, ctx, lane);
        bool bad = false;
        for (int i = (warp + NW - k0 % NW) % NW; i < n; i += NW) {
            if (*abort_flag) break;
            const int k = k0 + i, st = k % STAGES;
            if (!__all_sync(FULL, mbar_wait_bounded(&full_bar[st], (k / STAGES) & 1))) {
                if (lane == 0) {
                    record_error(PA_DEVERR_TIMEOUT);
                    *abort_flag = 1;
                }
                break;
            }
            if (stage[st].bad) {
                bad = true;
            } else {
                const int t0 = (first + at.block + i) * BS;
                if constexpr (QT == 0) {
                    split_consume_bf16<C, BS, G>(smem + st * C::STAGE_BYTES, max(0, first_tok - t0), min(BS, ctx - t0), t0,
                                                 qb, row, state, lane);
                } else {
                    SplitStage sc;
                    sc.k_scale = stage[st].k_scale;
                    sc.v_log2 = stage[st].v_log2;
                    sc.v_inv = stage[st].v_inv;
                    split_consume_q8<C, D, BS, QT>(smem + st * C::STAGE_BYTES, min(BS, ctx - t0), qb, kbias, k_factor, sc,
                                                   state, lane);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty_bar[st]);
        }
        k0 += n;
        x += n;

        // ---- the warps' states of this group ----
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            state.l[0] += __shfl_xor_sync(FULL, state.l[0], off);
            state.l[1] += __shfl_xor_sync(FULL, state.l[1], off);
        }
        if (lane == 0) bad_flag[warp] = bad;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int h = 2 * tq + j;
            if (h < G) {
                if (r8 == 0) {
                    cm[warp * G + h] = state.m[j];
                    cl[warp * G + h] = state.l[j];
                }
                float *dst = co + (size_t)(warp * G + h) * D;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if constexpr (QT == 0) {
                        dst[16 * mt + r8] = state.o[mt][j];
                        dst[16 * mt + r8 + 8] = state.o[mt][2 + j];
                    } else {
                        dst[16 * mt + 2 * r8] = state.o[mt][j];
                        dst[16 * mt + 2 * r8 + 1] = state.o[mt][2 + j];
                    }
                }
            }
        }
        consumers_sync<NW>();
        bool failed = *abort_flag != 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) failed = failed || bad_flag[w] != 0;
        const bool whole = at.block == 0 && n == at.nb;
        const long long group0 = x - n - at.block;                           // the group's first triple
        const int slot = split_slot(range, group0, blockIdx.x);
        const float nan = __int_as_float(0x7fc00000);
        for (int idx = tid; idx < G * D / 4; idx += NW * 32) {
            const int h = idx / (D / 4), d4 = idx % (D / 4);
            float M = cm[h], L = 0.f;
#pragma unroll
            for (int w = 1; w < NW; ++w) M = fmaxf(M, cm[w * G + h]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = cm[w * G + h] == M ? 1.f : exp2f(cm[w * G + h] - M);
                const float4 a = reinterpret_cast<const float4 *>(co + (w * G + h) * D)[d4];
                L += cl[w * G + h] * f;
                o = make_float4(fmaf(a.x, f, o.x), fmaf(a.y, f, o.y), fmaf(a.z, f, o.z), fmaf(a.w, f, o.w));
            }
            if (whole) {
                const float inv = failed ? nan : (L == 0.f ? 0.f : 1.f / L);
                *reinterpret_cast<uint2 *>(p.out + (head0 + h) * D + 4 * d4) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
                if (d4 == 0 && p.lse) p.lse[head0 + h] = failed ? nan : log2_sum(M, L);
            } else {
                if (failed) o = make_float4(nan, nan, nan, nan);
                reinterpret_cast<float4 *>(p.part_o + ((size_t)slot * G + h) * D)[d4] = o;
                if (d4 == 0) reinterpret_cast<float2 *>(p.part_ml)[(size_t)slot * G + h] = make_float2(M, failed ? nan : L);
            }
        }
        consumers_sync<NW>();                                                    // states read, partials written
        if (whole) continue;

        // ---- count; the CTA that completes the group merges it ----
        // the barrier orders all partial writes before thread 0's fence and count (release); whoever sees
        // the count complete fences before its threads read the others' partials (acquire)
        int c0, pieces;
        split_sharers(range, group0, at.nb, c0, pieces);
        if (tid == 0) {
            int *cnt = p.counters + (size_t)at.seq * p.h_kv + at.kvh;
            __threadfence();
            const int is_last = atomicAdd(cnt, 1) == pieces - 1;
            if (is_last) {
                *cnt = 0;                                                    // every CTA of the group has counted
                __threadfence();
            }
            *last_flag = is_last;
        }
        consumers_sync<NW>();
        if (!*last_flag) continue;
        // a warp for each head, a lane for each piece (and the one 32 further): weights 2^(m - M) / L
        for (int h = warp; h < G; h += NW) {
            float2 ml[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = lane + 32 * i;
                const float2 *from = reinterpret_cast<const float2 *>(p.part_ml);
                ml[i] = c < pieces ? __ldcg(from + (size_t)split_slot(range, group0, c0 + c) * G + h)
                                   : make_float2(-INFINITY, 0.f);
            }
            float M = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, off));
            const float w0 = ml[0].x == M ? 1.f : exp2f(ml[0].x - M), w1 = ml[1].x == M ? 1.f : exp2f(ml[1].x - M);
            float L = w0 * ml[0].y + w1 * ml[1].y;
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(FULL, L, off);
            const float inv = L == 0.f ? 0.f : 1.f / L;
            mw[h * kSplitMaxPieces + lane] = w0 * inv;
            mw[h * kSplitMaxPieces + lane + 32] = w1 * inv;
            if (lane == 0 && p.lse) p.lse[head0 + h] = log2_sum(M, L);
        }
        consumers_sync<NW>();
        for (int idx = tid; idx < G * D / 4; idx += NW * 32) {
            const int h = idx / (D / 4), d4 = idx % (D / 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            constexpr int R = 4;                                             // partials loaded at a time, added in order
            for (int q0 = 0; q0 < pieces; q0 += R) {
                float4 v[R];
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (q0 + i < pieces)
                        v[i] = __ldcg(reinterpret_cast<const float4 *>(p.part_o) +
                                      ((size_t)split_slot(range, group0, c0 + q0 + i) * G + h) * (D / 4) + d4);
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (q0 + i < pieces) {
                        const float w = mw[h * kSplitMaxPieces + q0 + i];
                        acc.x += w * v[i].x;
                        acc.y += w * v[i].y;
                        acc.z += w * v[i].z;
                        acc.w += w * v[i].w;
                    }
            }
            *reinterpret_cast<uint2 *>(p.out + (head0 + h) * D + 4 * d4) =
                make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        }
        consumers_sync<NW>();                                                    // mw / last_flag free for the next group
    }
}

}  // namespace pa
