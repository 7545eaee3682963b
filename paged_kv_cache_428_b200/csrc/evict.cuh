// evict.cuh -- what every cached token has been worth to attention, and eviction by it.
//
//   weights[s][k][t] += sum over the query heads h of KV head k of p[s][h][t]
// with p the softmax weights of a decode step.  The decode of decode_split.cuh leaves its logits x (log2 domain,
// fp32) and each row's log2 denominator; a second launch adds 2^(x - denominator).  Logits are 4 bytes for each
// query head and token beside 4 head_dim bytes of K and V for each KV head and token (3 % at 4 heads of 128),
// and mostly stay in L2 between the launches.
//
// Eviction keeps, for each (sequence, KV head), the last `recent` tokens and the heaviest of the older ones, in
// their order, and moves their rows to fresh blocks: a sequence's old blocks may be shared, and its rows move
// towards the front, so in place some would be overwritten before they are read.
#pragma once

#include <cooperative_groups.h>

#include "decode_split.cuh"

namespace pa {

// ---- decode that leaves its logits ------------------------------------------------------------
struct WeightsExt {
    struct Args {
        float *logits;             // [B][h_kv][row_tokens][G]
        int row_tokens;
    };
    template <int G>
    struct Row {
        float *base;
        float scale;
        int row_tokens, tq;
        __device__ __forceinline__ Row(const Args &a, const SplitParams &p, int seq, int kvh, int, int lane)
            : base(a.logits + ((size_t)seq * p.h_kv + kvh) * a.row_tokens * G), scale(p.qk_scale),
              row_tokens(a.row_tokens), tq(lane & 3)
        {
        }
        __device__ __forceinline__ float logit(float dot, int, int) const { return dot * scale; }
        __device__ __forceinline__ void keep(const float (&x)[4], int t, bool use0, bool use1) const
        {
            if (2 * tq >= G) return;
            if (use0 && t < row_tokens) put(t, x[0], x[1]);
            if (use1 && t + 8 < row_tokens) put(t + 8, x[2], x[3]);
        }
        __device__ __forceinline__ void put(int t, float a, float b) const
        {
            if constexpr (G == 1) base[t] = a;
            else *reinterpret_cast<float2 *>(base + (size_t)t * G + 2 * tq) = make_float2(a, b);
        }
    };
};

struct AddWeightsParams {
    const float *logits;           // [B][h_kv][row_tokens][G]
    const float *lse;              // [B][h_q]
    const int32_t *context_lens;
    float *weights;                // [B][h_kv][stride]
    int64_t stride;
    int max_tokens;                // counted at most
    int row_tokens;
    int h_kv;
};

constexpr int kAddThreads = 128, kAddPer = 4;          // threads, tokens of each

// grid (ceil(max_tokens / (threads * per)), h_kv, B).  A sequence whose denominator is not finite (a block outside
// the pool, NaN among its values) keeps its weights.
template <int G>
__global__ void __launch_bounds__(kAddThreads) add_weights_kernel(const AddWeightsParams p)
{
    const int kvh = blockIdx.y, seq = blockIdx.z;
    const int ctx = p.context_lens[seq];
    if (ctx > p.max_tokens && blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0) record_error(PA_DEVERR_BAD_LENGTH);
    const int n = min(ctx, p.max_tokens);
    const size_t row = (size_t)seq * p.h_kv + kvh;
    const int t0 = blockIdx.x * kAddThreads * kAddPer + threadIdx.x;
    if ((int)blockIdx.x * kAddThreads * kAddPer >= n) return;
    float lse[G];
    bool fine = true;
#pragma unroll
    for (int h = 0; h < G; ++h) {
        lse[h] = __ldcg(p.lse + row * G + h);
        fine = fine && fabsf(lse[h]) < INFINITY;
    }
    if (!fine) return;
    const float *x = p.logits + row * p.row_tokens * G;
    float *w = p.weights + row * p.stride;
    float v[kAddPer][G], old[kAddPer];
#pragma unroll
    for (int i = 0; i < kAddPer; ++i) {
        const int t = t0 + i * kAddThreads;
        if (t < n) {
            old[i] = w[t];
            if constexpr (G % 4 == 0) {
#pragma unroll
                for (int h = 0; h < G; h += 4) {
                    const float4 a = __ldcg(reinterpret_cast<const float4 *>(x + (size_t)t * G + h));
                    v[i][h] = a.x;
                    v[i][h + 1] = a.y;
                    v[i][h + 2] = a.z;
                    v[i][h + 3] = a.w;
                }
            } else {
#pragma unroll
                for (int h = 0; h < G; ++h) v[i][h] = __ldcg(x + (size_t)t * G + h);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kAddPer; ++i) {
        const int t = t0 + i * kAddThreads;
        if (t < n) {
            float sum = 0.f;
#pragma unroll
            for (int h = 0; h < G; ++h) sum += exp2f(v[i][h] - lse[h]);
            w[t] = old[i] + sum;
        }
    }
}

// ---- choosing what stays ------------------------------------------------------------------------
struct EvictParams {
    uint8_t *k_cache;
    uint8_t *v_cache;
    const float *weights;          // [B][h_kv][stride]
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *new_tables;
    int32_t *kept;                 // [B][h_kv][budget] old positions, -1 past the last
    float *new_weights;            // [B][h_kv][new_stride]
    int32_t *new_lens;             // [B]
    int64_t stride, new_stride;
    int max_blocks, new_max_blocks;
    int h_kv, block_size, num_blocks;
    int budget, recent;
    int slice_cap;                 // weights of one CTA that fit its shared memory
};

// What becomes of a sequence of ctx tokens: `older` of them compete for `need` places, the `last` ones stay.
// A context longer than its row of weights is refused as a whole.
struct EvictCounts {
    int size, last, older, need;
    __device__ __forceinline__ EvictCounts(const EvictParams &p, int seq)
    {
        int ctx = max(0, __ldg(p.context_lens + seq));
        if (ctx > p.stride) ctx = 0;
        size = min(ctx, p.budget);
        last = min(size, p.recent);
        older = ctx - last;
        need = size - last;
    }
};

// Order of the weights as unsigned numbers; what is not above 0 (NaN included) ranks as 0.
__device__ __forceinline__ uint32_t weight_key(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kSelectBins = 2048;
constexpr int kSelectMaxCluster = 8;
constexpr int kSelectSlice = 16384;                    // weights that one CTA keeps in shared memory

// One cluster for each (sequence, KV head); its CTAs hold slices of the row of weights in shared memory (or
// read them again from L2 where the row is longer than 8 slices).  The need-th largest key comes out of three
// passes over 11, 11 and 10 bits of it: a histogram of the keys that agree with the digits so far, added up over
// the cluster, and the digit in which the remaining count runs out.  Equal keys are taken from the front, by
// their rank among equals.  All counts are integers: the choice does not depend on timing.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams p)
{
    namespace cg = cooperative_groups;
    constexpr unsigned FULL = 0xffffffffu;
    extern __shared__ uint32_t keys[];                 // [slice_cap]
    __shared__ int hist[kSelectBins];
    __shared__ int warp_sum[kSelectWarps];
    __shared__ int found[2];                           // digit, keys in the digits above it
    __shared__ int counts[2];                          // this CTA's keys above the threshold, and equal to it
    __shared__ int warp_gt[kSelectWarps], warp_eq[kSelectWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = blockIdx.x, ranks = gridDim.x, kvh = blockIdx.y, seq = blockIdx.z;   // one cluster in x
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const EvictCounts n(p, seq);
    const size_t row = (size_t)seq * p.h_kv + kvh;
    const float *w = p.weights + row * p.stride;
    int32_t *kept = p.kept + row * p.budget;
    float *new_w = p.new_weights + row * p.new_stride;
    if (kvh == 0 && rank == 0 && tid == 0) {
        p.new_lens[seq] = n.size;
        if (__ldg(p.context_lens + seq) > p.stride) record_error(PA_DEVERR_BAD_LENGTH);
    }
    // what needs no choice: the last ones, and the end of the rows
    const int all = rank * kSelectThreads + tid, step = ranks * kSelectThreads;
    for (int j = all; j < n.last; j += step) {
        kept[n.need + j] = n.older + j;
        new_w[n.need + j] = w[n.older + j];
    }
    for (int j = n.size + all; j < p.budget; j += step) kept[j] = -1;
    for (int64_t j = n.size + all; j < p.new_stride; j += step) new_w[j] = 0.f;
    if (n.need == n.older) {                           // nobody goes
        for (int j = all; j < n.need; j += step) {
            kept[j] = j;
            new_w[j] = w[j];
        }
        return;                                        // the whole cluster
    }
    if (n.need == 0) return;

    const int slice = (n.older + ranks - 1) / ranks;
    const int first = min(n.older, rank * slice), len = min(n.older, first + slice) - first;
    const bool in_smem = slice <= p.slice_cap;
    if (in_smem)
        for (int i = tid; i < len; i += kSelectThreads) keys[i] = weight_key(__ldg(w + first + i));
    auto key_at = [&](int i) { return in_smem ? keys[i] : weight_key(__ldg(w + first + i)); };

    uint32_t prefix = 0, mask = 0;
    int remaining = n.need;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
        for (int b = tid; b < bins; b += kSelectThreads) hist[b] = 0;
        __syncthreads();
        for (int i0 = warp * 32; i0 < len; i0 += kSelectThreads) {
            const int i = i0 + lane;
            const uint32_t k = i < len ? key_at(i) : 0u;
            const bool in = i < len && (k & mask) == prefix;
            const int bin = in ? (int)((k >> shift) & (bins - 1)) : -1;
            // a warp of equal digits (weights that are all alike) adds once
            int same = 0;
            __match_all_sync(FULL, bin, &same);
            if (same) {
                if (in && lane == 0) atomicAdd(&hist[bin], 32);
            } else if (in) {
                atomicAdd(&hist[bin], 1);
            }
        }
        __syncthreads();
        if (ranks > 1) cluster.sync();
        // thread t has bins 4 t .. 4 t + 3, counted from the top
        int c[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int b = bins - 1 - (4 * tid + j);
            c[j] = 0;
            if (b >= 0) {
                if (ranks == 1) c[j] = hist[b];
                else
                    for (int r = 0; r < ranks; ++r) c[j] += *cluster.map_shared_rank(&hist[b], r);
            }
            sum += c[j];
        }
        int upto = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(FULL, upto, off);
            if (lane >= off) upto += y;
        }
        if (lane == 31) warp_sum[warp] = upto;
        __syncthreads();
        int above = upto - sum;
        for (int i = 0; i < warp; ++i) above += warp_sum[i];
        if (above < remaining && above + sum >= remaining) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (above < remaining && above + c[j] >= remaining) {
                    found[0] = bins - 1 - (4 * tid + j);
                    found[1] = above;
                }
                above += c[j];
            }
        }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        remaining -= found[1];
        if (ranks > 1) cluster.sync();                 // every CTA has read the histograms
    }

    // ---- the kept ones in order: warp w has a stretch of the slice ----
    const int part = (len + kSelectWarps - 1) / kSelectWarps;
    const int i_begin = min(len, warp * part), i_end = min(len, i_begin + part);
    int gt = 0, eq = 0;
    for (int i0 = i_begin; i0 < i_end; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < i_end ? key_at(i) : 0u;
        gt += __popc(__ballot_sync(FULL, i < i_end && k > prefix));
        eq += __popc(__ballot_sync(FULL, i < i_end && k == prefix));
    }
    if (lane == 0) {
        warp_gt[warp] = gt;
        warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        int a = 0, b = 0;
        for (int i = 0; i < kSelectWarps; ++i) {
            a += warp_gt[i];
            b += warp_eq[i];
        }
        counts[0] = a;
        counts[1] = b;
    }
    if (ranks > 1) cluster.sync();
    int gt_before = 0, eq_before = 0;
    for (int r = 0; r < rank; ++r) {
        gt_before += *cluster.map_shared_rank(&counts[0], r);
        eq_before += *cluster.map_shared_rank(&counts[1], r);
    }
    for (int i = 0; i < warp; ++i) {
        gt_before += warp_gt[i];
        eq_before += warp_eq[i];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = i_begin; i0 < i_end; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < i_end ? key_at(i) : 0u;
        const uint32_t g = __ballot_sync(FULL, i < i_end && k > prefix), e = __ballot_sync(FULL, i < i_end && k == prefix);
        const int g_pre = gt_before + __popc(g & below), e_pre = eq_before + __popc(e & below);
        if (i < i_end && (k > prefix || (k == prefix && e_pre < remaining))) {
            const int at = g_pre + min(e_pre, remaining);
            kept[at] = first + i;
            new_w[at] = __ldg(w + first + i);
        }
        gt_before += __popc(g);
        eq_before += __popc(e);
    }
    if (ranks > 1) cluster.sync();                     // `counts` read by every CTA before any of them leaves
}

// ---- moving the rows ------------------------------------------------------------------------------
constexpr int kMoveWarps = 8;

// grid (ceil(budget / rows of a CTA), h_kv, B).  LPR: 16-byte chunks of one row.  A warp moves 32 / LPR rows of K
// and of V at a time, four such steps in flight.
template <int LPR>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const EvictParams p)
{
    constexpr int RPW = 32 / LPR, U = 4, ROWS = RPW * U;       // rows of a warp
    const int kvh = blockIdx.y, seq = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const EvictCounts n(p, seq);
    const int j0 = (blockIdx.x * kMoveWarps + warp) * ROWS + lane / LPR;
    const int col = lane % LPR;
    if ((int)(blockIdx.x * kMoveWarps + warp) * ROWS >= n.size) return;
    const int32_t *kept = p.kept + ((size_t)seq * p.h_kv + kvh) * p.budget;
    const int32_t *from = p.block_tables + (size_t)seq * p.max_blocks, *to = p.new_tables + (size_t)seq * p.new_max_blocks;
    const uint4 *k = reinterpret_cast<const uint4 *>(p.k_cache), *v = reinterpret_cast<const uint4 *>(p.v_cache);
    int64_t src[U], dst[U];                                    // 16-byte chunks; -1: no row
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int j = j0 + u * RPW;
        src[u] = dst[u] = -1;
        if (j < n.size) {
            const int t = kept[j], sb = t / p.block_size, db = j / p.block_size;
            const int a = t >= 0 && sb < p.max_blocks ? __ldg(from + sb) : -1, b = db < p.new_max_blocks ? __ldg(to + db) : -1;
            if (a >= 0 && a < p.num_blocks && b >= 0 && b < p.num_blocks) {
                src[u] = (((int64_t)a * p.h_kv + kvh) * p.block_size + t % p.block_size) * LPR + col;
                dst[u] = (((int64_t)b * p.h_kv + kvh) * p.block_size + j % p.block_size) * LPR + col;
            } else if (col == 0) {
                record_error(PA_DEVERR_BAD_BLOCK);
            }
        }
    }
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (src[u] >= 0) {
            a[u] = __ldcs(k + src[u]);
            b[u] = __ldcs(v + src[u]);
        }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (src[u] >= 0) {
            reinterpret_cast<uint4 *>(p.k_cache)[dst[u]] = a[u];
            reinterpret_cast<uint4 *>(p.v_cache)[dst[u]] = b[u];
        }
}

}  // namespace pa
