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
    static constexpr bool kDependent = true;           // add_weights_kernel
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

constexpr int kMaxWeights = 1 << 30;                   // of one row: places are counted in 32 bits, in steps
constexpr int kAddThreads = 128, kAddPer = 4;          // threads, tokens of each

// grid (ceil(max_tokens / (threads * per)), h_kv, B).  Bound by latency (length, denominators and logits, 28 MB mostly
// from L2): 8.7 us for 64 sequences of 512..4096 tokens and 8 KV heads, partly behind the decode's end.  A sequence
// whose denominator is not finite (a block outside the pool, NaN among its values) keeps its weights.
template <int G>
__global__ void __launch_bounds__(kAddThreads) add_weights_kernel(const AddWeightsParams p)
{
    const int kvh = blockIdx.y, seq = blockIdx.z;
    const int ctx = p.context_lens[seq];
    pdl_wait();                                        // the decode is complete
    if (ctx > p.max_tokens && blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0) record_error(PA_DEVERR_BAD_LENGTH);
    const int n = min(ctx, p.max_tokens);
    const size_t row = (size_t)seq * p.h_kv + kvh;
    const int t0 = blockIdx.x * kAddThreads * kAddPer + threadIdx.x;
    if ((int)blockIdx.x * kAddThreads * kAddPer >= n) return;
    const float *x = p.logits + row * p.row_tokens * G;
    float *w = p.weights + row * p.stride;
    float v[kAddPer][G], old[kAddPer], lse[G];                 // all loads at once
#pragma unroll
    for (int i = 0; i < kAddPer; ++i) {
        const int t = t0 + i * kAddThreads;
        if (t < n) {
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
            old[i] = w[t];
        }
    }
    bool fine = true;
#pragma unroll
    for (int h = 0; h < G; ++h) {
        lse[h] = __ldcg(p.lse + row * G + h);
        fine = fine && fabsf(lse[h]) < INFINITY;
    }
    if (!fine) return;
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
    int longest;                   // context that the rows of weights, and the counts here, have room for
    int max_blocks, new_max_blocks;
    int h_kv, block_size, num_blocks;
    int budget, recent;
};

// What becomes of a sequence of ctx tokens: `older` of them compete for `need` places, the `last` ones stay.
// A context longer than its row of weights (or than kMaxWeights) is refused as a whole.
struct EvictCounts {
    int size, last, older, need;
    __device__ __forceinline__ EvictCounts(const EvictParams &p, int seq)
    {
        int ctx = max(0, __ldg(p.context_lens + seq));
        if (ctx > p.longest) ctx = 0;
        size = min(ctx, p.budget);
        last = min(size, p.recent);
        older = ctx - last;
        need = size - last;
    }
};

// Order of the weights as whole numbers; what is not above 0 (NaN included) ranks as 0.
__device__ __forceinline__ int weight_key(float w) { return w > 0.f ? __float_as_int(w) : 0; }

constexpr int kSelectBins = 2048;
constexpr int kSelectMaxCluster = 8;

// One cluster for each (sequence, KV head); its CTAs take slices of the row of weights.  Warp w of a CTA holds
// V x 32 neighbouring keys of its slice in registers (a row longer than NT * V keys for each CTA is read again,
// NT * V at a time, for every step below); -1 stands for no key.  The need-th largest key comes out of three
// passes over its upper 11, next 11 and last 10 bits: a histogram of the keys that agree with the digits so far,
// and the digit in which the remaining count runs out.  To find it the first warp of every CTA adds up, over
// the cluster, 32 sums of neighbouring bins, then the bins behind one of them (all bins of all CTAs would keep the
// paths between the SMs busy for longer than the rest takes).  Equal keys are taken from the front, by their
// rank among equals.  All counts are integers: the choice does not depend on timing.
//   Bound by instructions and barriers, not by the row's 4 bytes a token: 512 rows of 512..4096 keys 16 us, 16 rows of
// 32768..131072 26 us (load 4, three passes 11, counting 1.5, writing 5).
template <int NT, int V>
__global__ void __launch_bounds__(NT, 1024 / NT) evict_select_kernel(const EvictParams p)
{
    namespace cg = cooperative_groups;
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int NWARP = NT / 32;
    __shared__ __align__(16) int hist[3][kSelectBins];
    __shared__ int coarse[3][32];                      // sums of bins / 32 neighbouring bins
    __shared__ int found[3][2];                        // of each pass: the digit, keys in the digits above it
    __shared__ int counts[2];                          // this CTA's keys above the threshold, and equal to it
    __shared__ int warp_gt[NWARP], warp_eq[NWARP];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = blockIdx.x, ranks = gridDim.x, kvh = blockIdx.y, seq = blockIdx.z;   // one cluster in x
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();                           // the rows' copy may be set up meanwhile
    const EvictCounts n(p, seq);
    const size_t row = (size_t)seq * p.h_kv + kvh;
    const float *w = p.weights + row * p.stride;
    int32_t *kept = p.kept + row * p.budget;
    float *new_w = p.new_weights + row * p.new_stride;
    const bool choose = n.need != n.older && n.need > 0;        // else nobody goes, or only the last ones stay
    const int slice = (n.older + ranks - 1) / ranks;
    const int first = min(n.older, rank * slice), len = choose ? min(n.older, first + slice) - first : 0;
    const int chunks = choose ? (slice + NT * V - 1) / (NT * V) : 0;   // the same in every CTA of the cluster

    int key[V], diff = 0;                              // diff: bits in which the lane's keys differ
    int i0 = 0;                                        // place of key[0] of this lane in the slice
    auto load = [&](int chunk) {
        i0 = (chunk * NWARP + warp) * V * 32 + lane;
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = i0 + v * 32 < len ? weight_key(__ldg(w + first + i0 + v * 32)) : -1;
        diff = 0;
#pragma unroll
        for (int v = 1; v < V; ++v) diff |= key[v] ^ key[0];
    };
    if (chunks == 1) load(0);
    if (choose) {
#pragma unroll
        for (int h = 0; h < 3; ++h)
            for (int b = tid; b < kSelectBins / 4; b += NT) reinterpret_cast<int4 *>(hist[h])[b] = make_int4(0, 0, 0, 0);
    }
    if (kvh == 0 && rank == 0 && tid == 0) {
        p.new_lens[seq] = n.size;
        if (__ldg(p.context_lens + seq) > p.longest) record_error(PA_DEVERR_BAD_LENGTH);
    }
    // what needs no choice: the last ones, and the end of the rows
    const int all = rank * NT + tid, step = ranks * NT;
    for (int j = all; j < n.last; j += step) {
        kept[n.need + j] = n.older + j;
        new_w[n.need + j] = __ldg(w + n.older + j);
    }
    for (int j = n.size + all; j < p.budget; j += step) kept[j] = -1;
    for (int64_t j = n.size + all; j < p.new_stride; j += step) new_w[j] = 0.f;
    if (!choose) {                                     // the whole cluster
        for (int j = all; j < n.need; j += step) {
            kept[j] = j;
            new_w[j] = __ldg(w + j);
        }
        return;
    }
    __syncthreads();

    int prefix = 0, mask = 0;
    int remaining = n.need;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        // a key's first digit is below 1024 (its sign bit is 0); -1 goes to bin 2047, which nobody reads
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, digits = pass == 2 ? 1023 : 2047, bins = pass == 1 ? 2048 : 1024;
        for (int chunk = 0; chunk < chunks; ++chunk) {
            if (chunks > 1) load(chunk);
            // a warp of equal digits (weights that are all alike) adds once
            const int cared = mask | (digits << shift);
            if (__all_sync(FULL, ((diff | (key[0] ^ __shfl_sync(FULL, key[0], 0))) & cared) == 0)) {
                if (lane == 0 && (key[0] & mask) == prefix) atomicAdd(&hist[pass][(key[0] >> shift) & digits], 32 * V);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if ((key[v] & mask) == prefix) atomicAdd(&hist[pass][(key[v] >> shift) & digits], 1);
            }
        }
        __syncthreads();
        const int width = bins / 32;                   // 32 or 64
        for (int b = warp; b < 32; b += NWARP) {
            const int *from = hist[pass] + b * width + lane;
            const int sum = __reduce_add_sync(FULL, width == 64 ? from[0] + from[32] : from[0]);
            if (lane == 0) coarse[pass][b] = sum;
        }
        if (ranks > 1) cluster.sync();
        else __syncthreads();
        if (warp == 0) {
            auto over_cluster = [&](const int *at) {
                int sum = 0;
#pragma unroll
                for (int r = 0; r < kSelectMaxCluster; ++r)
                    if (r < ranks) sum += ranks > 1 ? *cluster.map_shared_rank(at, r) : *at;
                return sum;
            };
            // lane l: what lies above its (31 - l)-th stretch of values c; the lane in which `left` runs out
            auto runs_out = [&](int c, int left, int &above) {
                int upto = c;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(FULL, upto, off);
                    if (lane >= off) upto += y;
                }
                above = upto - c;
                return __ffs(__ballot_sync(FULL, above < left && upto >= left)) - 1;
            };
            int above, more;
            const int a = runs_out(over_cluster(&coarse[pass][31 - lane]), remaining, above);
            const int before = __shfl_sync(FULL, above, a), left = remaining - before;
            const int *fine = hist[pass] + (31 - a) * width;
            if (width == 64) {
                const int hi = over_cluster(fine + 63 - 2 * lane), lo = over_cluster(fine + 62 - 2 * lane);
                const int b = runs_out(hi + lo, left, more);
                const int c = __shfl_sync(FULL, hi, b), m = __shfl_sync(FULL, more, b);
                const bool second = m + c < left;
                if (lane == 0) {
                    found[pass][0] = (31 - a) * 64 + 63 - 2 * b - second;
                    found[pass][1] = before + m + (second ? c : 0);
                }
            } else {
                const int b = runs_out(over_cluster(fine + 31 - lane), left, more);
                if (lane == b) {
                    found[pass][0] = (31 - a) * 32 + 31 - b;
                    found[pass][1] = before + more;
                }
            }
        }
        __syncthreads();
        prefix |= found[pass][0] << shift;
        mask |= digits << shift;
        remaining -= found[pass][1];
    }

    // ---- the kept ones, in order ----
    // keys above the threshold and equal to it: of this warp's part of a chunk, of the CTA, of the CTAs before
    auto count = [&](int &gt, int &eq) {
        gt = eq = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            gt += key[v] > prefix;
            eq += key[v] == prefix;
        }
        gt = __reduce_add_sync(FULL, gt);
        eq = __reduce_add_sync(FULL, eq);
    };
    int gt = 0, eq = 0, gt_before = 0, eq_before = 0;
    if (ranks > 1) {
        int a = 0, b = 0;
        for (int chunk = 0; chunk < chunks; ++chunk) {
            if (chunks > 1) load(chunk);
            count(gt, eq);
            a += gt;
            b += eq;
        }
        if (lane == 0) {
            warp_gt[warp] = a;
            warp_eq[warp] = b;
        }
        __syncthreads();
        if (warp == 0) {
            a = __reduce_add_sync(FULL, lane < NWARP ? warp_gt[lane] : 0);
            b = __reduce_add_sync(FULL, lane < NWARP ? warp_eq[lane] : 0);
            if (lane == 0) {
                counts[0] = a;
                counts[1] = b;
            }
        }
        cluster.sync();
        const bool mine = lane < rank;
        gt_before = __reduce_add_sync(FULL, mine ? *cluster.map_shared_rank(&counts[0], mine ? lane : 0) : 0);
        eq_before = __reduce_add_sync(FULL, mine ? *cluster.map_shared_rank(&counts[1], mine ? lane : 0) : 0);
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int chunk = 0; chunk < chunks; ++chunk) {
        if (chunks > 1) load(chunk);
        if (chunks > 1 || ranks == 1) count(gt, eq);
        if (chunks > 1 || ranks == 1) {
            __syncthreads();                           // the previous chunk's counts have been read
            if (lane == 0) {
                warp_gt[warp] = gt;
                warp_eq[warp] = eq;
            }
            __syncthreads();
        }
        int g_at = gt_before + __reduce_add_sync(FULL, lane < warp ? warp_gt[lane] : 0);
        int e_at = eq_before + __reduce_add_sync(FULL, lane < warp ? warp_eq[lane] : 0);
        if (chunks > 1) {
            gt_before += __reduce_add_sync(FULL, lane < NWARP ? warp_gt[lane] : 0);
            eq_before += __reduce_add_sync(FULL, lane < NWARP ? warp_eq[lane] : 0);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t g = __ballot_sync(FULL, key[v] > prefix), e = __ballot_sync(FULL, key[v] == prefix);
            if (g | e) {
                const int g_pre = g_at + __popc(g & below), e_pre = e_at + __popc(e & below);
                if (key[v] > prefix || (key[v] == prefix && e_pre < remaining)) {
                    const int at = g_pre + min(e_pre, remaining), i = first + i0 + v * 32;
                    kept[at] = i;
                    // what is above 0 is its key; below that the weight itself
                    new_w[at] = key[v] ? __int_as_float(key[v]) : __ldg(w + i);
                }
                g_at += __popc(g);
                e_at += __popc(e);
            }
        }
    }
    if (ranks > 1) cluster.sync();                     // histograms and counts read by every CTA before any leaves
}

// ---- moving the rows ------------------------------------------------------------------------------
constexpr int kMoveWarps = 8;

// grid (CTAs for the rows that the host expects, at least one; h_kv, B).  LPR: 16-byte chunks of one row.  A warp moves
// 32 / LPR rows of K and of V at a time, four such steps in flight, and goes on behind the grid's last row where more
// stay (contexts above the host's bound).  Bound by HBM: 268 MB in 44 us, 6.1 TB/s.
template <int LPR>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const EvictParams p)
{
    constexpr int RPW = 32 / LPR, U = 4, ROWS = RPW * U;       // rows of a warp
    const int kvh = blockIdx.y, seq = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const EvictCounts n(p, seq);
    pdl_wait();                                                // the choice is complete
    const int col = lane % LPR, shift = __ffs(p.block_size) - 1, low = p.block_size - 1;     // a power of two
    const int32_t *kept = p.kept + ((size_t)seq * p.h_kv + kvh) * p.budget;
    const int32_t *from = p.block_tables + (size_t)seq * p.max_blocks, *to = p.new_tables + (size_t)seq * p.new_max_blocks;
    const uint4 *k = reinterpret_cast<const uint4 *>(p.k_cache), *v = reinterpret_cast<const uint4 *>(p.v_cache);
#pragma unroll 1
    for (unsigned first = (blockIdx.x * kMoveWarps + warp) * ROWS; first < (unsigned)n.size;
         first += gridDim.x * kMoveWarps * ROWS) {
        const int j0 = (int)first + lane / LPR;
        int64_t src[U], dst[U];                                // 16-byte chunks; -1: no row
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u * RPW;
            src[u] = dst[u] = -1;
            if (j < n.size) {
                const int t = kept[j], sb = t >> shift, db = j >> shift;
                const int a = t >= 0 && sb < p.max_blocks ? __ldg(from + sb) : -1;
                const int b = db < p.new_max_blocks ? __ldg(to + db) : -1;
                if (a >= 0 && a < p.num_blocks && b >= 0 && b < p.num_blocks) {
                    src[u] = (((int64_t)a * p.h_kv + kvh) * p.block_size + (t & low)) * LPR + col;
                    dst[u] = (((int64_t)b * p.h_kv + kvh) * p.block_size + (j & low)) * LPR + col;
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
}

}  // namespace pa
