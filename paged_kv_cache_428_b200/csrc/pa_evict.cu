// pa_evict.cu -- C-ABI calls of decode with attention weights and of eviction by them.
#include "evict.cuh"
#include "split_launch.cuh"

using namespace pa;

int pa::evict_errors(unsigned int *flags, int clear) { return collect_device_errors(flags, clear); }

namespace {

// Tokens that the logits of one (sequence, KV head) have room for.
int logit_tokens(int max_context_len) { return (max_context_len + 3) / 4 * 4; }

size_t logit_bytes(int num_seqs, int h_q, int max_context_len)
{
    return round256((size_t)num_seqs * h_q * logit_tokens(max_context_len) * sizeof(float));
}

template <int NT, int V>
int launch_select_as(const EvictParams &p, int num_seqs, int ranks, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ranks, p.h_kv, num_seqs);
    cfg.blockDim = dim3(NT);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<NT, V>, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Keys of a row in the registers of as few threads as hold them: 4096 a CTA of 256 threads up to clusters of 8,
// 16384 a CTA of 512 beyond.  More threads a CTA are faster alone but fill the SMs: 512 rows of up to 4096 in two
// waves, 24.6 us at 512 threads; 16 clusters of 8 for 131072 in two waves, 50 us at 1024.
int launch_select(const EvictParams &p, int num_seqs, int max_context_len, cudaStream_t st)
{
    int ranks = 1;
    while (ranks < kSelectMaxCluster && ranks * 4096 < max_context_len) ranks *= 2;
    if (max_context_len <= 1024) return launch_select_as<256, 4>(p, num_seqs, 1, st);
    if (max_context_len <= kSelectMaxCluster * 4096) return launch_select_as<256, 16>(p, num_seqs, ranks, st);
    return launch_select_as<512, 32>(p, num_seqs, kSelectMaxCluster, st);
}

template <int LPR>
int launch_move(const EvictParams &p, int num_seqs, int most, cudaStream_t st)
{
    const int rows = 32 / LPR * 4 * kMoveWarps;
    return launch_ex(evict_move_kernel<LPR>, dim3(std::max(1, (most + rows - 1) / rows), p.h_kv, num_seqs), dim3(kMoveWarps * 32), 0, st,
                     true, p);
}

bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

}  // namespace

extern "C" {

size_t pa_decode_weights_workspace_size(int num_seqs, int h_q, int h_kv, int head_dim, int max_context_len)
{
    if (!split_sizes_ok(num_seqs, h_q, h_kv, head_dim, max_context_len) || max_context_len > kMaxWeights) return 0;
    return split_layout(num_seqs, h_q, h_kv, head_dim, max_context_len).end + logit_bytes(num_seqs, h_q, max_context_len);
}

int pa_decode_weights(void *out, float *weights, int64_t weights_stride, const void *q, const void *k_cache,
                      const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                      int num_seqs, int max_context_len, int h_q, int h_kv, int head_dim, int block_size, int num_blocks,
                      float scale, int cache_dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    if (cache_dtype < PA_CACHE_BF16 || cache_dtype > PA_CACHE_INT8 || weights_stride < max_context_len) return PA_ERR_INVALID_ARG;
    if (cache_dtype != PA_CACHE_BF16 || max_context_len > kMaxWeights) return PA_ERR_UNSUPPORTED;
    const SplitCall c{out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, max_context_len,
                      h_q, h_kv, head_dim, block_size, num_blocks, scale, 0, workspace, workspace_bytes, stream};
    SplitParams p{};
    const bool sized = split_sizes_ok(num_seqs, h_q, h_kv, head_dim, max_context_len);
    int rc = split_prepare(p, c, sized ? logit_bytes(num_seqs, h_q, max_context_len) : 0);
    if (rc != PA_OK || num_seqs == 0) return rc;
    if (!weights) return PA_ERR_INVALID_ARG;
    if (h_kv > 65535) return PA_ERR_UNSUPPORTED;
    const SplitLayout lay = split_layout(num_seqs, h_q, h_kv, head_dim, max_context_len);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.lse = reinterpret_cast<float *>(ws + lay.lse);
    const WeightsExt::Args args{reinterpret_cast<float *>(ws + lay.end), logit_tokens(max_context_len)};
    rc = split_launch<0, WeightsExt>(c, p, args);
    if (rc != PA_OK) return rc;
    AddWeightsParams a{};
    a.logits = args.logits;
    a.lse = p.lse;
    a.context_lens = context_lens;
    a.weights = weights;
    a.stride = weights_stride;
    a.max_tokens = max_context_len;
    a.row_tokens = args.row_tokens;
    a.h_kv = h_kv;
    const dim3 grid(std::max(1, (max_context_len + kAddThreads * kAddPer - 1) / (kAddThreads * kAddPer)), h_kv, num_seqs);
    return switch_group(h_q / h_kv, [&](auto gc) {
        return launch_ex(add_weights_kernel<decltype(gc)::value>, grid, dim3(kAddThreads), 0,
                         static_cast<cudaStream_t>(stream), true, a);
    });
}

int pa_evict(void *k_cache, void *v_cache, const float *weights, int64_t weights_stride, const int32_t *block_tables,
             int max_blocks_per_seq, const int32_t *context_lens, const int32_t *new_block_tables, int new_max_blocks_per_seq,
             int num_seqs, int max_context_len, int budget, int recent, int h_kv, int head_dim, int block_size,
             int num_blocks, int cache_dtype, int32_t *kept, float *new_weights, int64_t new_weights_stride,
             int32_t *new_context_lens, void *stream)
{
    if (num_seqs < 0 || max_context_len < 0 || budget < 1 || recent < 0 || recent > budget || h_kv <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || new_max_blocks_per_seq <= 0 || cache_dtype < PA_CACHE_BF16 || cache_dtype > PA_CACHE_INT8)
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size)) return PA_ERR_UNSUPPORTED;
    const int most = std::min(budget, max_context_len);
    if (weights_stride < max_context_len || new_weights_stride < budget ||
        (long long)new_max_blocks_per_seq * block_size < most)
        return PA_ERR_INVALID_ARG;
    if (h_kv > 65535 || num_seqs > 65535 || max_context_len > kMaxWeights || budget > kMaxWeights) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!k_cache || !v_cache || !weights || !block_tables || !context_lens || !new_block_tables || !kept || !new_weights ||
        !new_context_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    // the old weights and lengths are read while the new ones are written
    const size_t rows = (size_t)num_seqs * h_kv;
    if (overlap(weights, rows * weights_stride * 4, new_weights, rows * new_weights_stride * 4) ||
        overlap(context_lens, (size_t)num_seqs * 4, new_context_lens, (size_t)num_seqs * 4))
        return PA_ERR_INVALID_ARG;
    EvictParams p{};
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.weights = weights;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.new_tables = new_block_tables;
    p.kept = kept;
    p.new_weights = new_weights;
    p.new_lens = new_context_lens;
    p.stride = weights_stride;
    p.longest = (int)std::min<int64_t>(weights_stride, kMaxWeights);
    p.new_stride = new_weights_stride;
    p.max_blocks = max_blocks_per_seq;
    p.new_max_blocks = new_max_blocks_per_seq;
    p.h_kv = h_kv;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.budget = budget;
    p.recent = recent;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rc = launch_select(p, num_seqs, max_context_len, st);
    if (rc != PA_OK) return rc;
    switch (head_dim * (cache_dtype == PA_CACHE_BF16 ? 2 : 1) / 16) {
    case 4: return launch_move<4>(p, num_seqs, most, st);
    case 8: return launch_move<8>(p, num_seqs, most, st);
    case 16: return launch_move<16>(p, num_seqs, most, st);
    default: return PA_ERR_UNSUPPORTED;
    }
}

}  // extern "C"
