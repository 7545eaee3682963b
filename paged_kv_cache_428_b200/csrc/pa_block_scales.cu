// pa_block_scales.cu -- C-ABI calls of the 8-bit cache with a scale for each block and KV head.
#include "block_scales.cuh"
#include "split_launch.cuh"

using namespace pa;

int pa::block_scales_errors(unsigned int *flags, int clear) { return collect_device_errors(flags, clear); }

namespace {

bool quantised(int cache_dtype) { return cache_dtype == PA_CACHE_E4M3 || cache_dtype == PA_CACHE_INT8; }

template <int D, int BS>
void launch_write(int cache_dtype, dim3 grid, const BlockScaleWriteParams &p, cudaStream_t st)
{
    if (cache_dtype == PA_CACHE_E4M3) write_block_scales_kernel<D, BS, 1><<<grid, kScaleWriteWarps * 32, 0, st>>>(p);
    else write_block_scales_kernel<D, BS, 2><<<grid, kScaleWriteWarps * 32, 0, st>>>(p);
}

template <int D>
void launch_write_block(int block_size, int cache_dtype, dim3 grid, const BlockScaleWriteParams &p, cudaStream_t st)
{
    if (block_size == 16) launch_write<D, 16>(cache_dtype, grid, p, st);
    else if (block_size == 32) launch_write<D, 32>(cache_dtype, grid, p, st);
    else launch_write<D, 64>(cache_dtype, grid, p, st);
}

}  // namespace

extern "C" {

int pa_reshape_and_cache_block_scales(const void *key, const void *value, int64_t key_stride, int64_t value_stride,
                                      void *k_cache, void *v_cache, float *k_scales, float *v_scales,
                                      const int64_t *slot_mapping, int num_tokens, int h_kv, int head_dim, int block_size,
                                      int num_blocks, int cache_dtype, void *stream)
{
    if (num_tokens < 0 || h_kv <= 0 || num_blocks <= 0 || !quantised(cache_dtype)) return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size)) return PA_ERR_UNSUPPORTED;
    const int64_t row = (int64_t)h_kv * head_dim;
    if (key_stride == 0) key_stride = row;
    if (value_stride == 0) value_stride = row;
    if (key_stride < row || value_stride < row || key_stride % 8 != 0 || value_stride % 8 != 0) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !k_scales || !v_scales || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    if (h_kv > 65535) return PA_ERR_UNSUPPORTED;
    BlockScaleWriteParams p{};
    p.key = static_cast<const __nv_bfloat16 *>(key);
    p.value = static_cast<const __nv_bfloat16 *>(value);
    p.key_stride = key_stride;
    p.value_stride = value_stride;
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.slot_mapping = slot_mapping;
    p.num_tokens = num_tokens;
    p.h_kv = h_kv;
    p.num_slots = (long long)num_blocks * block_size;
    // As many tokens a CTA as leave one CTA for each of the 8 places of an SM: a CTA takes its runs a few at a time, and
    // finding them costs about as much as writing one.  One-token runs of 8 heads of 128 into blocks of 64, in chunks of
    // 2, 8 and 64: 512 tokens 10, 11 and 51 us, 4096 tokens 56, 45 and 64; prompts of 4096 tokens 21, 13 and 11 us, of
    // 32768 (4, 8 and 64) 85, 61 and 45.
    const int sms = sm_count();
    if (sms < 1) return PA_ERR_CUDA;
    p.chunk = 2;
    while (p.chunk < kScaleWriteMaxChunk && (long long)num_tokens * h_kv >= (long long)2 * p.chunk * 8 * sms) p.chunk *= 2;
    const dim3 grid((num_tokens + p.chunk - 1) / p.chunk, h_kv);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (head_dim == 64) launch_write_block<64>(block_size, cache_dtype, grid, p, st);
    else launch_write_block<128>(block_size, cache_dtype, grid, p, st);
    return launch_status();
}

int pa_copy_block_scales(float *const *k_scales, float *const *v_scales, int num_layers, const int64_t *block_pairs,
                         int num_pairs, int h_kv, int num_blocks, void *stream)
{
    if (num_layers < 0 || num_pairs < 0 || num_blocks <= 0 || h_kv <= 0) return PA_ERR_INVALID_ARG;
    if (num_layers == 0 || num_pairs == 0) return PA_OK;
    if (!k_scales || !v_scales || !block_pairs) return PA_ERR_INVALID_ARG;
    for (int l = 0; l < num_layers; ++l)
        if (!k_scales[l] || !v_scales[l]) return PA_ERR_INVALID_ARG;
    for (int l0 = 0; l0 < num_layers; l0 += kScaleCopyMaxLayers) {
        const int nl = std::min(num_layers - l0, kScaleCopyMaxLayers);
        CopyScalesParams p{};
        for (int l = 0; l < nl; ++l) {
            p.k[l] = k_scales[l0 + l];
            p.v[l] = v_scales[l0 + l];
        }
        p.pairs = block_pairs;
        p.h_kv = h_kv;
        p.num_blocks = num_blocks;
        copy_scales_kernel<<<dim3(num_pairs, nl, 2), 32, 0, static_cast<cudaStream_t>(stream)>>>(p);
        const int rc = launch_status();
        if (rc != PA_OK) return rc;
    }
    return PA_OK;
}

int pa_validate_block_runs(const int64_t *slot_mapping, int num_tokens, int block_size, int num_blocks)
{
    if (num_tokens < 0 || block_size <= 0 || num_blocks <= 0 || (num_tokens > 0 && !slot_mapping)) return PA_ERR_INVALID_ARG;
    uint8_t *seen = static_cast<uint8_t *>(std::calloc((size_t)num_blocks, 1));
    if (!seen) return PA_ERR_OOM;
    int rc = PA_OK;
    int64_t before = -1;
    for (int t = 0; t < num_tokens && rc == PA_OK; ++t) {
        const int64_t block = slot_mapping[t] < 0 ? -1 : slot_mapping[t] / block_size;
        if (block >= num_blocks) rc = PA_ERR_INVALID_ARG;
        else if (block >= 0 && block != before) {
            if (seen[block]) rc = PA_ERR_INVALID_ARG;
            seen[block] = 1;
        }
        before = block;
    }
    std::free(seen);
    return rc;
}

size_t pa_decode_block_scales_workspace_size(int num_seqs, int h_q, int h_kv, int head_dim, int max_context_len)
{
    if (!split_sizes_ok(num_seqs, h_q, h_kv, head_dim, max_context_len)) return 0;
    return split_layout(num_seqs, h_q, h_kv, head_dim, max_context_len).end;
}

int pa_decode_block_scales(void *out, const void *q, const void *k_cache, const void *v_cache, const float *k_scales,
                           const float *v_scales, const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens, int num_seqs, int max_context_len, int h_q, int h_kv, int head_dim,
                           int block_size, int num_blocks, float scale, int cache_dtype, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    if (!quantised(cache_dtype)) return PA_ERR_INVALID_ARG;
    const SplitCall c{out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, max_context_len,
                      h_q, h_kv, head_dim, block_size, num_blocks, scale, 0, workspace, workspace_bytes, stream};
    SplitParams p{};
    const int rc = split_prepare(p, c, 0);
    if (rc != PA_OK || num_seqs == 0) return rc;
    if (!k_scales || !v_scales) return PA_ERR_INVALID_ARG;
    const BlockScalesExt::Args args{k_scales, v_scales};
    return cache_dtype == PA_CACHE_E4M3 ? split_launch<1, BlockScalesExt>(c, p, args)
                                        : split_launch<2, BlockScalesExt>(c, p, args);
}

}  // extern "C"
