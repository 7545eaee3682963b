// pa_scoremod.cu -- C-ABI calls of decode with modified scores.
#include "scoremod_decode.cuh"
#include "split_launch.cuh"

using namespace pa;

int pa::scoremod_errors(unsigned int *flags, int clear) { return collect_device_errors(flags, clear); }

extern "C" {

size_t pa_decode_scoremod_workspace_size(int num_seqs, int h_q, int h_kv, int head_dim, int max_context_len, int window)
{
    if (!split_sizes_ok(num_seqs, h_q, h_kv, head_dim, max_context_len) || window < 0) return 0;
    return split_layout(num_seqs, h_q, h_kv, head_dim, window > 0 ? std::min(window, max_context_len) : max_context_len).end;
}

int pa_decode_scoremod(void *out, const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
                       int max_blocks_per_seq, const int32_t *context_lens, int num_seqs, int max_context_len, int h_q,
                       int h_kv, int head_dim, int block_size, int num_blocks, float scale, float softcap,
                       const float *alibi_slopes, int window, int cache_dtype, void *workspace, size_t workspace_bytes,
                       void *stream)
{
    if (cache_dtype < PA_CACHE_BF16 || cache_dtype > PA_CACHE_INT8 || !valid_scores(scale, softcap)) return PA_ERR_INVALID_ARG;
    if (cache_dtype != PA_CACHE_BF16) return PA_ERR_UNSUPPORTED;
    const SplitCall c{out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, max_context_len,
                      h_q, h_kv, head_dim, block_size, num_blocks, scale, window, workspace, workspace_bytes, stream};
    SplitParams p{};
    const int rc = split_prepare(p, c, 0);
    if (rc != PA_OK || num_seqs == 0) return rc;
    const ScoreModExt::Args args{alibi_slopes, softcap > 0.f ? 2.f * p.qk_scale / softcap : 0.f, softcap * kLog2e};
    return split_launch<0, ScoreModExt>(c, p, args);
}

}  // extern "C"
