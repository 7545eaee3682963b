// pa_prefill_scoremod.cu -- C-ABI call of chunked prefill with modified scores.
#include "prefill_launch.cuh"
#include "scoremod_prefill.cuh"

using namespace pa;

int pa::prefill_scoremod_errors(unsigned int *flags, int clear) { return collect_device_errors(flags, clear); }

namespace {

template <int D, int BS, bool CAP, bool BIAS>
int dispatch_scoremod_group(int g, const PrefillParams &pp, int n, int mql, int *counters,
                            const PrefillScoreMod<CAP, BIAS> &mod, cudaStream_t st)
{
    return switch_group(g, [&](auto gc) {
        return launch_prefill_tc<D, BS, decltype(gc)::value, PrefillScoreMod<CAP, BIAS>>(pp, n, mql, counters, st, mod);
    });
}

template <int D, bool CAP, bool BIAS>
int dispatch_scoremod_block(int bs, int g, const PrefillParams &pp, int n, int mql, int *counters,
                            const PrefillScoreMod<CAP, BIAS> &mod, cudaStream_t st)
{
    if (bs == 16) return dispatch_scoremod_group<D, 16>(g, pp, n, mql, counters, mod, st);
    if (bs == 32) return dispatch_scoremod_group<D, 32>(g, pp, n, mql, counters, mod, st);
    return dispatch_scoremod_group<D, 64>(g, pp, n, mql, counters, mod, st);
}

template <bool CAP, bool BIAS>
int dispatch_scoremod(int d, int bs, int g, const PrefillParams &pp, int n, int mql, int *counters, float scale, float softcap,
                      const float *slopes, int window, const int32_t *prefix_lens, cudaStream_t st)
{
    PrefillScoreMod<CAP, BIAS> mod{};
    mod.slopes = slopes;
    mod.prefix_lens = prefix_lens;
    mod.window = window;
    if (CAP) {
        // y = raw score * in; logit = out * y q(y^2)
        const double in = (double)scale / softcap, to = (double)softcap * kLog2e;
        const double coef[3] = {PA_TANH_C0, PA_TANH_C1, PA_TANH_C2};
        mod.cap_in = (float)(2. * in * kLog2e);
        mod.cap_out = (float)to;
        mod.range = (float)std::min(PA_TANH_RANGE / in, 0x1p60);       // the polynomial squares scores
        double f = to * in;
        for (int i = 0; i < 3; ++i, f *= in * in) {
            mod.c[i] = (float)(coef[i] * f);
            // (scale / cap)^5 cap can pass fp32, and 0 times that is NaN: caps that small (1e-11 at a scale of 1 / 8) go
            // without the polynomial
            if (!std::isfinite(mod.c[i])) mod.range = -1.f;
        }
    }
    return d == 64 ? dispatch_scoremod_block<64>(bs, g, pp, n, mql, counters, mod, st)
                   : dispatch_scoremod_block<128>(bs, g, pp, n, mql, counters, mod, st);
}

}  // namespace

extern "C" {

int pa_prefill_scoremod(void *out, const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
                        int max_blocks_per_seq, const int32_t *query_start, const int32_t *context_lens, int num_seqs,
                        int max_query_len, int h_q, int h_kv, int head_dim, int block_size, int num_blocks, float scale,
                        float softcap, const float *alibi_slopes, int window, const int32_t *prefix_lens, int cache_dtype,
                        void *workspace, size_t workspace_bytes, void *stream)
{
    if (workspace == nullptr || workspace_bytes < kPrefillWorkspaceBytes || !aligned16(workspace)) return PA_ERR_WORKSPACE;
    if (num_seqs < 0 || max_query_len < 0 || h_q <= 0 || h_kv <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || window < 0 ||
        h_q % h_kv != 0 || !(scale >= 0x1p-64f) || !valid_scores(scale, softcap) || cache_dtype < PA_CACHE_BF16 ||
        cache_dtype > PA_CACHE_INT8)
        return PA_ERR_INVALID_ARG;
    if (cache_dtype != PA_CACHE_BF16) return PA_ERR_UNSUPPORTED;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size) || !supported_group(h_q / h_kv) ||
        h_kv > 65535 || num_seqs > 65535 || (long long)num_blocks * h_kv * block_size > INT_MAX)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || max_query_len == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !query_start || !context_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    PrefillParams pp{};
    pp.out = static_cast<__nv_bfloat16 *>(out);
    pp.q = static_cast<const __nv_bfloat16 *>(q);
    pp.k_cache = static_cast<const uint8_t *>(k_cache);
    pp.v_cache = static_cast<const uint8_t *>(v_cache);
    pp.block_tables = block_tables;
    pp.query_start = query_start;
    pp.context_lens = context_lens;
    pp.max_blocks_per_seq = max_blocks_per_seq;
    pp.h_q = h_q;
    pp.h_kv = h_kv;
    pp.num_blocks = num_blocks;
    pp.qk_scale = scale * kLog2e;
    const auto run = [&](auto cap, auto bias) {
        return dispatch_scoremod<decltype(cap)::value, decltype(bias)::value>(
            head_dim, block_size, h_q / h_kv, pp, num_seqs, max_query_len, static_cast<int *>(workspace), scale, softcap,
            alibi_slopes, window, prefix_lens, static_cast<cudaStream_t>(stream));
    };
    if (softcap > 0.f) return alibi_slopes ? run(std::true_type{}, std::true_type{}) : run(std::true_type{}, std::false_type{});
    return alibi_slopes ? run(std::false_type{}, std::true_type{}) : run(std::false_type{}, std::false_type{});
}

}  // extern "C"
