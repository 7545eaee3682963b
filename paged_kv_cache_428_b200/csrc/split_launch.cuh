// split_launch.cuh -- host side of the split decode (decode_split.cuh): workspace, checks, launch.
#pragma once

#include <algorithm>
#include <climits>

#include "decode_split.cuh"
#include "host_launch.cuh"

namespace pa {
namespace {

// Workspace: [kSplitMaxGroups counters][partial (m, l)][partial o][lse][what the call adds].  The counters have
// one place whatever the call's sizes are, so calls of different shapes, and of different kinds, can take
// turns on one workspace.
struct SplitLayout {
    size_t ml = 0, o = 0, lse = 0, end = 0;
};

constexpr size_t kSplitCounterBytes = (size_t)kSplitMaxGroups * sizeof(int);

// CTAs that a step of these sizes can use at most (known without the device, so that the workspace's size
// is too).
int split_ctas_bound(int num_seqs, int h_kv, int span)
{
    const long long pieces = (long long)span / kSplitMinTokens + 2;
    return (int)std::min<long long>(kSplitMaxCtas, pieces * num_seqs * h_kv);
}

SplitLayout split_layout(int num_seqs, int h_q, int h_kv, int head_dim, int span)
{
    const size_t slots = (size_t)2 * split_ctas_bound(num_seqs, h_kv, span) * (h_q / h_kv);
    SplitLayout L;
    L.ml = kSplitCounterBytes;
    L.o = L.ml + round256(slots * 2 * sizeof(float));
    L.lse = L.o + round256(slots * head_dim * sizeof(float));
    L.end = L.lse + round256((size_t)num_seqs * h_q * sizeof(float));
    return L;
}

bool split_sizes_ok(int num_seqs, int h_q, int h_kv, int head_dim, int max_context_len)
{
    return num_seqs > 0 && h_kv > 0 && h_q > 0 && h_q % h_kv == 0 && head_dim > 0 && max_context_len >= 0;
}

// Arguments that the split decodes share.
struct SplitCall {
    void *out;
    const void *q, *k_cache, *v_cache;
    const int32_t *block_tables;
    int max_blocks_per_seq;
    const int32_t *context_lens;
    int num_seqs, max_context_len, h_q, h_kv, head_dim, block_size, num_blocks;
    float scale;
    int window;
    void *workspace;
    size_t workspace_bytes;
    void *stream;
};

// PA_OK and the kernel's parameters, or what is wrong with the arguments.  `more`: bytes that the call needs
// behind the layout.
int split_prepare(SplitParams &p, const SplitCall &c, size_t more)
{
    if (c.num_seqs < 0 || c.max_context_len < 0 || c.h_q <= 0 || c.h_kv <= 0 || c.num_blocks <= 0 ||
        c.max_blocks_per_seq <= 0 || c.window < 0 || c.h_q % c.h_kv != 0 || !std::isfinite(c.scale * kLog2e))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(c.head_dim) || !supported_block_size(c.block_size) || !supported_group(c.h_q / c.h_kv))
        return PA_ERR_UNSUPPORTED;
    if (c.num_seqs == 0) return PA_OK;
    // the prefix sums of the launch's blocks and the tensor-map rows are 32-bit
    if (c.num_seqs > kSplitMaxSeqs || (long long)c.num_seqs * c.h_kv > kSplitMaxGroups ||
        (long long)c.num_seqs * ((long long)c.max_blocks_per_seq + 1) > INT_MAX ||
        (long long)c.num_blocks * c.h_kv * c.block_size > INT_MAX)
        return PA_ERR_UNSUPPORTED;
    if (!c.out || !c.q || !c.k_cache || !c.v_cache || !c.block_tables || !c.context_lens) return PA_ERR_INVALID_ARG;
    if (!aligned16(c.out) || !aligned16(c.q) || !aligned16(c.k_cache) || !aligned16(c.v_cache)) return PA_ERR_INVALID_ARG;
    const int span = c.window > 0 ? std::min(c.window, c.max_context_len) : c.max_context_len;
    const SplitLayout lay = split_layout(c.num_seqs, c.h_q, c.h_kv, c.head_dim, span);
    if (c.workspace == nullptr || !aligned16(c.workspace) || c.workspace_bytes < lay.end + more) return PA_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(c.workspace);
    p.out = static_cast<__nv_bfloat16 *>(c.out);
    p.q = static_cast<const __nv_bfloat16 *>(c.q);
    p.block_tables = c.block_tables;
    p.context_lens = c.context_lens;
    p.counters = reinterpret_cast<int *>(ws);
    p.part_ml = reinterpret_cast<float *>(ws + lay.ml);
    p.part_o = reinterpret_cast<float *>(ws + lay.o);
    p.lse = nullptr;
    p.max_blocks_per_seq = c.max_blocks_per_seq;
    p.num_seqs = c.num_seqs;
    p.h_q = c.h_q;
    p.h_kv = c.h_kv;
    p.num_blocks = c.num_blocks;
    p.window = c.window;
    p.qk_scale = c.scale * kLog2e;
    return PA_OK;
}

template <int D, int BS, int G, int QT, class Ext>
int split_launch_one(const SplitCall &c, const SplitParams &p, const typename Ext::Args &args)
{
    using SC = SplitConfig<D, BS, G, QT>;
    auto *kernel = paged_decode_split_kernel<D, BS, G, QT, Ext>;
    static std::atomic<unsigned long long> smem_set{0};
    int rc = allow_smem(kernel, SC::smem_bytes(kSplitMaxSeqs), smem_set);
    if (rc != PA_OK) return rc;
    const int smem = SC::smem_bytes(c.num_seqs), sms = sm_count();
    static thread_local int known_smem = -1, known = 0;       // the last answer (the GPUs of a host are alike)
    int per_sm = known;
    if (sms < 1) return PA_ERR_CUDA;
    if (known_smem != smem) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, SC::THREADS, smem) != cudaSuccess || per_sm < 1)
            return PA_ERR_CUDA;
        known_smem = smem;
        known = per_sm;
    }
    const int span = c.window > 0 ? std::min(c.window, c.max_context_len) : c.max_context_len;
    const int ctas = std::min(split_ctas_bound(c.num_seqs, c.h_kv, span), per_sm * sms);
    CUtensorMap mk, mv;
    rc = cached_cache_map(&mk, c.k_cache, c.num_blocks, c.h_kv, BS, D, QT == 0 ? 2 : 1);
    if (rc == PA_OK) rc = cached_cache_map(&mv, c.v_cache, c.num_blocks, c.h_kv, BS, D, QT == 0 ? 2 : 1);
    if (rc != PA_OK) return rc;
    return launch_ex(kernel, dim3(ctas), dim3(SC::THREADS), (size_t)smem, static_cast<cudaStream_t>(c.stream), false, p, args,
                     mk, mv);
}

template <int D, int QT, class Ext>
int split_launch_dim(const SplitCall &c, const SplitParams &p, const typename Ext::Args &args)
{
    return switch_group(c.h_q / c.h_kv, [&](auto gc) {
        constexpr int G = decltype(gc)::value;
        switch (c.block_size) {
        case 16: return split_launch_one<D, 16, G, QT, Ext>(c, p, args);
        case 32: return split_launch_one<D, 32, G, QT, Ext>(c, p, args);
        case 64: return split_launch_one<D, 64, G, QT, Ext>(c, p, args);
        default: return PA_ERR_UNSUPPORTED;
        }
    });
}

template <int QT, class Ext>
int split_launch(const SplitCall &c, const SplitParams &p, const typename Ext::Args &args)
{
    return c.head_dim == 64 ? split_launch_dim<64, QT, Ext>(c, p, args) : split_launch_dim<128, QT, Ext>(c, p, args);
}

}  // namespace
}  // namespace pa
