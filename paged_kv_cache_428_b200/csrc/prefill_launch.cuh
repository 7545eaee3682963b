// prefill_launch.cuh -- host side of the tcgen05 prefill kernel (prefill_tc.cuh): launch on either schedule.
#pragma once

#include <algorithm>
#include <climits>

#include "host_launch.cuh"
#include "prefill_tc.cuh"

namespace pa {
namespace {

// pa_prefill_ws: the claim counter and the finished-CTA counter, padded
constexpr size_t kPrefillWorkspaceBytes = 256;

template <int D, int BS, int G, class Mod = PrefillPlain>
int launch_prefill_tc(const PrefillParams &pp, int num_seqs, int max_query_len, int *counters, cudaStream_t st,
                      const Mod &mod = Mod{})
{
    using C = PrefillTcConfig<D, BS, G>;
    static std::atomic<unsigned long long> smem_set{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(smem_set.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(paged_prefill_tc_kernel<D, BS, G, Mod>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::SMEM) != cudaSuccess)
            return PA_ERR_CUDA;
        smem_set.fetch_or(bit, std::memory_order_release);
    }
    CUtensorMap mk, mv;
    int rc = cached_cache_map(&mk, pp.k_cache, pp.num_blocks, pp.h_kv, BS, D);
    if (rc == PA_OK) rc = cached_cache_map(&mv, pp.v_cache, pp.num_blocks, pp.h_kv, BS, D);
    if (rc != PA_OK) return rc;
    const int pairs = (prefill_tiles<C::TQ>(max_query_len) + C::NQ - 1) / C::NQ;
    const long long items = (long long)pairs * pp.h_kv * num_seqs;
    if (items > INT_MAX) return PA_ERR_UNSUPPORTED;
    PrefillSched sc{};
    sc.counters = counters;
    sc.num_seqs = num_seqs;
    sc.pairs_max = pairs;
    sc.total_items = (int)items;
    CUtensorMap mq;
    sc.q_tma = make_q_map(&mq, pp.q, pp.h_q, D, G, (long long)num_seqs * max_query_len) == PA_OK;
    if (!sc.q_tma) std::memset(&mq, 0, sizeof(mq));
    dim3 grid(pairs, pp.h_kv, num_seqs);                      // one CTA per item
    if (counters) {
        const int sms = sm_count();                              // one CTA per SM, claiming items
        if (sms <= 0) return PA_ERR_CUDA;
        grid = dim3((unsigned)std::min<long long>(sms, items));
    }
    paged_prefill_tc_kernel<D, BS, G, Mod><<<grid, C::THREADS, C::SMEM, st>>>(pp, sc, mk, mv, mq, mod);
    return launch_status();
}

}  // namespace
}  // namespace pa
