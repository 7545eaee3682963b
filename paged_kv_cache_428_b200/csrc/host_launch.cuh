// host_launch.cuh -- host-side helpers shared by the files that hold the C-ABI device calls:
// argument predicates, launches, tensor maps of the caches, dispatch on the head group.
#pragma once

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <type_traits>
#include <utility>

#include "common.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int launch_status()
{
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Launch `kernel`; with `pdl`, as a programmatic dependent of the grid before it on the stream
// (it may start while that grid runs; the kernel waits for it where it reads its results).
template <typename... KArgs, typename... Args>
int launch_ex(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool pdl,
              Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

bool supported_head_dim(int d) { return d == 64 || d == 128; }
bool supported_block_size(int bs) { return bs == 16 || bs == 32 || bs == 64; }
bool supported_group(int g) { return g == 1 || g == 2 || g == 4 || g == 8; }

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

bool env_flag(const char *name)
{
    const char *e = std::getenv(name);
    return e != nullptr && std::strcmp(e, "1") == 0;
}

// ---- tensor maps of the bf16 caches (2-D: rows of head_dim elements, 128B swizzle) -----
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled()
{
    static EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

// The cache viewed as [num_blocks * h_kv * block_size rows][head_dim] elements.  bf16: a box is
// 64 elements (128 bytes) by block_size rows, swizzled in 128-byte atoms (two boxes per row at
// head_dim 128).  One-byte codes: a box is a whole row (head_dim bytes) by block_size rows,
// 128-byte swizzle for 128-byte rows, 64-byte swizzle for 64-byte rows.
// box_rows: rows of one box (block_size for one KV head's tile; h_kv * block_size for a whole block).
int make_cache_map(CUtensorMap *map, const void *cache, int num_blocks, int h_kv, int block_size, int head_dim,
                   int elem_bytes, int box_rows)
{
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return PA_ERR_CUDA;
    const cuuint64_t dims[2] = {(cuuint64_t)head_dim, (cuuint64_t)num_blocks * h_kv * block_size};
    const cuuint64_t strides[1] = {(cuuint64_t)head_dim * elem_bytes};
    const cuuint32_t box[2] = {elem_bytes == 2 ? 64u : (cuuint32_t)head_dim, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType dt = elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUtensorMapSwizzle sw = (elem_bytes == 1 && head_dim == 64) ? CU_TENSOR_MAP_SWIZZLE_64B
                                                                       : CU_TENSOR_MAP_SWIZZLE_128B;
    const CUresult r = enc(map, dt, 2, const_cast<void *>(cache), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PA_OK : PA_ERR_CUDA;
}

// The prefill queries q [tokens][h_q][head_dim] as a 3-D map (head_dim, h_q, tokens) whose box is
// one query tile: 64 elements (128 bytes, 128-byte swizzle) x g heads x 128 / g tokens, landing as
// the swizzled Q tile the S products read.  `tokens` only bounds the coordinates: the kernel loads
// only tiles that lie inside their sequence's chunk.  q must be 16-byte aligned with 16-byte
// strides, else the encoding fails and the kernel copies every tile itself.
int make_q_map(CUtensorMap *map, const void *q, int h_q, int head_dim, int g, long long tokens)
{
    EncodeTiledFn enc = encode_tiled();
    if (!enc || tokens <= 0 || 128 % g != 0) return PA_ERR_CUDA;
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)h_q, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)h_q * head_dim * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)g, (cuuint32_t)(128 / g)};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PA_OK : PA_ERR_CUDA;
}

// Encoded maps of recently used caches (per host thread): a decode step reuses the same
// cache tensors call after call, and encoding costs host time on every launch otherwise.
struct CachedMap {
    const void *base = nullptr;
    int num_blocks = 0, h_kv = 0, block_size = 0, head_dim = 0, elem_bytes = 0, box_rows = 0;
    CUtensorMap map;
};

int cached_cache_map(CUtensorMap *map, const void *cache, int num_blocks, int h_kv, int block_size, int head_dim,
                     int elem_bytes = 2, int box_rows = 0)
{
    constexpr int kSlots = 8;
    static thread_local CachedMap slots[kSlots];
    static thread_local int next = 0;
    if (box_rows <= 0) box_rows = block_size;
    for (const CachedMap &c : slots) {
        if (c.base == cache && c.num_blocks == num_blocks && c.h_kv == h_kv && c.block_size == block_size &&
            c.head_dim == head_dim && c.elem_bytes == elem_bytes && c.box_rows == box_rows) {
            *map = c.map;
            return PA_OK;
        }
    }
    CachedMap &c = slots[next];
    next = (next + 1) % kSlots;
    const int rc = make_cache_map(&c.map, cache, num_blocks, h_kv, block_size, head_dim, elem_bytes, box_rows);
    if (rc != PA_OK) {
        c.base = nullptr;
        return rc;
    }
    c.base = cache;
    c.num_blocks = num_blocks;
    c.h_kv = h_kv;
    c.block_size = block_size;
    c.head_dim = head_dim;
    c.elem_bytes = elem_bytes;
    c.box_rows = box_rows;
    *map = c.map;
    return PA_OK;
}

struct SmCount {
    int dev = -1, count = 0;
};

int sm_count()
{
    static thread_local SmCount cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (cache.dev != dev) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
        cache.dev = dev;
        cache.count = n;
    }
    return cache.count;
}

template <class F>
int switch_group(int g, F &&f)
{
    switch (g) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    default: return PA_ERR_UNSUPPORTED;
    }
}

// Raise `kernel`'s dynamic shared memory limit on the current device, once per kernel and device
// (`done`: a static of the caller, one bit per device).
template <class K>
int allow_smem(K *kernel, int bytes, std::atomic<unsigned long long> &done)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
            return PA_ERR_CUDA;
        done.fetch_or(bit, std::memory_order_release);
    }
    return PA_OK;
}

// The error word of this translation unit's kernels: its bits are added to *flags, and cleared on
// request.  Each .cu file has a word of its own; pa_device_errors puts them together.
int collect_device_errors(unsigned int *flags, int clear)
{
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_errors, sizeof(v)) != cudaSuccess) return PA_ERR_CUDA;
    *flags |= v;
    if (clear && v != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_device_errors, &zero, sizeof(zero)) != cudaSuccess) return PA_ERR_CUDA;
    }
    return PA_OK;
}

// Scores are multiplied by scale * log2(e), and by 2 / cap more inside the tanh, and come out as cap * log2(e): all
// of these have to be numbers in fp32 (infinity times a score of 0 is NaN).  cap: 0 = none, else at least 2^-64.
bool valid_scores(float scale, float cap)
{
    if (!std::isfinite(scale * kLog2e) || !std::isfinite(cap * kLog2e) || !(cap == 0.f || cap >= 0x1p-64f)) return false;
    return cap == 0.f || std::isfinite(2.f * (scale * kLog2e) / cap);
}

}  // namespace

int block_scales_errors(unsigned int *flags, int clear);    // pa_block_scales.cu
int evict_errors(unsigned int *flags, int clear);           // pa_evict.cu
int scoremod_errors(unsigned int *flags, int clear);        // pa_scoremod.cu
int prefill_scoremod_errors(unsigned int *flags, int clear);    // pa_prefill_scoremod.cu

}  // namespace pa
