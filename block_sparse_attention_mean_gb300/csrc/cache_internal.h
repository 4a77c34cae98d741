// cache_internal.h -- declarations shared by the host checks (cache_api.cu) and the kernels of attention over packed
// sequences and paged caches (cache_rows.cu, cache_attention.cu, prompt_attention.cu). Not part of the public C ABI.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/bsa_cache.h"
#include "internal.h"

namespace bsa {

// Workspace of the four calls: the header of internal.h (its first word is the error word), then the tickets of
// bsa_cache_attention, which every call leaves zero, then whatever the call at hand keeps there.
constexpr int kCacheMaxCtas = 640;  // CTAs of a bsa_cache_attention launch
constexpr size_t kCacheCounter = kWsHeader - 2 * sizeof(uint32_t);  // two words of bsa_prompt_attention, zero between calls too
constexpr size_t kCacheTickets = kWsHeader;
constexpr size_t kCacheScratch = BSA_CACHE_ROWS_WORKSPACE;
static_assert(kCacheTickets + sizeof(uint32_t) * 3 * kCacheMaxCtas <= kCacheScratch, "room for the tickets");

// Lets a kernel use `bytes` of dynamic shared memory on the current device; `ready` remembers the devices where it may.
template <typename Kernel>
inline bool allow_shared_memory(Kernel kern, int bytes, std::atomic<uint64_t> &ready)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (ready.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    ready.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

struct PackedView {
    char *p;
    int64_t token, head;  // bytes
};

struct CacheView {
    char *k, *v;
    uint8_t *k_exp, *v_exp;
    int n_pages, page_shift, heads;
    bool e4m3;
};

struct TableView {
    const int32_t *pages;
    int64_t stride;
    int B, width;
};

struct CacheRowsArgs {
    CacheView cache;
    TableView table;
    PackedView k, v;
    const int32_t *kv_lens, *cu;  // cu nullptr: one token per sequence (write)
    int T, d;
    uint32_t *err;
};
bsa_status launch_cache_write(const CacheRowsArgs &a, cudaStream_t st);
bsa_status launch_cache_read(const CacheRowsArgs &a, cudaStream_t st);

struct CacheAttentionArgs {
    CacheView cache;
    TableView table;
    PackedView q, o;
    const int32_t *kv_lens;
    float *lse;
    int H, d;
    float scale;
    char *ws;
};
size_t cache_attention_workspace(int d);
bsa_status launch_cache_attention(const CacheAttentionArgs &a, cudaStream_t st);

struct PromptArgs {
    PackedView q, k, v, o;
    const int32_t *cu_q, *cu_k;
    float *lse;
    int Tq, Tk, B, H, Hk, d, causal;
    float scale;
    char *ws;
    uint64_t wait_limit_ns;
    uint32_t dbg_flags;
};
size_t prompt_workspace(int T, int B, int H, int Hk, int d);
bsa_status launch_prompt_attention(const PromptArgs &a, cudaStream_t st);

}  // namespace bsa
