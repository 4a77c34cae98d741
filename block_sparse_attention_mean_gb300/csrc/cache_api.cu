// cache_api.cu -- host side of the C ABI in bsa_cache.h: argument checks, the workspace's size and dispatch. Every check
// runs before any launch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "cache_internal.h"
#include "footprint.h"

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 39;  // bytes between tokens or heads: what a tensor map holds

bool valid_heads(int H, int Hk) { return Hk >= 1 && Hk <= 65535 && H >= Hk && H <= 65535 && H % Hk == 0; }

// the [T][heads][d] bf16 tensor t as a footprint and a view; false if it is unusable
bool packed_of(const bsa_packed *t, int64_t T, int heads, int d, Footprint *f, bsa::PackedView *v)
{
    if (!t || !make_footprint(t->ptr, T, t->token, heads, t->head, 1, 0, d, 2, f)) return false;
    if ((T > 1 && (t->token == 0 || f->stride[0] >= kMaxStride)) || (heads > 1 && (t->head == 0 || f->stride[1] >= kMaxStride)))
        return false;
    v->p = static_cast<char *>(t->ptr);
    v->token = f->stride[0];
    v->head = f->stride[1];
    return true;
}

bsa_status check_cache(const bsa_kv_cache *c, Tensors *all, bool written, bsa::CacheView *v)
{
    if (!c) return BSA_ERR_INVALID_ARG;
    if (c->kind != BSA_CACHE_BF16 && c->kind != BSA_CACHE_E4M3) return BSA_ERR_INVALID_ARG;
    if ((c->d != 64 && c->d != 128) || c->heads < 1 || c->heads > 65535 || c->n_pages < 1) return BSA_ERR_SHAPE;
    int shift = 4;
    while (shift <= 8 && 1 << shift != c->page_size) ++shift;
    if (shift > 8) return BSA_ERR_SHAPE;
    const bool e4m3 = c->kind == BSA_CACHE_E4M3;
    // the largest n_pages * heads * page_size * d stays below 2^63 bytes: 2^31 * 2^16 * 2^8 * 2^8
    const int64_t rows = static_cast<int64_t>(c->n_pages) * c->heads * c->page_size;
    if (rows > (int64_t(1) << 46)) return BSA_ERR_SHAPE;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return BSA_ERR_INVALID_ARG;
    if (e4m3 && (!c->k_exp || !c->v_exp || !aligned(c->k_exp, 16) || !aligned(c->v_exp, 16))) return BSA_ERR_INVALID_ARG;
    const int64_t bytes = rows * c->d * (e4m3 ? 1 : 2);
    for (const void *p : {static_cast<const void *>(c->k), static_cast<const void *>(c->v)})
        written ? all->writes(p, bytes) : all->reads(p, bytes);
    if (e4m3)
        for (const void *p : {static_cast<const void *>(c->k_exp), static_cast<const void *>(c->v_exp)})
            written ? all->writes(p, rows) : all->reads(p, rows);
    *v = bsa::CacheView{static_cast<char *>(c->k), static_cast<char *>(c->v), c->k_exp, c->v_exp, c->n_pages, shift, c->heads, e4m3};
    return BSA_OK;
}

bsa_status check_table(const bsa_page_table *t, Tensors *all, bsa::TableView *v)
{
    if (!t || !t->pages || !aligned(t->pages, 4)) return BSA_ERR_INVALID_ARG;
    if (t->B < 1 || t->width < 1) return BSA_ERR_SHAPE;
    if (t->B > 1 && (t->stride < t->width || t->stride > (INT64_MAX >> 34))) return BSA_ERR_INVALID_ARG;
    const int64_t stride = t->B > 1 ? t->stride : t->width;
    all->reads(t->pages, 4 * (static_cast<int64_t>(t->B - 1) * stride + t->width));
    *v = bsa::TableView{t->pages, stride, t->B, t->width};
    return BSA_OK;
}

// int32 [n], required
bool reads_ints(const int32_t *p, int64_t n, Tensors *all)
{
    if (!p || !aligned(p, 4)) return false;
    all->reads(p, 4 * n);
    return true;
}

// the workspace: present, aligned, of that size, and clear of everything else (it counts as an output)
bsa_status check_workspace(void *ws, size_t bytes, size_t need, Tensors *all)
{
    if (!ws || !aligned(ws, 256) || bytes < need) return BSA_ERR_WORKSPACE;
    all->writes(ws, static_cast<int64_t>(need));
    return BSA_OK;
}

bool scale_of(float scale, int d, float *out)
{
    if (!std::isfinite(scale) || scale < 0.0f) return false;
    *out = scale > 0.0f ? scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    return true;
}

// what bsa_cache_write and bsa_cache_read have in common
bsa_status check_rows(const bsa_kv_cache *cache, const bsa_packed *k, const bsa_packed *v, int dt, int T,
                      const bsa_page_table *table, void *workspace, size_t workspace_bytes, bool write, Tensors *all,
                      bsa::CacheRowsArgs *a)
{
    bsa_status s = check_cache(cache, all, write, &a->cache);
    if (s != BSA_OK) return s;
    if (dt != BSA_BF16) return BSA_ERR_DTYPE;
    if (T < 0) return BSA_ERR_SHAPE;
    s = check_table(table, all, &a->table);
    if (s != BSA_OK) return s;
    s = check_workspace(workspace, workspace_bytes, bsa::kCacheScratch, all);
    if (s != BSA_OK) return s;
    a->T = T;
    a->d = cache->d;
    a->err = static_cast<uint32_t *>(workspace);
    if (T == 0) return BSA_OK;
    Footprint f[2];
    if (!packed_of(k, T, cache->heads, cache->d, &f[0], &a->k) || !packed_of(v, T, cache->heads, cache->d, &f[1], &a->v))
        return BSA_ERR_INVALID_ARG;
    for (const Footprint &x : f) {
        if (write) {
            all->in[all->n_in++] = x;
        } else {
            all->may_be[all->n_out] = 0;
            all->out[all->n_out++] = x;
        }
    }
    return BSA_OK;
}

}  // namespace

extern "C" {

bsa_status bsa_cache_write(const bsa_kv_cache *cache, const bsa_packed *k, const bsa_packed *v, int dt, int T,
                           const bsa_page_table *table, const int32_t *kv_lens, const int32_t *cu, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    Tensors all;
    bsa::CacheRowsArgs a{};
    const bsa_status s = check_rows(cache, k, v, dt, T, table, workspace, workspace_bytes, true, &all, &a);
    if (s != BSA_OK) return s;
    if (!reads_ints(kv_lens, table->B, &all)) return BSA_ERR_INVALID_ARG;
    if (cu ? !reads_ints(cu, static_cast<int64_t>(table->B) + 1, &all) : T != table->B) return cu ? BSA_ERR_INVALID_ARG : BSA_ERR_SHAPE;
    if (!all.check()) return BSA_ERR_INVALID_ARG;
    a.kv_lens = kv_lens;
    a.cu = cu;
    return bsa::launch_cache_write(a, static_cast<cudaStream_t>(stream));
}

bsa_status bsa_cache_read(const bsa_kv_cache *cache, const bsa_page_table *table, const int32_t *cu, const bsa_packed *k,
                          const bsa_packed *v, int dt, int T, void *workspace, size_t workspace_bytes, void *stream)
{
    Tensors all;
    bsa::CacheRowsArgs a{};
    const bsa_status s = check_rows(cache, k, v, dt, T, table, workspace, workspace_bytes, false, &all, &a);
    if (s != BSA_OK) return s;
    if (!reads_ints(cu, static_cast<int64_t>(table->B) + 1, &all)) return BSA_ERR_INVALID_ARG;
    if (!all.check()) return BSA_ERR_INVALID_ARG;
    a.cu = cu;
    return bsa::launch_cache_read(a, static_cast<cudaStream_t>(stream));
}

bsa_status bsa_cache_attention(const bsa_kv_cache *cache, const bsa_packed *q, int dt, int H, const bsa_page_table *table,
                               const int32_t *kv_lens, float scale, const bsa_packed *O, float *LSE, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    Tensors all;
    bsa::CacheAttentionArgs a{};
    bsa_status s = check_cache(cache, &all, false, &a.cache);
    if (s != BSA_OK) return s;
    if (dt != BSA_BF16) return BSA_ERR_DTYPE;
    if (!valid_heads(H, cache->heads)) return BSA_ERR_SHAPE;
    s = check_table(table, &all, &a.table);
    if (s != BSA_OK) return s;
    Footprint fq, fo;
    if (!packed_of(q, table->B, H, cache->d, &fq, &a.q) || !packed_of(O, table->B, H, cache->d, &fo, &a.o)) return BSA_ERR_INVALID_ARG;
    all.in[all.n_in++] = fq;
    all.may_be[all.n_out] = 0;
    all.out[all.n_out++] = fo;
    if (LSE && !aligned(LSE, 4)) return BSA_ERR_INVALID_ARG;
    all.writes(LSE, 4 * static_cast<int64_t>(table->B) * H);
    if (!reads_ints(kv_lens, table->B, &all) || !scale_of(scale, cache->d, &a.scale)) return BSA_ERR_INVALID_ARG;
    s = check_workspace(workspace, workspace_bytes, bsa::kCacheScratch + bsa::cache_attention_workspace(cache->d), &all);
    if (s != BSA_OK) return s;
    if (!all.check()) return BSA_ERR_INVALID_ARG;
    // units of 64 tokens of all key heads and chunks of query heads are counted in 31 bits
    const int64_t chunks = static_cast<int64_t>(cache->heads) * ((H / cache->heads + 7) / 8);
    const double tokens = static_cast<double>(table->B) * table->width * cache->page_size;
    if ((tokens / 64 + 3.0 * table->B) * chunks > INT32_MAX) return BSA_ERR_SHAPE;
    a.kv_lens = kv_lens;
    a.lse = LSE;
    a.H = H;
    a.d = cache->d;
    a.ws = static_cast<char *>(workspace);
    return bsa::launch_cache_attention(a, static_cast<cudaStream_t>(stream));
}

// shapes of a prompt call or of its workspace
static bsa_status check_prompt_shape(int T, int B, int H, int Hk, int d)
{
    if ((d != 64 && d != 128) || T < 0 || B < 1 || !valid_heads(H, Hk) || H / Hk > 128) return BSA_ERR_SHAPE;
    // items (tiles of floor(128 / g) tokens) of all key heads are counted in 31 bits
    const int64_t items = T / (128 / (H / Hk)) + static_cast<int64_t>(B);
    return items * Hk <= INT32_MAX ? BSA_OK : BSA_ERR_SHAPE;
}

bsa_status bsa_prompt_attention(const bsa_packed *q, const bsa_packed *k, const bsa_packed *v, int dt, int T_q, int T_k, int B,
                                int H, int Hk, int d, const int32_t *cu_q, const int32_t *cu_k, int causal, float scale,
                                const bsa_packed *O, float *LSE, void *workspace, size_t workspace_bytes, void *stream)
{
    bsa_status s = check_prompt_shape(T_q, B, H, Hk, d);
    if (s != BSA_OK) return s;
    if (T_k < 0) return BSA_ERR_SHAPE;
    if (dt != BSA_BF16) return BSA_ERR_DTYPE;
    Tensors all;
    bsa::PromptArgs a{};
    if (!reads_ints(cu_q, static_cast<int64_t>(B) + 1, &all) || !reads_ints(cu_k, static_cast<int64_t>(B) + 1, &all)) return BSA_ERR_INVALID_ARG;
    if (!scale_of(scale, d, &a.scale)) return BSA_ERR_INVALID_ARG;
    if (LSE && !aligned(LSE, 4)) return BSA_ERR_INVALID_ARG;
    s = check_workspace(workspace, workspace_bytes, bsa::kCacheScratch + bsa::prompt_workspace(T_q, B, H, Hk, d), &all);
    if (s != BSA_OK) return s;
    if (T_q == 0) return BSA_OK;
    Footprint f[4];
    if (!packed_of(q, T_q, H, d, &f[0], &a.q) || !packed_of(O, T_q, H, d, &f[3], &a.o)) return BSA_ERR_INVALID_ARG;
    all.in[all.n_in++] = f[0];
    if (T_k > 0) {
        if (!packed_of(k, T_k, Hk, d, &f[1], &a.k) || !packed_of(v, T_k, Hk, d, &f[2], &a.v)) return BSA_ERR_INVALID_ARG;
        all.in[all.n_in++] = f[1];
        all.in[all.n_in++] = f[2];
    }
    all.may_be[all.n_out] = 0;
    all.out[all.n_out++] = f[3];
    all.writes(LSE, 4 * static_cast<int64_t>(T_q) * H);
    if (!all.check()) return BSA_ERR_INVALID_ARG;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.lse = LSE;
    a.Tq = T_q, a.Tk = T_k, a.B = B, a.H = H, a.Hk = Hk, a.d = d, a.causal = causal != 0;
    a.ws = static_cast<char *>(workspace);
    bsa::current_debug_config(&a.dbg_flags, &a.wait_limit_ns);
    return bsa::launch_prompt_attention(a, static_cast<cudaStream_t>(stream));
}

bsa_status bsa_cache_workspace_size(int T, int B, int H, int Hk, int d, size_t *bytes)
{
    if (!bytes) return BSA_ERR_INVALID_ARG;
    const bsa_status s = check_prompt_shape(T, B, H, Hk, d);
    if (s != BSA_OK) return s;
    const size_t one = bsa::cache_attention_workspace(d), whole = bsa::prompt_workspace(T, B, H, Hk, d);
    *bytes = bsa::kCacheScratch + (one > whole ? one : whole);
    return BSA_OK;
}

}  // extern "C"
