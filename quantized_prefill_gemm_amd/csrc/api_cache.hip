// C ABI of the operators over a paged cache of keys and values (declared in include/qpg.h): argument
// validation, device check, then the kernel launches. Nothing here allocates, frees, prints or synchronises.
#include <math.h>

#include "qpg_cache.h"

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;       // 256 threads to a row, < 2^32 threads in a launch
constexpr int64_t kMaxSequences = (int64_t)1 << 20;
constexpr int64_t kMaxLength = (int64_t)1 << 30;     // a token's place plus a tile is an int
constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxWords = 1024;
constexpr int64_t kMaxInt = (int64_t)1 << 31;
constexpr int64_t kMaxGroups = (int64_t)1 << 24;     // an attention's workgroups, which it divides as f32
constexpr int64_t kMaxThreads = (int64_t)1 << 32;    // of a launch

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool type_ok(int t) { return t == QPG_F32 || t == QPG_F16 || t == QPG_BF16; }
int status_of(hipError_t e) { return e == hipSuccess ? QPG_OK : QPG_EHIP; }

bool dim_ok(int64_t dim) { return dim >= 8 && dim <= 256 && dim % 8 == 0; }

bool cache_ok(const qpg_cache* c)
{
    if (!c || !c->k || !c->v || (c->type != QPG_F16 && c->type != QPG_BF16)) return false;
    if (c->pages < 1 || c->pages >= kMaxInt || c->heads < 1 || c->heads > kMaxHeads || !dim_ok(c->dim)) return false;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256) return false;
    const int64_t block = c->heads * c->page * c->dim;
    return c->k_stride >= block && c->v_stride >= block && c->k_stride % 8 == 0 && c->v_stride % 8 == 0 &&
           c->k_stride <= kMaxStride && c->v_stride <= kMaxStride;
}

bool batch_ok(const qpg_batch* b, int64_t page)
{
    if (!b || !b->table || !b->lens || !b->offsets) return false;
    return b->B >= 1 && b->B <= kMaxSequences && b->T >= 1 && b->T < kMaxRows && b->width >= 1 && b->width <= kMaxLength / page;
}

bool batch_aligned(const qpg_batch* b) { return aligned(b->table, 4) && aligned(b->lens, 4) && aligned(b->offsets, 4); }

bool heads_ok(int64_t T, int64_t heads, int64_t kv)
{
    return heads >= kv && heads <= kMaxHeads && heads % kv == 0 && T < kMaxInt / heads;
}

int attention(const qpg_cache* cache, const qpg_batch* batch, const qpg_scores* scores, const void* q, int64_t heads,
              const int64_t* tree, int64_t words, const int32_t* positions, void* y, int y_type, void* ws, hipStream_t s)
{
    if (!cache_ok(cache) || !batch_ok(batch, cache->page) || !scores || !q || !y || !type_ok(y_type)) return QPG_EINVAL;
    if (!heads_ok(batch->T, heads, cache->heads)) return QPG_EINVAL;
    if (!(scores->scale > 0.0f) || !isfinite(scores->scale) || !(scores->cap >= 0.0f) || !isfinite(scores->cap) ||
        scores->window < 0)
        return QPG_EINVAL;
    // the kernel's factors, in powers of two
    if (!isfinite(1.5f * scores->scale) || !isfinite(3.0f * scores->cap) ||
        (scores->cap > 0.0f && !isfinite(3.0f * scores->scale / scores->cap)))
        return QPG_EINVAL;
    int64_t threads;
    if (qpg_cache_attention_grid(batch->T, batch->B, heads, cache->heads, cache->dim, batch->width * cache->page, &threads) >=
            kMaxGroups ||
        threads >= kMaxThreads)
        return QPG_EINVAL;
    if (!ws && qpg_cache_attention_bytes(batch->T, batch->B, heads, cache->heads, cache->dim, batch->width * cache->page))
        return QPG_EINVAL;
    if (!aligned(cache->k, 16) || !aligned(cache->v, 16) || !aligned(q, 16) || !aligned(y, 16) || !aligned(ws, 16) ||
        !batch_aligned(batch) || !aligned(scores->slopes, 4) || !aligned(scores->prefix, 4) || !aligned(tree, 8) ||
        !aligned(positions, 4))
        return QPG_EALIGN;
    const int rc = qpg_check_device();
    if (rc != QPG_OK) return rc;
    return status_of(qpg_launch_cache_attention(*cache, *batch, *scores, q, heads, tree, words, positions, y, y_type, ws, s));
}

}  // namespace

extern "C" {

int cache_append(const qpg_cache* cache, const qpg_batch* batch, const void* q, const void* k, const void* v, int type,
                 int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t heads, const int32_t* positions,
                 const float* freqs, int64_t rot, int adjacent, const float* q_norm, const float* k_norm, float eps,
                 void* y, qpg_stream_t stream)
{
    if (!cache_ok(cache) || !batch_ok(batch, cache->page) || !k || !v || !type_ok(type)) return QPG_EINVAL;
    if (heads != 0 && (!q || !y || !heads_ok(batch->T, heads, cache->heads))) return QPG_EINVAL;
    if (rot < 0 || rot > cache->dim || rot % 8 || (rot && !freqs) || !(eps >= 0.0f) || !isfinite(eps)) return QPG_EINVAL;
    const int64_t kv = cache->heads * cache->dim;
    if (batch->T > 1 && (k_stride < kv || v_stride < kv || q_stride < heads * cache->dim)) return QPG_EINVAL;
    if (q_stride < 0 || k_stride < 0 || v_stride < 0 || q_stride > kMaxStride || k_stride > kMaxStride ||
        v_stride > kMaxStride)
        return QPG_EINVAL;
    const uintptr_t a = qpg::type_bytes(type);
    if (!aligned(cache->k, 16) || !aligned(cache->v, 16) || !aligned(y, 16) || !aligned(q, a) || !aligned(k, a) ||
        !aligned(v, a) || !batch_aligned(batch) || !aligned(positions, 4) || !aligned(freqs, 4) || !aligned(q_norm, 4) ||
        !aligned(k_norm, 4))
        return QPG_EALIGN;
    const int rc = qpg_check_device();
    if (rc != QPG_OK) return rc;
    return status_of(qpg_launch_cache_append(*cache, *batch, q, k, v, type, q_stride, k_stride, v_stride, heads, positions,
                                             freqs, rot, adjacent, q_norm, k_norm, eps, y,
                                             reinterpret_cast<hipStream_t>(stream)));
}

size_t qpg_cache_attention_bytes(int64_t T, int64_t B, int64_t heads, int64_t cache_heads, int64_t dim, int64_t length)
{
    if (T < 1 || T >= kMaxRows || B < 1 || B > kMaxSequences || cache_heads < 1 || cache_heads > kMaxHeads ||
        !heads_ok(T, heads, cache_heads) || !dim_ok(dim) || length < 1 || length > kMaxLength)
        return 0;
    const int splits = qpg_cache_attention_splits(T, B, heads, cache_heads, dim, length);
    return splits > 1 ? (size_t)splits * (size_t)(T * heads) * (size_t)(dim * 4 + 8) : 0;
}

int cache_attention(const qpg_cache* cache, const qpg_batch* batch, const qpg_scores* scores, const void* q, int64_t heads,
                    void* y, int y_type, void* ws, qpg_stream_t stream)
{
    return attention(cache, batch, scores, q, heads, nullptr, 0, nullptr, y, y_type, ws,
                     reinterpret_cast<hipStream_t>(stream));
}

int cache_attention_tree(const qpg_cache* cache, const qpg_batch* batch, const qpg_scores* scores, const void* q,
                         int64_t heads, const int64_t* tree, int64_t words, const int32_t* positions, void* y, int y_type,
                         void* ws, qpg_stream_t stream)
{
    if (!tree || !positions || words < 1 || words > kMaxWords || !scores || scores->prefix) return QPG_EINVAL;
    return attention(cache, batch, scores, q, heads, tree, words, positions, y, y_type, ws,
                     reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
