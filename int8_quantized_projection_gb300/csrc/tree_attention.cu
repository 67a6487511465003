// tree_attention.cu -- the entry points of q8_tree_attention: checks, the
// workspace's layout and the choice of the kernel.
#include <cfloat>
#include <cmath>

#include "attn_common.cuh"

namespace {

using q8::AttnArgs;
using q8::kAttnCtas;

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Workspace {
    size_t ml, desc, bytes;
};

Workspace workspace(int rows, int d)
{
    Workspace w;
    w.ml = up256(size_t(2) * kAttnCtas * rows * d * 4);
    w.desc = w.ml + up256(size_t(2) * kAttnCtas * rows * 8);
    w.bytes = w.desc + size_t(2) * kAttnCtas * 16;
    return w;
}

// Packed rows of a unit, by the most a sequence and head can have.  Measured with 28 heads on 4, head_dim 128, 8 sequences
// of up to 16001 keys (136 / 70 MB, 20 / 10 us of HBM), f16 / int8: for 7 rows 30.2 / 23.5 us with 8 rows a unit, 35.5 / 36.4
// with 16, 36.5 / 56.5 with 128; for 14 rows 36.7 / 37.6 us with 16 rows a unit, 36.6 / 56.4 with 128.
int rows_of(int64_t max_rows) { return max_rows <= 8 ? 8 : max_rows <= 16 ? 16 : 128; }

// CTAs of a unit that join without the workspace, or 0.
int cluster_of(int64_t max_rows, const q8_kv_cache *c, int64_t batch, int64_t max_len)
{
    const int rows = rows_of(max_rows);
    const int64_t units = batch * c->kv_heads * ((max_rows + rows - 1) / rows);
    if (units > (1 << 20)) return 0;  // counted in 32 bits
    return rows == 128 ? q8::attn_tiles_cluster(units, max_len) : q8::attn_rows_cluster(rows, units, max_len);
}

} // namespace

static bool attn_shape_ok(const q8_kv_cache *c, int64_t heads, int64_t max_fresh)
{
    return heads >= 1 && heads % c->kv_heads == 0 && heads / c->kv_heads <= 64 && max_fresh >= 1 &&
           max_fresh < (int64_t(1) << 24);
}

extern "C" size_t q8_tree_attention_workspace_bytes(const q8_kv_cache *cache, int64_t heads, int64_t max_fresh)
{
    if (q8::kv_cache_status(cache) == Q8_ERR_ARG || !attn_shape_ok(cache, heads, max_fresh)) return 0;
    return workspace(rows_of(max_fresh * (heads / cache->kv_heads)), cache->head_dim).bytes;
}

extern "C" int q8_tree_attention_needs_workspace(const q8_kv_cache *cache, int64_t heads, int64_t batch, int64_t max_fresh,
                                                 int64_t max_len)
{
    if (q8::kv_cache_status(cache) == Q8_ERR_ARG || !attn_shape_ok(cache, heads, max_fresh) || batch < 1 ||
        batch > Q8_KV_MAX_BATCH || max_len < 1)
        return 1;
    return cluster_of(max_fresh * (heads / cache->kv_heads), cache, batch, max_len) == 0;
}

extern "C" int q8_tree_attention(const q8_kv_cache *cache, int64_t layer, const float *q, int64_t heads, float scale,
                                 const int32_t *table, int64_t max_pages, const int32_t *cached, const int32_t *starts,
                                 int64_t batch, const int64_t *masks, int64_t tokens, int64_t max_fresh,
                                 int64_t max_len, float *y, int8_t *qs, uint32_t *ds, void *workspace_,
                                 size_t workspace_bytes, void *stream)
{
    if (!cache || !q || !table || !cached || !starts || (!y && !qs) || (qs == nullptr) != (ds == nullptr))
        return Q8_ERR_ARG;
    const int cst = q8::kv_cache_status(cache);
    if (cst == Q8_ERR_ARG) return cst;
    if (layer < 0 || layer >= cache->layers || !attn_shape_ok(cache, heads, max_fresh) || batch < 1 ||
        batch > Q8_KV_MAX_BATCH || tokens < 1 || tokens >= (int64_t(1) << 31) || max_fresh > tokens ||
        max_len < max_fresh || max_len >= (int64_t(1) << 31) - 4096 || max_pages < 1 ||
        max_pages >= (int64_t(1) << 31) || (masks && max_fresh > Q8_TREE_MAX_NODES))
        return Q8_ERR_ARG;
    const float scale2 = scale * 1.4426950408889634f;  // the weights are powers of two
    if (!(fabsf(scale2) <= FLT_MAX)) return Q8_ERR_ARG;
    const int group = static_cast<int>(heads / cache->kv_heads);
    const int rows = rows_of(max_fresh * group);
    // the line of tiles and units' heads is counted in 32 bits
    const double line = double(batch) * cache->kv_heads * ((max_fresh * group + rows - 1) / rows) *
                        ((max_len + 127) / 128 + 8);
    if (line > 2.0e9) return Q8_ERR_ARG;
    const Workspace w = workspace(rows, cache->head_dim);
    const int cluster = cluster_of(max_fresh * group, cache, batch, max_len);
    if (!cluster && (!workspace_ || workspace_bytes < w.bytes)) return Q8_ERR_ARG;
    if (cst != Q8_OK) return cst;
    const void *all[] = {q, table, cached, starts, masks, y, qs, ds, workspace_};
    for (const void *p : all)
        if (!q8::aligned16(p)) return Q8_ERR_ALIGN;
    if (!q8::device_is_sm103()) return Q8_ERR_DEVICE;

    const int D = cache->head_dim;
    const bool i8 = cache->dtype == Q8_KV_INT8;
    const int64_t lr = q8::kv_layer_rows(*cache), eb = q8::kv_element_bytes(*cache);
    const uint8_t *kp = static_cast<const uint8_t *>(cache->k) + layer * lr * D * eb;
    const uint8_t *vp = static_cast<const uint8_t *>(cache->v) + layer * lr * D * eb;
    uint8_t *ws = static_cast<uint8_t *>(workspace_);
    q8::AttnCall c;
    c.a = {q, table, cached, starts, reinterpret_cast<const long long *>(masks),
           i8 ? cache->k_scale + layer * lr : nullptr, i8 ? cache->v_scale + layer * lr : nullptr,
           reinterpret_cast<const uint16_t *>(vp), y, qs, ds, reinterpret_cast<float *>(ws),
           reinterpret_cast<float2 *>(ws + w.ml), reinterpret_cast<int4 *>(ws + w.desc), tokens,
           static_cast<int>(batch), static_cast<int>(heads), cache->kv_heads, group, static_cast<int>(max_pages),
           cache->page_size, static_cast<int>(cache->n_pages), static_cast<int>(max_fresh),
           static_cast<int>(max_len), q8::kv_inverse(group), cluster, scale2};
    c.k = kp, c.v = vp, c.layer_rows = lr, c.dim = D, c.int8 = i8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return rows == 128 ? q8::attn_tiles_launch(c, s) : q8::attn_rows_launch(c, rows, s);
}
