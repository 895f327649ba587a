// C-ABI entry points of the paged 8-bit K/V cache and the attention of single
// query tokens over it: host-side validation and launches.  Nothing here
// allocates device memory or synchronises with the device.
#include <cmath>
#include <cstdint>

#include "bsattn_internal.h"

namespace {

using bsattn::kTile;

bool misaligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// The cache's shape (its pointers are checked by check_cache).
bsattn_status check_cache_shape(const bsattn_kv_cache *c) {
    if (!c) return BSATTN_ERR_INVALID_ARG;
    if (c->dtype != BSATTN_KV_E4M3 && c->dtype != BSATTN_KV_INT8) return BSATTN_ERR_INVALID_ARG;
    if (c->num_pages < 0 || c->H <= 0) return BSATTN_ERR_INVALID_ARG;
    if (c->D != 64 && c->D != 128) return BSATTN_ERR_UNSUPPORTED;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return BSATTN_ERR_UNSUPPORTED;
    // rows are numbered in 32 bits
    if ((long long)c->num_pages * c->H > INT32_MAX / c->page_size) return BSATTN_ERR_INVALID_ARG;
    return BSATTN_OK;
}

bsattn_status check_cache(const bsattn_kv_cache *c) {
    bsattn_status st = check_cache_shape(c);
    if (st != BSATTN_OK) return st;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return BSATTN_ERR_INVALID_ARG;
    if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 16) || misaligned(c->v_scale, 16))
        return BSATTN_ERR_INVALID_ARG;
    return BSATTN_OK;
}

bsattn::CacheView view(const bsattn_kv_cache *c) {
    bsattn::CacheView w = {};
    w.k = static_cast<uint8_t *>(c->k);
    w.v = static_cast<uint8_t *>(c->v);
    w.ks = c->k_scale;
    w.vs = c->v_scale;
    w.num_pages = c->num_pages;
    for (w.page_shift = 4; (1 << w.page_shift) < c->page_size; ++w.page_shift) {}
    w.H = c->H;
    w.D = c->D;
    w.int8 = c->dtype == BSATTN_KV_INT8 ? 1 : 0;
    return w;
}

// A page table; a row's positions (cols pages) are numbered in 32 bits.
bsattn_status check_table(const int32_t *table, int32_t stride, int32_t cols, int32_t page_size,
                          bool may_be_empty) {
    if (cols < 0 || (cols == 0 && !may_be_empty) || stride < cols) return BSATTN_ERR_INVALID_ARG;
    if (cols > 0 && !table) return BSATTN_ERR_INVALID_ARG;
    if (cols > (INT32_MAX - kTile) / page_size) return BSATTN_ERR_INVALID_ARG;
    return BSATTN_OK;
}

bsattn_status decode_impl(const void *q, int64_t q_stride, int32_t B, int32_t Hq,
                          const bsattn_kv_cache *cache, const int32_t *prefix_table, int32_t prefix_len,
                          const int32_t *page_table, int32_t table_stride, int32_t table_cols,
                          const int32_t *seqlens, const bsattn_meta *meta, const int32_t *kv_valid_len,
                          float softmax_scale, void *out, bsattn_out_dtype out_dtype, float *lse,
                          void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream) {
    bsattn_status st = check_cache(cache);
    if (st != BSATTN_OK) return st;
    if (B <= 0 || Hq <= 0 || Hq % cache->H) return BSATTN_ERR_INVALID_ARG;
    if (!q || !out || !lse || !seqlens || !workspace) return BSATTN_ERR_INVALID_ARG;
    if (misaligned(q, 16) || misaligned(out, 16) || misaligned(workspace, 256)) return BSATTN_ERR_INVALID_ARG;
    if (q_stride < (int64_t)Hq * cache->D || q_stride % 8) return BSATTN_ERR_INVALID_ARG;
    if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return BSATTN_ERR_INVALID_ARG;
    if (out_dtype != BSATTN_OUT_BF16 && out_dtype != BSATTN_OUT_F32) return BSATTN_ERR_INVALID_ARG;
    if (prefix_len < 0 || (prefix_len > 0 && !prefix_table)) return BSATTN_ERR_INVALID_ARG;
    if ((st = check_table(page_table, table_stride, table_cols, cache->page_size, prefix_len > 0)) != BSATTN_OK) return st;
    if (prefix_len > INT32_MAX - kTile) return BSATTN_ERR_INVALID_ARG;
    size_t need = 0;
    if ((st = bsattn_decode_workspace_size(cache, B, Hq, prefix_len, &need)) != BSATTN_OK) return st;
    if (workspace_bytes < need) return BSATTN_ERR_INVALID_ARG;

    bsattn::DecodeParams p = {};
    p.c = view(cache);
    p.q = static_cast<const uint16_t *>(q);
    p.q_stride = q_stride;
    p.B = B;
    p.Hq = Hq;
    p.G = Hq / cache->H;
    p.table = page_table;
    p.table_stride = table_stride;
    p.table_cols = table_cols;
    p.seqlens = seqlens;
    p.prefix_table = prefix_table;
    p.prefix_len = prefix_len;
    if (meta) {
        if ((st = bsattn::check_meta_desc(meta)) != BSATTN_OK) return st;
        if (meta->tile_m != kTile || meta->tile_n != kTile) return BSATTN_ERR_UNSUPPORTED;
        if (meta->B != B || meta->H != cache->H) return BSATTN_ERR_INVALID_ARG;
        if (meta->varlen ? meta->total_m_blocks != B : meta->num_m != 1) return BSATTN_ERR_INVALID_ARG;
        if (kv_valid_len && meta->num_n <= 0) return BSATTN_ERR_INVALID_ARG;
        p.has_lists = 1;
        p.lists_varlen = meta->varlen;
        p.list_n = meta->num_n;
        p.total_n = meta->total_n_blocks;
        p.full_cnt = meta->full_cnt;
        p.full_idx = meta->full_idx;
        p.mask_cnt = meta->mask_cnt;
        p.mask_idx = meta->mask_idx;
        p.cu_off = meta->cu_block_idx_offsets;
        p.vl = kv_valid_len;
    } else if (kv_valid_len) {
        return BSATTN_ERR_INVALID_ARG;  // it belongs to the listed tiles
    }
    p.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634074);
    p.out = out;
    p.out_f32 = out_dtype == BSATTN_OUT_F32 ? 1 : 0;
    p.lse = lse;
    p.err = err_flag;
    p.ws = static_cast<uint8_t *>(workspace);
    const cudaError_t e = bsattn::launch_decode(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

bsattn_status bsattn_kv_append(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                               int32_t total, int32_t B, const int32_t *cu_seqlens,
                               const int32_t *page_table, int32_t table_stride, int32_t table_cols,
                               const int32_t *seqlens, const bsattn_kv_cache *cache,
                               int32_t *err_flag, void *stream) {
    bsattn_status st = check_cache(cache);
    if (st != BSATTN_OK) return st;
    if (B <= 0 || total < 0 || (!cu_seqlens && total != B)) return BSATTN_ERR_INVALID_ARG;
    if (!seqlens || (total > 0 && (!k || !v))) return BSATTN_ERR_INVALID_ARG;
    if (misaligned(k, 16) || misaligned(v, 16)) return BSATTN_ERR_INVALID_ARG;
    const int64_t row = (int64_t)cache->H * cache->D;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return BSATTN_ERR_INVALID_ARG;
    if ((st = check_table(page_table, table_stride, table_cols, cache->page_size, false)) != BSATTN_OK) return st;
    if (total == 0 && !err_flag) return BSATTN_OK;  // else the offsets are still checked
    bsattn::AppendParams p = {};
    p.c = view(cache);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.total = total;
    p.B = B;
    p.cu = cu_seqlens;
    p.table = page_table;
    p.table_stride = table_stride;
    p.table_cols = table_cols;
    p.seqlens = seqlens;
    p.err = err_flag;
    const cudaError_t e = bsattn::launch_append(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

bsattn_status bsattn_kv_read(const bsattn_kv_cache *cache, const int32_t *page_table,
                             int32_t table_stride, int32_t table_cols, int32_t B,
                             const int32_t *cu_seqlens, int32_t total, void *k, void *v,
                             int32_t *err_flag, void *stream) {
    bsattn_status st = check_cache(cache);
    if (st != BSATTN_OK) return st;
    if (B <= 0 || total < 0 || !cu_seqlens || (total > 0 && (!k || !v))) return BSATTN_ERR_INVALID_ARG;
    if (misaligned(k, 16) || misaligned(v, 16)) return BSATTN_ERR_INVALID_ARG;
    if ((st = check_table(page_table, table_stride, table_cols, cache->page_size, false)) != BSATTN_OK) return st;
    if (total == 0 && !err_flag) return BSATTN_OK;  // else the offsets are still checked
    bsattn::ReadParams p = {};
    p.c = view(cache);
    p.table = page_table;
    p.table_stride = table_stride;
    p.table_cols = table_cols;
    p.total = total;
    p.B = B;
    p.cu = cu_seqlens;
    p.k = static_cast<uint16_t *>(k);
    p.v = static_cast<uint16_t *>(v);
    p.err = err_flag;
    const cudaError_t e = bsattn::launch_read(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

bsattn_status bsattn_decode_workspace_size(const bsattn_kv_cache *cache, int32_t B, int32_t Hq,
                                           int32_t prefix_len, size_t *bytes) {
    if (!bytes) return BSATTN_ERR_INVALID_ARG;
    *bytes = 0;
    bsattn_status st = check_cache_shape(cache);
    if (st != BSATTN_OK) return st;
    if (B <= 0 || Hq <= 0 || Hq % cache->H || prefix_len < 0) return BSATTN_ERR_INVALID_ARG;
    if (Hq / cache->H > 128) return BSATTN_ERR_UNSUPPORTED;
    if ((long long)B * Hq > INT32_MAX / 256) return BSATTN_ERR_INVALID_ARG;
    *bytes = bsattn::decode_workspace_bytes(B, cache->H, Hq / cache->H, cache->D, prefix_len);
    return BSATTN_OK;
}

bsattn_status bsattn_decode(const void *q, int64_t q_stride, int32_t B, int32_t Hq,
                            const bsattn_kv_cache *cache, const int32_t *page_table,
                            int32_t table_stride, int32_t table_cols, const int32_t *seqlens,
                            const bsattn_meta *meta, const int32_t *kv_valid_len,
                            float softmax_scale, void *out, bsattn_out_dtype out_dtype, float *lse,
                            void *workspace, size_t workspace_bytes, int32_t *err_flag, void *stream) {
    return decode_impl(q, q_stride, B, Hq, cache, nullptr, 0, page_table, table_stride, table_cols, seqlens,
                       meta, kv_valid_len, softmax_scale, out, out_dtype, lse, workspace, workspace_bytes,
                       err_flag, stream);
}

bsattn_status bsattn_decode_shared_prefix(const void *q, int64_t q_stride, int32_t B, int32_t Hq,
                                          const bsattn_kv_cache *cache, const int32_t *prefix_table,
                                          int32_t prefix_len, const int32_t *page_table,
                                          int32_t table_stride, int32_t table_cols,
                                          const int32_t *seqlens, const bsattn_meta *meta,
                                          const int32_t *kv_valid_len, float softmax_scale, void *out,
                                          bsattn_out_dtype out_dtype, float *lse, void *workspace,
                                          size_t workspace_bytes, int32_t *err_flag, void *stream) {
    return decode_impl(q, q_stride, B, Hq, cache, prefix_table, prefix_len, page_table, table_stride,
                       table_cols, seqlens, meta, kv_valid_len, softmax_scale, out, out_dtype, lse, workspace,
                       workspace_bytes, err_flag, stream);
}

}  // extern "C"
