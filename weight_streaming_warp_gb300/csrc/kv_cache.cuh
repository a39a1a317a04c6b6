// kv_cache.cuh -- the paged KV cache as the kernels see it, and its host checks.
#pragma once

#include "common.cuh"

namespace wsw {

// One row (head_dim values of one position and KV head) starts at
// base + page * page_stride + offset * pos_stride + head * head_stride, in bytes.
struct KvView {
    unsigned char *k, *v;    // codes for q8_0
    unsigned char *kd, *vd;  // q8_0 scales
    int64_t page_stride, pos_stride, head_stride;
    int64_t d_page_stride, d_pos_stride, d_head_stride;
    int num_pages;
    int page_shift;  // log2(page_size)
    int heads, head_dim;
};

inline int check_kv_cache(const wsw_kv_cache *c, KvView *out) {
    if (!c || !c->k || !c->v) return WSW_ERR_INVALID_ARG;
    if (c->dtype != WSW_F16 && c->dtype != WSW_BF16 && c->dtype != WSW_Q8_0) return WSW_ERR_UNSUPPORTED;
    const bool q8 = c->dtype == WSW_Q8_0;
    if (q8 && (!c->kd || !c->vd)) return WSW_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->page_size < 1 || c->heads < 1 || c->head_dim < 1 || c->page_stride < 0 ||
        c->pos_stride < 0 || c->head_stride < 0)
        return WSW_ERR_INVALID_ARG;
    if (q8 && (c->d_page_stride < 0 || c->d_pos_stride < 0 || c->d_head_stride < 0)) return WSW_ERR_INVALID_ARG;
    if (c->num_pages >= (int64_t(1) << 31) || c->page_size > 65536 || (c->page_size & (c->page_size - 1)) ||
        c->heads > 65535 || (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256))
        return WSW_ERR_UNSUPPORTED;
    const int64_t esize = q8 ? 1 : 2;
    const uint64_t al = reinterpret_cast<uint64_t>(c->k) | reinterpret_cast<uint64_t>(c->v) |
                        static_cast<uint64_t>((c->page_stride | c->pos_stride | c->head_stride) * esize);
    if (al & 15) return WSW_ERR_MISALIGNED;
    *out = KvView{};
    out->k = static_cast<unsigned char *>(c->k);
    out->v = static_cast<unsigned char *>(c->v);
    out->page_stride = c->page_stride * esize;
    out->pos_stride = c->pos_stride * esize;
    out->head_stride = c->head_stride * esize;
    if (q8) {
        const uint64_t dal = reinterpret_cast<uint64_t>(c->kd) | reinterpret_cast<uint64_t>(c->vd) |
                             static_cast<uint64_t>((c->d_page_stride | c->d_pos_stride | c->d_head_stride) * 2);
        if (dal & static_cast<uint64_t>(c->head_dim / 16 - 1)) return WSW_ERR_MISALIGNED;
        out->kd = reinterpret_cast<unsigned char *>(c->kd);
        out->vd = reinterpret_cast<unsigned char *>(c->vd);
        out->d_page_stride = c->d_page_stride * 2;
        out->d_pos_stride = c->d_pos_stride * 2;
        out->d_head_stride = c->d_head_stride * 2;
    }
    out->num_pages = static_cast<int>(c->num_pages);
    while ((int64_t(1) << out->page_shift) < c->page_size) ++out->page_shift;
    out->heads = static_cast<int>(c->heads);
    out->head_dim = static_cast<int>(c->head_dim);
    return WSW_OK;
}

}  // namespace wsw
