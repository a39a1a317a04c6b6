// attn_paged.cu -- host entry of the paged decode attention (kernel: attn_paged.cuh).
#include <cfloat>
#include <cmath>

#include "attn_paged.cuh"

namespace wsw {
namespace paged {

#define WSW_PAGED_DECLARE(CT, X3)                                                                       \
    template <> cudaError_t launch_type<CT, X3, false>(const Args &, int, cudaStream_t, bool, int64_t); \
    template <> cudaError_t launch_type<CT, X3, true>(const Args &, int, cudaStream_t, bool, int64_t);
WSW_PAGED_DECLARE(WSW_F16, false)
WSW_PAGED_DECLARE(WSW_BF16, false)
WSW_PAGED_DECLARE(WSW_BF16, true)
WSW_PAGED_DECLARE(WSW_Q8_0, false)

namespace {
constexpr size_t kCounterBytes = 2048;
static_assert(3 * kCtas * 4 <= kCounterBytes, "counters");
// groups of up to 8 query heads keep their residuals in the other 8 rows of a 16-row tile
int rows_of(int64_t group) { return group <= 8 ? 8 : 16; }
int warps_of(int64_t head_dim) { return head_dim == 256 ? 4 : 12; }  // at most
size_t record_bytes(int rows, int64_t head_dim) { return static_cast<size_t>(rows) * (head_dim + 4) * 4; }
}  // namespace
}  // namespace paged
}  // namespace wsw

extern "C" size_t wsw_attn_paged_decode_workspace_bytes(int64_t requests, int64_t q_heads, int64_t kv_heads,
                                                        int64_t head_dim) {
    using namespace wsw::paged;
    if (requests < 0 || requests > 65535 || kv_heads < 1 || kv_heads > 65535 || q_heads < kv_heads ||
        q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return 0;
    // counters, two records per CTA, one per warp
    return kCounterBytes + static_cast<size_t>(kCtas) * (2 + warps_of(head_dim)) *
                               record_bytes(rows_of(q_heads / kv_heads), head_dim);
}

namespace wsw {
namespace paged {

int prepare(const void *q, int32_t dtype, int64_t requests, int64_t q_heads, const wsw_kv_cache *cache,
            const int32_t *table, int64_t max_pages, int64_t table_stride, const int32_t *lens, float scale,
            float softcap, int64_t window, const float *slopes, void *out, float *lse, int32_t *err_flag, Args *args,
            int *rows, int64_t *tiles) {
    Args &a = *args;
    a = Args{};
    int st = check_kv_cache(cache, &a.kv);
    if (st != WSW_OK) return st;
    if (dtype != WSW_F32 && dtype != WSW_F16 && dtype != WSW_BF16) return WSW_ERR_UNSUPPORTED;
    if (requests < 0 || q_heads < 1 || q_heads % a.kv.heads != 0 || max_pages < 0 || table_stride < max_pages ||
        !std::isfinite(scale * kLog2e) || !std::isfinite(softcap) || softcap < 0.f || window < 0)
        return WSW_ERR_INVALID_ARG;
    constexpr int64_t lim = int64_t(1) << 31;
    // Positions and page numbers are 32 bits: a tile's positions and a window of 64 + 32 table entries run past
    // the last position (page_size 1: an entry's number past 2^31 - 1 was read at a negative offset), a step of
    // the CTA past a row's last vector of four.
    constexpr int64_t most = lim - 4096;
    if (requests > 65535 || q_heads >= lim || requests * q_heads >= lim || q_heads * (a.kv.head_dim / 4) > most ||
        max_pages > most || (max_pages << a.kv.page_shift) > most || window >= lim)
        return WSW_ERR_UNSUPPORTED;
    if (requests == 0) return WSW_OK;
    if (!q || !out || !lens || (max_pages > 0 && !table)) return WSW_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) ||
        ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(lse) |
          reinterpret_cast<uintptr_t>(slopes) | reinterpret_cast<uintptr_t>(err_flag)) & 3))
        return WSW_ERR_MISALIGNED;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.slopes = slopes;
    a.table = table;
    a.lens = lens;
    a.err = err_flag;
    a.table_stride = table_stride;
    a.scale2 = scale * kLog2e;
    // A cap so large that softcap log2 e or scale / softcap leaves fp32's normal range bends only scores of
    // |q . K| above 2^114: none.  (As a cap, inf * tanh(0) made every result NaN.)
    // A cap so small that scale / softcap, or its product with 2 log2 e, leaves it at the other end cuts every score but 0, to +-
    // softcap: a quarter of the largest value does the same.  (As it was, 0 * inf made rows of zeros NaN.)
    const float most_in = FLT_MAX / 4;
    const float in = softcap > 0.f ? std::fmin(std::fmax(scale / softcap, -most_in), most_in) : 0.f;
    const bool capped = std::isfinite(softcap * kLog2e) && std::fabs(in) >= FLT_MIN;
    a.cap_in = capped ? in : 0.f;
    a.cap_out = capped ? softcap * kLog2e : 0.f;
    a.requests = static_cast<int>(requests);
    a.q_heads = static_cast<int>(q_heads);
    a.group = static_cast<int>(q_heads / cache->heads);
    *rows = rows_of(a.group);
    a.passes = (a.group + *rows - 1) / *rows;
    a.max_len = static_cast<int>(max_pages << a.kv.page_shift);
    a.window = window > 0 ? static_cast<int>(window) : 0x7fffffff;
    a.dtype = dtype;
    // the longest possible list
    const int64_t seen = a.max_len < a.window ? a.max_len : a.window;
    *tiles = requests * cache->heads * a.passes * ((seen + 15) / 16 + kPair);
    if (*tiles >= lim - 65536) return WSW_ERR_UNSUPPORTED;  // tiles are counted in 32 bits
    return WSW_OK;
}

void place(Args *a, void *ws, int rows) {
    unsigned char *w = static_cast<unsigned char *>(ws);
    a->cnt = reinterpret_cast<unsigned *>(w);
    a->rec = reinterpret_cast<float *>(w + kCounterBytes);
    a->wrec = a->rec + static_cast<size_t>(kCtas) * 2 * record_bytes(rows, a->kv.head_dim) / 4;
}

template <bool Rest>
cudaError_t launch_cache(const Args &a, int cache_dtype, int rows, int64_t tiles, cudaStream_t s, bool pdl) {
    if (cache_dtype == WSW_F16) return launch_type<WSW_F16, false, Rest>(a, rows, s, pdl, tiles);
    if (cache_dtype == WSW_Q8_0) return launch_type<WSW_Q8_0, false, Rest>(a, rows, s, pdl, tiles);
    if (a.dtype == WSW_F32) return launch_type<WSW_BF16, true, Rest>(a, rows, s, pdl, tiles);
    return launch_type<WSW_BF16, false, Rest>(a, rows, s, pdl, tiles);
}
cudaError_t launch_paged(const Args &a, int cache_dtype, int rows, int64_t tiles, cudaStream_t s, bool pdl) {
    return a.ml ? launch_cache<true>(a, cache_dtype, rows, tiles, s, pdl) : launch_cache<false>(a, cache_dtype, rows, tiles, s, pdl);
}

}  // namespace paged
}  // namespace wsw

extern "C" int wsw_attn_paged_decode(const void *q, int32_t dtype, int64_t requests, int64_t q_heads,
                                     const wsw_kv_cache *cache, const int32_t *table, int64_t max_pages,
                                     int64_t table_stride, const int32_t *lens, float scale, float softcap,
                                     int64_t window, const float *slopes, void *out, float *lse, int32_t *err_flag,
                                     void *ws, size_t ws_bytes, void *stream, const wsw_launch_opts *opts) {
    using namespace wsw;
    using namespace wsw::paged;
    Opts o;
    int st = resolve_opts(opts, &o);
    if (st != WSW_OK) return st;
    Args a;
    int rows = 0;
    int64_t tiles = 0;
    st = prepare(q, dtype, requests, q_heads, cache, table, max_pages, table_stride, lens, scale, softcap, window, slopes,
                 out, lse, err_flag, &a, &rows, &tiles);
    if (st != WSW_OK || requests == 0) return st;
    if (!ws) return WSW_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(ws) & 15) return WSW_ERR_MISALIGNED;
    if (ws_bytes < wsw_attn_paged_decode_workspace_bytes(requests, q_heads, cache->heads, cache->head_dim))
        return WSW_ERR_WORKSPACE;
    place(&a, ws, rows);
    DeviceInfo di;
    if (!device_info(&di, &st)) return st;
    const cudaError_t e = launch_paged(a, cache->dtype, rows, tiles, static_cast<cudaStream_t>(stream), o.pdl);
    return e == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
}
