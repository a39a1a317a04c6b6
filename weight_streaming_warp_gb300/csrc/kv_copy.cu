// kv_copy.cu -- pages of a paged KV cache copied within it, for every layer in one launch.
//
// Copy e moves the first fill[e] positions of page src[e] (all of it without `fill`) to page
// dst[e], K and V and q8_0 scales, in each of the caches.  Bytes: each copied one read and
// written, HBM-bound.  The number of copies is on the device, so the CTAs are persistent and
// take units of (copy, cache, K or V, part) in turn; a part is about kPart bytes of rows of
// head_dim values, in the order in which they lie in memory, moved in 16-byte vectors, kUnroll
// of a thread in flight: 64 KB on an SM with four CTAs of 128 threads.  (28800 whole pages of 64 KB: 460 us, 6.5 TB/s;
// twice as many bytes in flight 20 to 60% slower, half as many 25%; four vectors of 256 threads 472 us.  Pages of
// which half is filled: 64 x 8 rows of 4 heads and 4 layers 27 us, 35 so.)
#include "kv_cache.cuh"

namespace wsw {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 8;
constexpr int kPart = kThreads * kUnroll * 16;
constexpr int kCaches = 32;  // of one launch

struct Layer {
    unsigned char *k, *v, *kd, *vd;
    int64_t page_stride, pos_stride, head_stride;        // bytes
    int64_t d_page_stride, d_pos_stride, d_head_stride;
    int num_pages, heads, row, q8;  // row: bytes of head_dim values
};
struct CopyArgs {
    Layer layer[kCaches];
    const int32_t *src, *dst, *fill, *count;
    int32_t *err;
    int layers, most, shift, parts, kinds;
};

// Vectors [v0, v1) of the rows of `n` positions, of W bytes each, 1 << vs of them in a row.
template <typename V>
__device__ __forceinline__ void move(const unsigned char *from, unsigned char *to, int64_t pos_stride,
                                     int64_t head_stride, int heads, int n, int vs, int64_t v0, int64_t v1) {
    // the smaller stride is the inner one
    const bool by_head = head_stride > pos_stride;
    const unsigned inner = by_head ? n : heads;
    const int64_t si = by_head ? pos_stride : head_stride, so = by_head ? head_stride : pos_stride;
    // row / inner by a product, one too small at most, since less than 2^-32 of 1 / inner is lost and row < 2^32 (fork and
    // copy of 64 x 8 rows: 35.1 us with divisions, 34.5 so)
    const unsigned per = 0xffffffffu / max(inner, 1u);
    for (int64_t v = v0 + threadIdx.x; v < v1; v += kThreads * kUnroll) {
        V x[kUnroll];
        int64_t at[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t i = v + u * kThreads;
            const unsigned row = static_cast<unsigned>(i >> vs), q = __umulhi(row, per), left = row - q * inner;
            const unsigned o = q + (left >= inner);
            at[u] = o * so + (left >= inner ? left - inner : left) * si + (i & ((1 << vs) - 1)) * static_cast<int64_t>(sizeof(V));
            if (i < v1) x[u] = *reinterpret_cast<const V *>(from + at[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (v + u * kThreads < v1) *reinterpret_cast<V *>(to + at[u]) = x[u];
    }
}

// A unit of work: copy, cache, K, V or their scales, part.
struct Unit {
    int src, dst, fill, layer, kind, part;
};

__global__ void __launch_bounds__(kThreads, 4) kv_copy_kernel(const __grid_constant__ CopyArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int n = min(max(*a.count, 0), a.most);
    const int64_t each = static_cast<int64_t>(a.layers) * a.kinds * a.parts, units = n * each;
    auto fetch = [&](int64_t u) {
        Unit x{};
        if (u >= units) return x;
        const int e = static_cast<int>(u / each);
        int in = static_cast<int>(u - e * each);
        x.src = a.src[e];
        x.dst = a.dst[e];
        x.fill = a.fill ? a.fill[e] : 1 << a.shift;
        x.part = in % a.parts;
        in /= a.parts;
        x.kind = in % a.kinds;
        x.layer = in / a.kinds;
        return x;
    };
    Unit next = fetch(blockIdx.x);
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const Unit x = next;
        next = fetch(u + gridDim.x);  // its pages' numbers on their way during this unit's copies
        const Layer &l = a.layer[x.layer];
        const bool scales = x.kind >= 2;
        if (scales && !l.q8) continue;
        const bool ok = static_cast<unsigned>(x.src) < static_cast<unsigned>(l.num_pages) &&
                        static_cast<unsigned>(x.dst) < static_cast<unsigned>(l.num_pages);
        if (!ok && a.err && threadIdx.x == 0) atomicOr(a.err, 1);
        if (!ok || x.src == x.dst) continue;
        const int filled = min(max(x.fill, 0), 1 << a.shift);
        unsigned char *base = scales ? (x.kind == 2 ? l.kd : l.vd) : (x.kind == 0 ? l.k : l.v);
        const int64_t page = scales ? l.d_page_stride : l.page_stride;
        const int64_t pos = scales ? l.d_pos_stride : l.pos_stride, head = scales ? l.d_head_stride : l.head_stride;
        const unsigned char *from = base + x.src * page;
        unsigned char *to = base + x.dst * page;
        const int width = scales ? l.row / 16 : 16;             // of a vector; a row's scales are one
        const int vs = scales ? 0 : 31 - __clz(l.row / 16);
        const int64_t all = (static_cast<int64_t>(filled) * l.heads) << vs;
        const int64_t v0 = all * x.part / a.parts, v1 = all * (x.part + 1) / a.parts;
        if (width == 16) move<uint4>(from, to, pos, head, l.heads, filled, vs, v0, v1);
        else if (width == 8) move<uint2>(from, to, pos, head, l.heads, filled, vs, v0, v1);
        else move<uint32_t>(from, to, pos, head, l.heads, filled, vs, v0, v1);
    }
}

}  // namespace
}  // namespace wsw

extern "C" int wsw_kv_page_copy(const int32_t *src, const int32_t *dst, const int32_t *fill, const int32_t *count,
                                int64_t copies, const wsw_kv_cache *const *caches, int64_t n_caches,
                                int32_t *err_flag, void *stream, const wsw_launch_opts *opts) {
    using namespace wsw;
    Opts o;
    int st = resolve_opts(opts, &o);
    if (st != WSW_OK) return st;
    if (copies < 0 || n_caches < 0 || (n_caches > 0 && !caches)) return WSW_ERR_INVALID_ARG;
    if (copies >= (int64_t(1) << 31) || n_caches > 65536) return WSW_ERR_UNSUPPORTED;
    KvView view;
    for (int64_t i = 0; i < n_caches; ++i) {
        st = check_kv_cache(caches[i], &view);
        if (st != WSW_OK) return st;
        if (caches[i]->page_size != caches[0]->page_size) return WSW_ERR_INVALID_ARG;
    }
    if (copies == 0 || n_caches == 0) return WSW_OK;
    if (!src || !dst || !count) return WSW_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(fill) |
         reinterpret_cast<uintptr_t>(count) | reinterpret_cast<uintptr_t>(err_flag)) & 3)
        return WSW_ERR_MISALIGNED;
    DeviceInfo di;
    if (!device_info(&di, &st)) return st;
    CopyArgs a;
    a.src = src; a.dst = dst; a.fill = fill; a.count = count; a.err = err_flag;
    a.most = static_cast<int>(copies);
    bool pdl = o.pdl;
    for (int64_t first = 0; first < n_caches; first += kCaches) {
        a.layers = static_cast<int>(n_caches - first < kCaches ? n_caches - first : kCaches);
        a.kinds = 2;
        int64_t bytes = 0;
        for (int i = 0; i < a.layers; ++i) {
            check_kv_cache(caches[first + i], &view);
            const bool q8 = caches[first + i]->dtype == WSW_Q8_0;
            const int row = view.head_dim * (q8 ? 1 : 2);
            a.layer[i] = Layer{view.k, view.v, view.kd, view.vd, view.page_stride, view.pos_stride, view.head_stride,
                               view.d_page_stride, view.d_pos_stride, view.d_head_stride, view.num_pages, view.heads,
                               row, q8 ? 1 : 0};
            a.shift = view.page_shift;
            if (q8) a.kinds = 4;
            const int64_t b = (static_cast<int64_t>(row) * view.heads) << view.page_shift;
            if (b > bytes) bytes = b;
        }
        a.parts = static_cast<int>(bytes < kPart ? 1 : bytes / kPart > 65536 ? 65536 : bytes / kPart);
        const int64_t units = copies * a.layers * a.kinds * a.parts, most = static_cast<int64_t>(di.sm_count) * 4;
        const cudaError_t e = launch(kv_copy_kernel, dim3(static_cast<unsigned>(units < most ? units : most)),
                                     dim3(kThreads), 0, static_cast<cudaStream_t>(stream), pdl, a);
        if (e != cudaSuccess) return WSW_ERR_CUDA;
    }
    return WSW_OK;
}
