// kv_compact.cu -- the pages of a cache that nobody lists any more become the free list, and
// the others move together to the front of the pool.
//
//   live(p): some row's first ceil(len / P) entries list p, or held[p];  N = number of live pages
//   the k-th live page p >= N that is not held moves to the k-th other page below N, both in
//   ascending order, while k < max_moves; the tables follow, copy k says which page to copy
//   free list: the pages not live then, in ascending order, in the last places of `free_pages`
//
// Nothing is counted from one call to the next: what is free is what the rows do not list.  Bytes:
// the entries in (and out, with moves), a mark and a held byte a page, the free list; two passes over the
// tables and three over the marks with barriers in between, so one cluster (a CTA alone for little), whose
// barriers cost half a microsecond.  With pages' prefix counts of live, moving and filled ones a
// free page's place needs no scan of its own: p - live(p) + moved(p) - filled(p) lie below it.
#include "kv_rows.cuh"

namespace wsw {
namespace {

constexpr int kThreads = 1024;
constexpr int kSegment = 256;  // entries of a row that a warp takes
constexpr int64_t kMaxPages = int64_t(1) << 26;

struct CompactArgs {
    const int32_t *seq, *table;
    const uint8_t *held;
    int32_t *table_out, *free_pages, *head, *src, *dst, *count, *err;
    uint8_t *mark;       // [pages rounded up to 16]
    int32_t *to;         // [pages] where each page goes (with moves)
    int *sums;           // [3][16] of the CTAs
    int64_t table_stride, out_stride;
    int rows, shift, max_pages, pages, max_moves;
};

__device__ __forceinline__ unsigned bytes_set(unsigned w) {  // of bytes 0 or 1
    return __popc(w & 0x01010101u);
}
__device__ __forceinline__ unsigned nonzero(unsigned w) {    // bytes to 0 or 1
    w |= w >> 4;
    w |= w >> 2;
    w |= w >> 1;
    return w & 0x01010101u;
}

__global__ void __launch_bounds__(kThreads, 1) kv_compact_kernel(const CompactArgs a) {
    __shared__ int scan_sm[33];
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
    const int cta = blockIdx.x, ncta = gridDim.x;
    auto barrier = [&] {
        if (ncta > 1) cluster_barrier();
        else __syncthreads();
    };
    pdl_launch_dependents();
    pdl_wait();
    // a thread has `per` times sixteen consecutive pages
    const int vecs = (a.pages + 15) >> 4, threads = ncta * nt, me = cta * nt + tid;
    const int per = (vecs + threads - 1) / threads;
    const int v0 = min(me * per, vecs), v1 = min(v0 + per, vecs);
    uint4 *marks = reinterpret_cast<uint4 *>(a.mark);
    for (int v = me; v < vecs; v += threads) marks[v] = make_uint4(0u, 0u, 0u, 0u);
    barrier();

    // ---- marks
    int err = 0;
    const int segments = (a.max_pages + kSegment - 1) / kSegment;
    const int64_t tasks = static_cast<int64_t>(a.rows) * segments;
    // every entry that a row uses: f(row's offsets in and out, entry's number, entry)
    auto entries = [&](auto f) {
        for (int64_t t = me >> 5; t < tasks; t += threads >> 5) {
            // neighbouring warps take neighbouring rows: the long ones' ends spread
            const int s = static_cast<int>(t / a.rows), r = static_cast<int>(t - static_cast<int64_t>(s) * a.rows);
            const int n = a.seq[r];
            const int need = n < 0 ? 0 : pages_of(n, a.shift);
            if (n < 0 || need > a.max_pages) {
                err |= 2;
                continue;
            }
            const int32_t *row = a.table + r * a.table_stride;
            const int first = s * kSegment;
            int e[kSegment / 32];
#pragma unroll
            for (int i = 0; i < kSegment / 32; ++i) {
                const int j = first + 32 * i + lane;
                e[i] = j < need ? row[j] : 0;
            }
#pragma unroll
            for (int i = 0; i < kSegment / 32; ++i) {
                const int j = first + 32 * i + lane;
                if (j < need) f(r, j, e[i]);
            }
        }
    };
    entries([&](int, int, int page) {
        if (static_cast<unsigned>(page) < static_cast<unsigned>(a.pages)) a.mark[page] = 1;
        else err |= 1;
    });
    if (err && a.err) atomicOr(a.err, err);
    barrier();

    // ---- live pages
    auto held16 = [&](int v) {  // 0 or 1 in each byte; a page past the last one reads as held, not live
        uint4 h = make_uint4(0u, 0u, 0u, 0u);
        if (!a.held) return h;
        if (16 * v + 16 <= a.pages && (reinterpret_cast<uintptr_t>(a.held) & 15) == 0) {
            h = reinterpret_cast<const uint4 *>(a.held)[v];
            h.x = nonzero(h.x); h.y = nonzero(h.y); h.z = nonzero(h.z); h.w = nonzero(h.w);
        } else {
            unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (16 * v + i < a.pages) w[i >> 2] |= (a.held[16 * v + i] != 0 ? 1u : 0u) << (8 * (i & 3));
            h = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return h;
    };
    int live = 0, total;
    for (int v = v0; v < v1; ++v) {
        const uint4 m = __ldcg(marks + v), h = held16(v);
        live += bytes_set(m.x | h.x) + bytes_set(m.y | h.y) + bytes_set(m.z | h.z) + bytes_set(m.w | h.w);
    }
    constexpr int kNoCap = 0x7fffffff;
    int live_before = block_scan(live, kNoCap, scan_sm, &total);
    // the other CTAs' totals: what came before, and all
    auto exchange = [&](int which, int mine, int *before, int *all) {
        if (tid == 0) a.sums[which * 16 + cta] = mine;
        barrier();
        *before = *all = 0;
        for (int i = 0; i < ncta; ++i) {
            const int x = __ldcg(a.sums + which * 16 + i);
            if (i < cta) *before += x;
            *all += x;
        }
    };
    int before, many;
    exchange(0, total, &before, &many);
    live_before += before;

    // ---- moves
    auto is = [](const uint4 &w, int i) {
        const unsigned x = i < 4 ? w.x : i < 8 ? w.y : i < 12 ? w.z : w.w;
        return (x >> (8 * (i & 3))) & 1u;
    };
    int out_before = 0, in_before = 0, moves = 0;
    if (a.max_moves > 0) {
        int out = 0, in = 0;
        for (int v = v0; v < v1; ++v) {
            const uint4 m = __ldcg(marks + v), h = held16(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int p = 16 * v + i;
                const bool held = is(h, i), listed = is(m, i);
                out += listed && !held && p >= many;
                in += !listed && !held && p < many;
            }
        }
        int out_total, in_total, ignore, all_in;
        out_before = block_scan(out, kNoCap, scan_sm, &out_total);
        in_before = block_scan(in, kNoCap, scan_sm, &in_total);
        if (tid == 0) a.sums[32 + cta] = in_total;
        exchange(1, out_total, &before, &moves);
        out_before += before;
        ignore = all_in = 0;
        for (int i = 0; i < ncta; ++i) {
            const int x = __ldcg(a.sums + 32 + i);
            if (i < cta) ignore += x;
            all_in += x;
        }
        in_before += ignore;
        moves = min(min(moves, all_in), a.max_moves);
        int o = out_before, k = in_before;
        for (int v = v0; v < v1; ++v) {
            const uint4 m = __ldcg(marks + v), h = held16(v);
            for (int i = 0; i < 16; ++i) {
                const int p = 16 * v + i;
                const bool held = is(h, i), listed = is(m, i);
                if (listed && !held && p >= many && o < moves) a.src[o++] = p;
                else if (!listed && !held && p < many && k < moves) a.dst[k++] = p;
            }
        }
    }
    if (cta == 0 && tid == 0) {
        *a.head = many;
        *a.count = moves;
    }
    if (moves > 0) barrier();  // src and dst

    // ---- the free list, and where each page goes
    const int first_free = many;  // the list's last pages - many places
    int l = live_before, o = min(out_before, moves), k = min(in_before, moves);
    for (int v = v0; v < v1; ++v) {
        const uint4 m = __ldcg(marks + v), h = held16(v);
        for (int i = 0; i < 16; ++i) {
            const int p = 16 * v + i;
            if (p >= a.pages) break;
            const bool held = is(h, i), listed = is(m, i), lives = held || listed;
            const bool goes = listed && !held && p >= many && o < moves;
            const bool filled = !lives && p < many && k < moves;
            if (goes || (!lives && !filled)) a.free_pages[first_free + p - l + o - k] = p;
            if (moves > 0) a.to[p] = goes ? __ldcg(a.dst + o) : p;
            l += lives;
            o += goes;
            k += filled;
        }
    }
    if (a.max_moves == 0) return;

    // ---- the tables
    if (moves > 0) barrier();
    entries([&](int r, int j, int page) {
        const bool ok = moves > 0 && static_cast<unsigned>(page) < static_cast<unsigned>(a.pages);
        a.table_out[r * a.out_stride + j] = ok ? __ldcg(a.to + page) : page;
    });
}

size_t mark_bytes(int64_t pages) { return (static_cast<size_t>(pages) + 15) / 16 * 16; }
constexpr size_t kSumBytes = 3 * 16 * 4;

}  // namespace
}  // namespace wsw

extern "C" size_t wsw_kv_page_compact_workspace_bytes(int64_t num_pages) {
    using namespace wsw;
    if (num_pages < 1 || num_pages > kMaxPages) return 0;
    return kSumBytes + mark_bytes(num_pages) + static_cast<size_t>(num_pages) * 4;
}

extern "C" int wsw_kv_page_compact(const int32_t *seq_len, int64_t requests, const int32_t *table, int64_t max_pages,
                                   int64_t table_stride, int64_t page_size, int64_t num_pages, const uint8_t *held,
                                   int64_t max_moves, int32_t *table_out, int64_t out_stride, int32_t *free_pages,
                                   int32_t *head, int32_t *src, int32_t *dst, int32_t *count, int32_t *err_flag,
                                   void *ws, size_t ws_bytes, void *stream, const wsw_launch_opts *opts) {
    using namespace wsw;
    Opts o;
    int st = resolve_opts(opts, &o);
    if (st != WSW_OK) return st;
    if (requests < 0 || max_pages < 0 || table_stride < max_pages || page_size < 1 || num_pages < 1 || max_moves < 0 ||
        (max_moves > 0 && out_stride < max_pages))
        return WSW_ERR_INVALID_ARG;
    if (requests > 65535 || max_pages > (int64_t(1) << 31) - (1 << 20) || num_pages > kMaxPages || page_size > 65536 ||
        (page_size & (page_size - 1)) || max_moves >= (int64_t(1) << 31) || table_stride > (int64_t(1) << 40) ||
        out_stride > (int64_t(1) << 40))
        return WSW_ERR_UNSUPPORTED;
    const bool entries = requests > 0 && max_pages > 0;
    if (!free_pages || !head || !count || !ws || (requests > 0 && !seq_len) || (entries && !table) ||
        (max_moves > 0 && (!src || !dst || (entries && !table_out))))
        return WSW_ERR_INVALID_ARG;
    uintptr_t al = 0;
    for (const void *p : {static_cast<const void *>(seq_len), static_cast<const void *>(table),
                          static_cast<const void *>(table_out), static_cast<const void *>(free_pages),
                          static_cast<const void *>(head), static_cast<const void *>(src),
                          static_cast<const void *>(dst), static_cast<const void *>(count),
                          static_cast<const void *>(err_flag)})
        al |= reinterpret_cast<uintptr_t>(p);
    if ((al & 3) || (reinterpret_cast<uintptr_t>(ws) & 15)) return WSW_ERR_MISALIGNED;
    if (max_moves > 0 && entries && !(table_out == table && out_stride == table_stride) &&
        overlap(table, ((requests - 1) * table_stride + max_pages) * 4, table_out,
                ((requests - 1) * out_stride + max_pages) * 4))
        return WSW_ERR_INVALID_ARG;
    if (ws_bytes < wsw_kv_page_compact_workspace_bytes(num_pages)) return WSW_ERR_WORKSPACE;
    DeviceInfo di;
    if (!device_info(&di, &st)) return st;
    CompactArgs a;
    a.seq = seq_len; a.table = table; a.held = held;
    a.table_out = table_out; a.free_pages = free_pages; a.head = head;
    a.src = src; a.dst = dst; a.count = count; a.err = err_flag;
    unsigned char *w = static_cast<unsigned char *>(ws);
    a.sums = reinterpret_cast<int *>(w);
    a.mark = w + kSumBytes;
    a.to = reinterpret_cast<int32_t *>(a.mark + mark_bytes(num_pages));
    a.table_stride = table_stride; a.out_stride = out_stride;
    a.rows = static_cast<int>(requests);
    a.shift = 0;
    while ((int64_t(1) << a.shift) < page_size) ++a.shift;
    a.max_pages = static_cast<int>(max_pages);
    a.pages = static_cast<int>(num_pages);
    a.max_moves = static_cast<int>(max_moves);
    static ClusterChoice choice;
    unsigned ncta = 1;
    if (cluster_ctas(choice, reinterpret_cast<const void *>(kv_compact_kernel), kThreads, 0, di.device, &ncta) !=
        cudaSuccess)
        return WSW_ERR_CUDA;
    if (requests * max_pages <= 8192 && num_pages <= 8192) ncta = 1;
    const cudaError_t e = launch_cluster(kv_compact_kernel, ncta, ncta, kThreads, 0, static_cast<cudaStream_t>(stream),
                                         o.pdl, a);
    return e == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
}
