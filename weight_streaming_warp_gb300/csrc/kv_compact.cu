// kv_compact.cu -- the pages of a cache that nobody lists any more become the free list, and
// the others move together to the front of the pool.
//
//   live(p): some row's first ceil(len / P) entries list p, or held[p];  N = number of live pages
//   the k-th live page p >= N that is not held moves to the k-th other page below N, both in
//   ascending order, while k < max_moves; the tables follow, copy k says which page to copy
//   free list: the pages not live then, in ascending order, in the last places of `free_pages`
//
// Nothing is counted from one call to the next: what is free is what the rows do not list.  Bytes:
// the entries in (and out, with moves), a held byte a page, the free list.  One cluster, of which each CTA has
// a run of the pages as bits in shared memory: it reads all entries and marks those of its own
// run (marks as bytes in memory, each CTA's entries scattered over them, took 9 us of 16 for 64 rows
// of 380 entries: an SM sends a scattered store every 8 cycles or so; all CTAs' reads are 1 us).  A warp
// takes 32 pages at a time, a lane each, so that ranks are ballots; with the counts of live, moving and
// filled pages before a page its place in the free list needs no scan of its own: p - live + moved -
// filled pages lie below it.  The CTAs exchange their counts through the workspace, a barrier
// of the cluster (1 us) for each exchange.  Bound: these dependent steps (64 rows of 380 entries, freeing only, 9.6 us;
// 40 rows of 88 entries with their moves 14 us under a profiler's serialised launches).
#include "kv_rows.cuh"

namespace wsw {
namespace {

constexpr int kThreads = 1024;
constexpr int kSegment = 256;  // entries of a row that a warp takes
constexpr int64_t kMaxPages = int64_t(1) << 22;  // two bits each in the shared memory of 8 CTAs

struct CompactArgs {
    const int32_t *seq, *table;
    const uint8_t *held;
    int32_t *table_out, *free_pages, *head, *src, *dst, *count, *err;
    int32_t *to;         // [pages] where a page that may move goes
    int *sums;           // [3][16] of the CTAs
    int64_t table_stride, out_stride;
    int rows, shift, max_pages, pages, max_moves, run;  // run: pages of a warp, a multiple of 32
};

__global__ void __launch_bounds__(kThreads, 1) kv_compact_kernel(const CompactArgs a) {
    extern __shared__ uint32_t bits[];  // [words of the CTA] listed pages, then held ones
    __shared__ int scan_sm[33];
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
    const int cta = blockIdx.x, ncta = gridDim.x;
    auto barrier = [&] {
        if (ncta > 1) cluster_barrier();
        else __syncthreads();
    };
    const int own_words = a.run / 32 * (nt >> 5);
    uint32_t *listed_bits = bits, *held_bits = bits + own_words;
    const unsigned first_page = static_cast<unsigned>(cta) * (a.run * (nt >> 5)), own_pages = 32u * own_words;
    for (int i = tid; i < own_words; i += nt) listed_bits[i] = 0u;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t start = static_cast<int64_t>(first_page) + static_cast<int64_t>(tid >> 5) * a.run;
    const int p0 = static_cast<int>(min(start, static_cast<int64_t>(a.pages)));
    const int p1 = static_cast<int>(min(start + a.run, static_cast<int64_t>(a.pages)));
    uint32_t *listed_run = listed_bits + (tid >> 5) * (a.run / 32), *held_run = held_bits + (tid >> 5) * (a.run / 32);
    for (int base = p0, w = 0; base < p1; base += 128, w += 4) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = base + 32 * i + lane;
            h[i] = a.held && p < p1 ? a.held[p] : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = __ballot_sync(WSW_FULL_MASK, h[i]);
            if (lane == 0 && base + 32 * i < p1) held_run[w + i] = h[i];
        }
    }
    __syncthreads();

    // ---- marks
    int err = 0;
    const int segments = max((a.max_pages + kSegment - 1) / kSegment, 1);  // one for the lengths at least
    const int64_t tasks = static_cast<int64_t>(a.rows) * segments;
    // every entry that a row uses, shared among warps first, first + step, ...: f(row, entry's number, entry)
    auto entries = [&](int64_t from, int step, auto f) {
        for (int64_t t = from; t < tasks; t += step) {
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
    entries(tid >> 5, nt >> 5, [&](int, int, int page) {
        const unsigned at = static_cast<unsigned>(page) - first_page;
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.pages)) err |= 1;
        else if (at < own_pages) atomicOr(&listed_bits[at >> 5], 1u << (at & 31));
    });
    if (err && a.err && cta == 0) atomicOr(a.err, err);
    __syncthreads();

    // f(page, whether a row lists it, whether it is held) for the warp's pages, all lanes together
    auto pages = [&](auto f) {
        for (int base = p0, w = 0; base < p1; base += 32, ++w)
            f(base + lane, (listed_run[w] >> lane) & 1u, (held_run[w] >> lane) & 1u);
    };
    const uint32_t below = (1u << lane) - 1;
    auto count = [&](bool x) { return __popc(__ballot_sync(WSW_FULL_MASK, x)); };
    auto rank = [&](bool x) { return __popc(__ballot_sync(WSW_FULL_MASK, x) & below); };
    // what the block's earlier warps and the earlier CTAs have of a warp's count, and all
    auto exchange = [&](int which, int mine, int *before) {
        int total;
        const int own = block_scan(lane == 0 ? mine : 0, 0x7fffffff, scan_sm, &total);
        *before = __shfl_sync(WSW_FULL_MASK, own, 0);
        if (tid == 0) a.sums[which * 16 + cta] = total;
    };
    auto collect = [&](int which, int *before, int *all) {
        const int x = lane < ncta ? __ldcg(a.sums + which * 16 + lane) : 0;
        *before += __reduce_add_sync(WSW_FULL_MASK, lane < cta ? x : 0);
        *all = __reduce_add_sync(WSW_FULL_MASK, x);
    };

    // ---- live pages
    int live = 0, live_before, many;
    for (int w = lane; w < (p1 - p0 + 31) / 32; w += 32) live += __popc(listed_run[w] | held_run[w]);
    live = __reduce_add_sync(WSW_FULL_MASK, live);
    exchange(0, live, &live_before);
    barrier();
    collect(0, &live_before, &many);

    // ---- moves
    int out_before = 0, in_before = 0, moves = 0;
    if (a.max_moves > 0) {
        int out = 0, in = 0, holes;
        pages([&](int p, bool listed, bool held) {
            out += count(listed && !held && p >= many);
            in += count(!listed && !held && p < many);
        });
        exchange(1, out, &out_before);
        exchange(2, in, &in_before);
        barrier();
        collect(1, &out_before, &moves);
        collect(2, &in_before, &holes);
        moves = min(min(moves, holes), a.max_moves);
        int o = out_before, k = in_before;
        pages([&](int p, bool listed, bool held) {
            const bool goes = listed && !held && p >= many, fills = !listed && !held && p < many;
            const int ro = o + rank(goes), rk = k + rank(fills);
            if (goes && ro < moves) a.src[ro] = p;
            if (fills && rk < moves) a.dst[rk] = p;
            o += count(goes);
            k += count(fills);
        });
    }
    if (cta == 0 && tid == 0) {
        *a.head = many;
        *a.count = moves;
    }
    if (moves > 0) barrier();  // src and dst

    // ---- the free list, and where each page goes
    int l = live_before, o = out_before, k = in_before;
    pages([&](int p, bool listed, bool held) {
        const bool lives = listed || held;
        const bool out = listed && !held && p >= many, in = !lives && p < many;
        const int rl = l + rank(lives), ro = o + rank(out), rk = k + rank(in);
        const bool goes = out && ro < moves, filled = in && rk < moves;
        if (p < a.pages) {
            // in the list's last pages - many places
            if (goes || (!lives && !filled)) a.free_pages[many + p - rl + min(ro, moves) - min(rk, moves)] = p;
            if (moves > 0 && out) a.to[p] = goes ? __ldcg(a.dst + ro) : p;
        }
        l += count(lives);
        o += count(out);
        k += count(in);
    });
    if (a.max_moves == 0) return;

    // ---- the tables: pages below N stay, as do held ones
    if (moves > 0) barrier();
    entries(cta * (nt >> 5) + (tid >> 5), ncta * (nt >> 5), [&](int r, int j, int page) {
        int to = page;
        if (moves > 0 && page >= many && page < a.pages && !(a.held && a.held[page])) to = __ldcg(a.to + page);
        a.table_out[r * a.out_stride + j] = to;
    });
}

constexpr size_t kSumBytes = 3 * 16 * 4;

}  // namespace
}  // namespace wsw

extern "C" size_t wsw_kv_page_compact_workspace_bytes(int64_t num_pages) {
    using namespace wsw;
    if (num_pages < 1 || num_pages > kMaxPages) return 0;
    return kSumBytes + static_cast<size_t>(num_pages) * 4;
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
    a.to = reinterpret_cast<int32_t *>(w + kSumBytes);
    a.table_stride = table_stride; a.out_stride = out_stride;
    a.rows = static_cast<int>(requests);
    a.shift = 0;
    while ((int64_t(1) << a.shift) < page_size) ++a.shift;
    a.max_pages = static_cast<int>(max_pages);
    a.pages = static_cast<int>(num_pages);
    a.max_moves = static_cast<int>(max_moves);
    static ClusterChoice choice;
    unsigned ncta = 1;
    constexpr int kMost = static_cast<int>(kMaxPages / 8 * 2 / 8);  // bytes of bits with 8 CTAs
    static_assert(kMost <= 200 * 1024, "shared memory");
    if (cluster_ctas(choice, reinterpret_cast<const void *>(kv_compact_kernel), kThreads, kMost + 2048, di.device, &ncta) !=
        cudaSuccess)
        return WSW_ERR_CUDA;
    // little is done sooner without barriers between CTAs
    if (requests * max_pages <= 4096 && num_pages <= 8192) ncta = 1;
    const int64_t warps = static_cast<int64_t>(ncta) * (kThreads / 32);
    a.run = static_cast<int>(((num_pages + warps - 1) / warps + 31) / 32 * 32);
    const size_t smem = static_cast<size_t>(a.run) / 32 * (kThreads / 32) * 2 * 4;
    const cudaError_t e = launch_cluster(kv_compact_kernel, ncta, ncta, kThreads, smem, static_cast<cudaStream_t>(stream),
                                         o.pdl, a);
    return e == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
}
