// kv_fork.cu -- rows of a block table that continue other rows: the children of a step share
// their parents' full pages, and each but the first gets a page of its own for a partly
// filled last one.
//
//   n = seq_len[parent[i]];  table_out[i][j] = table[parent[i]][j] for j < ceil(n / P)
//   a partly filled last page (n % P > 0) stays with the lowest child of its row; the k-th of
//   the others, in row order, takes free[head + k] and leaves (old page, new page, n % P) as copy k
//
// Bytes: the entries of the old rows in, of the new ones out, 4 each.  A tile of columns of all
// the old rows goes through shared memory before the new rows' are written, so that the new
// table may be the old one; what it costs is little: 64 rows of 512 pages are 256 KB.  Lengths
// and the free list's head may be updated in place, too: then the CTAs are one cluster and a
// barrier lies between the last read and the first write, else there are as many as tiles.
#include "kv_rows.cuh"

namespace wsw {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxRows = 8192;      // four words of shared memory for each row at most
constexpr int kMaxSmem = 226 * 1024;

struct ForkArgs {
    const int32_t *parent, *seq, *free_pages, *head, *table;
    int32_t *table_out, *len_out, *head_out;
    int32_t *src, *dst, *fill, *count, *err;
    int64_t table_stride, out_stride;
    int children, rows, n_free, shift, max_pages;
    int col_shift;  // log2 of a tile's columns
};

__global__ void __launch_bounds__(kThreads, 1) kv_fork_kernel(const ForkArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ int scan_sm[33];
    __shared__ int err_sm, most_sm;
    const int tid = threadIdx.x, nt = blockDim.x, cta = blockIdx.x;
    int32_t *par = sm;                     // [children] old row, -1: none
    int32_t *len = par + a.children;       // [children] positions
    int32_t *rank = len + a.children;      // [children] its copy's number, -1: none
    int32_t *lowest = rank + a.children;   // [rows] first child
    int32_t *stage = lowest + a.rows;      // [rows][columns] of the old table
    pdl_launch_dependents();
    for (int r = tid; r < a.rows; r += nt) lowest[r] = 0x7fffffff;
    if (tid == 0) err_sm = most_sm = 0;
    pdl_wait();
    __syncthreads();

    const int head = *a.head;
    const int avail = head < 0 || head > a.n_free ? 0 : a.n_free - head;
    const int part = (1 << a.shift) - 1;
    auto fits = [&](int n) { return n >= 0 && pages_of(n, a.shift) <= a.max_pages; };
    int err = 0, most = 0;
    for (int r = tid; r < a.rows; r += nt) {
        const int n = a.seq[r];
        if (fits(n)) most = max(most, pages_of(n, a.shift));
    }
    for (int i = tid; i < a.children; i += nt) {
        int p = a.parent[i], n = 0;
        if (p < -1 || p >= a.rows) {
            err |= 1;
            p = -1;
        }
        if (p >= 0) {
            n = a.seq[p];
            if (!fits(n)) {
                err |= 2;
                p = -1;
                n = 0;
            }
        }
        if (n & part) atomicMin(&lowest[p], i);
        par[i] = p;
        len[i] = n;
    }
    if (most > 0) atomicMax(&most_sm, most);
    __syncthreads();
    const int per = (a.children + nt - 1) / nt;
    const int i0 = min(tid * per, a.children), i1 = min(i0 + per, a.children);
    int mine = 0, total;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) mine += (len[i] & part) && lowest[par[i]] != i;
    int at = block_scan(mine, kMaxRows, scan_sm, &total);
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const bool own = (len[i] & part) && lowest[par[i]] != i;
        rank[i] = own ? at : -1;
        if (own && at++ >= avail) {  // no page for it: an empty row
            err |= 8;
            rank[i] = par[i] = -1;
            len[i] = 0;
        }
    }
    if (err) atomicOr(&err_sm, err);
    __syncthreads();
    const int copies = min(total, avail), columns = most_sm;
    unsigned in_cluster;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(in_cluster));
    if (in_cluster > 1) cluster_barrier();  // every CTA has read the lengths and the head

    if (cta == 0) {
        if (tid == 0) {
            *a.head_out = head + copies;
            *a.count = copies;
            if (err_sm && a.err) atomicOr(a.err, err_sm);
        }
        for (int i = tid; i < a.children; i += nt) a.len_out[i] = len[i];
    }
    const int width = 1 << a.col_shift;
#pragma unroll 1
    for (int j0 = cta << a.col_shift; j0 < columns; j0 += static_cast<int>(gridDim.x) << a.col_shift) {
        const int c = tid & (width - 1), j = j0 + c, step = nt >> a.col_shift;
#pragma unroll 8
        for (int r = tid >> a.col_shift; r < a.rows; r += step)
            if (j < columns) stage[(r << a.col_shift) + c] = a.table[r * a.table_stride + j];
        __syncthreads();
#pragma unroll 2
        for (int i = tid >> a.col_shift; i < a.children; i += step) {
            if (j >= columns) continue;
            const int need = pages_of(len[i], a.shift), k = rank[i];
            int v = j < need ? stage[(par[i] << a.col_shift) + c] : -1;
            if (k >= 0 && j == need - 1) {
                a.src[k] = v;
                v = a.free_pages[head + k];
                a.dst[k] = v;
                a.fill[k] = len[i] & part;
            }
            a.table_out[i * a.out_stride + j] = v;
        }
        __syncthreads();
    }
}

}  // namespace
}  // namespace wsw

extern "C" int wsw_kv_page_fork(const int32_t *parent, int64_t children, const int32_t *seq_len, int64_t requests,
                                const int32_t *free_pages, int64_t n_free, const int32_t *head, int64_t page_size,
                                const int32_t *table, int64_t max_pages, int64_t table_stride, int32_t *table_out,
                                int64_t out_stride, int32_t *len_out, int32_t *head_out, int32_t *src, int32_t *dst,
                                int32_t *fill, int32_t *count, int32_t *err_flag, void *stream,
                                const wsw_launch_opts *opts) {
    using namespace wsw;
    Opts o;
    int st = resolve_opts(opts, &o);
    if (st != WSW_OK) return st;
    if (children < 0 || requests < 0 || n_free < 0 || max_pages < 0 || page_size < 1 || table_stride < max_pages ||
        out_stride < max_pages)
        return WSW_ERR_INVALID_ARG;
    if (!head || !head_out || !count || (n_free > 0 && !free_pages) || (requests > 0 && !seq_len) ||
        (requests > 0 && max_pages > 0 && !table))
        return WSW_ERR_INVALID_ARG;
    if (children > 0 && (!parent || !len_out || !src || !dst || !fill || (max_pages > 0 && !table_out)))
        return WSW_ERR_INVALID_ARG;
    constexpr int64_t lim = int64_t(1) << 31;
    if (children > kMaxRows || requests > kMaxRows || n_free >= lim - 1 || max_pages > lim - (1 << 20) ||
        page_size > 65536 || (page_size & (page_size - 1)))
        return WSW_ERR_UNSUPPORTED;
    // in 64 bits beyond any real table: the strides' products fit
    if (table_stride > (int64_t(1) << 40) || out_stride > (int64_t(1) << 40)) return WSW_ERR_UNSUPPORTED;
    uintptr_t al = 0;
    for (const void *p : {static_cast<const void *>(parent), static_cast<const void *>(seq_len),
                          static_cast<const void *>(free_pages), static_cast<const void *>(head),
                          static_cast<const void *>(table), static_cast<const void *>(table_out),
                          static_cast<const void *>(len_out), static_cast<const void *>(head_out),
                          static_cast<const void *>(src), static_cast<const void *>(dst),
                          static_cast<const void *>(fill), static_cast<const void *>(count),
                          static_cast<const void *>(err_flag)})
        al |= reinterpret_cast<uintptr_t>(p);
    if (al & 3) return WSW_ERR_MISALIGNED;
    // the new table is the old one, or lies elsewhere
    auto extent = [&](int64_t rows, int64_t stride) { return rows > 0 ? ((rows - 1) * stride + max_pages) * 4 : 0; };
    const bool same = table_out == table && out_stride == table_stride;
    if (!same && overlap(table, extent(requests, table_stride), table_out, extent(children, out_stride)))
        return WSW_ERR_INVALID_ARG;
    if (len_out != seq_len && overlap(seq_len, requests * 4, len_out, children * 4)) return WSW_ERR_INVALID_ARG;
    DeviceInfo di;
    if (!device_info(&di, &st)) return st;
    ForkArgs a;
    a.parent = parent; a.seq = seq_len; a.free_pages = free_pages; a.head = head; a.table = table;
    a.table_out = table_out; a.len_out = len_out; a.head_out = head_out;
    a.src = src; a.dst = dst; a.fill = fill; a.count = count; a.err = err_flag;
    a.table_stride = table_stride; a.out_stride = out_stride;
    a.children = static_cast<int>(children); a.rows = static_cast<int>(requests);
    a.n_free = static_cast<int>(n_free); a.max_pages = static_cast<int>(max_pages);
    a.shift = 0;
    while ((int64_t(1) << a.shift) < page_size) ++a.shift;
    // a sector of 8 entries wide, so that there are many tiles (64 x 8 rows of 130 pages: 8.1 us, lines of 32 16 us),
    // and narrower for many rows
    const int64_t words = 3 * children + requests;
    a.col_shift = 3;
    while (a.col_shift > 0 && (words + (requests << a.col_shift)) * 4 > kMaxSmem) --a.col_shift;
    const size_t smem = static_cast<size_t>(words + (requests << a.col_shift)) * 4;
    static_assert((4 * kMaxRows + 2 * kMaxRows) * 4 <= kMaxSmem, "tile");
    static ClusterChoice choice;
    unsigned ncta = 1;
    if (cluster_ctas(choice, reinterpret_cast<const void *>(kv_fork_kernel), kThreads, kMaxSmem, di.device, &ncta) !=
        cudaSuccess)
        return WSW_ERR_CUDA;
    const bool in_place = len_out == seq_len || head_out == head;
    const int64_t tiles = (max_pages + (int64_t(1) << a.col_shift) - 1) >> a.col_shift;
    unsigned ctas, cluster = 1;
    if (tiles <= 1) ctas = 1;
    else if (in_place) ctas = cluster = ncta;
    else ctas = static_cast<unsigned>(tiles < di.sm_count ? tiles : di.sm_count);
    const cudaError_t e = launch_cluster(kv_fork_kernel, ctas, cluster, kThreads, smem, static_cast<cudaStream_t>(stream),
                                         o.pdl, a);
    return e == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
}
