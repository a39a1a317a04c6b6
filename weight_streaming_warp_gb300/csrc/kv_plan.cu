// kv_plan.cu -- block table and slot map of a serving step, built on the GPU from the
// requests' lengths.
//
//   cu(r)   = sum of new lengths before r           (tokens of the step, in request order)
//   need(r) = ceil((len + new) / P) - ceil(len / P) (pages that r opens)
//   off(r)  = sum of need before r; new page j of r is free[head + off(r) + j - ceil(len / P)]
//   slot    = page(position / P) * P + position % P, position = len + i for token cu(r) + i
//
// Two exclusive scans over the requests, then independent writes; the bytes (16 per
// request, 12 per token) are a few hundred nanoseconds of HBM time at any size served, so
// the launch and the dependent steps (lengths, two scans, table entry, slot) are the time.
// One launch of one cluster, of 16 CTAs where the device holds one, else 8: every CTA scans all the
// requests into its own shared memory (no exchange, no workspace), a cluster barrier puts every
// length read before the first write, so that the new lengths may overwrite the old (a call whose
// lengths go elsewhere takes the same form), and the CTAs share the writes.
// The sums saturate just beyond what can be served, so they fit in 32 bits whatever the
// lengths.  A thread takes four consecutive tokens (one while there are threads for all): one binary search in shared memory (a
// search for each token made 130000 tokens of 1000 requests bound by instructions, 18 us), one
// table read for each page that they touch.  64 requests of one token each take 3.9 us, 130000
// tokens of 1000 requests 10.5 us (clusters of 8 CTAs 13.7 us).
#include "cluster_choice.h"
#include "common.cuh"

namespace wsw {
namespace {

constexpr int kMaxRequests = 16384;  // three words of shared memory each
constexpr int kThreads = 1024;

struct PlanArgs {
    const int32_t *seq, *add;
    const int32_t *free_pages, *head;
    int32_t *table;
    int32_t *positions;
    int64_t *slots;
    int32_t *cu, *len_out, *head_out, *err;
    int64_t table_stride;
    int requests, n_free, shift, max_pages, tokens;
};

// pages of `len` < 2^31 positions
__device__ __forceinline__ int pages_of(int len, int shift) {
    return static_cast<int>((static_cast<unsigned>(len) + (1u << shift) - 1) >> shift);
}

// a + b, at most cap < 2^31 (a, b <= cap)
__device__ __forceinline__ int add_sat(int a, int b, int cap) {
    const unsigned s = static_cast<unsigned>(a) + static_cast<unsigned>(b);
    return s < static_cast<unsigned>(cap) ? static_cast<int>(s) : cap;
}

// Exclusive saturating prefix of v <= cap over the block's threads, and the block's total.
// Every thread calls it; sm holds 33 values.
__device__ __forceinline__ int block_scan(int v, int cap, int *sm, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(WSW_FULL_MASK, x, d);
        if (lane >= d) x = add_sat(x, y, cap);
    }
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = lane < warps ? sm[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(WSW_FULL_MASK, w, d);
            if (lane >= d) w = add_sat(w, y, cap);
        }
        sm[lane + 1] = w;
        if (lane == 0) sm[0] = 0;
    }
    __syncthreads();
    *total = sm[32];
    const int x_before = __shfl_up_sync(WSW_FULL_MASK, x, 1);
    const int before = add_sat(sm[warp], lane ? x_before : 0, cap);
    __syncthreads();  // sm may be reused
    return before;
}

// The last i with a[i] <= x[j] for each of N values (a is ascending, n entries, a[0] <= x)
template <int N>
__device__ __forceinline__ void find(const int32_t *a, int n, const int (&x)[N], int (&at)[N]) {
    int top = 1;
    while (top < n) top <<= 1;
#pragma unroll
    for (int j = 0; j < N; ++j) at[j] = 0;
#pragma unroll 1
    for (int step = top >> 1; step > 0; step >>= 1)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int i = at[j] + step;
            if (i < n && a[i] <= x[j]) at[j] = i;
        }
}

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const PlanArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ int scan_sm[33];
    __shared__ int used_sm, err_sm;
    const int R = a.requests, tid = threadIdx.x, nt = blockDim.x;
    int32_t *cu = sm;             // [R + 1] tokens before each request, cut at a.tokens
    int32_t *off = sm + R + 1;    // [R + 1] new pages before each request
    int32_t *len = off + R + 1;   // [R] cached length, -1 for a request that is not served
    const int ncta = gridDim.x, cta = blockIdx.x;
    const int step = ncta * nt;
    if (tid == 0) used_sm = err_sm = 0;
    pdl_launch_dependents();
    pdl_wait();

    const int head = *a.head;
    const int avail = head < 0 || head > a.n_free ? 0 : a.n_free - head;
    // a thread takes `per` consecutive requests
    const int per = (R + nt - 1) / nt;
    const int r0 = min(tid * per, R), r1 = min(r0 + per, R);
    const int tok_cap = a.tokens + 1, page_cap = avail + 1;  // < 2^31: what does not fit any more
    int err = 0, sum = 0;
    for (int r = tid; r < R; r += nt) {
        const int s = a.seq[r], n = a.add[r];
        const bool bad = s < 0 || n < 0;
        if (bad) err |= 1;
        len[r] = bad ? -1 : s;
        off[r] = bad ? 0 : n;  // the new length, until the page scan replaces it
    }
    __syncthreads();
#pragma unroll 1
    for (int r = r0; r < r1; ++r) sum = add_sat(sum, min(off[r], tok_cap), tok_cap);
    int total;
    int at = block_scan(sum, tok_cap, scan_sm, &total);
    sum = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        const int n = off[r], s = len[r];
        cu[r] = min(at, a.tokens);
        at = add_sat(at, min(n, tok_cap), tok_cap);
        int need = 0;
        if (s >= 0) {
            if (n > 0x7fffffff - s || pages_of(s + n, a.shift) > a.max_pages) { err |= 2; len[r] = -1; }
            else if (at > a.tokens) { err |= 4; len[r] = -1; }
            else need = pages_of(s + n, a.shift) - pages_of(s, a.shift);
        }
        off[r] = need;  // at most max_pages
        sum = add_sat(sum, min(need, page_cap), page_cap);
    }
    if (tid == 0) cu[R] = min(total, a.tokens);
    int before = block_scan(sum, page_cap, scan_sm, &total), used = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        const int need = min(off[r], page_cap), after = add_sat(before, need, page_cap);
        if (need > 0) {
            if (after > avail) { err |= 8; len[r] = -1; }
            else used = after;
        }
        off[r] = before;
        before = after;
    }
    if (used > 0) atomicMax(&used_sm, used);  // served requests come first
    if (err) atomicOr(&err_sm, err);
    __syncthreads();
    if (ncta > 1) {  // every CTA of the cluster has read its lengths
        asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
    const int granted = used_sm;

    if (cta == 0 && tid == 0) {
        *a.head_out = head + granted;
        a.cu[R] = cu[R];
        if (err_sm && a.err) atomicOr(a.err, err_sm);
    }
    const int first = cta * nt + tid;
    // the new length of a request is added here, from its own tokens: cu is not cut below a
    // served request's end
    for (int r = first; r < R; r += step) {
        a.cu[r] = cu[r];
        if (len[r] >= 0) a.len_out[r] = len[r] + (cu[r + 1] - cu[r]);
        else if (a.len_out != a.seq) a.len_out[r] = a.seq[r];
    }
    // four places of the thread at a time, their searches and reads in flight together
    const int rounds = (granted + 4 * step - 1) / (4 * step);
#pragma unroll 1
    for (int k = 0; k < rounds; ++k) {
        int i[4], r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) i[j] = min(first + (4 * k + j) * step, granted - 1);  // the last one again
        find(off, R, i, r);
        int32_t page[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) page[j] = a.free_pages[head + i[j]];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            a.table[r[j] * a.table_stride + pages_of(len[r[j]], a.shift) + (i[j] - off[r[j]])] = page[j];
    }
    const int filled = cu[R];
    const int group = a.tokens > step ? 4 : 1;
    const bool wide = group == 4 && ((reinterpret_cast<uintptr_t>(a.positions) | reinterpret_cast<uintptr_t>(a.slots)) & 15) == 0;
#pragma unroll 1
    for (int64_t base = group * static_cast<int64_t>(first); base < a.tokens; base += group * static_cast<int64_t>(step)) {
        const int t0 = static_cast<int>(base);
        const int x[1] = {t0};
        int at0[1];
        find(cu, R > 0 ? R : 1, x, at0);
        int r = at0[0], end = t0 < filled ? cu[r + 1] : 0, page = -1, page_key = -1;
        int pos[4];
        int64_t slot[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + i;
            pos[i] = -1;
            slot[i] = -1;
            if (i >= group || t >= filled) continue;
            while (t >= end) {  // cu[R] = filled > t
                end = cu[++r + 1];
                page_key = -1;
            }
            const int s = len[r];
            if (s < 0) continue;
            pos[i] = s + (t - cu[r]);
            const int q = pos[i] >> a.shift;
            if (q != page_key) {
                const int have = pages_of(s, a.shift);
                page = q < have ? a.table[r * a.table_stride + q] : a.free_pages[head + off[r] + (q - have)];
                page_key = q;
            }
            if (page >= 0) slot[i] = (int64_t(page) << a.shift) + (pos[i] & ((1 << a.shift) - 1));
        }
        if (wide && t0 + 4 <= a.tokens) {
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            reinterpret_cast<longlong2 *>(a.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
            reinterpret_cast<longlong2 *>(a.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < group && t0 + i < a.tokens) {
                    a.positions[t0 + i] = pos[i];
                    a.slots[t0 + i] = slot[i];
                }
        }
    }
}

constexpr int kMaxSmem = (3 * kMaxRequests + 2) * 4;

// Sets the kernel's options on the current device, once, and says how many CTAs a cluster can have.
cudaError_t cluster_ctas(int device, unsigned *ctas) {
    static ClusterChoice choice;
    const void *kernel = reinterpret_cast<const void *>(kv_plan_kernel);
    const cudaError_t e = ensure_smem(kernel, kMaxSmem);
    if (e != cudaSuccess) return e;
    *ctas = choice.of(device, [kernel] {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 16;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kMaxSmem;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        return clusters > 0;
    });
    return cudaSuccess;
}

}  // namespace
}  // namespace wsw

extern "C" int wsw_kv_page_plan(const int32_t *seq_len, const int32_t *new_len, int64_t requests,
                                const int32_t *free_pages, int64_t n_free, const int32_t *head, int64_t page_size,
                                int32_t *table, int64_t max_pages, int64_t table_stride, int64_t tokens,
                                int32_t *positions, int64_t *slots, int32_t *cu, int32_t *len_out,
                                int32_t *head_out, int32_t *err_flag, void *stream, const wsw_launch_opts *opts) {
    using namespace wsw;
    Opts o;
    int st = resolve_opts(opts, &o);
    if (st != WSW_OK) return st;
    if (requests < 0 || n_free < 0 || tokens < 0 || max_pages < 0 || page_size < 1 || table_stride < max_pages)
        return WSW_ERR_INVALID_ARG;
    if (!head || !head_out || !cu || (n_free > 0 && !free_pages) || (tokens > 0 && (!positions || !slots)))
        return WSW_ERR_INVALID_ARG;
    if (requests > 0 && (!seq_len || !new_len || !len_out || (max_pages > 0 && !table))) return WSW_ERR_INVALID_ARG;
    constexpr int64_t lim = int64_t(1) << 31;
    // threads step in rounds of up to 4 * 16 * kThreads places, the last one past the tokens and the new pages
    // (no more than the tokens): it stays below 2^31
    constexpr int64_t most = lim - (int64_t(1) << 20);
    static_assert(4 * 16 * kThreads < (1 << 20), "rounds");
    if (requests > kMaxRequests || tokens > most || n_free >= lim - 1 || max_pages >= lim || page_size > 65536 ||
        (page_size & (page_size - 1)))
        return WSW_ERR_UNSUPPORTED;
    const uintptr_t al = reinterpret_cast<uintptr_t>(seq_len) | reinterpret_cast<uintptr_t>(new_len) |
                         reinterpret_cast<uintptr_t>(free_pages) | reinterpret_cast<uintptr_t>(head) |
                         reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(positions) |
                         reinterpret_cast<uintptr_t>(cu) | reinterpret_cast<uintptr_t>(len_out) |
                         reinterpret_cast<uintptr_t>(head_out) | reinterpret_cast<uintptr_t>(err_flag);
    if ((al & 3) || (reinterpret_cast<uintptr_t>(slots) & 7)) return WSW_ERR_MISALIGNED;
    DeviceInfo di;
    if (!device_info(&di, &st)) return st;
    PlanArgs a;
    a.seq = seq_len; a.add = new_len; a.free_pages = free_pages; a.head = head; a.table = table;
    a.positions = positions; a.slots = slots; a.cu = cu; a.len_out = len_out; a.head_out = head_out; a.err = err_flag;
    a.table_stride = table_stride;
    a.requests = static_cast<int>(requests);
    a.n_free = static_cast<int>(n_free);
    a.max_pages = static_cast<int>(max_pages);
    a.tokens = static_cast<int>(tokens);
    a.shift = 0;
    while ((int64_t(1) << a.shift) < page_size) ++a.shift;
    const int smem = static_cast<int>((3 * requests + 2) * 4);
    unsigned ncta = 1;
    if (cluster_ctas(di.device, &ncta) != cudaSuccess) return WSW_ERR_CUDA;
    if (tokens <= 2048) ncta = 1;  // while its threads see few tokens each, else the largest cluster
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    const int64_t want = requests > tokens / ncta ? requests : tokens / ncta;
    cfg.gridDim = dim3(ncta);
    cfg.blockDim = dim3(want > 512 ? kThreads : want > 128 ? 512 : 128);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ncta;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    if (o.pdl) {
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kv_plan_kernel, a) == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
}
