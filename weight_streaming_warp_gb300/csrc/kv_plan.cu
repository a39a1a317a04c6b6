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
// One launch of one cluster: every CTA scans all the requests into its own shared memory
// (no exchange, no workspace), a cluster barrier puts every length read before the first
// write, so that the new lengths may overwrite the old, and the CTAs share the writes.
// Tokens find their request by binary search in shared memory, four consecutive ones per
// thread with one search.
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

__device__ __forceinline__ int64_t pages_of(int64_t len, int shift) {
    return (len + (int64_t(1) << shift) - 1) >> shift;
}

// Exclusive prefix of v over the block's threads, and the block's total.  Every thread
// calls it; sm holds 33 values.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *sm, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(WSW_FULL_MASK, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t w = lane < warps ? sm[lane] : 0;
        const int64_t own = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(WSW_FULL_MASK, w, d);
            if (lane >= d) w += y;
        }
        sm[lane] = w - own;
        if (lane == 31) sm[32] = w;
    }
    __syncthreads();
    *total = sm[32];
    const int64_t before = sm[warp] + x - v;
    __syncthreads();  // sm may be reused
    return before;
}

// The last i with a[i] <= x, for a[0] <= x (a is ascending, n entries).
__device__ __forceinline__ int find(const int32_t *a, int n, int x) {
    int lo = 0, hi = n;  // a[lo] <= x < a[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const PlanArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ int64_t scan_sm[33];
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
    const int64_t avail = head < 0 || head > a.n_free ? 0 : a.n_free - head;
    // a thread takes `per` consecutive requests
    const int per = (R + nt - 1) / nt;
    const int r0 = min(tid * per, R), r1 = min(r0 + per, R);
    int err = 0;
    int64_t sum = 0;
    for (int r = r0; r < r1; ++r) {
        const int s = a.seq[r], n = a.add[r];
        const bool bad = s < 0 || n < 0;
        if (bad) err |= 1;
        len[r] = bad ? -1 : s;
        off[r] = bad ? 0 : n;  // the new length, until the page scan replaces it
        sum += bad ? 0 : n;
    }
    int64_t total;
    int64_t at = block_scan(sum, scan_sm, &total);
    sum = 0;
    for (int r = r0; r < r1; ++r) {
        const int n = off[r], s = len[r];
        cu[r] = static_cast<int32_t>(at < a.tokens ? at : a.tokens);
        at += n;
        int64_t need = 0;
        if (s >= 0) {
            const int64_t want = pages_of(int64_t(s) + n, a.shift);
            if (want > a.max_pages || int64_t(s) + n > 0x7fffffff) { err |= 2; len[r] = -1; }
            else if (at > a.tokens) { err |= 4; len[r] = -1; }
            else need = want - pages_of(s, a.shift);
        }
        off[r] = static_cast<int32_t>(need);  // at most max_pages
        sum += need;
    }
    if (tid == 0) cu[R] = static_cast<int32_t>(total < a.tokens ? total : a.tokens);
    int64_t before = block_scan(sum, scan_sm, &total), used = 0;
    for (int r = r0; r < r1; ++r) {
        const int need = off[r];
        if (need > 0) {
            if (before + need > avail) { err |= 8; len[r] = -1; }
            else used = before + need;
        }
        // past the end of the free list the exact offset does not matter
        off[r] = static_cast<int32_t>(before < 0x7fffffff ? before : 0x7fffffff);
        before += need;
    }
    if (tid == 0) off[R] = 0x7fffffff;
    if (used > 0) atomicMax(&used_sm, static_cast<int>(used));  // served requests come first
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
    for (int i = first; i < granted; i += step) {
        const int r = find(off, R, i);
        const int64_t j = pages_of(len[r], a.shift) + (i - off[r]);
        a.table[r * a.table_stride + j] = a.free_pages[head + i];
    }
    const int filled = cu[R];
    for (int64_t t0 = int64_t(first) * 4; t0 < a.tokens; t0 += int64_t(step) * 4) {
        int32_t pos[4];
        int64_t slot[4];
        int r = t0 < filled ? find(cu, R, static_cast<int>(t0)) : R;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = t0 + i;
            pos[i] = -1;
            slot[i] = -1;
            if (t >= filled) continue;
            while (t >= cu[r + 1]) ++r;  // cu[R] = filled > t
            if (len[r] < 0) continue;
            const int p = len[r] + static_cast<int>(t - cu[r]);
            const int have = static_cast<int>(pages_of(len[r], a.shift)), j = p >> a.shift;
            const int page = j < have ? a.table[r * a.table_stride + j] : a.free_pages[head + off[r] + (j - have)];
            pos[i] = p;
            if (page >= 0) slot[i] = (int64_t(page) << a.shift) + (p & ((1 << a.shift) - 1));
        }
        if (t0 + 4 <= a.tokens && ((reinterpret_cast<uintptr_t>(a.positions) | reinterpret_cast<uintptr_t>(a.slots)) & 15) == 0) {
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            reinterpret_cast<longlong2 *>(a.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
            reinterpret_cast<longlong2 *>(a.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t0 + i < a.tokens) {
                    a.positions[t0 + i] = pos[i];
                    a.slots[t0 + i] = slot[i];
                }
        }
    }
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
    if (requests > kMaxRequests || n_free >= lim || tokens >= lim || max_pages >= lim || page_size > 65536 ||
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
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kv_plan_kernel), smem);
    if (e != cudaSuccess) return WSW_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    const unsigned ncta = tokens > 8192 ? 8 : 1;
    const int64_t want = requests > (tokens + 3) / 4 ? requests : (tokens + 3) / 4;
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
