// attn_prefix.cu -- host entry of the attention over shared prefixes, its plan and its join.
//
// Four launches, each behind the one before: the plan (which requests share what, and the list
// of tiles), the prefixes (attn_prefix.cuh), the rest of each request's positions
// (attn_paged.cuh, from first[r] on) and the join:
//   M = max_i m_i;  out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i;  lse = ln 2 (M + log2 sum_i ...)
// over the pieces i of a row's prefix and the rest.  A row reads its pieces' (m, l) first, a lane each,
// then their sums; a piece's maximum and sum stay apart until here, so that no logarithm is rounded
// in between.
#include "attn_prefix.cuh"
#include "kv_rows.cuh"

namespace wsw {
namespace prefix {

#define WSW_PREFIX_DECLARE(CT) template <> cudaError_t launch_prefix<CT>(const Args &, int, cudaStream_t, int);
WSW_PREFIX_DECLARE(WSW_F16)
WSW_PREFIX_DECLARE(WSW_BF16)
WSW_PREFIX_DECLARE(WSW_Q8_0)

namespace {

constexpr int kMaxGroups = 16384;  // three words of shared memory each
constexpr int kPlanThreads = 1024;
constexpr int64_t kEachBytes = int64_t(128) << 20;
// Tiles that a piece costs.  16 x 4 requests of 4 x 8 heads behind 4096 positions, bf16: 57 us with none, 56 with 3, 54 with 7, 55 with
// 14; 1 x 256 behind 8192, q8_0: 89, 85, 84, 85.  (CTAs with a single piece each, where there are enough for that, lengthened
// the plan: 6 us more for 16 x 4.)
constexpr int kPiece = 7;

// Parts of q by types.
int q_parts(int dtype, int cache) {
    if (dtype == WSW_F32) return cache == WSW_BF16 ? 3 : 2;
    return dtype == WSW_F16 && cache == WSW_BF16 ? 2 : 1;
}
// Row tiles of a unit.  Two read K and V half as often, for groups of more than 128 rows a head (several parts of q would leave
// no room for the ring), but an SM's two slots then work on one tile: they pay from some kRowTiles tiles of 128 rows and
// 128 positions for each SM.  4 heads of 128, bf16, group 8, us with one and with two: 32 requests behind 8192 / 32768
// positions 31 / 50 and 37 / 58 (3 / 13 tiles), 64 behind 32768 65 and 66 (27), 128 behind 8192 / 16384 / 32768 41 / 59 / 96
// and 44 / 59 / 92 (13 / 27 / 54), 256 behind 32768 166 and 153 (108).
constexpr int kRowTiles = 20;
int row_tiles(int64_t requests, int64_t group, int64_t groups, int parts, int64_t heads, int64_t max_len) {
    const int64_t rows = requests * group;
    return parts == 1 && rows > 128 * groups && heads * (rows / 128) * (max_len / 128) > kRowTiles * kCtas ? 2 : 1;
}

struct PlanArgs {
    const int32_t *cu, *prefix, *lens;
    int *begin, *off, *used, *rep, *stride, *run;  // as Plan
    int2 *start;
    int *first;    // [requests] where the rest begins
    int4 *pieces;  // [requests] what the join needs of its group (Pieces); rows 0: it shares nothing
    int32_t *err;
    int requests, groups, max_len, heads, group, unit_rows, tile;
};

__global__ void __launch_bounds__(kPlanThreads, 1) prefix_plan_kernel(const PlanArgs a) {
    extern __shared__ int sm[];
    __shared__ int scan_sm[33];
    int *begin = sm, *used = begin + a.groups + 1, *off = used + a.groups;
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    pdl_wait();
    // ---- the groups' bounds: cu cut to [0, requests], and never below the one before
    const int per = (a.groups + nt) / nt;  // of groups + 1
    const int i0 = min(tid * per, a.groups + 1), i1 = min(i0 + per, a.groups + 1);
    int err = 0, most = 0;
    for (int i = i0; i < i1; ++i) most = max(most, min(max(a.cu[i], 0), a.requests));
    int upto = most;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(WSW_FULL_MASK, upto, d);
        if (lane >= d) upto = max(upto, y);
    }
    if (lane == 31) scan_sm[warp] = upto;
    __syncthreads();
    int before = __shfl_up_sync(WSW_FULL_MASK, upto, 1);
    if (lane == 0) before = 0;
    for (int w = 0; w < warp; ++w) before = max(before, scan_sm[w]);
    for (int i = i0; i < i1; ++i) {
        const int x = a.cu[i];
        before = max(before, min(max(x, 0), a.requests));
        if (before != x) err |= 4;
        begin[i] = before;
    }
    __syncthreads();
    // ---- the prefixes
    const int g0 = min(i0, a.groups), g1 = min(i1, a.groups);
    auto units = [&](int g) {  // of a KV head
        return ((begin[g + 1] - begin[g]) * a.group + a.unit_rows - 1) / a.unit_rows;
    };
    auto tiles = [&](int g) { return (used[g] + a.tile - 1) / a.tile; };
    auto group_of = [&](int r) {  // the last group that begins at r or before
        int lo = 0, n = a.groups;
        while (n > 1) {
            const int half = n >> 1;
            if (begin[lo + half] <= r) lo += half;
            n -= half;
        }
        return lo;
    };
    auto reaches = [&](int r, int n) { return min(a.lens[r], a.max_len) >= n; };
    // The prefix is read through the first request that reaches it, mostly the group's first (off has it for a while).
    bool look = false;
    for (int g = g0; g < g1; ++g) {
        const int x = a.prefix[g], n = min(max(x, 0), a.max_len);
        if (n != x) err |= 4;
        // one request has nobody to share with
        const bool shares = n > 0 && begin[g + 1] - begin[g] > 1, at_once = shares && reaches(begin[g], n);
        used[g] = at_once ? n : shares ? -n : 0;
        off[g] = at_once ? begin[g] : 0x7fffffff;
        look |= shares && !at_once;
    }
    // Else all requests look together (four rows behind 60000 unused ones of their group: 0.5 ms a call, as
    // one thread's loop 3.9; with the unused rows outside 0.38).
    if (__syncthreads_or(look)) {
        for (int r = begin[0] + tid; r < begin[a.groups]; r += nt) {
            const int g = group_of(r);
            if (used[g] < 0 && reaches(r, -used[g])) atomicMin(&off[g], r);
        }
        __syncthreads();
    }
    int sum = 0, count = 0;
    for (int g = g0; g < g1; ++g) {
        used[g] = off[g] < a.requests ? abs(used[g]) : 0;
        a.used[g] = used[g];
        a.rep[g] = off[g] < a.requests ? off[g] : 0;
        if (used[g] > 0) {
            count += a.heads * units(g);
            sum += a.heads * units(g) * tiles(g);
        }
    }
    // ---- the list: a piece of a unit costs its CTA kPiece tiles beside its own (start, queries, its sums' way out), so
    // that units have as many places more
    int total, all_units;
    block_scan(sum, 0x7fffffff, scan_sm, &total);
    block_scan(count, 0x7fffffff, scan_sm, &all_units);
    int run = (total + kPiece * all_units + kCtas - 1) / kCtas;
    run = max(run, 1);
    auto stride = [&](int g) { return used[g] == 0 ? 0 : tiles(g) + kPiece; };
    sum = 0;
    for (int g = g0; g < g1; ++g) sum += a.heads * units(g) * stride(g);
    int at = block_scan(sum, 0x7fffffff, scan_sm, &total);
    for (int g = g0; g < g1; ++g) {
        a.off[g] = off[g] = at;
        a.begin[g] = begin[g];
        a.stride[g] = stride(g);
        at += a.heads * units(g) * stride(g);
    }
    if (tid == 0) {
        a.off[a.groups] = total;
        a.begin[a.groups] = begin[a.groups];
        a.run[0] = run;
    }
    if (err && a.err) atomicOr(a.err, err);
    __syncthreads();
    // ---- where each CTA begins: the last group whose part begins there or before
    for (int c = tid; c < kCtas; c += nt) {
        const int64_t pos = static_cast<int64_t>(c) * run;
        int lo = 0, n = a.groups;
        while (n > 1) {
            const int half = n >> 1;
            if (off[lo + half] <= pos) lo += half;
            n -= half;
        }
        a.start[c] = pos < total ? make_int2(lo, static_cast<int>(pos) - off[lo]) : make_int2(-1, 0);
    }
    // ---- each request's part
    for (int r = tid; r < a.requests; r += nt) {
        const int lo = group_of(r);
        const bool in = r >= begin[0] && r < begin[a.groups];
        const bool shares = in && used[lo] > 0 && reaches(r, used[lo]);
        a.first[r] = shares ? used[lo] : 0;
        a.pieces[r] = shares ? make_int4((begin[lo + 1] - begin[lo]) * a.group, (r - begin[lo]) * a.group, off[lo], used[lo])
                             : make_int4(0, 0, 0, 0);
    }
}

struct JoinArgs {
    const int *run;      // [1] places of a CTA; 0: a wait ran out
    const int4 *pieces;  // [requests]: query rows of its group per KV head, its own ones' place there, the group's place
                         // in the list, its prefix's positions
    const float *rec, *whole;
    const float *rest;   // [rows][D]
    const float2 *ml;    // [rows]
    void *out;
    float *lse;
    int q_heads, group, row_shift, tile_shift, dtype;  // log2 of a unit's rows, of a tile's positions
};

// A warp for each query head of a request.
template <int D>
__global__ void __launch_bounds__(256) prefix_join_kernel(const JoinArgs a) {
    constexpr int N = D / 32, kRec = D + kHead;  // values of a lane
    using V = std::conditional_t<N == 4, float4, float2>;
    const int lane = threadIdx.x & 31;
    const int req = blockIdx.y, head = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t row = static_cast<int64_t>(req) * a.q_heads + head;
    pdl_launch_dependents();
    pdl_wait();
    if (head >= a.q_heads) return;
    const int4 of = a.pieces[req];
    const int run = *a.run;
    const V rest = *reinterpret_cast<const V *>(a.rest + row * D + lane * N);
    const float2 ml = a.ml[row];
    float s[N], m = ml.x, l = ml.y;
    const float *r = reinterpret_cast<const float *>(&rest);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = r[i] * l;  // the rest comes divided by its sum
    if (of.x > 0 && run == 0) l = __int_as_float(0x7fc00000);
    if (of.x > 0 && run > 0) {
        const int unit_rows = 1 << a.row_shift, nt = ((of.w - 1) >> a.tile_shift) + 1;
        const int kv = head / a.group, in = of.y + head - kv * a.group;
        const int unit = kv * (((of.x - 1) >> a.row_shift) + 1) + (in >> a.row_shift);
        const int stride = nt + kPiece;
        const int first = of.z + unit * stride, c0 = first / run, c1 = (first + nt - 1) / run;
        const int n = c1 - c0 + 1;
        // piece k: a unit that one CTA has whole, or of CTA c0 + k its last piece (k = 0) or its first
        const int64_t apart = static_cast<int64_t>(2) * unit_rows * kRec;
        const float *one = n == 1 ? a.whole + row * kRec
                                  : a.rec + (static_cast<int64_t>(c0) * 2 * unit_rows + (in & (unit_rows - 1))) * kRec;
        // four at a time: their sums and values on their way together, then raised to a common maximum
        for (int k0 = 0; k0 < n; k0 += 4) {
            float2 pml[4];
            V v[4];
            float mx = m;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float *p = n == 1 ? one : one + (k0 + k) * apart + (k0 + k == 0 ? static_cast<int64_t>(unit_rows) * kRec : 0);
                pml[k] = make_float2(-INFINITY, 0.f);
                if (k0 + k < n) {
                    pml[k] = *reinterpret_cast<const float2 *>(p);
                    v[k] = *reinterpret_cast<const V *>(p + kHead + lane * N);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) mx = fmaxf(mx, pml[k].x);
            const float f = paged::weight(m, mx);
            l *= f;
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = f == 0.f ? 0.f : s[i] * f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k0 + k >= n) break;
                const float w = paged::weight(pml[k].x, mx);
                const float *x = reinterpret_cast<const float *>(&v[k]);
#pragma unroll
                for (int i = 0; i < N; ++i) s[i] = w == 0.f ? s[i] : fmaf(x[i], w, s[i]);
                l = fmaf(pml[k].y, w, l);
            }
            m = mx;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (lane == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * paged::kLn2;
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] *= inv;
    const int64_t at = row * D + lane * N;
    if (a.dtype == WSW_F32) {
        *reinterpret_cast<V *>(static_cast<float *>(a.out) + at) = *reinterpret_cast<const V *>(s);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at + i) = paged::pack16(a.dtype, s[i], s[i + 1]);
    }
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// The workspace: the paged attention's part first (its counters stay at the beginning whatever the sizes),
// the plan, the prefixes' pieces and whole units, the rest's results.
struct Room {
    size_t plan, rec, whole, rest, ml, bytes;
};
Room room(int64_t requests, int64_t groups, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
    Room w;
    const size_t rows = static_cast<size_t>(requests) * q_heads, rec = static_cast<size_t>(head_dim + kHead) * 4;
    // the most that any types and lengths need
    const int rt = row_tiles(requests, q_heads / kv_heads, groups, 1, kv_heads, int64_t(1) << 31);
    w.plan = align256(wsw_attn_paged_decode_workspace_bytes(requests, q_heads, kv_heads, head_dim));
    w.rec = w.plan + align256((2 * kCtas + 4 * static_cast<size_t>(requests) + 5 * (static_cast<size_t>(groups) + 1) + 1 +
                               static_cast<size_t>(requests)) * 4);
    w.whole = w.rec + static_cast<size_t>(kCtas) * 2 * rt * 128 * rec;
    w.rest = w.whole + align256(rows * rec);
    w.ml = w.rest + align256(rows * head_dim * 4);
    w.bytes = w.ml + rows * 8;
    return w;
}

}  // namespace
}  // namespace prefix
}  // namespace wsw

extern "C" size_t wsw_attn_paged_prefix_workspace_bytes(int64_t requests, int64_t groups, int64_t q_heads,
                                                        int64_t kv_heads, int64_t head_dim) {
    using namespace wsw::prefix;
    if (requests < 0 || groups < 1 || groups > kMaxGroups || (head_dim != 64 && head_dim != 128) ||
        wsw_attn_paged_decode_workspace_bytes(requests, q_heads, kv_heads, head_dim) == 0)
        return 0;
    return room(requests, groups, q_heads, kv_heads, head_dim).bytes;
}

extern "C" int wsw_attn_paged_prefix(const void *q, int32_t dtype, int64_t requests, int64_t q_heads,
                                     const wsw_kv_cache *cache, const int32_t *table, int64_t max_pages,
                                     int64_t table_stride, const int32_t *lens, const int32_t *cu_groups,
                                     int64_t groups, const int32_t *prefix_len, int32_t share, float scale,
                                     float softcap, const float *slopes, void *out, float *lse, int32_t *err_flag, void *ws,
                                     size_t ws_bytes, void *stream, const wsw_launch_opts *opts) {
    using namespace wsw;
    using namespace wsw::prefix;
    Opts o;
    int st = resolve_opts(opts, &o);
    if (st != WSW_OK) return st;
    paged::Args rest;
    int rows = 0;
    int64_t list = 0;
    st = paged::prepare(q, dtype, requests, q_heads, cache, table, max_pages, table_stride, lens, scale, softcap, 0, slopes,
                        out, lse, err_flag, &rest, &rows, &list);
    if (st != WSW_OK) return st;
    if (groups < 1 || (share != 0 && share != 1)) return WSW_ERR_INVALID_ARG;
    if (groups > kMaxGroups || rest.kv.head_dim == 256) return WSW_ERR_UNSUPPORTED;
    if (requests == 0) return WSW_OK;
    if (!cu_groups || !prefix_len || !ws) return WSW_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(cu_groups) | reinterpret_cast<uintptr_t>(prefix_len)) & 3) ||
        (reinterpret_cast<uintptr_t>(ws) & 255))
        return WSW_ERR_MISALIGNED;
    const int64_t kv_heads = cache->heads, group = rest.group;
    // places of the longest list, units * (longest + kPiece) of tiles of 64 positions or more, are counted in 32 bits; the limit
    // is above them, longest <= max_len / 64 + 1
    const int64_t units = kv_heads * (requests * group / 128 + groups), longest = (rest.max_len + 63) / 64;
    if (requests * q_heads > (int64_t(1) << 30) || units * (rest.max_len / 16 + 9) >= (int64_t(1) << 31) - 65536)
        return WSW_ERR_UNSUPPORTED;
    const Room w = room(requests, groups, q_heads, kv_heads, cache->head_dim);
    if (ws_bytes < w.bytes) return WSW_ERR_WORKSPACE;
    DeviceInfo di;
    if (!device_info(&di, &st)) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned char *base = static_cast<unsigned char *>(ws);
    paged::place(&rest, ws, rows);
    // What all requests list of a prefix comes from HBM once anyhow while it stays in L2, and four launches cost 9 us
    // more than one: 4 heads of 128, bf16, group 8, one prefix of 8192 for 4 / 8 / 16 requests (68 / 135 / 271 MB in all) 30 /
    // 31 / 32 us shared and 22 / 25 / 39 each on its own; 16 prefixes of 1024 / 2048 / 4096 for 4 each (143 / 277 / 546 MB) 31 /
    // 37 / 53 and 25 / 38 / 60; fp32 over q8_0, 8 / 16 / 32 requests behind 8192 (72 / 143 / 286 MB) 39 / 41 / 42 and 31 / 42 / 65.
    // Lengths stay on the device: the table's width stands for them.
    const int64_t row_bytes = 2 * kv_heads * (cache->dtype == WSW_Q8_0 ? cache->head_dim * 17 / 16 : cache->head_dim * 2);
    if (!share && requests * static_cast<int64_t>(rest.max_len) <= kEachBytes / row_bytes)
        return paged::launch_paged(rest, cache->dtype, rows, list, s, o.pdl) == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;

    const int rt = row_tiles(requests, group, groups, q_parts(dtype, cache->dtype), kv_heads, rest.max_len);
    PlanArgs p;
    p.cu = cu_groups; p.prefix = prefix_len; p.lens = lens; p.err = err_flag;
    p.pieces = reinterpret_cast<int4 *>(base + w.plan);
    p.start = reinterpret_cast<int2 *>(p.pieces + requests);
    p.begin = reinterpret_cast<int *>(p.start + kCtas);
    p.off = p.begin + groups + 1;
    p.used = p.off + groups + 1;
    p.rep = p.used + groups + 1;
    p.stride = p.rep + groups + 1;
    p.run = p.stride + groups + 1;
    p.first = p.run + 1;
    p.requests = rest.requests; p.groups = static_cast<int>(groups); p.max_len = rest.max_len;
    p.heads = rest.kv.heads; p.group = rest.group; p.unit_rows = 128 * rt; p.tile = tile_positions(dtype == WSW_F32, cache->dtype, rt);
    const int plan_smem = static_cast<int>((3 * groups + 1) * 4);
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(prefix_plan_kernel), (3 * kMaxGroups + 1) * 4);
    if (e == cudaSuccess)
        e = launch(prefix_plan_kernel, dim3(1), dim3(requests > 256 || groups > 256 ? kPlanThreads : 256), plan_smem, s, o.pdl, p);
    if (e != cudaSuccess) return WSW_ERR_CUDA;

    Args a;
    a.q = q; a.slopes = slopes; a.table = table; a.lens = lens; a.err = err_flag;
    a.plan = Plan{p.begin, p.off, p.used, p.rep, p.stride, p.run, p.start};
    a.rec = reinterpret_cast<float *>(base + w.rec);
    a.whole = reinterpret_cast<float *>(base + w.whole);
    a.kv = rest.kv;
    a.table_stride = table_stride;
    a.scale2 = std::fabs(rest.scale2);
    a.cap_in = std::fabs(rest.cap_in);
    a.cap_out = rest.cap_out;
    a.q_heads = rest.q_heads; a.group = rest.group; a.groups = p.groups; a.max_len = rest.max_len;
    a.dtype = dtype;
    a.negative = scale < 0.f;
    const int64_t most = units * (longest + kPiece);  // places of the list
    const int ctas = static_cast<int>(most < kCtas ? most : kCtas);
    if (cache->dtype == WSW_F16) e = launch_prefix<WSW_F16>(a, rt, s, ctas);
    else if (cache->dtype == WSW_BF16) e = launch_prefix<WSW_BF16>(a, rt, s, ctas);
    else e = launch_prefix<WSW_Q8_0>(a, rt, s, ctas);
    if (e != cudaSuccess) return WSW_ERR_CUDA;

    rest.first = p.first;
    rest.out = base + w.rest;
    rest.ml = reinterpret_cast<float2 *>(base + w.ml);
    e = paged::launch_paged(rest, cache->dtype, rows, list, s, true);
    if (e != cudaSuccess) return WSW_ERR_CUDA;

    JoinArgs j;
    j.run = p.run;
    j.pieces = p.pieces;
    j.rec = a.rec; j.whole = a.whole;
    j.rest = reinterpret_cast<const float *>(rest.out); j.ml = rest.ml;
    j.out = out; j.lse = lse;
    j.q_heads = rest.q_heads; j.group = rest.group; j.dtype = dtype;
    j.row_shift = rt == 2 ? 8 : 7;
    j.tile_shift = p.tile == 128 ? 7 : 6;
    const dim3 grid(static_cast<unsigned>((q_heads + 7) / 8), static_cast<unsigned>(requests));
    e = rest.kv.head_dim == 64 ? launch(prefix_join_kernel<64>, grid, dim3(256), 0, s, true, j)
                               : launch(prefix_join_kernel<128>, grid, dim3(256), 0, s, true, j);
    return e == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
}
