// logprobs.cu -- log probability, rank, entropy and top alternatives of each row of
// logits, in one pass.
//
//   y_j = scale x_j;  lse = ln sum exp(y_j);  logprob = y_t - lse
//   entropy = ln S - E / S with S = sum e_j, E = sum e_j (y_j - m), e_j = exp(y_j - m)
//   (-sum p ln p with p = e / S; a peaked row's terms are both small, which leaves an absolute error of
//   about 2^-24: what of S - 1 is below that is lost in S)
//
// One pass: a thread keeps a running maximum m, S and E in fp32 over its vectors (kept in
// the log2 domain, e = 2^((x - m) scale log2 e)); when m grows by D (log2 units), S and E
// become f S and f (E - D S), f = 2^-D.  The rank is a count of the values
// that reach the token's logit, 16-bit ones compared and counted in pairs.
//
// Top k: topk_rows.cuh.
//
// Rows are split over CTAs when there are few; each split leaves (m, S, E, count, k keys) in
// the workspace and the row's last CTA joins them in a fixed order.
//
// Bound: the logits once, but a bf16 logit's arithmetic costs more issue slots than its two
// bytes cost of HBM's time.  2047 rows of 50021: bf16 63 us with 5 alternatives (3.3 TB/s) and
// 47 us with none, fp32 75 and 70 us (5.4 and 5.8 TB/s); sorted rows, the worst order, take 145 us
// (bf16, rising).  One row of 152064 fp32
// values: 11 us with 20 alternatives, 4.4 us with none; 64 rows with 8: 18 us.
#include <cmath>

#include "topk_rows.cuh"

namespace wsw {
namespace {

using namespace topk;

struct LpArgs {
    const void *x;
    const int32_t *tokens;
    float *logprob, *lse, *entropy, *top_logprob;
    int32_t *rank, *top_id;
    unsigned *cnt;  // [rows] arrival counters (zero between calls)
    float *part;    // [rows][splits][rec] records
    int64_t ld, rows;
    float scale, c;  // c = scale log2 e
    int vocab, top, splits, chunk, rec;
};

// the same among T's values, for an x that is one
template <typename T>
__device__ __forceinline__ float above_in(float x) {
    if constexpr (sizeof(T) == 4) {
        return above(x);
    } else {
        if (!(x < INFINITY)) return NAN;
        constexpr bool bf = Elem<T>::kBf16;
        if (x == 0.f) return bf ? __uint_as_float(1u << 16) : __half2float(__ushort_as_half(1));
        const uint16_t b = bf ? __float_as_uint(x) >> 16 : __half_as_ushort(__float2half_rn(x));
        const uint16_t n = static_cast<uint16_t>(b + (x > 0.f ? 1 : -1));
        return bf ? __uint_as_float(static_cast<uint32_t>(n) << 16) : __half2float(__ushort_as_half(n));
    }
}

// Counts a tile's values from a bound up.  16-bit values are compared and counted in pairs (at
// most 16 of each half: exact); the bound is one of their type's values, or NaN for nothing.
template <typename T>
struct Counter {
    using Pair = typename Elem<T>::Pair;
    Pair n = Elem<T>::pair(0.f);
    __device__ static Pair bound(float b) { return Elem<T>::pair(b); }
    __device__ void add(const uint4 &raw, const float (&)[8], Pair b) {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) n = __hadd2(n, __hge2(*reinterpret_cast<const Pair *>(&w[i]), b));
    }
    __device__ int total() const {
        const float2 f = Elem<T>::floats(n);
        return static_cast<int>(f.x + f.y);
    }
};
template <>
struct Counter<float> {
    int n = 0;
    __device__ static float bound(float b) { return b; }
    __device__ void add(const uint4 &, const float (&x)[4], float b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) n += x[i] >= b;
    }
    __device__ int total() const { return n; }
};

// Results of a row from its sums; keys: its top, in order.  Every thread calls it with
// thread 0's sums and count in sm.sums[0], sm.count[0].
__device__ __forceinline__ void finish(const LpArgs &a, Shared &sm, int64_t row, float xt) {
    const Sums r = sm.sums[0];
    const float ln_s = logf(r.s);
    const bool none = r.s == 0.f;  // nothing but -inf
    const int tid = threadIdx.x;
    if (tid == 0) {
        a.lse[row] = none ? -INFINITY : fmaf(r.m, a.scale, ln_s);
        a.entropy[row] = none ? 0.f : ln_s - r.e / r.s * kLn2;
        if (a.tokens) {
            const int t = a.tokens[row];
            const bool ok = t >= 0 && t < a.vocab;
            a.logprob[row] = !ok ? NAN : none ? -INFINITY : (xt - r.m) * a.scale - ln_s;
            a.rank[row] = ok ? sm.count[0] : -1;
        }
    }
    if (tid < a.top) {
        const uint64_t key = tid < min(sm.n, kCap) ? sm.best[tid] : 0;
        const float x = unord(static_cast<uint32_t>(key >> 32));
        a.top_id[row * a.top + tid] = key ? static_cast<int>(~static_cast<uint32_t>(key)) : -1;
        a.top_logprob[row * a.top + tid] = none ? -INFINITY : !key ? NAN : (x - r.m) * a.scale - ln_s;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 8 : 6) logprobs_kernel(const LpArgs a) {
    constexpr int V = Elem<T>::kVec;
    constexpr int kTile = kThreads * kUnroll * V;  // values per tile (4096 or 8192)
    __shared__ Shared sm;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.splits;
    const int split = static_cast<int>(blockIdx.x - row * a.splits);
    pdl_launch_dependents();
    pdl_wait();
    const T *x = static_cast<const T *>(a.x) + row * a.ld;
    // The row as 16-byte vectors: `lead` values come before the first.  The split takes the
    // vectors of [lo, hi); the first split also the values before them, the last one those
    // after the last whole vector: at most V - 1 each, one for each of the first threads.
    const int lead = min(static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T)), a.vocab);
    const int64_t begin = lead + static_cast<int64_t>(split) * a.chunk;
    const int whole = lead + (a.vocab - lead) / V * V;  // end of the last whole vector
    const int lo = static_cast<int>(min(begin, static_cast<int64_t>(whole)));
    const int hi = static_cast<int>(min(begin + a.chunk, static_cast<int64_t>(whole)));
    const float c = a.c;
    const int k = a.top;

    uint4 raw[kUnroll];
    auto fetch = [&](int tile0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int at = tile0 + (u * kThreads + tid) * V;
            raw[u] = make_uint4(Elem<T>::kLow, Elem<T>::kLow, Elem<T>::kLow, Elem<T>::kLow);
            if (at < hi) raw[u] = __ldg(reinterpret_cast<const uint4 *>(x + at));
        }
    };
    fetch(lo);

    // rank: x_j >= xt for j < t, x_j >= the next value for j > t; NaN: nothing counts.  A vector
    // that holds t counts as after it; its equal values before t are added here.
    const int t = a.tokens ? a.tokens[row] : -1;
    const bool has_t = t >= 0 && t < a.vocab;
    const float xt = has_t ? Elem<T>::get(x, t) : NAN;
    const float xt_next = above(xt);
    const auto ge_t = Counter<T>::bound(xt), gt_t = Counter<T>::bound(above_in<T>(xt)), none = Counter<T>::bound(NAN);
    int count = 0;
    if (tid == 64 && has_t && t >= lo && t < hi)
        for (int i = lo + (t - lo) / V * V; i < t; ++i) count += Elem<T>::get(x, i) == xt;
    Sums s{-FLT_MAX, 0.f, 0.f};
    if (tid == 0) {
        sm.n = sm.nvec = 0;
        sm.thr = -INFINITY;
    }
    __syncthreads();
    {
        int i = -1;
        if (split == 0 && tid < lead) i = tid;
        if (split == a.splits - 1 && tid >= 32 && tid - 32 < a.vocab - whole) i = whole + tid - 32;
        if (i >= 0) {
            const float v = Elem<T>::get(x, i);
            count += v >= (i < t ? xt : xt_next);
            if (!(v == -INFINITY)) {
                s.m = fmaxf(v, -FLT_MAX);
                s.s = v != v || v == INFINITY ? NAN : 1.f;
            }
            if (k > 0) push(sm, key_of(v, i));
        }
    }
    const uint64_t c2 = f2(c, c);

    int since = 0, filled = 0;  // tiles since the buffer was looked at, candidates known then
    int group0 = lo;
    bool first = true;
    float thr = -INFINITY;
    for (int tile0 = lo; tile0 < hi; tile0 += kTile) {
        float v[kUnroll][V];
        float vm[kUnroll];
        Counter<T> counted;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            Elem<T>::unpack(raw[u], v[u]);
            const int at = tile0 + (u * kThreads + tid) * V;
            counted.add(raw[u], v[u], at >= hi ? none : at + V <= t ? ge_t : gt_t);
        }
        count += counted.total();
        if (tile0 + kTile < hi) fetch(tile0 + kTile);  // in flight during this tile's arithmetic
        float tm = -INFINITY;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            vm[u] = fmaxf(v[u][0], v[u][1]);
#pragma unroll
            for (int i = 2; i < V; i += 2) vm[u] = max3(vm[u], v[u][i], v[u][i + 1]);
            tm = fmaxf(tm, vm[u]);
        }
        if (tm > s.m) raise(s, tm, c);
        const uint64_t nm2 = f2(-s.m, -s.m);
        uint64_t ss = 0ull, ee = 0ull;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                uint64_t d2 = f2(v[u][i], v[u][i + 1]);
                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d2) : "l"(nm2));
                asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d2) : "l"(c2));
                float d0, d1;
                asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(d2));
                d0 = max_nan(d0, -200.f);  // 2^-200 is 0, and 0 times -200 too
                d1 = max_nan(d1, -200.f);
                const uint64_t e2 = f2(ex2(d0), ex2(d1));
                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(ss) : "l"(e2));
                asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(ee) : "l"(e2), "l"(f2(d0, d1)));
            }
        {
            float x0, x1;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(ss));
            s.s += x0 + x1;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(ee));
            s.e += x0 + x1;
        }
        if (k == 0) continue;
        // what reaches the first tile's bound; after a cut, only what beats the k-th best
        if (first) thr = reached_by(sm, tm, k);
        if (tm >= thr) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int at = tile0 + (u * kThreads + tid) * V;
                if (!(vm[u] >= thr) || at >= hi) continue;
                filled = atomicAdd(&sm.nvec, 1);
                if (filled >= kVecs) continue;
                sm.vec[filled] = pack<T>(v[u]);
                sm.vec_at[filled] = at;
            }
        }
        if (!first && ++since < kLook && tile0 + kTile < hi) continue;
        // one answer for the whole block (a large k's bound is loose: it is cut after the first of
        // several tiles)
        const bool last = tile0 + kTile >= hi;
        if (__syncthreads_or(filled > kKeep || last || (first && k > 8))) {
            const int end = min(tile0 + kTile, hi);
            select(sm, x, group0, end, thr, k, LoadAligned{});
            group0 = end;
            thr = after_cut(sm, end, k);
        }
        first = false;
        since = filled = 0;
    }
    if (k > 0 && lo >= hi) {
        __syncthreads();
        cut(sm, k);
    }
    s = block_sums(sm, s, count, c);
    if (tid == 0) {
        sm.sums[0] = s;
        sm.count[0] = count;
    }
    __syncthreads();
    if (a.splits == 1) {
        finish(a, sm, row, xt);
        return;
    }

    float *rec = a.part + (row * a.splits + split) * a.rec;
    if (tid == 0) *reinterpret_cast<float4 *>(rec) = make_float4(s.m, s.s, s.e, __int_as_float(count));
    if (tid < k) reinterpret_cast<uint64_t *>(rec + 4)[tid] = tid < sm.n ? sm.best[tid] : 0;
    // the block barrier orders the record before thread 0's arrival, whose release publishes
    // it; the last arrival's acquire orders the reads below after every record
    __syncthreads();
    if (tid == 0) {
        unsigned old;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(a.cnt + row) : "memory");
        sm.last = old == static_cast<unsigned>(a.splits - 1);
    }
    __syncthreads();
    if (!sm.last) return;
    const float *recs = a.part + row * a.splits * a.rec;
    s = Sums{-FLT_MAX, 0.f, 0.f};
    count = 0;
    for (int i = tid; i < a.splits; i += kThreads) {
        const float4 r = __ldcg(reinterpret_cast<const float4 *>(recs + static_cast<int64_t>(i) * a.rec));
        s = join(s, Sums{r.x, r.y, r.z}, c);
        count += __float_as_int(r.w);
    }
    if (k > 0) join_keys(sm, recs, a.rec, a.splits, k);
    s = block_sums(sm, s, count, c);
    __syncthreads();
    if (tid == 0) {
        sm.sums[0] = s;
        sm.count[0] = count;
        a.cnt[row] = 0u;  // ready for the next call
    }
    __syncthreads();
    finish(a, sm, row, xt);
}

// Rows are split only while there are at most kTargetCtas / 2 of them.  The counters' place does
// not depend on the sizes: one workspace serves calls of different sizes in turn.
constexpr size_t kCounterBytes = 2048;
static_assert(kTargetCtas / 2 * 4 <= kCounterBytes, "counters");

}  // namespace
}  // namespace wsw

extern "C" size_t wsw_token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int64_t top) {
    using namespace wsw;
    constexpr int64_t lim = int64_t(1) << 31;
    if (rows < 1 || vocab < 1 || rows >= lim || vocab >= lim || top < 0 || top > kMaxTop) return 0;
    int splits, chunk;
    split_rows(rows, vocab, &splits, &chunk);
    if (splits == 1) return 0;
    return kCounterBytes + static_cast<size_t>(rows) * splits * record_floats(top) * 4;
}

extern "C" int wsw_token_logprobs(const void *logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                                  const int32_t *tokens, float scale, int32_t top, float *logprob, int32_t *rank,
                                  float *lse, float *entropy, float *top_logprob, int32_t *top_id, void *ws,
                                  size_t ws_bytes, void *stream, const wsw_launch_opts *opts) {
    using namespace wsw;
    Opts o;
    int st = resolve_opts(opts, &o);
    if (st != WSW_OK) return st;
    if (dtype != WSW_F32 && dtype != WSW_F16 && dtype != WSW_BF16) return WSW_ERR_UNSUPPORTED;
    if (rows < 0 || vocab < 1 || ld < vocab || !std::isfinite(scale * kLog2e) || !(scale > 0.f) || top < 0 || top > vocab)
        return WSW_ERR_INVALID_ARG;
    constexpr int64_t lim = int64_t(1) << 31;
    if (top > kMaxTop || vocab >= lim - 65536 || rows >= lim) return WSW_ERR_UNSUPPORTED;
    if (rows == 0) return WSW_OK;
    if (!logits || !lse || !entropy || (tokens && (!logprob || !rank)) || (!tokens && (logprob || rank)) ||
        (top > 0 && (!top_logprob || !top_id)))
        return WSW_ERR_INVALID_ARG;
    const uintptr_t al = reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(logprob) |
                         reinterpret_cast<uintptr_t>(rank) | reinterpret_cast<uintptr_t>(lse) |
                         reinterpret_cast<uintptr_t>(entropy) | reinterpret_cast<uintptr_t>(top_logprob) |
                         reinterpret_cast<uintptr_t>(top_id);
    if ((al & 3) || (reinterpret_cast<uintptr_t>(logits) & (dtype == WSW_F32 ? 3 : 1))) return WSW_ERR_MISALIGNED;
    const size_t need = wsw_token_logprobs_workspace_bytes(rows, vocab, top);
    if (need > 0) {
        if (!ws || ws_bytes < need) return WSW_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(ws) & 15) return WSW_ERR_MISALIGNED;
    }
    DeviceInfo di;
    if (!device_info(&di, &st)) return st;
    LpArgs a;
    a.x = logits; a.tokens = tokens;
    a.logprob = logprob; a.lse = lse; a.entropy = entropy; a.top_logprob = top_logprob;
    a.rank = rank; a.top_id = top_id;
    a.cnt = static_cast<unsigned *>(ws);
    a.part = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + (need ? kCounterBytes : 0));
    a.ld = ld; a.rows = rows;
    a.scale = scale;
    a.c = scale * kLog2e;
    a.vocab = static_cast<int>(vocab);
    a.top = top;
    a.rec = record_floats(top);
    split_rows(rows, vocab, &a.splits, &a.chunk);
    const int64_t ctas = rows * a.splits;
    if (ctas >= lim) return WSW_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(ctas));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == WSW_F32) e = launch(logprobs_kernel<float>, grid, dim3(kThreads), 0, s, o.pdl, a);
    else if (dtype == WSW_F16) e = launch(logprobs_kernel<__half>, grid, dim3(kThreads), 0, s, o.pdl, a);
    else e = launch(logprobs_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, o.pdl, a);
    return e == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
}
