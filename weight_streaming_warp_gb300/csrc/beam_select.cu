// beam_select.cu -- the next beams of every request from all its beams' logits, in one pass.
//
//   s[b][j] = score[b] + scale x[b][j] - lse_b,  lse_b = ln sum_i exp(scale x[b][i])
//   the candidates (b, j) in order of s; the first `beams` that do not end become the beams
//
// Nothing beyond a row's k = beams * (1 + end tokens) largest logits can be chosen: an end token
// takes one place in each row at most.  So a row is streamed once, as for its log probabilities
// (topk_rows.cuh), with its sum and its k best kept; rows are split over CTAs when there are few.
// The last CTA of a row joins its splits, the last row of a request merges the rows' lists: a lane
// holds the head of each beam's list, and a step finds the best head with two warp-wide
// maxima.
//
// The order of near candidates of different beams hangs on the difference of their lse, so that more
// than fp32 of it counts: a thread's sum of some hundred terms is fp32 (the errors of single terms,
// 2^-22 at most, have no common sign), the sums of threads and CTAs, the logarithm and the
// scores are 64 bits.  lse is off by some 1e-8, and by what the rounding of scale log2 e to
// fp32 (6e-8 at most) makes of the mean of the log probabilities, which all beams have nearly in
// common.  Rows of different alignment are summed in another order: beams whose k best are the
// same logits of the same tokens, and whose sums differ by less than 2^-20, count as equal,
// so that copies of a beam tie and rank by index.
//
// Bound: the logits once; as the log probabilities with alternatives, by the selection's dependent steps
// for few rows and by instructions for 16-bit logits.
#include "topk_rows.cuh"

namespace wsw {
namespace {

using namespace topk;

constexpr int kMaxBeams = 32;
constexpr int kMaxEnds = 8;
constexpr int kMaxRequests = 16384;

struct BeamArgs {
    const void *x;
    const float *scores;
    int32_t *parent, *token, *end_parent, *end_token;
    float *score, *end_score;
    unsigned *row_cnt, *req_cnt;  // arrival counters, zero between calls
    float *part;                  // [rows][splits][rec]: maximum, sum (64 bits), keys
    uint64_t *lists;              // [rows][1 + k]: lse (64 bits), keys
    int64_t ld;
    double scale;
    float c;                      // scale log2 e
    int vocab, beams, k, splits, chunk, rec, n_ends;
    int32_t ends[kMaxEnds];
};

struct BeamShared {
    Shared top;
    uint64_t cand[kMaxBeams * kMaxTop];  // order-preserving scores, 0: no candidate
    double sum[kWarps];
    double lse[kMaxBeams];
    float max[kWarps];
    int last;
};

__device__ __forceinline__ uint64_t ord64(double s) {
    if (!(s > -INFINITY) || !(s < INFINITY)) return 0;  // -inf, NaN
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(s + 0.0));
    return (u >> 63) ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ float unord64(uint64_t k) {
    return static_cast<float>(__longlong_as_double(static_cast<long long>((k >> 63) ? k & ~(1ull << 63) : ~k)));
}

// Arrive at a counter; whether this is the last of `expected` arrivals.  The block barrier before
// orders the block's writes before thread 0's arrival, whose release publishes them; the last
// one's acquire, and the barrier after, order the reads behind every arrival.
__device__ __forceinline__ bool arrive(unsigned *cnt, int expected, int *flag) {
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned old;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(cnt) : "memory");
        *flag = old == static_cast<unsigned>(expected - 1);
        if (*flag) *cnt = 0u;  // ready for the next call
    }
    __syncthreads();
    return *flag;
}

// The block's maximum and sum from the threads' (m, s), the sum in 64 bits; all threads get them.
__device__ __forceinline__ void block_total(const BeamArgs &a, BeamShared &sm, float m, double s, float &mx, double &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    mx = m;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mx = max_nan(mx, __shfl_xor_sync(WSW_FULL_MASK, mx, d));
    if (lane == 0) sm.max[warp] = mx;
    __syncthreads();
    mx = sm.max[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = max_nan(mx, sm.max[w]);
    total = s == 0. ? 0. : s * static_cast<double>(ex2((m - mx) * a.c));
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) total += __shfl_xor_sync(WSW_FULL_MASK, total, d);
    if (lane == 0) sm.sum[warp] = total;
    __syncthreads();
    total = 0.;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sm.sum[w];
}

// The request's answer, once all its rows' lists are there.  Every thread calls it.
__device__ __forceinline__ void merge(const BeamArgs &a, BeamShared &sm, int64_t request) {
    const int tid = threadIdx.x, k = a.k, n = a.beams * k;
    uint64_t *keys = sm.top.buf;
    static_assert(kMaxBeams * kMaxTop <= kCap, "keys");
    const uint64_t *lists = a.lists + request * a.beams * (1 + k);
    for (int i = tid; i < n; i += kThreads) {
        const int b = i / k;
        keys[i] = __ldcg(lists + i + b + 1);
    }
    if (tid < a.beams) sm.lse[tid] = __longlong_as_double(static_cast<long long>(__ldcg(lists + tid * (1 + k))));
    __syncthreads();
    // copies of a beam: the first one's lse
    double lse = 0.;
    if (tid < a.beams) {
        lse = sm.lse[tid];
        for (int b = 0; b < tid; ++b) {
            if (!(fabs(sm.lse[b] - lse) <= 9.5367431640625e-7)) continue;
            int i = 0;
            while (i < k && keys[b * k + i] == keys[tid * k + i]) ++i;
            if (i < k) continue;
            lse = sm.lse[b];
            break;
        }
    }
    __syncthreads();
    if (tid < a.beams) sm.lse[tid] = lse;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const int b = i / k;
        const double x = static_cast<double>(unord(static_cast<uint32_t>(keys[i] >> 32)));
        const double sc = static_cast<double>(a.scores[request * a.beams + b]);
        sm.cand[i] = keys[i] ? ord64(sc + (a.scale * x - sm.lse[b])) : 0;
    }
    __syncthreads();
    if (tid >= 32) return;
    const int64_t out = request * a.beams;
    int at = 0, alive = 0, ended = 0;
    uint64_t own = tid < a.beams ? sm.cand[tid * k] : 0;
#pragma unroll 1
    for (int rank = 0; alive < a.beams; ++rank) {
        const unsigned hi = static_cast<unsigned>(own >> 32);
        const unsigned mh = __reduce_max_sync(WSW_FULL_MASK, hi);
        if (mh == 0) break;  // no candidate is left (one has its highest bit or the next ones set)
        const unsigned lo = hi == mh ? static_cast<unsigned>(own) : 0;
        const unsigned ml = __reduce_max_sync(WSW_FULL_MASK, lo);
        const int best = __ffs(__ballot_sync(WSW_FULL_MASK, hi == mh && lo == ml)) - 1;  // ties: the lowest beam
        int token = 0;
        bool ends = false;
        if (tid == best) {
            token = static_cast<int>(~static_cast<uint32_t>(keys[tid * k + at]));
            for (int i = 0; i < a.n_ends; ++i) ends |= token == a.ends[i];
        }
        ends = __any_sync(WSW_FULL_MASK, ends);
        if (tid == best) {
            const int32_t row = static_cast<int32_t>(out + tid);
            if (!ends) {
                a.parent[out + alive] = row;
                a.token[out + alive] = token;
                a.score[out + alive] = unord64(own);
            } else if (rank < a.beams) {
                a.end_parent[out + ended] = row;
                a.end_token[out + ended] = token;
                a.end_score[out + ended] = unord64(own);
            }
            own = ++at < k ? sm.cand[tid * k + at] : 0;
        }
        alive += !ends;
        ended += ends && rank < a.beams;
    }
    // the places without a candidate
    for (int i = alive + tid; i < a.beams; i += 32) {
        a.parent[out + i] = a.token[out + i] = -1;
        a.score[out + i] = -INFINITY;
    }
    for (int i = ended + tid; a.end_parent && i < a.beams; i += 32) {
        a.end_parent[out + i] = a.end_token[out + i] = -1;
        a.end_score[out + i] = -INFINITY;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 8 : 6) beam_kernel(const __grid_constant__ BeamArgs a) {
    constexpr int V = Elem<T>::kVec;
    constexpr int kTile = kThreads * kUnroll * V;
    __shared__ BeamShared sm;
    Shared &top = sm.top;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.splits;
    const int split = static_cast<int>(blockIdx.x - row * a.splits);
    pdl_launch_dependents();
    pdl_wait();
    const T *x = static_cast<const T *>(a.x) + row * a.ld;
    // The row as 16-byte vectors behind `lead` values: the split takes the vectors of [lo, hi); the first
    // split also the values before them, the last one those after the last whole vector.
    const int lead = min(static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T)), a.vocab);
    const int64_t begin = lead + static_cast<int64_t>(split) * a.chunk;
    const int whole = lead + (a.vocab - lead) / V * V;
    const int lo = static_cast<int>(min(begin, static_cast<int64_t>(whole)));
    const int hi = static_cast<int>(min(begin + a.chunk, static_cast<int64_t>(whole)));
    const int k = a.k;

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
    float m = -FLT_MAX, s = 0.f;  // m >= -FLT_MAX: x - m is never (-inf) - (-inf)
    if (tid == 0) {
        top.n = top.nvec = 0;
        top.thr = -INFINITY;
    }
    __syncthreads();
    {
        int i = -1;
        if (split == 0 && tid < lead) i = tid;
        if (split == a.splits - 1 && tid >= 32 && tid - 32 < a.vocab - whole) i = whole + tid - 32;
        if (i >= 0) {
            const float v = Elem<T>::get(x, i);
            if (!(v == -INFINITY)) {
                m = fmaxf(v, -FLT_MAX);
                s = v != v || v == INFINITY ? NAN : 1.f;
            }
            push(top, key_of(v, i));
        }
    }
    const uint64_t c2 = f2(a.c, a.c);

    int since = 0, filled = 0;  // tiles since the buffer was looked at, candidates known then
    int group0 = lo;
    bool first = true;
    float thr = -INFINITY;
    for (int tile0 = lo; tile0 < hi; tile0 += kTile) {
        float v[kUnroll][V];
        float vm[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) Elem<T>::unpack(raw[u], v[u]);
        if (tile0 + kTile < hi) fetch(tile0 + kTile);  // in flight during this tile's arithmetic
        float tm = -INFINITY;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            vm[u] = fmaxf(v[u][0], v[u][1]);
#pragma unroll
            for (int i = 2; i < V; i += 2) vm[u] = max3(vm[u], v[u][i], v[u][i + 1]);
            tm = fmaxf(tm, vm[u]);
        }
        if (tm > m) {
            s = s == 0.f ? 0.f : s * ex2((m - tm) * a.c);  // before the first value the difference may be -inf
            m = tm;
        }
        const uint64_t nm2 = f2(-m, -m);
        uint64_t ss = 0ull;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                uint64_t d2 = f2(v[u][i], v[u][i + 1]);
                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d2) : "l"(nm2));
                asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d2) : "l"(c2));
                float d0, d1;
                asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(d2));
                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(ss) : "l"(f2(ex2(d0), ex2(d1))));
            }
        {
            float x0, x1;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(ss));
            s += x0 + x1;
        }
        // what reaches the first tile's bound; after a cut, only what beats the k-th best
        if (first) thr = reached_by(top, tm, k);
        if (tm >= thr) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int at = tile0 + (u * kThreads + tid) * V;
                if (!(vm[u] >= thr) || at >= hi) continue;
                filled = atomicAdd(&top.nvec, 1);
                if (filled >= kVecs) continue;
                top.vec[filled] = pack<T>(v[u]);
                top.vec_at[filled] = at;
            }
        }
        if (!first && ++since < kLook && tile0 + kTile < hi) continue;
        const bool last = tile0 + kTile >= hi;
        if (__syncthreads_or(filled > kKeep || last || (first && k > 8))) {
            const int end = min(tile0 + kTile, hi);
            select(top, x, group0, end, thr, k);
            group0 = end;
            thr = after_cut(top, end, k);
        }
        first = false;
        since = filled = 0;
    }
    if (lo >= hi) {
        __syncthreads();
        cut(top, k);
    }
    float mx;
    double total;
    block_total(a, sm, m, static_cast<double>(s), mx, total);
    if (a.splits > 1) {
        float *rec = a.part + (row * a.splits + split) * a.rec;
        if (tid == 0) {
            rec[0] = mx;
            reinterpret_cast<double *>(rec)[1] = total;
        }
        if (tid < k) reinterpret_cast<uint64_t *>(rec + 4)[tid] = tid < top.n ? top.best[tid] : 0;
        if (!arrive(a.row_cnt + row, a.splits, &sm.last)) return;
        const float *recs = a.part + row * a.splits * a.rec;
        m = -FLT_MAX;
        double sum = 0.;
        static_assert(kTargetCtas / 2 >= kThreads, "several splits a thread");
        for (int i = tid; i < a.splits; i += kThreads) {
            const float *r = recs + static_cast<int64_t>(i) * a.rec;
            const float rm = __ldcg(r);
            const double rs = __ldcg(reinterpret_cast<const double *>(r) + 1);
            const float mn = max_nan(m, rm);
            sum = (sum == 0. ? 0. : sum * static_cast<double>(ex2((m - mn) * a.c))) +
                  (rs == 0. ? 0. : rs * static_cast<double>(ex2((rm - mn) * a.c)));
            m = mn;
        }
        join_keys(top, recs, a.rec, a.splits, k);
        block_total(a, sm, m, sum, mx, total);
    }
    // the row's list; a row of nothing but -inf, with a NaN or with +inf has no candidate: lse -inf or NaN
    uint64_t *list = a.lists + row * (1 + k);
    if (tid == 0) list[0] = static_cast<uint64_t>(__double_as_longlong(a.scale * static_cast<double>(mx) + log(total)));
    if (tid < k) list[1 + tid] = tid < min(top.n, kCap) ? top.best[tid] : 0;
    const int64_t request = row / a.beams;
    if (arrive(a.req_cnt + request, a.beams, &sm.last)) merge(a, sm, request);
}

constexpr size_t kRowCounters = 2048;
static_assert(kTargetCtas / 2 * 4 <= kRowCounters, "counters");
// the counters' places do not depend on the sizes: one workspace serves calls of different sizes in turn
constexpr size_t kCounterBytes = kRowCounters + kMaxRequests * 4;

int64_t list_length(int64_t beams, int64_t vocab, int64_t n_ends) {
    const int64_t k = beams * (1 + n_ends);
    return k < vocab ? k : vocab;
}

}  // namespace
}  // namespace wsw

extern "C" size_t wsw_beam_select_workspace_bytes(int64_t requests, int64_t beams, int64_t vocab, int64_t n_ends) {
    using namespace wsw;
    constexpr int64_t lim = int64_t(1) << 31;
    if (requests < 1 || requests > kMaxRequests || beams < 1 || beams > kMaxBeams || vocab < 1 || vocab >= lim - 65536 ||
        n_ends < 0 || n_ends > kMaxEnds || beams * (1 + n_ends) > kMaxTop)
        return 0;
    int splits, chunk;
    const int64_t rows = requests * beams, k = list_length(beams, vocab, n_ends);
    split_rows(rows, vocab, &splits, &chunk);
    const size_t records = splits > 1 ? static_cast<size_t>(rows) * splits * record_floats(k) * 4 : 0;
    return kCounterBytes + records + static_cast<size_t>(rows) * (1 + k) * 8;
}

extern "C" int wsw_beam_select(const void *logits, int32_t dtype, int64_t requests, int64_t beams, int64_t vocab,
                               int64_t ld, const float *scores, const int32_t *end_tokens, int64_t n_ends, float scale,
                               int32_t *parent, int32_t *token, float *score, int32_t *end_parent, int32_t *end_token,
                               float *end_score, void *ws, size_t ws_bytes, void *stream, const wsw_launch_opts *opts) {
    using namespace wsw;
    Opts o;
    int st = resolve_opts(opts, &o);
    if (st != WSW_OK) return st;
    if (dtype != WSW_F32 && dtype != WSW_F16 && dtype != WSW_BF16) return WSW_ERR_UNSUPPORTED;
    if (requests < 0 || beams < 1 || vocab < 1 || ld < vocab || n_ends < 0 || (n_ends > 0 && !end_tokens) ||
        !std::isfinite(scale * kLog2e) || !(scale > 0.f))
        return WSW_ERR_INVALID_ARG;
    if (requests > kMaxRequests || beams > kMaxBeams || n_ends > kMaxEnds || beams * (1 + n_ends) > kMaxTop ||
        vocab >= (int64_t(1) << 31) - 65536)
        return WSW_ERR_UNSUPPORTED;
    if (requests == 0) return WSW_OK;
    if (!logits || !scores || !parent || !token || !score || !ws) return WSW_ERR_INVALID_ARG;
    if ((n_ends > 0 && !end_parent) || !end_parent != !end_token || !end_parent != !end_score) return WSW_ERR_INVALID_ARG;
    uintptr_t al = 0;
    for (const void *p : {static_cast<const void *>(scores), static_cast<const void *>(parent),
                          static_cast<const void *>(token), static_cast<const void *>(score),
                          static_cast<const void *>(end_parent), static_cast<const void *>(end_token),
                          static_cast<const void *>(end_score)})
        al |= reinterpret_cast<uintptr_t>(p);
    if ((al & 3) || (reinterpret_cast<uintptr_t>(logits) & (dtype == WSW_F32 ? 3 : 1)) ||
        (reinterpret_cast<uintptr_t>(ws) & 15))
        return WSW_ERR_MISALIGNED;
    if (ws_bytes < wsw_beam_select_workspace_bytes(requests, beams, vocab, n_ends)) return WSW_ERR_WORKSPACE;
    DeviceInfo di;
    if (!device_info(&di, &st)) return st;
    BeamArgs a;
    a.x = logits; a.scores = scores;
    a.parent = parent; a.token = token; a.score = score;
    a.end_parent = end_parent; a.end_token = end_token; a.end_score = end_score;
    a.ld = ld;
    a.scale = static_cast<double>(scale);
    a.c = static_cast<float>(a.scale * 1.4426950408889634);
    a.vocab = static_cast<int>(vocab);
    a.beams = static_cast<int>(beams);
    a.k = static_cast<int>(list_length(beams, vocab, n_ends));
    a.n_ends = static_cast<int>(n_ends);
    for (int64_t i = 0; i < n_ends; ++i) a.ends[i] = end_tokens[i];
    const int64_t rows = requests * beams;
    split_rows(rows, vocab, &a.splits, &a.chunk);
    a.rec = record_floats(a.k);
    unsigned char *w = static_cast<unsigned char *>(ws);
    a.row_cnt = reinterpret_cast<unsigned *>(w);
    a.req_cnt = reinterpret_cast<unsigned *>(w + kRowCounters);
    a.part = reinterpret_cast<float *>(w + kCounterBytes);
    a.lists = reinterpret_cast<uint64_t *>(w + kCounterBytes +
                                           (a.splits > 1 ? static_cast<size_t>(rows) * a.splits * a.rec * 4 : 0));
    const dim3 grid(static_cast<unsigned>(rows * a.splits));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == WSW_F32) e = launch(beam_kernel<float>, grid, dim3(kThreads), 0, s, o.pdl, a);
    else if (dtype == WSW_F16) e = launch(beam_kernel<__half>, grid, dim3(kThreads), 0, s, o.pdl, a);
    else e = launch(beam_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, o.pdl, a);
    return e == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
}
