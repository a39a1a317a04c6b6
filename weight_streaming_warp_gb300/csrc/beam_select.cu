// beam_select.cu -- the next beams of every request from all its beams' logits, in one pass.
//
//   s[b][j] = score[b] + scale x[b][j] - lse_b,  lse_b = ln sum_i exp(scale x[b][i])
//   the candidates (b, j) in order of s; the first `beams` that do not end become the beams
//
// Nothing beyond a row's k = beams + end tokens largest logits can matter: an end token takes one place
// in each row, and behind `beams` others nothing is chosen or reported.  So a row is streamed once, as for its log probabilities
// (topk_rows.cuh), with its sum and its k best kept; rows are split over CTAs when there are few.
// Each CTA leaves its part's maximum, sum and k best keys; the last CTA of a request merges the lists of
// all its beams' parts: a score that enough candidates reach comes from the heads of the lists,
// whatever reaches it is ranked, and the ranks answer.  (Rows joined first, then the request: 3 us more.)
//
// The order of near candidates of different beams hangs on the difference of their lse, so that more
// than fp32 of it counts.  A tile's terms, 8 or 16 of each half of a pair, are added in fp32; the sums of tiles, threads
// and CTAs, their factors when a maximum is raised, the logarithm and the scores are pairs of fp32 (some 45 bits: FP64 has
// a hundredth of fp32's rate here, and 900 scores of four operations took 5 us), and scale log2 e is one.  (A thread's sum in
// fp32 lost what was below half its last place tile after tile, always downward: 1.4e-6 of a row of 152064 behind a peak of
// 20.)  lse is off by 2^-22 (a term's power), 15 2^-24 (a tile's additions), and 2 2^-24 ln 2 |t| (the two roundings of a
// term's exponent t; its mean is below the entropy and kLag, 26): 2^-18 at most.  Nearly all of it comes
// with either sign: rows of 152064 normal values, flat, rising, behind a peak or but two, are off by 5e-9 to 5e-8 in the root
// mean square and 2e-7 at most, the beams' differences by half of that (5e-8 to 1.4e-6 and 2.4e-6 with fp32 sums and factors,
// at 1 us less of 30).  Value i of every row is the same thread's in the same order, whatever the row's alignment, so that equal rows have
// equal sums, bit for bit: copies of a beam tie and rank by index.  Rows that do not lie on 16 bytes take a vector from
// two loads, the second from L1.  (60 x 10 x 50021, of which seven bf16 rows in eight and three fp32 rows in four do not:
// 32.6 and 45.1 us; with the vectors of each row as they lie in memory 4 and 8 less, and sums of copies that differ.  The
// second vector by shuffles: 3 and 17 more.)
//
// Bound: the logits once; as the log probabilities with alternatives, by the selection's dependent steps
// for few rows (1 x 4 x 152064 fp32 11.3 us; the logits alone are 0.4) and by instructions and the selection's
// barriers for many (60 x 10 x 50024 bf16 27.5 us, 2.2 TB/s; 150 x 4 x 50000 fp32 33 us, 3.7 TB/s).
#include <algorithm>
#include <limits>

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
    unsigned *cnt;                // [requests] arrival counters, zero between calls
    float *part;                  // [rows][splits][rec]: maximum, sum (64 bits), keys
    int64_t ld;
    float scale, c, c_lo;         // c + c_lo = scale log2 e, c_lo > 0
    int vocab, beams, want, k, splits, chunk, rec, n_ends;  // want: candidates that can matter, k: of a row
    int32_t ends[kMaxEnds];
};

// A value as the sum of two fp32, |l| at most half a step of h.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {  // a + b, exact
    const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
    return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}
__device__ __forceinline__ Two renorm(float h, float l) {   // |l| <= |h|
    const float s = __fadd_rn(h, l);
    return Two{s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    const Two s = two_sum(a.h, b.h);
    return renorm(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Two operator*(Two a, float f) {
    const float p = __fmul_rn(a.h, f);
    return renorm(p, __fmaf_rn(a.l, f, __fmaf_rn(a.h, f, -p)));
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
    const float p = __fmul_rn(a.h, b.h);
    return renorm(p, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.h, -p))));
}
// a / b of positive values: the quotient's remainder, divided again
__device__ __forceinline__ Two operator/(Two a, Two b) {
    const float q = __fdiv_rn(a.h, b.h);
    const Two r = a + b * -q;
    return renorm(q, __fdiv_rn(__fadd_rn(r.h, r.l), b.h));
}
// ln x, x >= 1 or 0 or NaN: x = 2^e f with f in [0.7, 1.42), ln f = 2 (t + t^3 / 3 + t^5 / 5 + ...), t = (f - 1) / (f + 1),
// |t| < 0.18; the terms from t^5 on need fp32 alone, and end where they are below 2^-45.
__device__ __forceinline__ Two ln(Two x) {
    if (!(x.h > 0.f) || !(x.h < INFINITY)) return Two{x.h == 0.f ? -INFINITY : NAN, 0.f};
    int e = static_cast<int>(__float_as_uint(x.h) >> 23) - 127;
    if ((__float_as_uint(x.h) & 0x7fffffu) > 0x350000u) ++e;  // from 1.414 on
    const float unit = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const Two f{x.h * unit, x.l * unit};
    const Two t = (f + Two{-1.f, 0.f}) / (f + Two{1.f, 0.f});
    const Two t2 = t * t;
    const float y = t2.h;
    float p = 1.f / 15.f;
    p = fmaf(p, y, 1.f / 13.f);
    p = fmaf(p, y, 1.f / 11.f);
    p = fmaf(p, y, 1.f / 9.f);
    p = fmaf(p, y, 1.f / 7.f);
    p = fmaf(p, y, 1.f / 5.f);
    // 1 / 3 and ln 2 in two parts
    const Two series = Two{1.f, 0.f} + t2 * (Two{0.33333334f, -9.934108e-9f} + Two{p * y, 0.f});
    return Two{0.69314718f, -1.9046543e-9f} * static_cast<float>(e) + t * series * 2.f;
}

struct BeamShared {
    Shared top;                // its buf holds the lists' keys in the end
    uint64_t score[kCap];      // of each key, 0: no candidate
    uint16_t at[kCap];         // the places of those that reach the threshold
    uint64_t best[2][kMaxTop]; // the best so far, in order: scores, and their
    int2 tag[2][kMaxTop];      // lists and tokens; two sets in turn
    alignas(16) uint32_t group[kThreads];
    uint32_t reach;
    Two sum[kMaxBeams], base[kMaxBeams];
    float max[kMaxBeams];
    int last, n;
};

// The maximum in use lags behind a thread's by up to so much (log2), so that factors, which are pairs, are rare.
constexpr float kLag = 8.f;

// order-preserving bits of a finite score; 0: no candidate
__device__ __forceinline__ uint64_t ord2(Two s) {
    if (!(s.h > -INFINITY) || !(s.h < INFINITY)) return 0;  // -inf, NaN
    return (static_cast<uint64_t>(ord(s.h)) << 32) | ord(s.l);
}

// (m, s) of a set raised to the maximum mx: s 2^y of y = (m - mx) scale log2 e = i + f, |f| <= 0.5, by the exponential series
// of z = f ln 2: the terms from z^3 on, 0.007 at most, need fp32 alone, and end where they are below 2^-32.
__device__ __forceinline__ Two raised(const BeamArgs &a, float m, Two s, float mx) {
    if (s.h == 0.f || m == mx) return s;
    const Two d = two_sum(m, -mx);
    if (!(d.h * a.c > -125.f)) return m != m || mx != mx ? Two{NAN, 0.f} : Two{0.f, 0.f};
    const Two y = d * Two{a.c, a.c_lo};
    const float i = rintf(y.h);
    const Two z = renorm(y.h - i, y.l) * Two{0.69314718f, -1.9046543e-9f}, z2 = z * z;
    const float x = z.h;
    float p = 1.f / 40320.f;
    p = fmaf(p, x, 1.f / 5040.f);
    p = fmaf(p, x, 1.f / 720.f);
    p = fmaf(p, x, 1.f / 120.f);
    p = fmaf(p, x, 1.f / 24.f);
    p = fmaf(p, x, 1.f / 6.f);
    const Two power = Two{1.f, 0.f} + (z + Two{z2.h * 0.5f, z2.l * 0.5f} + Two{p * x * z2.h, 0.f});
    const float unit = __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(i)) << 23);
    return s * Two{power.h * unit, power.l * unit};
}
// The maximum and sum of groups of W lanes; every lane gets its group's.
template <int W = 32>
__device__ __forceinline__ void warp_total(const BeamArgs &a, float &m, Two &s) {
    float mx = m;
#pragma unroll
    for (int d = W / 2; d >= 1; d >>= 1) mx = max_nan(mx, __shfl_xor_sync(WSW_FULL_MASK, mx, d));
    s = raised(a, m, s, mx);
    m = mx;
#pragma unroll
    for (int d = W / 2; d >= 1; d >>= 1)
        s = s + Two{__shfl_xor_sync(WSW_FULL_MASK, s.h, d), __shfl_xor_sync(WSW_FULL_MASK, s.l, d)};
}

__device__ __forceinline__ bool is_end(const BeamArgs &a, int token) {
    bool ends = false;
#pragma unroll 1
    for (int i = 0; i < a.n_ends; ++i) ends |= token == a.ends[i];
    return ends;
}

// Each of the request's beams: score - ln S and its maximum, from its parts.
__device__ __forceinline__ void beam_sums(const BeamArgs &a, BeamShared &sm, const float *recs, int64_t request) {
    const int tid = threadIdx.x, lane = tid & 31;
#pragma unroll 1
    for (int b = tid >> 5; b < a.beams; b += kWarps) {
        float m = -FLT_MAX;
        Two sum{0.f, 0.f};
#pragma unroll 1
        for (int i = lane; i < a.splits; i += 32) {
            const float *r = recs + (static_cast<int64_t>(b) * a.splits + i) * a.rec;
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(r));
            const float mn = max_nan(m, v.x);
            sum = raised(a, m, sum, mn) + raised(a, v.x, Two{v.z, v.w}, mn);
            m = mn;
        }
        if (a.splits > 1) warp_total(a, m, sum);
        if (lane == 0) {
            sm.max[b] = m;
            sm.sum[b] = sum;
        }
    }
    __syncthreads();
    // a row of nothing but -inf, with a NaN or with +inf has no candidate: ln S -inf or NaN
    if (tid >= a.beams) return;  // a barrier follows
    const Two l = ln(sm.sum[tid]);
    sm.base[tid] = Two{a.scores[request * a.beams + tid], 0.f} + Two{-l.h, -l.l};
}

// The request's answer, once all its rows' parts are there.  Every thread calls it.  (The loops are not
// unrolled: of code that runs once, fetching is the larger part.)
__device__ __forceinline__ void merge(const BeamArgs &a, BeamShared &sm, int64_t request) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.k, want = a.want;
    const int lists = a.beams * a.splits;  // at most kThreads
    static_assert(kMaxBeams <= kThreads && 3 * kThreads <= kCap, "keys in buf");
    const float *recs = a.part + request * lists * a.rec;
    uint64_t *keys = sm.top.buf;
    // the first keys of each list, three a thread
    constexpr int kEach = 3;
    const int some = min(k, kEach * kThreads / lists), here = lists * some;
    auto key_at = [&](int i, int d0) {
        const int list = i / some, d = d0 + i - list * some;
        return d < k ? __ldcg(reinterpret_cast<const uint64_t *>(recs + static_cast<int64_t>(list) * a.rec + 4) + d) : 0;
    };
    uint64_t got[kEach];  // on their way while the sums are taken
#pragma unroll
    for (int u = 0; u < kEach; ++u) got[u] = tid + u * kThreads < here ? key_at(tid + u * kThreads, 0) : 0;
    if (tid == 0) sm.n = 0;
    beam_sums(a, sm, recs, request);
    int set = 0, have = 0;  // the best so far
    uint64_t thr = 1;       // a score that a candidate has to reach
    for (int d0 = 0;; d0 += some) {
#pragma unroll
        for (int u = 0; u < kEach; ++u)
            if (tid + u * kThreads < here) keys[tid + u * kThreads] = got[u];
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < here; i += kThreads) {
            const int b = i / some / a.splits;
            const uint64_t key = keys[i];
            // score - ln S + scale (x - m): the difference and its product are exact pairs
            const Two d = two_sum(unord(static_cast<uint32_t>(key >> 32)), -sm.max[b]);
            const Two p = d * a.scale;
            sm.score[i] = key && p.h > -INFINITY ? ord2(sm.base[b] + p) : 0;
        }
        __syncthreads();
        if (d0 == 0) {
            // a score that `beams` candidates that do not end reach (what is below it is neither chosen nor
            // reported), from a candidate a thread, the first few of each list
            const int depth = min(kThreads / lists, some), at = tid / depth * some + tid % depth;
            uint64_t own = 0;
            if (tid < lists * depth && !is_end(a, static_cast<int>(~static_cast<uint32_t>(keys[at])))) own = sm.score[at];
            // their order by a word each, whose last bits keep them apart: the bound is that much lower
            static_assert(kThreads == 128, "seven bits");
            const uint32_t word = (static_cast<uint32_t>(own >> 32) & ~127u) | (127 - tid);
            sm.group[tid] = word;
            __syncthreads();
            int more = 0;
#pragma unroll 4
            for (int j = 0; j < kThreads / 4; ++j) {
                const uint4 o = reinterpret_cast<const uint4 *>(sm.group)[j];
                more += (o.x > word) + (o.y > word) + (o.z > word) + (o.w > word);
            }
            if (more == a.beams - 1) sm.reach = word & ~127u;
            __syncthreads();
            thr = static_cast<uint64_t>(sm.reach) << 32;
            thr = max(thr, static_cast<uint64_t>(1));  // 0: fewer candidates than that
        }
        // ---- the candidates that reach it, ranked
#pragma unroll 1
        for (int i = tid; i < here; i += kThreads)
            if (sm.score[i] >= thr) sm.at[atomicAdd(&sm.n, 1)] = static_cast<uint16_t>(i);
        __syncthreads();
        const int n = sm.n, all = n + have;
        auto score_of = [&](int i) { return i < n ? sm.score[sm.at[i]] : sm.best[set][i - n]; };
        // Equal scores: the lower beam, then the lower token.  Lists are in the order of beams and tokens, and
        // each in its own, so that it is the lower list, then the one before in it (an earlier round's).
        auto list_of = [&](int i) { return i < n ? sm.at[i] / some : sm.tag[set][i - n].x; };
        auto comes_first = [&](int j, int i) {
            if ((j < n) == (i < n)) return j < n ? sm.at[j] < sm.at[i] : j < i;
            return j < n ? list_of(j) < list_of(i) : list_of(j) <= list_of(i);
        };
#pragma unroll 1
        for (int i = tid; i < all; i += kThreads) {
            const uint64_t mine = score_of(i);
            int before = 0;
#pragma unroll 2
            for (int j = 0; j < all; ++j) {
                const uint64_t o = score_of(j);
                before += o > mine;
                if (o == mine && j != i) before += comes_first(j, i);
            }
            if (before < want) {
                sm.best[set ^ 1][before] = mine;
                sm.tag[set ^ 1][before] = i < n ? make_int2(list_of(i), static_cast<int>(~static_cast<uint32_t>(keys[sm.at[i]])))
                                                : sm.tag[set][i - n];
            }
        }
        __syncthreads();
        set ^= 1;
        have = min(all, want);
        if (have == want) thr = max(thr, sm.best[set][want - 1]);
        // again where a list's last key here reaches it, too
        bool again = false;
#pragma unroll 1
        for (int i = tid; i < lists; i += kThreads) again |= sm.score[i * some + some - 1] >= thr;
        if (d0 + some >= k || !__syncthreads_or(again)) break;
        if (tid == 0) sm.n = 0;
#pragma unroll
        for (int u = 0; u < kEach; ++u) got[u] = tid + u * kThreads < here ? key_at(tid + u * kThreads, d0 + some) : 0;
    }
    if (tid >= 32) return;
    // ---- in order: a lane for each of the best
    const int64_t out = request * a.beams;
    const bool there = lane < have;
    const int2 tag = there ? sm.tag[set][lane] : make_int2(0, 0);
    const int token = tag.y, row = static_cast<int>(out) + tag.x / a.splits;
    const bool ends = there && is_end(a, token);
    const uint32_t alive = __ballot_sync(WSW_FULL_MASK, there && !ends), ended = __ballot_sync(WSW_FULL_MASK, ends && lane < a.beams);
    const uint32_t below = (1u << lane) - 1;
    const int at = __popc(alive & below), at_end = __popc(ended & below);
    const float s = there ? unord(static_cast<uint32_t>(sm.best[set][lane] >> 32)) : 0.f;
    if (there && !ends && at < a.beams) {
        a.parent[out + at] = row;
        a.token[out + at] = token;
        a.score[out + at] = s;
    }
    if (ends && lane < a.beams) {
        a.end_parent[out + at_end] = row;
        a.end_token[out + at_end] = token;
        a.end_score[out + at_end] = s;
    }
    // the places without a candidate
    if (lane < a.beams && lane >= __popc(alive)) {
        a.parent[out + lane] = a.token[out + lane] = -1;
        a.score[out + lane] = -INFINITY;
    }
    if (a.end_parent && lane < a.beams && lane >= __popc(ended)) {
        a.end_parent[out + lane] = a.end_token[out + lane] = -1;
        a.end_score[out + lane] = -INFINITY;
    }
}

// 16 bytes at any multiple of T's size, `behind` bytes behind a multiple of 16: of one or two vectors there, both of
// which hold some of them.
struct LoadAnywhere {
    int behind;
    __device__ __forceinline__ static uint4 first(const void *p, int behind) {
        return __ldg(reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(p) - behind));
    }
    // the bytes from `behind` on of a and the vector b after it
    __device__ __forceinline__ static uint4 join(const uint4 &a, const uint4 &b, int behind) {
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        if (behind & 8) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (behind & 4) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        if (behind & 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ uint4 operator()(const void *p) const {
        const uint4 a = first(p, behind);
        if (behind == 0) return a;
        return join(a, first(static_cast<const unsigned char *>(p) + 16, behind), behind);
    }
};

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
    // The row as vectors of 16 bytes: the split takes those of [lo, hi), the last one also the values behind the last
    // whole vector.
    const int behind = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15);
    const int64_t begin = static_cast<int64_t>(split) * a.chunk;
    const int whole = a.vocab / V * V;
    const int lo = static_cast<int>(min(begin, static_cast<int64_t>(whole)));
    const int hi = static_cast<int>(min(begin + a.chunk, static_cast<int64_t>(whole)));
    const int k = a.k;

    uint4 raw[kUnroll];
    auto fetch = [&](int tile0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int at = tile0 + (u * kThreads + tid) * V;
            raw[u] = make_uint4(Elem<T>::kLow, Elem<T>::kLow, Elem<T>::kLow, Elem<T>::kLow);
            if (at < hi) raw[u] = LoadAnywhere::first(x + at, behind);
        }
    };
    fetch(lo);
    float m = -FLT_MAX;  // m >= -FLT_MAX: x - m is never (-inf) - (-inf)
    Two sum{0.f, 0.f};
    if (tid == 0) {
        top.n = top.nvec = 0;
        top.thr = -INFINITY;
    }
    __syncthreads();
    if (split == a.splits - 1 && tid >= 32 && tid - 32 < a.vocab - whole) {
        const int i = whole + tid - 32;
        const float v = Elem<T>::get(x, i);
        if (!(v == -INFINITY)) {
            m = fmaxf(v, -FLT_MAX);
            sum.h = v != v || v == INFINITY ? NAN : 1.f;
        }
        push(top, key_of(v, i));
    }
    const uint64_t c2 = f2(a.c, a.c), c2_lo = f2(a.c_lo, a.c_lo);

    int since = 0, filled = 0;  // tiles since the buffer was looked at, candidates known then
    int group0 = lo;
    bool first = true;
    float thr = -INFINITY;
    for (int tile0 = lo; tile0 < hi; tile0 += kTile) {
        float v[kUnroll][V];
        float vm[kUnroll];
        if (behind) {
            uint4 next[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int at = tile0 + (u * kThreads + tid) * V;
                next[u] = raw[u];
                if (at < hi) next[u] = LoadAnywhere::first(x + at + V, behind);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) raw[u] = LoadAnywhere::join(raw[u], next[u], behind);
        }
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
        if ((tm - m) * a.c > kLag) {
            sum = raised(a, m, sum, tm);
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
                uint64_t lo;  // of a masked value (-inf) as d2 c is, since c_lo > 0
                asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(lo) : "l"(d2), "l"(c2_lo));
                asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(d2) : "l"(c2), "l"(lo));
                float d0, d1;
                asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(d2));
                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(ss) : "l"(f2(ex2(d0), ex2(d1))));
            }
        {
            float x0, x1;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(ss));
            sum = sum + two_sum(x0, x1);
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
            select(top, x, group0, end, thr, k, LoadAnywhere{behind});
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
    // the block's maximum and sum
    warp_total(a, m, sum);
    if ((tid & 31) == 0) {
        sm.max[tid >> 5] = m;
        sm.sum[tid >> 5] = sum;
    }
    __syncthreads();
    float *rec = a.part + (row * a.splits + split) * a.rec;
    if (tid < 32) {
        m = sm.max[tid % kWarps];
        sum = sm.sum[tid % kWarps];
        warp_total<kWarps>(a, m, sum);
        if (tid == 0) *reinterpret_cast<float4 *>(rec) = make_float4(m, 0.f, sum.h, sum.l);
    }
    if (tid < k) reinterpret_cast<uint64_t *>(rec + 4)[tid] = tid < top.n ? top.best[tid] : 0;
    // the block barrier orders the record before thread 0's arrival, whose release publishes
    // it; the last arrival's acquire orders the reads behind it after every record
    __syncthreads();
    const int64_t request = row / a.beams;
    if (tid == 0) {
        unsigned old;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(a.cnt + request) : "memory");
        sm.last = old == static_cast<unsigned>(a.beams * a.splits - 1);
        if (sm.last) a.cnt[request] = 0u;  // ready for the next call
    }
    __syncthreads();
    if (sm.last) merge(a, sm, request);
}

// the counters' place does not depend on the sizes: one workspace serves calls of different sizes in turn
constexpr size_t kCounterBytes = kMaxRequests * 4;

// A row's splits: those of the log probabilities, but no more than 128 lists of a request, so that the merge
// fetches three keys of each at once.  152064 fp32 logits with an end token, us with up to 608 lists and with 128: 1 x 4
// 11.7 and 11.3, 1 x 8 19.2 and 15.6, 4 x 8 19.3 and 17.1, 1 x 16 31.6 and 29.3, 2 x 16 35.0 and 35.5 (64 lists: 13.0,
// 18.5, 19.3, 31.7 and 33.1).
void beam_splits(int64_t rows, int64_t beams, int64_t vocab, int *splits, int *chunk) {
    split_rows(rows, vocab, splits, chunk);
    const int64_t most = kThreads / beams;  // 4 at least
    if (*splits <= most) return;
    const int64_t ch = ((vocab + most - 1) / most + 31) / 32 * 32;
    *chunk = static_cast<int>(ch);
    *splits = static_cast<int>((vocab + ch - 1) / ch);
}

int64_t list_length(int64_t beams, int64_t n_ends, int64_t vocab) { return beams + n_ends < vocab ? beams + n_ends : vocab; }

}  // namespace
}  // namespace wsw

extern "C" size_t wsw_beam_select_workspace_bytes(int64_t requests, int64_t beams, int64_t vocab, int64_t n_ends) {
    using namespace wsw;
    constexpr int64_t lim = int64_t(1) << 31;
    if (requests < 1 || requests > kMaxRequests || beams < 1 || beams > kMaxBeams || vocab < 1 || vocab >= lim - 65536 ||
        n_ends < 0 || n_ends > kMaxEnds || beams * (1 + n_ends) > kMaxTop)
        return 0;
    int splits, chunk;
    const int64_t rows = requests * beams, k = list_length(beams, n_ends, vocab);
    beam_splits(rows, beams, vocab, &splits, &chunk);
    return kCounterBytes + static_cast<size_t>(rows) * splits * record_floats(k) * 4;
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
    a.scale = scale;
    const double c = static_cast<double>(scale) * 1.4426950408889634;
    a.c = static_cast<float>(c);
    if (static_cast<double>(a.c) >= c) a.c = std::nextafter(a.c, 0.f);
    a.c_lo = std::max(static_cast<float>(c - a.c), std::numeric_limits<float>::denorm_min());
    a.vocab = static_cast<int>(vocab);
    a.beams = static_cast<int>(beams);
    a.want = static_cast<int>(beams * (1 + n_ends));
    a.k = static_cast<int>(list_length(beams, n_ends, vocab));
    a.n_ends = static_cast<int>(n_ends);
    for (int64_t i = 0; i < n_ends; ++i) a.ends[i] = end_tokens[i];
    const int64_t rows = requests * beams;
    beam_splits(rows, beams, vocab, &a.splits, &a.chunk);
    a.rec = record_floats(a.k);
    unsigned char *w = static_cast<unsigned char *>(ws);
    a.cnt = reinterpret_cast<unsigned *>(w);
    a.part = reinterpret_cast<float *>(w + kCounterBytes);
    const dim3 grid(static_cast<unsigned>(rows * a.splits));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == WSW_F32) e = launch(beam_kernel<float>, grid, dim3(kThreads), 0, s, o.pdl, a);
    else if (dtype == WSW_F16) e = launch(beam_kernel<__half>, grid, dim3(kThreads), 0, s, o.pdl, a);
    else e = launch(beam_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, o.pdl, a);
    return e == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
}
