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
// Top k: only values above a threshold that is never above the k-th best of what was seen
// are kept, their whole 16-byte vector at first, in shared memory.  The first threshold is the k-th largest of the
// maxima of 32 groups of threads over the first tile (k distinct values are at least as
// large), which leaves k to some tens of candidates a tile.  Once
// there are more than kKeep vectors, their values become keys and the keys are cut to the k
// best, which raises the threshold to the k-th best value so far.  Keys are 64 bits, the
// value's order-preserving bits over the complemented index, so that they are distinct and
// equal values rank by index.  Tiles that bring too many vectors (logits that rise along the row, or a
// part of the vocabulary well above the rest) are read again, against a new bound from
// their own groups' maxima (2047 x 50021 bf16, 5 alternatives, a tenth of the row raised by two
// deviations: 226 us when they were read in pieces of 992 values with a cut each, 92 so).
//
// Rows are split over CTAs when there are few; each split leaves (m, S, E, count, k keys) in
// the workspace and the row's last CTA joins them in a fixed order.
//
// Bound: the logits once, but a bf16 logit's arithmetic costs more issue slots than its two
// bytes cost of HBM's time.  2047 rows of 50021: bf16 63 us with 5 alternatives (3.3 TB/s) and
// 47 us with none, fp32 75 and 70 us (5.4 and 5.8 TB/s); sorted rows, the worst order, take 145 us
// (bf16, rising).  One row of 152064 fp32
// values: 11 us with 20 alternatives, 4.4 us with none; 64 rows with 8: 18 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "common.cuh"

namespace wsw {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kUnroll = 4;      // 16-byte vectors per thread and tile
constexpr int kCap = 1024;      // keys
constexpr int kVecs = 112;      // candidate vectors: at most 8 keys each, beside k and the row's ends
constexpr int kKeep = 20;       // make keys of them beyond this
constexpr int kLook = 2;        // look at their number every so many tiles
constexpr int kPiece = 224;     // values of a piece
constexpr int kThin = 96;       // keys that are worth thinning before a cut
static_assert(kVecs * 8 + kMaxTop + 16 <= kCap && kPiece + kMaxTop + 16 <= kCap, "keys");
constexpr int kTargetCtas = 608;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// order-preserving bits of a value: a < b exactly when ord(a) < ord(b), -0 as 0, NaN lowest
__device__ __forceinline__ uint32_t ord(float x) {
    if (x != x) return 1u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unord(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key_of(float x, int i) {
    return (static_cast<uint64_t>(ord(x)) << 32) | static_cast<uint32_t>(~i);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// two fp32 values in one register pair, for the packed arithmetic
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kVec = 4;
    static constexpr uint32_t kLow = 0xff800000u;  // -inf in every element of a word
    __device__ static float get(const float *p, int64_t i) { return p[i]; }
    __device__ static void unpack(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
};
template <>
struct Elem<__half> {
    static constexpr int kVec = 8;
    static constexpr bool kBf16 = false;
    using Pair = __half2;
    __device__ static Pair pair(float x) { return __float2half2_rn(x); }
    __device__ static float2 floats(Pair p) { return __half22float2(p); }
    static constexpr uint32_t kLow = 0xfc00fc00u;
    __device__ static float get(const __half *p, int64_t i) { return __half2float(p[i]); }
    __device__ static void unpack(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static constexpr bool kBf16 = true;
    using Pair = __nv_bfloat162;
    __device__ static Pair pair(float x) { return __float2bfloat162_rn(x); }
    __device__ static float2 floats(Pair p) { return __bfloat1622float2(p); }
    static constexpr uint32_t kLow = 0xff80ff80u;
    __device__ static float get(const __nv_bfloat16 *p, int64_t i) { return __bfloat162float(p[i]); }
    __device__ static void unpack(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16lo(w[i]);
            x[2 * i + 1] = bf16hi(w[i]);
        }
    }
};

// unpack's inverse (exact: the values came from it)
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[Elem<T>::kVec]) {
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (Elem<T>::kBf16) {
                w[i] = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
            } else {
                const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// the least value above x (above -inf: -FLT_MAX; above +inf: nothing, NaN)
__device__ __forceinline__ float above(float x) {
    if (x == 0.f) return __uint_as_float(1u);
    return x < INFINITY ? __uint_as_float(__float_as_uint(x) + (x > 0.f ? 1 : -1)) : NAN;
}

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

// Running sums of one thread, then of larger sets.  m >= -FLT_MAX, so that x - m is never
// (-inf) - (-inf).
struct Sums {
    float m, s, e;
};
__device__ __forceinline__ void raise(Sums &a, float mn, float c) {
    const float d = (a.m - mn) * c;  // <= 0, log2 units
    const float f = ex2(d);
    // before the first value s = e = 0 and d may be -inf
    a.e = a.s == 0.f ? 0.f : f * fmaf(d < -300.f ? -300.f : d, a.s, a.e);
    a.s *= f;
    a.m = mn;
}
__device__ __forceinline__ Sums join(Sums a, Sums b, float c) {
    const float mn = max_nan(a.m, b.m);
    raise(a, mn, c);
    raise(b, mn, c);
    return Sums{mn, a.s + b.s, a.e + b.e};
}

struct Shared {
    uint4 vec[kVecs];
    int vec_at[kVecs];
    int nvec;      // may pass kVecs: then the tiles are read again
    uint64_t buf[kCap];
    uint64_t best[kMaxTop];
    float group[kMaxTop];
    Sums sums[kWarps];
    int count[kWarps];
    int n;         // keys in buf
    float thr;
    int last;
};

// A value that at least k <= 32 of the block's values reach, from the threads' maxima: the k-th
// largest maximum of 32 groups of neighbouring threads.  Every thread calls it and gets it.
__device__ __forceinline__ float reached_by(Shared &sm, float mx, int k) {
#pragma unroll
    for (int d = kThreads / 64; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(WSW_FULL_MASK, mx, d));
    if (threadIdx.x % (kThreads / 32) == 0) sm.group[threadIdx.x / (kThreads / 32)] = mx;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const float own = sm.group[lane];
    int larger = 0;
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
        const float o = sm.group[j];
        larger += o > own || (o == own && j < lane);
    }
    return __shfl_sync(WSW_FULL_MASK, own, __ffs(__ballot_sync(WSW_FULL_MASK, larger == k - 1)) - 1);
}

// Cut the buffer to its k best keys, in order, and set the threshold.  Every thread calls it.
__device__ __forceinline__ void cut(Shared &sm, int k) {
    const int n = sm.n;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t own = sm.buf[i];
        int above = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) above += sm.buf[j] > own;
        if (above < k) sm.best[above] = own;
    }
    __syncthreads();
    const int kept = min(n, k);
    if (static_cast<int>(threadIdx.x) < kept) sm.buf[threadIdx.x] = sm.best[threadIdx.x];
    if (threadIdx.x == 0) {
        sm.n = kept;
        if (kept == k) sm.thr = fmaxf(sm.thr, unord(static_cast<uint32_t>(sm.best[k - 1] >> 32)));
    }
    __syncthreads();
}

// The least value that can still be among the k best, from a cut and with [.., end) behind: one above
// the k-th best, but its equal where that one is of the row's last few values, which are read first
// and rank after an equal value before them.
__device__ __forceinline__ float after_cut(const Shared &sm, int end, int k) {
    if (sm.n == k && static_cast<int>(~static_cast<uint32_t>(sm.best[k - 1])) >= end) return sm.thr;
    return above(sm.thr);
}

__device__ __forceinline__ void push(Shared &sm, uint64_t key) { sm.buf[atomicAdd(&sm.n, 1)] = key; }

// The keys of buf that can be among the k best, by the k-th largest of 32 groups' maxima: some 30
// of any number of distinct values, so that the cut's n * n stays small.  Every thread calls it.
__device__ __forceinline__ void thin(Shared &sm, int n, int k) {
    uint64_t own[kCap / kThreads];
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < kCap / kThreads; ++j) {
        const int i = threadIdx.x + j * kThreads;
        own[j] = i < n ? sm.buf[i] : 0;
        if (own[j]) mx = fmaxf(mx, unord(static_cast<uint32_t>(own[j] >> 32)));
    }
    const uint64_t least = static_cast<uint64_t>(ord(reached_by(sm, mx, k))) << 32;  // a barrier: all have read buf
    if (threadIdx.x == 0) sm.n = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kCap / kThreads; ++j)
        if (own[j] && own[j] >= least) push(sm, own[j]);
    __syncthreads();
}

// The candidates' values from thr up become keys, and the keys are cut.  When there were too many
// vectors for their place, the values [from, end) of the row are read again: those that the k-th
// largest of 32 groups' maxima reaches, which some tens do in any order of distinct values; what
// many equal ones still overflow goes in pieces that cannot, a cut before each.  Every thread calls it
// after a barrier behind the candidates.
template <typename T>
__device__ __forceinline__ void select(Shared &sm, const T *x, int from, int end, float thr, int k) {
    constexpr int V = Elem<T>::kVec;
    const int tid = threadIdx.x, n0 = sm.n, nvec = sm.nvec;
    if (nvec <= kVecs) {
        for (int e = tid; e < nvec * V; e += kThreads) {
            const float y = Elem<T>::get(reinterpret_cast<const T *>(sm.vec), e);
            if (y >= thr) push(sm, key_of(y, sm.vec_at[e / V] + e % V));
        }
    } else {
        const int nv = (end - from) / V;
        float mx = -INFINITY;
        float v[V];
#pragma unroll 2
        for (int i = tid; i < nv; i += kThreads) {
            Elem<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(x + from) + i), v);
#pragma unroll
            for (int u = 0; u < V; ++u) mx = fmaxf(mx, v[u]);
        }
        const float bound = fmaxf(thr, reached_by(sm, mx, k));  // a barrier: all have read sm.n, sm.nvec
        bool full = !(mx >= bound);
#pragma unroll 1
        for (int i = tid; i < nv && !full; i += kThreads) {
            Elem<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(x + from) + i), v);
#pragma unroll
            for (int u = 0; u < V; ++u) {
                if (!(v[u] >= bound)) continue;
                const int to = atomicAdd(&sm.n, 1);
                full = to >= kCap;
                if (!full) sm.buf[to] = key_of(v[u], from + i * V + u);
            }
        }
        __syncthreads();
        if (sm.n > kCap) {
            __syncthreads();
            if (tid == 0) sm.n = n0;
#pragma unroll 1
            for (int p = from; p < end; p += kPiece) {
                __syncthreads();
                cut(sm, k);
                const uint64_t floor = sm.n == k ? sm.best[k - 1] : 0;
                const int pe = min(p + kPiece, end);
                mx = -INFINITY;
                for (int i = p + tid; i < pe; i += kThreads) mx = fmaxf(mx, Elem<T>::get(x, i));
                const uint64_t least = static_cast<uint64_t>(ord(reached_by(sm, mx, k))) << 32;
                for (int i = p + tid; i < pe; i += kThreads) {
                    const uint64_t key = key_of(Elem<T>::get(x, i), i);
                    if (key >= least && key > floor) push(sm, key);
                }
            }
        }
    }
    __syncthreads();
    const int n = sm.n;
    if (n > kThin) {
        __syncthreads();
        thin(sm, n, k);
    }
    if (tid == 0) sm.nvec = 0;
    cut(sm, k);
}

// The block's sums and count, valid in thread 0.
__device__ __forceinline__ Sums block_sums(Shared &sm, Sums a, int &count, float c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        Sums b;
        b.m = __shfl_xor_sync(WSW_FULL_MASK, a.m, d);
        b.s = __shfl_xor_sync(WSW_FULL_MASK, a.s, d);
        b.e = __shfl_xor_sync(WSW_FULL_MASK, a.e, d);
        a = join(a, b, c);
        count += __shfl_xor_sync(WSW_FULL_MASK, count, d);
    }
    if (lane == 0) {
        sm.sums[warp] = a;
        sm.count[warp] = count;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kWarps; ++i) {
            a = join(a, sm.sums[i], c);
            count += sm.count[i];
        }
    }
    return a;
}

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
            select(sm, x, group0, end, thr, k);
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
    if (k > 0) {
        // The splits' keys are in order.  A key that k of them reach: the k-th largest of the
        // splits' best, or with fewer splits the least of their ceil(k / splits)-th.
        auto key_at = [&](int sp, int i) {
            return __ldcg(reinterpret_cast<const uint64_t *>(recs + static_cast<int64_t>(sp) * a.rec + 4) + i);
        };
        const int depth = (k + a.splits - 1) / a.splits, keys = a.splits * k;
        if (tid == 0) {
            sm.n = 0;
            sm.thr = -INFINITY;
        }
        for (int i = tid; i < a.splits; i += kThreads) sm.buf[i] = key_at(i, depth - 1);
        __syncthreads();
        for (int i = tid; i < a.splits; i += kThreads) {
            const uint64_t own = sm.buf[i];
            int more = 0;  // ties (absent keys are 0) by index
            for (int j = 0; j < a.splits; ++j) more += sm.buf[j] > own || (sm.buf[j] == own && j < i);
            if (more == min(k, a.splits) - 1) sm.best[0] = own;
        }
        __syncthreads();
        const uint64_t thr = sm.best[0];
        for (int base = 0; base < keys; base += kCap - kMaxTop) {
            const int end = min(base + kCap - kMaxTop, keys);
            const uint64_t floor = base > 0 && sm.n == k ? sm.best[k - 1] : 0;
            constexpr int kEach = (kCap - kMaxTop + kThreads - 1) / kThreads;
            uint64_t got[kEach];  // a thread's keys, on their way together
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const int i = base + tid + j * kThreads, sp = i / k;
                got[j] = i < end ? key_at(sp, i - sp * k) : 0;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                if (base + tid + j * kThreads < end && got[j] >= thr && got[j] > floor) push(sm, got[j]);
            __syncthreads();
            cut(sm, k);
        }
    }
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

// Splits of a row: about kTargetCtas CTAs over all rows, each of 4096 values or more.  From 305 rows on
// each is one CTA's.  Rows of 152064 bf16 values, one CTA each and split over 1824 CTAs: with 5 alternatives 305
// rows 42 and 39 us, 400 44 and 47, 608 51 and 60, 912 69 and 79; without them 33 and 28, 35 and 33, 43 and 44, 60
// and 61 us.
void split_rows(int64_t rows, int64_t vocab, int *splits, int *chunk) {
    int64_t n = kTargetCtas / rows;
    const int64_t most = (vocab + 4095) / 4096;
    if (n > most) n = most;
    if (n < 1) n = 1;
    const int64_t ch = ((vocab + n - 1) / n + 31) / 32 * 32;
    *chunk = static_cast<int>(ch);
    *splits = static_cast<int>((vocab + ch - 1) / ch);
}
int record_floats(int64_t top) { return static_cast<int>(4 + 2 * ((top + 1) / 2 * 2)); }
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
