// topk_rows.cuh -- the largest values of long rows, kept while the rows stream by: what the calls
// on logits share.
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
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "common.cuh"

namespace wsw {
namespace topk {

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

// 16 bytes at a 16-byte boundary
struct LoadAligned {
    template <typename T>
    __device__ __forceinline__ uint4 operator()(const T *p) const { return __ldg(reinterpret_cast<const uint4 *>(p)); }
};

// The candidates' values from thr up become keys, and the keys are cut.  When there were too many
// vectors for their place, the values [from, end) of the row are read again: those that the k-th
// largest of 32 groups' maxima reaches, which some tens do in any order of distinct values; what
// many equal ones still overflow goes in pieces that cannot, a cut before each.  Every thread calls it
// after a barrier behind the candidates.  load(p): the 16 bytes of values from p on.
template <typename T, typename Load>
__device__ __forceinline__ void select(Shared &sm, const T *x, int from, int end, float thr, int k, Load load) {
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
            Elem<T>::unpack(load(x + from + i * V), v);
#pragma unroll
            for (int u = 0; u < V; ++u) mx = fmaxf(mx, v[u]);
        }
        const float bound = fmaxf(thr, reached_by(sm, mx, k));  // a barrier: all have read sm.n, sm.nvec
        bool full = !(mx >= bound);
#pragma unroll 1
        for (int i = tid; i < nv && !full; i += kThreads) {
            Elem<T>::unpack(load(x + from + i * V), v);
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

// The k best keys of a row's splits, from their records (rec floats apart, the keys behind four of
// them, in order, 0 where there are fewer): in sm.best, their number in sm.n.  Every thread calls it.
__device__ __forceinline__ void join_keys(Shared &sm, const float *recs, int rec, int splits, int k) {
    const int tid = threadIdx.x;
    // The splits' keys are in order.  A key that k of them reach: the k-th largest of the
    // splits' best, or with fewer splits the least of their ceil(k / splits)-th.
    auto key_at = [&](int sp, int i) {
        return __ldcg(reinterpret_cast<const uint64_t *>(recs + static_cast<int64_t>(sp) * rec + 4) + i);
    };
    const int depth = (k + splits - 1) / splits, keys = splits * k;
    if (tid == 0) {
        sm.n = 0;
        sm.thr = -INFINITY;
    }
    for (int i = tid; i < splits; i += kThreads) sm.buf[i] = key_at(i, depth - 1);
    __syncthreads();
    for (int i = tid; i < splits; i += kThreads) {
        const uint64_t own = sm.buf[i];
        int more = 0;  // ties (absent keys are 0) by index
        for (int j = 0; j < splits; ++j) more += sm.buf[j] > own || (sm.buf[j] == own && j < i);
        if (more == min(k, splits) - 1) sm.best[0] = own;
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

// ------------------------------------------------------------------- host --

// Splits of a row: about kTargetCtas CTAs over all rows, each of 4096 values or more.  From 305 rows on
// each is one CTA's.  Rows of 152064 bf16 values, one CTA each and split over 1824 CTAs: with 5 alternatives 305
// rows 42 and 39 us, 400 44 and 47, 608 51 and 60, 912 69 and 79; without them 33 and 28, 35 and 33, 43 and 44, 60
// and 61 us.
inline void split_rows(int64_t rows, int64_t vocab, int *splits, int *chunk) {
    int64_t n = kTargetCtas / rows;
    const int64_t most = (vocab + 4095) / 4096;
    if (n > most) n = most;
    if (n < 1) n = 1;
    const int64_t ch = ((vocab + n - 1) / n + 31) / 32 * 32;
    *chunk = static_cast<int>(ch);
    *splits = static_cast<int>((vocab + ch - 1) / ch);
}
inline int record_floats(int64_t top) { return static_cast<int>(4 + 2 * ((top + 1) / 2 * 2)); }

}  // namespace topk
}  // namespace wsw
