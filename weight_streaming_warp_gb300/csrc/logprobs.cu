// logprobs.cu -- log probability, rank, entropy and top alternatives of each row of
// logits, in one pass.
//
//   y_j = scale x_j;  lse = ln sum exp(y_j);  logprob = y_t - lse
//   entropy = ln S - E / S with S = sum e_j, E = sum e_j (y_j - m), e_j = exp(y_j - m)
//   (-sum p ln p with p = e / S; it stays exact for a peaked row, where both terms are small)
//
// One pass: a thread keeps a running maximum m, S and E in fp32 over its vectors (kept in
// the log2 domain, e = 2^((x - m) scale log2 e)); when m grows by D (log2 units), S and E
// become f S and f (E - D S), f = 2^-D.  The rank is a count, taken only in vectors whose
// maximum reaches the token's logit.
//
// Top k: only values above a threshold that is never above the k-th best of what was seen
// enter a candidate buffer in shared memory.  The first threshold is the k-th largest of
// the 256 threads' maxima over the first tile (k distinct values are at least as large),
// which leaves about k candidates of 8192.  Between tiles the buffer is cut to its k best
// keys once it holds more than kKeep, which raises the threshold.  Keys are 64 bits, the
// value's order-preserving bits over the complemented index, so that they are distinct and
// equal values rank by index.  A tile that overflows the buffer (a long run of equal or
// rising values) is read again in pieces that cannot.
//
// Rows are split over CTAs when there are few; each split leaves (m, S, E, count, k keys) in
// the workspace and the row's last CTA joins them in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "common.cuh"

namespace wsw {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kUnroll = 4;      // 16-byte vectors per thread and tile
constexpr int kCap = 1024;      // candidate buffer
constexpr int kKeep = 256;      // cut the buffer between tiles beyond this
constexpr int kTargetCtas = 304;
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

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kVec = 4;
    __device__ static float get(const float *p, int64_t i) { return p[i]; }
    __device__ static void unpack(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
};
template <>
struct Elem<__half> {
    static constexpr int kVec = 8;
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
    uint64_t buf[kCap];
    uint64_t best[kMaxTop];
    float mx[kThreads];
    Sums sums[kWarps];
    int count[kWarps];
    int n;         // candidates in buf (may pass kCap: then the tile is read again)
    float thr;
    int last;
};

// The k-th largest of n distinct-by-index values v (ties ordered by index), 1 <= k <= n: every
// thread calls it; the result goes to sm.thr.
__device__ __forceinline__ void kth_of_maxima(Shared &sm, int k) {
    __syncthreads();
    const float own = sm.mx[threadIdx.x];
    int above = 0;
    for (int i = 0; i < kThreads; ++i) {
        const float o = sm.mx[i];
        above += o > own || (o == own && i < static_cast<int>(threadIdx.x));
    }
    if (above == k - 1) sm.thr = own;
    __syncthreads();
}

// Cut the buffer to its k best keys, in order, and set the threshold.  Every thread calls it.
__device__ __forceinline__ void cut(Shared &sm, int k) {
    const int n = min(sm.n, kCap);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t own = sm.buf[i];
        int above = 0;
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

// Returns how many candidates there are now (beyond kCap they are dropped).
__device__ __forceinline__ int push(Shared &sm, uint64_t key) {
    const int at = atomicAdd(&sm.n, 1);
    if (at < kCap) sm.buf[at] = key;
    return at + 1;
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
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LpArgs a) {
    constexpr int V = Elem<T>::kVec;
    constexpr int kTile = kThreads * kUnroll * V;  // values per tile
    __shared__ Shared sm;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.splits;
    const int split = static_cast<int>(blockIdx.x - row * a.splits);
    pdl_launch_dependents();
    pdl_wait();
    const T *x = static_cast<const T *>(a.x) + row * a.ld;
    // positions of 16-byte vectors: the row's first `lead` values come before the first one.
    // Vector v covers values lead + v V ...; v = -1 and the last one may be partial.
    const int lead = static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T));
    const int64_t begin = static_cast<int64_t>(split) * a.chunk;  // in values, before the shift by lead
    const int lo = begin == 0 ? 0 : static_cast<int>(min(begin + lead, static_cast<int64_t>(a.vocab)));
    const int hi = static_cast<int>(min(begin + a.chunk + lead, static_cast<int64_t>(a.vocab)));
    const float c = a.c;
    const int k = a.top;

    const int t = a.tokens ? a.tokens[row] : -1;
    const bool has_t = t >= 0 && t < a.vocab;
    const float xt = has_t ? Elem<T>::get(x, t) : INFINITY;  // nothing is above it, so nothing is counted
    Sums s{-FLT_MAX, 0.f, 0.f};
    int count = 0;
    if (tid == 0) {
        sm.n = 0;
        sm.thr = -INFINITY;
    }

    // Each tile covers values [tile0, tile0 + kTile) with tile0 congruent to lead modulo V; the
    // first starts at or before lo.
    const int tile_first = lo - (((lo - lead) % V + V) % V);
    bool first = true;
    for (int64_t tile0 = tile_first; tile0 < hi; tile0 += kTile) {
        float v[kUnroll][V];
        float vm[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t at = tile0 + (static_cast<int64_t>(u) * kThreads + tid) * V;
            if (at >= lo && at + V <= hi) {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(x + at));
                Elem<T>::unpack(w, v[u]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) v[u][i] = at + i >= lo && at + i < hi ? Elem<T>::get(x, at + i) : -INFINITY;
            }
        }
        float tm = -INFINITY;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            vm[u] = v[u][0];
#pragma unroll
            for (int i = 1; i < V; ++i) vm[u] = fmaxf(vm[u], v[u][i]);
            tm = fmaxf(tm, vm[u]);
        }
        if (tm > s.m) raise(s, tm, c);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = max_nan((v[u][i] - s.m) * c, -200.f);  // 2^-200 is 0, and 0 times -200 too
                const float e = ex2(d);
                s.s += e;
                s.e = fmaf(e, d, s.e);
            }
        if (tm >= xt) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t at = tile0 + (static_cast<int64_t>(u) * kThreads + tid) * V;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    count += at + i >= lo && at + i < hi && (v[u][i] > xt || (v[u][i] == xt && at + i < t));
            }
        }
        if (k > 0) {
            if (first) {
                sm.mx[tid] = tm;
                kth_of_maxima(sm, k);
            }
            const float thr = sm.thr;
            int filled = 0;
            if (first ? tm >= thr : tm > thr) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int64_t at = tile0 + (static_cast<int64_t>(u) * kThreads + tid) * V;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (at + i >= lo && at + i < hi && (first ? v[u][i] >= thr : v[u][i] > thr))
                            filled = push(sm, key_of(v[u][i], static_cast<int>(at) + i));
                }
            }
            // one answer for the whole block; inside, nobody pushes until all have read sm.n
            const bool over = __syncthreads_or(filled > kKeep);
            const int n = over ? sm.n : 0;
            if (n > kCap) {
                // too many: drop this tile's candidates and take the tile again in pieces of
                // kCap - kMaxTop values, cutting after each
                __syncthreads();
                if (tid == 0) {
                    int kept = 0;
                    for (int i = 0; i < kCap && !first; ++i) {
                        const int idx = static_cast<int>(~static_cast<uint32_t>(sm.buf[i]));
                        if (idx < tile0) sm.buf[kept++] = sm.buf[i];
                    }
                    sm.n = kept;
                }
                __syncthreads();
                cut(sm, k);
                for (int64_t p = tile0; p < tile0 + kTile; p += kCap - kMaxTop) {
                    const uint64_t floor = sm.n == k ? sm.best[k - 1] : 0;
                    const int64_t end = min(p + (kCap - kMaxTop), tile0 + kTile);
                    __syncthreads();
                    for (int64_t i = p + tid; i < end; i += kThreads)
                        if (i >= lo && i < hi) {
                            const uint64_t key = key_of(Elem<T>::get(x, i), static_cast<int>(i));
                            if (key > floor) push(sm, key);
                        }
                    __syncthreads();
                    cut(sm, k);
                }
            } else if (over) {
                cut(sm, k);
            }
            first = false;
        }
    }
    if (k > 0) {
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
        // the same selection over the splits' keys
        if (tid == 0) {
            sm.n = 0;
            sm.thr = -INFINITY;
        }
        const int keys = a.splits * k;
        float tm = -INFINITY;
        for (int i = tid; i < keys; i += kThreads) {
            const int sp = i / k;
            const uint64_t key =
                __ldcg(reinterpret_cast<const uint64_t *>(recs + static_cast<int64_t>(sp) * a.rec + 4) + (i - sp * k));
            if (key >> 32 > 1) tm = fmaxf(tm, unord(static_cast<uint32_t>(key >> 32)));
        }
        sm.mx[tid] = tm;
        kth_of_maxima(sm, k);
        const uint64_t thr = static_cast<uint64_t>(ord(sm.thr)) << 32;
        for (int base = 0; base < keys; base += kCap - kMaxTop) {
            const int end = min(base + kCap - kMaxTop, keys);
            const uint64_t floor = base > 0 && sm.n == k ? sm.best[k - 1] : 0;
            __syncthreads();
            for (int i = base + tid; i < end; i += kThreads) {
                const int sp = i / k;
                const uint64_t key = __ldcg(
                    reinterpret_cast<const uint64_t *>(recs + static_cast<int64_t>(sp) * a.rec + 4) + (i - sp * k));
                if (key >= thr && key > floor) push(sm, key);
            }
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

// Splits of a row: about kTargetCtas CTAs over all rows, each of 4096 values or more.
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
constexpr size_t kCounterBytes = 1024;
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
    if (rows < 0 || vocab < 1 || ld < vocab || !std::isfinite(scale) || !(scale > 0.f) || top < 0 || top > vocab)
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
