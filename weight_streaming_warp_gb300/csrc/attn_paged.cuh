// attn_paged.cuh -- attention of one new token per request over a paged KV cache.
//
//   y_p = scale q . K_p (capped by softcap tanh(. / softcap), minus slope (n - 1 - p))
//   out = sum_p 2^(y_p - m) V_p / sum_p 2^(y_p - m), y in log2 units, m = max_p y_p
//
// Bound: every seen K and V byte once (2 head_dim values per position and KV head) against
// 2 * group multiply-adds per value; HBM bandwidth for any group up to 16.  So the layout of
// the work is about keeping loads in flight on every SM whatever the requests' lengths:
//  * One list of tiles.  A tile is 16 (q8_0: 32) positions of one pair (request, KV head); the tiles of
//    all pairs, in order, are cut into equal runs for 152 CTAs and those into equal runs for
//    their warps.  Nothing is launched per request and no SM waits for a long one; lengths are
//    read on the device, each CTA scanning them once.  A cut that falls into a pair of at most
//    kWhole positions moves to the nearer end of it: sharing a pair between CTAs costs 4 us at its
//    end, as much as so many tiles.  In long lists a pair counts kPair tiles more than it has:
//    its queries, its end and its last, partial tile cost a warp about as much (256 x 512
//    positions of 8 heads: with none the CTAs with the most pairs took 66 us, the median 46, and
//    the call 70 us; 58 us now).
//  * Each warp streams its run through a private ring of shared-memory stages with cp.async,
//    across pair boundaries without a drain, and keeps its own softmax (running maximum, sum,
//    value sums) in registers: no block barrier until its run ends.
//  * A pair that lies in one warp's run is written by that warp.  Otherwise the warps leave
//    (m, l, sums) records, the CTA joins its own, and when a pair spans CTAs the last of each
//    group of kGroup CTAs to arrive (a counter in the workspace) joins the group's records, and
//    the last group's CTA the groups', always in tile order, so that results do not depend on
//    timing.  (One CTA joining 147 records of eight rows took 15 us: 42 bytes a nanosecond of
//    one SM's loads.)  A CTA has at most two pairs that it shares with others.
//
// Measured, 4 KV heads of 128: 64 requests of up to 8192 positions, bf16, group 10, 111 us
// (4.9 TB/s, bound by latency with 8 warps on an SM); 32 of up to 32768, q8_0, group 8, 120 us (4.9
// TB/s, bound by instructions); the same in bf16 180 us (6.1 TB/s); one of 32768 binary16 positions, group 8,
// 24 us, of which 8 us are the two levels of joins; three short ones (head_dim 64) 8.7 us.
//
// Products on m16n8k16 tensor-core tiles with fp32 sums.  Up to eight query heads of a KV head
// share a 16-row operand as high parts (rows 0..7) and residuals (8..15) of q and of the
// weights; 9 to 16 take 16 rows and a second product for the residuals; more take several
// passes over the pair.  The maximum in use is raised, and the sums rescaled, only when a tile
// exceeds it by more than kLazy; binary16 weights, then up to 2^(kLazy + shift), stay in its
// range (a weight is off by 2^-22 of itself or 2^-32 of the largest).  bf16 weights end at 1 there:
// a value sum overflows where the sum of the values themselves would.  A query row enters
// binary16 times the power of two that brings its largest value to 2^14 .. 2^15, so that any fp32
// or bf16 row keeps 22 bits.  Over bf16 pages two parts are 16 bits, enough for a 16-bit result and
// exact for a 16-bit q; under fp32 queries q and the weights are three parts, exact, with one product more
// each (with two: results off by 4e-6.  32 x 32768, group 8: 175 us, with two parts 181; 64 ragged of group
// 10 126 and 113, three short ones 10.3 and 9.3 us).  q8_0 rows stay codes in shared memory and become binary16(scale *
// code) in registers, the value the one-pass dequantizer writes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_cache.cuh"

namespace wsw {
namespace paged {

constexpr int kWhole = 512;    // pairs of up to so many positions stay in one CTA
constexpr int kPair = 4;       // tiles that the beginning and end of a pair count for
constexpr float kLazy = 8.f;   // log2: the running maximum may lag by so much
constexpr int kGroup = 12;     // CTAs whose records are joined first
constexpr int kCtas = 152;     // runs of the tile list: one CTA per SM of a 152-SM part
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kSmemMax = 226 * 1024;

struct Args {
    const void *q;
    void *out;
    float *lse;
    const float *slopes;
    const int32_t *table, *lens;
    int32_t *err;
    // arrival counters, zero between calls: [kCtas][2] of a pair within a group of CTAs, by its
    // record there, then [kCtas] of a pair's groups, by its first CTA
    unsigned *cnt;
    float *rec;     // [kCtas][2][rows][D + 4] what a CTA leaves of its shared pairs
    float *wrec;    // [kCtas][warps][rows][D (+ 4)] what a warp leaves of its first pair
    KvView kv;
    int64_t table_stride;
    float scale2;     // scale log2 e
    float cap_in;     // scale / softcap, 0: not capped
    float cap_out;    // softcap log2 e
    int requests, q_heads, group, passes;  // passes = ceil(group / rows)
    int max_len, window;                   // window > 0
    int dtype;                             // of q and out
};

// Shape of one variant: cache type, head_dim, query rows (8 or 16), third parts of q and the weights
// (bf16 pages under fp32 queries).
template <int CT, int D, int RT, bool X3>
struct Cfg {
    static constexpr bool q8 = CT == WSW_Q8_0;
    // q8_0 is bound by the instructions that turn codes into values: tiles of 32 positions share
    // the bookkeeping and the softmax's reductions among more of them, and the smaller rows
    // leave room for 12 warps (32 x 32768 positions, group 8: 16-position tiles 150 us, 32
    // with 8, 10, 12 warps 126, 147, 124 us)
    static constexpr int warps = D == 256 ? 4 : q8 && RT == 8 ? 12 : 8;
    static constexpr int threads = warps * 32;
    static constexpr int row_bytes = q8 ? D : 2 * D;
    static constexpr int pieces = row_bytes / 16;      // 16-byte pieces of a row
    static constexpr int scale_bytes = q8 ? D / 16 : 0;
    static constexpr int tile = q8 && D <= 128 ? 32 : 16;           // positions
    static constexpr int kv_bytes = tile * row_bytes;   // K (or V) rows of a tile
    static constexpr int stage = 2 * kv_bytes + 2 * tile * scale_bytes;
    static constexpr int ksteps = D / 16;
    static constexpr bool q_smem = D == 256;            // q's high parts: registers if they fit
    static constexpr int qfrag = ksteps * 512;          // bytes of one warp's A fragments
    static constexpr int xfrag = X3 && q_smem ? ksteps * RT * 32 : 0;  // of q's third parts: as q's high parts
    static constexpr int q_bytes = (q_smem ? qfrag : 0) + (RT == 16 ? qfrag : 0) + xfrag;
    static constexpr int fit = (kSmemMax - warps * q_bytes) / (warps * stage);
    static constexpr int stages = fit < 6 ? fit : 6;
    static constexpr int ring = stages * stage;
    // the joins at the end keep weights where q was, or behind the rings
    static constexpr int smem = warps * (ring + q_bytes) + (q_bytes == 0 ? 4096 : 0);
    static constexpr float shift = CT == WSW_BF16 ? -kLazy : 7.f;  // log2 of the weights' scale
    static constexpr int rec = D + 4;                   // floats of a CTA's record row: m, l, 2 pad, sums
    // of a warp's: sums, padded against bank conflicts if two records fit into the warp's ring
    static constexpr int srec = 2 * RT * (D + 4) * 4 <= ring ? D + 4 : D;
    static_assert(stages >= 2 && 2 * RT * srec * 4 <= ring && ring % 16 == 0, "ring");
    static_assert(2 * warps <= 32 && 3 * 2 * warps * RT * 4 <= 4096 && smem <= 227 * 1024, "joins");
    static_assert(40 * RT * 4 + RT * 8 <= warps * ring, "joins");
};

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// copies of 16 (or 4, 8) bytes that write zeros and read nothing when !valid
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
template <int B>
__device__ __forceinline__ void cp_small(uint32_t dst, const void *src, bool valid) {
    if constexpr (B == 16) cp16(dst, src, valid);
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(B), "r"(valid ? B : 0)
                     : "memory");
}
__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p) : "memory");
}
template <int CT>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (CT == WSW_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same with an operand of third parts: rows 0..7 alone where the other rows are residuals
template <int CT, int RT>
__device__ __forceinline__ void mma_third(float (&d)[4], const uint32_t (&t)[RT / 4], uint32_t b0, uint32_t b1) {
    if constexpr (RT == 8) {
        const uint32_t a[4] = {t[0], 0u, t[1], 0u};
        mma<CT>(d, a, b0, b1);
    } else {
        mma<CT>(d, t, b0, b1);
    }
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (x, y) as a pair of 16-bit values, and what the rounding left of each as another pair
template <int CT>
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    if constexpr (CT == WSW_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(x - bf16lo(hi), y - bf16hi(hi));
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}
// (x, y) as three pairs of bf16, exact: each cut leaves the bits that the next ones take
__device__ __forceinline__ void split3(float x, float y, uint32_t &hi, uint32_t &lo, uint32_t &third) {
    hi = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
    x -= bf16lo(hi);
    y -= bf16hi(hi);
    lo = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
    third = __byte_perm(__float_as_uint(x - bf16lo(lo)), __float_as_uint(y - bf16hi(lo)), 0x7632);
}
// Two codes, bytes `sel` picks from w (biased by 128), times the scales in d: 0x6400 + u is
// 1024 + u in binary16, so both steps before the product are exact.
__device__ __forceinline__ uint32_t dequant2(uint32_t biased, uint32_t sel, __half2 d) {
    const uint32_t h = __byte_perm(biased, 0x64646464u, sel);
    const uint32_t bias = 0x64806480u;  // 1152
    const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&bias)), d);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// (x, y) in the output's 16-bit type
__device__ __forceinline__ uint32_t pack16(int dtype, float x, float y) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    const __half2 h = __floats2half2_rn(x, y);
    return dtype == WSW_BF16 ? *reinterpret_cast<const uint32_t *>(&b) : *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void store_out4(const Args &a, int64_t i, float4 v) {
    if (a.dtype == WSW_F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + i) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + i) =
            make_uint2(pack16(a.dtype, v.x, v.y), pack16(a.dtype, v.z, v.w));
}
__device__ __forceinline__ float lse_of(float m, float l, float shift) {
    return l == 0.f ? -INFINITY : (m + log2f(l) - shift) * kLn2;
}
// weight of a record with maximum m against the common maximum
__device__ __forceinline__ float weight(float m, float mx) { return m == -INFINITY ? 0.f : ex2(m - mx); }

// Where a warp is in the tile list: request, head and pass, tile of the pair.
struct Cursor {
    int g;       // its place in the list, in tiles and the pairs' extra counts before them
    int r, hp, t, nt;
    int start, len;  // seen positions are [start, len)
};
// A piece of a pair left as a record: the pair, its first tile's place and its tile count.
struct Piece {
    int pstart;
    int r, hp, nt;  // r = -1: none
};

__device__ __forceinline__ int clipped_len(const Args &a, int r) {
    const int n = a.lens[r];
    return n < 0 ? 0 : n > a.max_len ? a.max_len : n;
}
template <int T>
__device__ __forceinline__ int tiles_of(const Args &a, int len) {
    const int seen = len < a.window ? len : a.window;
    return seen / T + (seen % T != 0);
}
template <int T>
__device__ __forceinline__ void set_request(const Args &a, Cursor &c, int r) {
    c.r = r;
    c.len = clipped_len(a, r);
    c.nt = tiles_of<T>(a, c.len);
    c.start = c.len > a.window ? c.len - a.window : 0;
}
// The next tile of the list; the caller knows that there is one.
template <int T>
__device__ __forceinline__ void advance(const Args &a, Cursor &c, int extra) {
    ++c.g;
    if (++c.t < c.nt) return;
    c.t = 0;
    c.g += extra;
    if (++c.hp < a.kv.heads * a.passes) return;
    c.hp = 0;
    int r = c.r;
    do set_request<T>(a, c, ++r);
    while (c.nt == 0 && r + 1 < a.requests);
}

template <int CT, int D, int RT, bool X3>
__global__ void __launch_bounds__(Cfg<CT, D, RT, X3>::threads, 1) attn_paged_kernel(const __grid_constant__ Args a) {
    using C = Cfg<CT, D, RT, X3>;
    constexpr int W = C::warps, NT = C::threads, T = C::tile;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int2 scan[W];
    struct Place {
        int req, off, nt;  // a request, the place in its part of the list, its pairs' tiles
    };
    __shared__ Place cut[2], place[W];  // of the CTA's cuts, of the warps' first tiles
    __shared__ Piece pieces[2 * W];
    __shared__ float2 piece_ml[2 * W][RT];  // (m, l) of each piece's rows
    __shared__ uint32_t seen_mask[W][C::stages];
    __shared__ int last[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x;
    const int HP = a.kv.heads * a.passes;
    if (tid < 2 * W) pieces[tid].r = -1;
    pdl_launch_dependents();
    pdl_wait();

    // ---- the tile list (below 2^31 tiles): each thread counts a run of requests, a scan
    // places the runs
    const int per = (a.requests + NT - 1) / NT;
    const int r0 = min(tid * per, a.requests), r1 = min(r0 + per, a.requests);
    int mine = 0, mine_n = 0, nt0 = 0;  // tiles, pairs; nt0: of request r0
    bool cut_len = false;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
        const int n = a.lens[r], clipped = min(max(n, 0), a.max_len);
        cut_len |= n != clipped;
        const int nt = tiles_of<T>(a, clipped);
        if (r == r0) nt0 = nt;
        mine += nt * HP;
        mine_n += nt > 0 ? HP : 0;
    }
    if (cut_len && cta == 0 && a.err) atomicOr(a.err, 2);
    int upto = mine, upto_n = mine_n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(WSW_FULL_MASK, upto, d), y_n = __shfl_up_sync(WSW_FULL_MASK, upto_n, d);
        if (lane >= d) {
            upto += y;
            upto_n += y_n;
        }
    }
    if (lane == 31) scan[warp] = make_int2(upto, upto_n);
    __syncthreads();
    int total = 0, total_n = 0, before = upto - mine, before_n = upto_n - mine_n;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int2 x = scan[w];
        if (w < warp) {
            before += x.x;
            before_n += x.y;
        }
        total += x.x;
        total_n += x.y;
    }
    // a few tiles for each warp at least: there latency counts, not balance
    const int extra = total >= 4 * kCtas * W ? kPair : 0;
    mine += extra * mine_n;
    before += extra * before_n;
    total += extra * total_n;
    const int run = max((total + kCtas - 1) / kCtas, W);  // of a CTA
    auto counted = [&](int nt) { return nt > 0 ? nt + extra : 0; };  // a pair's length in the list
    // what the list has at s, from the thread whose requests hold it
    auto locate = [&](int s, Place &p) {
        if (s < before || s >= before + mine) return;
        int at = before, r = r0, nt = nt0;
#pragma unroll 1
        while (s >= at + counted(nt) * HP) {
            at += counted(nt) * HP;
            nt = tiles_of<T>(a, clipped_len(a, ++r));
        }
        p = Place{r, s - at, nt};
    };
    const int raw_b = static_cast<int>(min(static_cast<int64_t>(cta) * run, static_cast<int64_t>(total)));
    const int raw_e = static_cast<int>(min(static_cast<int64_t>(cta + 1) * run, static_cast<int64_t>(total)));
    locate(raw_b, cut[0]);
    locate(raw_e, cut[1]);
    __syncthreads();
    // a cut just inside a long pair moves to its end, too: a CTA that shares two pairs with
    // others ends with two joins, worth some 20 tiles
    const int margin = min(run / 8, 16);
    auto snapped = [&](int s, const Place &p) {
        if (s >= total || s == 0) return s;
        const int n = counted(p.nt), t = p.off % n;
        if (p.nt <= kWhole / T) return s - t + (2 * t > n ? n : 0);
        return t <= margin ? s - t : n - t <= margin ? s - t + n : s;
    };
    const int b = snapped(raw_b, cut[0]), e = snapped(raw_e, cut[1]);
    const int n_cta = e - b;
    auto first_tile = [&](int w) { return b + static_cast<int>(static_cast<int64_t>(n_cta) * w / W); };
    if (before < e && before + mine > b) {
#pragma unroll 1
        for (int w = 0; w < W; ++w) locate(first_tile(w), place[w]);
    }
    // requests that see nothing
#pragma unroll 1
    for (int r = cta; r < a.requests; r += gridDim.x) {
        if (clipped_len(a, r) > 0) continue;
        const int64_t head = static_cast<int64_t>(r) * a.q_heads;
#pragma unroll 1
        for (int i = tid; i < a.q_heads * (D / 4); i += NT) store_out4(a, head * D + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
#pragma unroll 1
        for (int i = tid; a.lse && i < a.q_heads; i += NT) a.lse[head + i] = -INFINITY;
    }
    __syncthreads();
    if (n_cta == 0) return;

    const int wb = first_tile(warp), we = first_tile(warp + 1);
    unsigned char *ring = smem + warp * C::ring;
    const uint32_t ring_s = smem_addr(ring);
    unsigned char *qsm = smem + W * C::ring + warp * C::q_bytes;
    uint4 *q_hi_sm = reinterpret_cast<uint4 *>(qsm);
    uint4 *q_lo_sm = reinterpret_cast<uint4 *>(qsm + (C::q_smem ? C::qfrag : 0));
    uint32_t *q_third_sm = reinterpret_cast<uint32_t *>(qsm + C::q_bytes - C::xfrag);

    if (wb < we) {
        Cursor uc;  // the tile in use
        const Place at_first = place[warp];
        set_request<T>(a, uc, at_first.req);
        {
            const int n = counted(uc.nt);
            uc.hp = at_first.off / n;
            const int in = at_first.off - uc.hp * n;
            uc.t = max(in - extra, 0);
            uc.g = wb - in + extra + uc.t;  // we or beyond: no tile here
        }
        Cursor ic = uc;  // the next tile to copy
        const int page_mask = (1 << a.kv.page_shift) - 1;

        // The request's page numbers from wbase on, 64 of them over the lanes, loaded well before
        // their copies: a table read on the way to each copy would double its latency.
        int wreq = -1, wbase = 0, win0 = -1, win1 = -1;
        auto entries = [&](int i) {  // page numbers i + lane
            i += lane;
            return i <= (ic.len - 1) >> a.kv.page_shift ? a.table[ic.r * a.table_stride + i] : -1;
        };
        auto look_up = [&]() {
            const int i0 = (ic.start + ic.t * T) >> a.kv.page_shift;
            if (ic.r != wreq || i0 < wbase || i0 >= wbase + 64) {
                wreq = ic.r;
                wbase = i0;
                win0 = entries(wbase);
                win1 = entries(wbase + 32);
            } else if (i0 >= wbase + 32) {
                wbase += 32;
                win0 = win1;
                win1 = entries(wbase + 32);
            }
        };
        look_up();
        int ist = 0;
        auto issue = [&]() {
            if (ic.g < we) {
                constexpr uint32_t kAll = T == 32 ? 0xffffffffu : (1u << (T & 31)) - 1;
                const int p0 = ic.start + ic.t * T, p = p0 + (lane & (T - 1));
                const int rel = (p >> a.kv.page_shift) - wbase;
                const int pg0 = __shfl_sync(WSW_FULL_MASK, win0, rel & 31), pg1 = __shfl_sync(WSW_FULL_MASK, win1, rel & 31);
                const int page = rel < 32 ? pg0 : pg1;
                const bool in = p < ic.len;
                const bool ok = in && static_cast<unsigned>(page) < static_cast<unsigned>(a.kv.num_pages);
                const uint32_t valid = __ballot_sync(WSW_FULL_MASK, ok) & kAll;
                if (in && !ok && a.err) atomicOr(a.err, 1);
                const int64_t at = ok ? page * a.kv.page_stride + (p & page_mask) * a.kv.pos_stride : 0;
                const int h = a.passes == 1 ? ic.hp : ic.hp / a.passes;
                const unsigned char *kb = a.kv.k + h * a.kv.head_stride, *vb = a.kv.v + h * a.kv.head_stride;
                const uint32_t stg = ring_s + ist * C::stage;
                constexpr int kRows = 32 / C::pieces;  // rows per round of the warp
                const int c = lane % C::pieces, rr = lane / C::pieces;
                auto swizzled = [&](int row) {
                    const int sw = C::pieces >= 8 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
                    return stg + row * C::row_bytes + sw * 16;
                };
                if (valid == kAll && (p0 & page_mask) + T - 1 <= page_mask) {
                    // the whole tile in one page: its rows are pos_stride apart
                    const int64_t o = __shfl_sync(WSW_FULL_MASK, at, 0) + rr * a.kv.pos_stride + c * 16;
                    const unsigned char *kp = kb + o, *vp = vb + o;
#pragma unroll
                    for (int i = 0; i < T / kRows; ++i) {
                        const uint32_t dst = swizzled(i * kRows + rr);
                        cp16(dst, kp, true);
                        cp16(dst + C::kv_bytes, vp, true);
                        kp += kRows * a.kv.pos_stride;
                        vp += kRows * a.kv.pos_stride;
                    }
                } else {
#pragma unroll 2
                    for (int i = 0; i < T / kRows; ++i) {
                        const int row = i * kRows + rr;
                        const int64_t o = __shfl_sync(WSW_FULL_MASK, at, row);
                        const bool v = (valid >> row) & 1;
                        const uint32_t dst = swizzled(row);
                        cp16(dst, kb + o + c * 16, v);
                        cp16(dst + C::kv_bytes, vb + o + c * 16, v);
                    }
                }
                if constexpr (C::q8 && T == 32) {  // a lane for each position's scales
                    const int64_t dat = ok ? page * a.kv.d_page_stride + (p & page_mask) * a.kv.d_pos_stride +
                                                 h * a.kv.d_head_stride : 0;
                    const uint32_t dst = stg + 2 * C::kv_bytes + lane * C::scale_bytes;
                    cp_small<C::scale_bytes>(dst, a.kv.kd + dat, ok);
                    cp_small<C::scale_bytes>(dst + T * C::scale_bytes, a.kv.vd + dat, ok);
                } else if constexpr (C::q8) {  // lanes 0..15: K scales, 16..31: V scales
                    const int64_t dat = ok ? page * a.kv.d_page_stride + (p & page_mask) * a.kv.d_pos_stride +
                                                 h * a.kv.d_head_stride : 0;
                    cp_small<C::scale_bytes>(stg + 2 * C::kv_bytes + lane * C::scale_bytes,
                                             (lane < 16 ? a.kv.kd : a.kv.vd) + dat, ok);
                }
                if (lane == 0) seen_mask[warp][ist] = valid;
                if (++ist == C::stages) ist = 0;
                if (ic.g + 1 + (ic.t == ic.nt - 1 ? extra : 0) >= we) {
                    ic.g = we;
                } else {
                    advance<T>(a, ic, extra);
                    look_up();
                    if (ic.t == 0) {  // a new pair: its queries on their way to L1
                        const int hn = a.passes == 1 ? ic.hp : ic.hp / a.passes, gn = (ic.hp - hn * a.passes) * RT;
                        const int esize = a.dtype == WSW_F32 ? 4 : 2;
                        const int bytes = min(RT, a.group - gn) * D * esize;
                        const unsigned char *qp = static_cast<const unsigned char *>(a.q) +
                            ((static_cast<int64_t>(ic.r) * a.q_heads + hn * a.group + gn) * D) * esize;
                        for (int i = lane * 128; i < bytes; i += 32 * 128)
                            asm volatile("prefetch.global.L1 [%0];" ::"l"(qp + i));
                    }
                }
            }
            cp_commit();  // one group per step, empty past the end
        };
        const int gq = lane >> 2, tq = lane & 3;
        uint32_t qa[C::q_smem ? 1 : C::ksteps][4];
        uint32_t q3[X3 && !C::q_smem ? C::ksteps : 1][RT / 4];  // third parts, of rows 0..7 (and 8..15)
        float m[RT / 8], l[RT / 8], slope[RT / 8];
        float unit[RT / 8];  // of a score's product sum, over softcap if that is used (not bf16)
        float o[D / 8][4];
        bool q_lo = false;   // RT 16: q has residuals
        int t_first = 0;     // first tile of the piece
        bool fresh = true;   // a new pair begins
        bool first_left = false;  // the first piece is in the workspace
        int rst = 0;
        const int mi = lane >> 3, mr = lane & 7;

        // the first turns only fill the ring
#pragma unroll 1
        for (int fill = 1 - C::stages; uc.g < we; ++fill) {
            __syncwarp();  // every lane is done reading the stage that the next copy reuses
            issue();
            if (fill < 0) continue;
            if (fresh) {
                fresh = false;
                t_first = uc.t;
                const int h = uc.hp / a.passes, g0 = (uc.hp - h * a.passes) * RT;
                const int64_t head0 = static_cast<int64_t>(uc.r) * a.q_heads + h * a.group + g0;
                bool some = false;
                // every load of a batch is issued before the first is used
                constexpr int kB = C::ksteps < 8 ? C::ksteps : 8;
                float2 qv[kB][2][RT / 8];
                auto load = [&](int k0) {
                    auto at = [&](int kt, int x, int row) -> int64_t {
                        // natural order for 16-bit rows; for q8_0 lane tq owns dimensions
                        // tq D / 4 ..., four of them per step
                        const int d = C::q8 ? tq * (D / 4) + 4 * (k0 + kt) + 2 * x : 16 * (k0 + kt) + 8 * x + 2 * tq;
                        return ((head0 + row) * D + d) >> 1;
                    };
                    if (a.dtype == WSW_F32) {
#pragma unroll
                        for (int i = 0; i < kB * 2 * (RT / 8); ++i) {
                            const int kt = i / (RT / 4), x = (i / (RT / 8)) & 1, y = i % (RT / 8);
                            qv[kt][x][y] = g0 + gq + 8 * y < a.group
                                               ? reinterpret_cast<const float2 *>(a.q)[at(kt, x, gq + 8 * y)]
                                               : make_float2(0.f, 0.f);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < kB * 2 * (RT / 8); ++i) {
                            const int kt = i / (RT / 4), x = (i / (RT / 8)) & 1, y = i % (RT / 8);
                            qv[kt][x][y].x = __uint_as_float(
                                g0 + gq + 8 * y < a.group
                                    ? reinterpret_cast<const uint32_t *>(a.q)[at(kt, x, gq + 8 * y)] : 0u);
                        }
#pragma unroll
                        for (int i = 0; i < kB * 2 * (RT / 8); ++i) {
                            float2 &v = qv[i / (RT / 4)][(i / (RT / 8)) & 1][i % (RT / 8)];
                            const uint32_t u = __float_as_uint(v.x);
                            v = a.dtype == WSW_BF16 ? make_float2(bf16lo(u), bf16hi(u))
                                                    : __half22float2(*reinterpret_cast<const __half2 *>(&u));
                        }
                    }
                };
                float up[RT / 8];
#pragma unroll
                for (int y = 0; y < RT / 8; ++y) {
                    up[y] = 1.f;  // bf16 has fp32's range
                    unit[y] = a.cap_in != 0.f ? a.cap_in : a.scale2;
                }
                if constexpr (CT != WSW_BF16) {
                    float top[RT / 8];
#pragma unroll
                    for (int y = 0; y < RT / 8; ++y) top[y] = 0.f;
#pragma unroll 1
                    for (int k0 = 0; k0 < C::ksteps; k0 += kB) {
                        load(k0);
#pragma unroll
                        for (int i = 0; i < kB * 2 * (RT / 8); ++i) {
                            const float2 v = qv[i / (RT / 4)][(i / (RT / 8)) & 1][i % (RT / 8)];
                            top[i % (RT / 8)] = fmaxf(top[i % (RT / 8)], fmaxf(fabsf(v.x), fabsf(v.y)));
                        }
                    }
#pragma unroll
                    for (int y = 0; y < RT / 8; ++y) {
                        top[y] = fmaxf(top[y], __shfl_xor_sync(WSW_FULL_MASK, top[y], 1));
                        top[y] = fmaxf(top[y], __shfl_xor_sync(WSW_FULL_MASK, top[y], 2));
                        const int e = max(static_cast<int>(__float_as_uint(top[y]) >> 23), 15);
                        up[y] = __uint_as_float((268u - e) << 23);           // 2^(14 - (e - 127))
                        unit[y] *= __uint_as_float((e - 14u) << 23);         // its inverse
                    }
                }
#pragma unroll
                for (int k0 = 0; k0 < C::ksteps; k0 += kB) {
                    if (CT == WSW_BF16 || C::ksteps > kB) load(k0);
#pragma unroll
                    for (int j = 0; j < kB; ++j) {
                        const int kt = k0 + j;
                        uint32_t hi[4], lo[4], third[RT / 4];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {  // the fragment's two column halves
#pragma unroll
                            for (int y = 0; y < RT / 8; ++y) {
                                const float2 v = qv[j][x][y];
                                uint32_t vh, vl;
                                if constexpr (X3) split3(v.x, v.y, vh, vl, third[x * (RT / 8) + y]);
                                else split<CT>(v.x * up[y], v.y * up[y], vh, vl);
                                if constexpr (RT == 8) {
                                    hi[2 * x] = vh;
                                    hi[2 * x + 1] = vl;
                                } else {
                                    hi[2 * x + y] = vh;
                                    lo[2 * x + y] = vl;
                                    some |= (vl & 0x7fff7fffu) != 0;
                                }
                            }
                        }
                        if constexpr (C::q_smem) q_hi_sm[kt * 32 + lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) qa[kt][i] = hi[i];
                        }
                        if constexpr (RT == 16) q_lo_sm[kt * 32 + lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        if constexpr (X3) {
#pragma unroll
                            for (int i = 0; i < RT / 4; ++i) {
                                if constexpr (C::q_smem) q_third_sm[(kt * (RT / 4) + i) * 32 + lane] = third[i];
                                else q3[kt][i] = third[i];
                            }
                        }
                    }
                }
                if constexpr (RT == 16) q_lo = __any_sync(WSW_FULL_MASK, some);
#pragma unroll
                for (int y = 0; y < RT / 8; ++y) {
                    m[y] = -INFINITY;
                    l[y] = 0.f;
                    const int row = g0 + gq + 8 * y;
                    slope[y] = a.slopes && row < a.group ? a.slopes[h * a.group + row] * kLog2e : 0.f;
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
            }
            cp_wait<C::stages - 1>();
            __syncwarp();  // the tile's pieces copied by every lane are visible
            const uint32_t stg = ring_s + rst * C::stage;
            const unsigned char *stg_p = ring + rst * C::stage;
            const uint32_t valid = seen_mask[warp][rst];
            if (++rst == C::stages) rst = 0;

            // ---- scores, in blocks of 8 positions
            constexpr int NB = T / 8;
            float sc[NB][4];
#pragma unroll
            for (int n = 0; n < NB; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
            auto q_frag = [&](int kt, uint32_t (&qf)[4]) {
                if constexpr (C::q_smem) {
                    const uint4 u = q_hi_sm[kt * 32 + lane];
                    qf[0] = u.x; qf[1] = u.y; qf[2] = u.z; qf[3] = u.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) qf[i] = qa[kt][i];
                }
            };
            // d += q_kt K^T for one block, its two registers b0 and b1
            auto score = [&](float (&d)[4], int kt, uint32_t b0, uint32_t b1) {
                uint32_t qf[4];
                q_frag(kt, qf);
                mma<CT>(d, qf, b0, b1);
                if constexpr (RT == 16) {
                    if (q_lo) {
                        const uint4 u = q_lo_sm[kt * 32 + lane];
                        const uint32_t ql[4] = {u.x, u.y, u.z, u.w};
                        mma<CT>(d, ql, b0, b1);
                    }
                }
                if constexpr (X3) {
                    uint32_t t[RT / 4];
#pragma unroll
                    for (int i = 0; i < RT / 4; ++i) {
                        if constexpr (C::q_smem) t[i] = q_third_sm[(kt * (RT / 4) + i) * 32 + lane];
                        else t[i] = q3[kt][i];
                    }
                    mma_third<CT, RT>(d, t, b0, b1);
                }
            };
            if constexpr (!C::q8) {
                static_assert(C::q8 || NB == 2, "blocks");
                float sd[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // the odd steps: a second chain
                const int pos = 8 * (mi >> 1) + mr;
#pragma unroll
                for (int kt = 0; kt < C::ksteps; ++kt) {
                    uint32_t kb[4];
                    const int ch = 2 * kt + (mi & 1);
                    ldsm4(kb, stg + pos * C::row_bytes + ((ch ^ (pos & 7)) << 4));
                    score(kt & 1 ? sd[0] : sc[0], kt, kb[0], kb[1]);
                    score(kt & 1 ? sd[1] : sc[1], kt, kb[2], kb[3]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[0][i] += sd[0][i];
                    sc[1][i] += sd[1][i];
                }
            } else {
                constexpr int kVec = D / 64;  // 16-byte pieces per lane and row
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    uint32_t w[4 * kVec];
                    __half2 ds[D == 256 ? 2 : 1];
                    const int row = 8 * n + gq;
#pragma unroll
                    for (int i = 0; i < kVec; ++i) {
                        const int ch = tq * kVec + i;
                        const int sw = C::pieces >= 8 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3);
                        const uint4 u = *reinterpret_cast<const uint4 *>(stg_p + row * C::row_bytes + sw * 16);
                        w[4 * i] = u.x ^ 0x80808080u;
                        w[4 * i + 1] = u.y ^ 0x80808080u;
                        w[4 * i + 2] = u.z ^ 0x80808080u;
                        w[4 * i + 3] = u.w ^ 0x80808080u;
                    }
                    const __half *sp = reinterpret_cast<const __half *>(stg_p + 2 * C::kv_bytes + row * C::scale_bytes);
                    if constexpr (D == 64) ds[0] = __half2half2(sp[tq >> 1]);
                    else if constexpr (D == 128) ds[0] = __half2half2(sp[tq]);
                    else {
                        ds[0] = __half2half2(sp[2 * tq]);
                        ds[1] = __half2half2(sp[2 * tq + 1]);
                    }
#pragma unroll
                    for (int kt = 0; kt < C::ksteps; ++kt) {
                        const int bl = D == 256 ? kt >> 3 : 0;
                        score(sc[n], kt, dequant2(w[kt], 0x4140, ds[bl]), dequant2(w[kt], 0x4342, ds[bl]));
                    }
                }
            }

            // ---- softmax: lane (gq, tq) holds positions 8 n + 2 tq + {0, 1} of rows gq, gq + 8
            const int p0 = uc.start + uc.t * T;
            uint32_t ph[NB / 2][4], pl[NB / 2][4], pt[NB / 2][RT / 4];
            float al[RT / 8];
            bool raised = false;
#pragma unroll
            for (int y = 0; y < RT / 8; ++y) {
                float s[2 * NB];
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int pi = 8 * n + 2 * tq + j;
                        float x = RT == 8 ? sc[n][j] + sc[n][2 + j] : sc[n][2 * y + j];
                        if constexpr (CT == WSW_BF16) {
                            x = a.cap_in != 0.f ? a.cap_out * tanhf(x * a.cap_in) : x * a.scale2;
                        } else {
                            x *= unit[y];
                            if (a.cap_in != 0.f) x = a.cap_out * tanhf(x);
                        }
                        if (a.slopes) x = fmaf(-slope[y], static_cast<float>(uc.len - 1 - (p0 + pi)), x);
                        s[2 * n + j] = (valid >> pi) & 1 ? x : -INFINITY;
                    }
                float mt = s[0];
#pragma unroll
                for (int i = 1; i < 2 * NB; ++i) mt = fmaxf(mt, s[i]);
                mt = fmaxf(mt, __shfl_xor_sync(WSW_FULL_MASK, mt, 1));
                mt = fmaxf(mt, __shfl_xor_sync(WSW_FULL_MASK, mt, 2));
                const bool raise = mt > m[y] + kLazy;  // m = -inf: by anything visible
                al[y] = raise ? ex2(m[y] - mt) : 1.f;
                raised |= raise;
                if (raise) m[y] = mt;
                const float ref = m[y] == -INFINITY ? 0.f : m[y] - C::shift;  // nothing seen yet: all weights 0
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const float p_0 = ex2(s[2 * n] - ref), p_1 = ex2(s[2 * n + 1] - ref);
                    sum += p_0 + p_1;
                    uint32_t &hi = ph[n / 2][2 * (n & 1) + y];
                    uint32_t &lo = RT == 8 ? ph[n / 2][2 * (n & 1) + 1] : pl[n / 2][2 * (n & 1) + y];
                    if constexpr (X3) split3(p_0, p_1, hi, lo, pt[n / 2][(n & 1) * (RT / 8) + y]);
                    else split<CT>(p_0, p_1, hi, lo);
                }
                l[y] = fmaf(l[y], al[y], sum);
            }
            if (__any_sync(WSW_FULL_MASK, raised)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][0] *= al[0];
                    o[n][1] *= al[0];
                    o[n][2] *= al[RT / 8 - 1];
                    o[n][3] *= al[RT / 8 - 1];
                }
            }

            // ---- value sums, 16 positions at a time
#pragma unroll
            for (int t16 = 0; t16 < T / 16; ++t16) {
                auto add = [&](int n, uint32_t b0, uint32_t b1) {
                    mma<CT>(o[n], ph[t16], b0, b1);
                    if constexpr (RT == 16) mma<CT>(o[n], pl[t16], b0, b1);
                    if constexpr (X3) mma_third<CT, RT>(o[n], pt[t16], b0, b1);
                };
                const int vpos = 16 * t16 + 8 * (mi & 1) + mr;
                if constexpr (!C::q8) {
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        uint32_t vb[4];
                        const int ch = 2 * j + (mi >> 1);
                        ldsm4_t(vb, stg + C::kv_bytes + vpos * C::row_bytes + ((ch ^ (vpos & 7)) << 4));
                        add(2 * j, vb[0], vb[1]);
                        add(2 * j + 1, vb[2], vb[3]);
                    }
                } else {
                    // a transposed 16-bit matrix element is a pair of codes: dimensions 16 c + 2 i and
                    // + 1 of one position.  Bytes 0 and 2 of a register are the even dimension at
                    // positions 2 tq and 2 tq + 1, bytes 1 and 3 the odd one: two column blocks.
                    const unsigned char *vs = stg_p + 2 * C::kv_bytes + T * C::scale_bytes;
                    constexpr int kBl = D / 32;
                    __half dv[4][kBl];  // scales of positions 2 tq, 2 tq + 1, 8 + 2 tq, 9 + 2 tq
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 16 * t16 + 8 * (i >> 1) + 2 * tq + (i & 1);
                        const __half *sp = reinterpret_cast<const __half *>(vs + row * C::scale_bytes);
                        if constexpr (kBl == 2) *reinterpret_cast<uint32_t *>(dv[i]) = *reinterpret_cast<const uint32_t *>(sp);
                        else if constexpr (kBl == 4) *reinterpret_cast<uint2 *>(dv[i]) = *reinterpret_cast<const uint2 *>(sp);
                        else *reinterpret_cast<uint4 *>(dv[i]) = *reinterpret_cast<const uint4 *>(sp);
                    }
#pragma unroll
                    for (int j = 0; j < kBl; ++j) {
                        uint32_t vb[4];
                        const int ch = 2 * j + (mi >> 1);
                        const int sw = C::pieces >= 8 ? ch ^ (vpos & 7) : ch ^ ((vpos >> 1) & 3);
                        ldsm4_t(vb, stg + C::kv_bytes + vpos * C::row_bytes + (sw << 4));
                        const __half2 d0 = __halves2half2(dv[0][j], dv[1][j]), d1 = __halves2half2(dv[2][j], dv[3][j]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) vb[i] ^= 0x80808080u;
#pragma unroll
                        for (int pc = 0; pc < 2; ++pc) {
                            add(4 * j + 2 * pc, dequant2(vb[2 * pc], 0x4240, d0), dequant2(vb[2 * pc + 1], 0x4240, d1));
                            add(4 * j + 2 * pc + 1, dequant2(vb[2 * pc], 0x4341, d0), dequant2(vb[2 * pc + 1], 0x4341, d1));
                        }
                    }
                }
            }

            // ---- the end of the pair, or of the run
            const bool pair_end = uc.t == uc.nt - 1, run_end = uc.g + 1 + (pair_end ? extra : 0) >= we;
            if (!pair_end && !run_end) {
                ++uc.t;
                ++uc.g;
                continue;
            }
            fresh = true;
            const int h = uc.hp / a.passes, g0 = (uc.hp - h * a.passes) * RT;
            const bool whole = pair_end && t_first == 0;
            float *rec = nullptr;
            if (!whole) {
                if (run_end) {  // the run's last piece: into the ring, which no copy uses any more
                    cp_wait<0>();
                    __syncwarp();
                    rec = reinterpret_cast<float *>(ring);
                } else {
                    rec = a.wrec + static_cast<int64_t>(cta * W + warp) * RT * C::srec;
                    first_left = true;
                }
                if (lane == 0) pieces[2 * warp + run_end] = Piece{uc.g - uc.t, uc.r, uc.hp, uc.nt};
            }
#pragma unroll
            for (int y = 0; y < RT / 8; ++y) {
                l[y] += __shfl_xor_sync(WSW_FULL_MASK, l[y], 1);
                l[y] += __shfl_xor_sync(WSW_FULL_MASK, l[y], 2);
                const int row = gq + 8 * y;
                if (g0 + row >= a.group) continue;
                const int64_t head = static_cast<int64_t>(uc.r) * a.q_heads + h * a.group + g0 + row;
                const float inv = l[y] == 0.f ? 0.f : 1.f / l[y], f = whole ? inv : 1.f;
                float v[D / 8][2];
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) v[n][x] = (RT == 8 ? o[n][x] + o[n][2 + x] : o[n][2 * y + x]) * f;
                if (tq == 0) {
                    if (!whole) piece_ml[2 * warp + run_end][row] = make_float2(m[y], l[y]);
                    else if (a.lse) a.lse[head] = lse_of(m[y], l[y], C::shift);
                }
                // lane tq's dimensions: 2 tq, 2 tq + 1 of every eight, or (q8_0) 4 tq .. 4 tq + 3 of sixteen
                if (!whole || a.dtype == WSW_F32) {
                    float *dst = whole ? static_cast<float *>(a.out) + head * D : rec + row * C::srec;
                    dst += C::q8 ? 4 * tq : 2 * tq;
#pragma unroll
                    for (int n = 0; n < D / 8; n += C::q8 ? 2 : 1) {
                        if constexpr (C::q8)
                            *reinterpret_cast<float4 *>(dst + 8 * n) = make_float4(v[n][0], v[n + 1][0], v[n][1], v[n + 1][1]);
                        else
                            *reinterpret_cast<float2 *>(dst + 8 * n) = make_float2(v[n][0], v[n][1]);
                    }
                } else {
                    uint16_t *dst = static_cast<uint16_t *>(a.out) + head * D + (C::q8 ? 4 * tq : 2 * tq);
#pragma unroll
                    for (int n = 0; n < D / 8; n += C::q8 ? 2 : 1) {
                        if constexpr (C::q8)
                            *reinterpret_cast<uint2 *>(dst + 8 * n) =
                                make_uint2(pack16(a.dtype, v[n][0], v[n + 1][0]), pack16(a.dtype, v[n][1], v[n + 1][1]));
                        else
                            *reinterpret_cast<uint32_t *>(dst + 8 * n) = pack16(a.dtype, v[n][0], v[n][1]);
                    }
                }
            }
            if (run_end) break;
            advance<T>(a, uc, extra);
        }
        // the first piece's record joins the last one's in the ring
        if (first_left) {
            __syncwarp();
            const float4 *src = reinterpret_cast<const float4 *>(a.wrec + static_cast<int64_t>(cta * W + warp) * RT * C::srec);
            float4 *dst = reinterpret_cast<float4 *>(ring) + RT * C::srec / 4;
            constexpr int kPer = RT * C::srec / 4 / 32;  // whole rounds of the warp
#pragma unroll 8
            for (int i = 0; i < kPer; ++i) dst[i * 32 + lane] = src[i * 32 + lane];
            if (lane < RT * C::srec / 4 - kPer * 32) dst[kPer * 32 + lane] = src[kPer * 32 + lane];
        }
    }
    __syncthreads();

    // ---- join the warps' records, pair by pair in tile order: the weights of a pair's
    // records first, then independent sums
    constexpr int kCols = D / 4;
    float *wgt = reinterpret_cast<float *>(smem + W * C::ring);  // [2 W][RT] weights, then [2 W][RT] (m, l)
    float2 *joined = reinterpret_cast<float2 *>(wgt + 2 * W * RT);
    __shared__ uint32_t pair_set[2 * W];  // each pair's pieces, and its first one
    __shared__ int pair_first[2 * W];
    // a lane for each piece: the pieces of a pair are neighbours
    const bool have = lane < 2 * W && pieces[lane < 2 * W ? lane : 0].r >= 0;
    const int key = have ? pieces[lane].pstart : -1;
    const uint32_t all = __ballot_sync(WSW_FULL_MASK, have);
    const uint32_t upto_me = (2u << lane) - 1, below = all & (upto_me >> 1);
    const int key_below = __shfl_sync(WSW_FULL_MASK, key, below ? 31 - __clz(below) : lane);
    const bool is_first = have && !(below && key == key_below);
    const uint32_t firsts = __ballot_sync(WSW_FULL_MASK, is_first), later = firsts & ~upto_me;
    const int pairs = __popc(firsts);
    const bool open = is_first && !(key >= b && key + pieces[lane < 2 * W ? lane : 0].nt <= e);
    const uint32_t open_set = __ballot_sync(WSW_FULL_MASK, open);  // pairs shared with other CTAs: at most two
    const int my_first = 31 - __clz((firsts & upto_me) | 1u), my_pair = __popc(firsts & upto_me) - 1;
    const uint32_t set = all & ~((1u << my_first) - 1) & (later ? (1u << (__ffs(later) - 1)) - 1 : 0xffffffffu);
    const int my_last = set ? 31 - __clz(set) : lane;  // of this lane's pair
    if (warp == 0 && is_first) {
        pair_set[my_pair] = set;
        pair_first[my_pair] = lane;
    }
    // a warp for each row: maximum and sum along the neighbours of a pair (a lane without a
    // piece counts as its pair's, with no weight)
    const int run_key = have ? key : key_below;
#pragma unroll 1
    for (int row = warp; row < RT; row += W) {
        const float2 ml = have ? piece_ml[lane < 2 * W ? lane : 0][row] : make_float2(-INFINITY, 0.f);
        float mx = ml.x;
#pragma unroll
        for (int d = 1; d < 2 * W; d <<= 1) {
            const float y = __shfl_up_sync(WSW_FULL_MASK, mx, d);
            const int k = __shfl_up_sync(WSW_FULL_MASK, run_key, d);
            if (lane >= d && k == run_key) mx = fmaxf(mx, y);
        }
        mx = __shfl_sync(WSW_FULL_MASK, mx, my_last);
        const float f = weight(ml.x, mx);
        float l = ml.y * f;
#pragma unroll
        for (int d = 1; d < 2 * W; d <<= 1) {
            const float y = __shfl_up_sync(WSW_FULL_MASK, l, d);
            const int k = __shfl_up_sync(WSW_FULL_MASK, run_key, d);
            if (lane >= d && k == run_key) l += y;
        }
        l = __shfl_sync(WSW_FULL_MASK, l, my_last);
        if (have) wgt[lane * RT + row] = f;
        if (is_first) joined[my_pair * RT + row] = make_float2(mx, l);
    }
    __syncthreads();
    // a thread keeps its place in the records and takes the pairs in turn
    constexpr int kUnits = RT * kCols, kTurns = NT / kUnits > 1 ? NT / kUnits : 1;
#pragma unroll 1
    for (int u = tid; u < kTurns * kUnits; u += NT) {
        const int v = u % kUnits, row = v / kCols, c4 = v % kCols;
#pragma unroll 1
        for (int j = u / kUnits; j < pairs; j += kTurns) {
            const Piece pc = pieces[pair_first[j]];
            const int h = a.passes == 1 ? pc.hp : pc.hp / a.passes, g0 = (pc.hp - h * a.passes) * RT;
            if (g0 + row >= a.group) continue;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (uint32_t m = pair_set[j]; m; m &= m - 1) {
                const int k = __ffs(m) - 1;
                const float f = wgt[k * RT + row];
                const float4 x = *reinterpret_cast<const float4 *>(
                    reinterpret_cast<const float *>(smem + (k >> 1) * C::ring) + ((k & 1 ? 0 : RT) + row) * C::srec + 4 * c4);
                s.x = fmaf(x.x, f, s.x);
                s.y = fmaf(x.y, f, s.y);
                s.z = fmaf(x.z, f, s.z);
                s.w = fmaf(x.w, f, s.w);
            }
            const float2 ml = joined[j * RT + row];
            if (pc.pstart >= b && pc.pstart + pc.nt <= e) {
                const int64_t head = static_cast<int64_t>(pc.r) * a.q_heads + h * a.group + g0 + row;
                const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
                store_out4(a, head * D + 4 * c4, make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv));
                if (c4 == 0 && a.lse) a.lse[head] = lse_of(ml.x, ml.y, C::shift);
            } else {
                float *r = a.rec + static_cast<int64_t>(cta * 2 + (pc.pstart < b ? 0 : 1)) * RT * C::rec + row * C::rec;
                *reinterpret_cast<float4 *>(r + 4 + 4 * c4) = s;
                if (c4 == 0) *reinterpret_cast<float2 *>(r) = ml;
            }
        }
    }
    const int nshared = __popc(open_set);
    Piece shared_a = pieces[0], shared_b = pieces[0];
    if (nshared > 0) shared_a = pieces[__ffs(open_set) - 1];
    if (nshared > 1) shared_b = pieces[31 - __clz(open_set)];
    __syncthreads();
    if (nshared == 0) return;

    // ---- pairs shared with other CTAs (at most two): first the group's CTAs, then the groups.
    // The block barrier above orders this CTA's records before thread 0's arrival, whose
    // release publishes them; its acquire, and the barrier after it, order the reads below
    // after every arrival.
    auto arrive = [](unsigned *cnt, int expected) {
        unsigned old;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(cnt) : "memory");
        const bool is_last = old == static_cast<unsigned>(expected - 1);
        if (is_last) *cnt = 0u;  // ready for the next call
        return is_last;
    };
    const int group0 = cta / kGroup * kGroup;  // the group's first CTA
    // the CTAs of a long pair's first and last tiles, by the cuts as they were moved
    auto first_cta = [&](const Piece &pc) {
        const int c = pc.pstart / run;
        return c + ((c + 1) * run - (pc.pstart - extra) <= margin);
    };
    auto last_cta = [&](const Piece &pc) {
        const int end = pc.pstart + pc.nt, c = (end - 1) / run;
        return c - (end - c * run <= margin);
    };
    if (tid < nshared) {
        const Piece pc = tid == 0 ? shared_a : shared_b;
        const int f = first_cta(pc), c0 = max(f, group0), c1 = min(last_cta(pc), group0 + kGroup - 1);
        last[tid] = arrive(a.cnt + 2 * c0 + (c0 == f), c1 - c0 + 1);
    }
    __syncthreads();
    for (int sp = 0; sp < nshared; ++sp) {
        if (!last[sp]) continue;
        const Piece pc = sp == 0 ? shared_a : shared_b;
        const int f = first_cta(pc), t = last_cta(pc);
        const int h = pc.hp / a.passes, g0 = (pc.hp - h * a.passes) * RT;
        const int rows = min(RT, a.group - g0);
        const int groups = t / kGroup - f / kGroup + 1;
        // level 0: the group's CTAs; level 1: the groups, each at its first CTA's record
#pragma unroll 1
        for (int level = 0; level < 2; ++level) {
            const int c0 = level == 0 ? max(f, group0) : f;
            const int n = level == 0 ? min(t, group0 + kGroup - 1) - c0 + 1 : groups;
            const bool final = level == 1 || groups == 1;
            // record k; a pair begins in its first CTA's second record
            auto record = [&](int k) -> float * {
                const int c = level == 0 ? c0 + k : k == 0 ? f : (f / kGroup + k) * kGroup;
                return a.rec + (static_cast<int64_t>(c) * 2 + (c == f)) * RT * C::rec;
            };
            constexpr int kMost = kGroup > (kCtas + kGroup - 1) / kGroup + 1 ? kGroup : (kCtas + kGroup - 1) / kGroup + 1;
            static_assert(kMost <= 64, "records");
            constexpr int kAhead = kMost < 20 ? kMost : 20;  // of a thread's records on their way at once
            float *w = reinterpret_cast<float *>(smem);                // [kMost][RT] weights
            float2 *jn = reinterpret_cast<float2 *>(w + kMost * RT);   // [RT] joined (m, l)
            const int apart = (level == 0 ? 2 : 2 * kGroup) * RT * C::rec;  // from the second record on
            const float *r0 = record(0), *r1 = record(1);
            auto part = [&](int k, int at) { return (k == 0 ? r0 : r1 + (k - 1) * apart) + at; };
#pragma unroll 1
            for (int u = tid; u - tid < kUnits; u += NT) {
                const int row = u / kCols, c4 = u % kCols, at = row * C::rec + 4 + 4 * c4;
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                for (int k0 = 0; k0 < n; k0 += kAhead) {
                    float4 xa[kAhead];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k)
                        if (k0 + k < n && row < rows) xa[k] = __ldcg(reinterpret_cast<const float4 *>(part(k0 + k, at)));
                    if (u == tid && k0 == 0) {  // meanwhile the weights, a warp for each row
#pragma unroll 1
                        for (int wr = warp; wr < rows; wr += W) {
                            const float2 none = make_float2(-INFINITY, 0.f);
                            const float2 x = lane < n ? __ldcg(reinterpret_cast<const float2 *>(part(lane, wr * C::rec))) : none;
                            const float2 y = lane + 32 < n
                                ? __ldcg(reinterpret_cast<const float2 *>(part(lane + 32, wr * C::rec))) : none;
                            float mx = fmaxf(x.x, y.x);
#pragma unroll
                            for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(WSW_FULL_MASK, mx, d));
                            const float fx = weight(x.x, mx), fy = weight(y.x, mx);
                            float l = fmaf(x.y, fx, y.y * fy);
#pragma unroll
                            for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(WSW_FULL_MASK, l, d);
                            if (lane < n) w[lane * RT + wr] = fx;
                            if (lane + 32 < n) w[(lane + 32) * RT + wr] = fy;
                            if (lane == 0) jn[wr] = make_float2(mx, l);
                        }
                        __syncthreads();
                    }
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        if (k0 + k >= n || row >= rows) break;
                        const float g = w[(k0 + k) * RT + row];
                        s.x = fmaf(xa[k].x, g, s.x);
                        s.y = fmaf(xa[k].y, g, s.y);
                        s.z = fmaf(xa[k].z, g, s.z);
                        s.w = fmaf(xa[k].w, g, s.w);
                    }
                }
                if (row >= rows) continue;
                const float2 ml = jn[row];
                if (final) {
                    const int64_t head = static_cast<int64_t>(pc.r) * a.q_heads + h * a.group + g0 + row;
                    const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
                    store_out4(a, head * D + 4 * c4, make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv));
                    if (c4 == 0 && a.lse) a.lse[head] = lse_of(ml.x, ml.y, C::shift);
                } else {
                    // the group's record takes the place of its first CTA's: this thread has read
                    // what it writes, and everyone the (m, l)
                    float *r = record(0);
                    *reinterpret_cast<float4 *>(r + at) = s;
                    if (c4 == 0) *reinterpret_cast<float2 *>(r + row * C::rec) = ml;
                }
            }
            __syncthreads();
            if (final) break;
            if (tid == 0) last[sp] = arrive(a.cnt + 2 * kCtas + f, groups);
            __syncthreads();
            if (!last[sp]) break;
        }
    }
}

template <int CT, bool X3>
cudaError_t launch_type(const Args &a, int rows, cudaStream_t s, bool pdl, int64_t tiles);

template <int CT, int D, int RT, bool X3>
cudaError_t launch_one(const Args &a, cudaStream_t s, bool pdl, int64_t tiles) {
    using C = Cfg<CT, D, RT, X3>;
    const auto kernel = attn_paged_kernel<CT, D, RT, X3>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kernel), C::smem);
    if (e != cudaSuccess) return e;
    // no more CTAs than `tiles`, the most that there can be, fill
    const int64_t want = (tiles + C::warps - 1) / C::warps, ctas = want < 1 ? 1 : want > kCtas ? kCtas : want;
    return launch(kernel, dim3(static_cast<unsigned>(ctas)), dim3(C::threads), C::smem, s, pdl, a);
}

#define WSW_PAGED_TYPE(CT, X3)                                                                       \
    template <>                                                                                      \
    cudaError_t launch_type<CT, X3>(const Args &a, int rows, cudaStream_t s, bool pdl, int64_t tiles) {   \
        switch (a.kv.head_dim * 2 + (rows == 16)) {                                                  \
            case 128: return launch_one<CT, 64, 8, X3>(a, s, pdl, tiles);                             \
            case 129: return launch_one<CT, 64, 16, X3>(a, s, pdl, tiles);                            \
            case 256: return launch_one<CT, 128, 8, X3>(a, s, pdl, tiles);                            \
            case 257: return launch_one<CT, 128, 16, X3>(a, s, pdl, tiles);                           \
            case 512: return launch_one<CT, 256, 8, X3>(a, s, pdl, tiles);                            \
            default: return launch_one<CT, 256, 16, X3>(a, s, pdl, tiles);                            \
        }                                                                                            \
    }

}  // namespace paged
}  // namespace wsw
