// attn_prefix.cuh -- attention of the requests of a group over the prefix that they share: K and V read
// once for all of them, on the fifth-generation tensor cores.
//
//   x = scale q . K_p (capped by softcap tanh(. / softcap), minus slope (n - 1 - p)), log2 units
//   m = max_p x,  l = sum_p 2^(x - m),  O = sum_p 2^(x - m) V_p       over the positions p < prefix
// The rest of each request's positions is the paged decode attention's (attn_paged.cuh), and a last
// kernel joins the parts (attn_prefix.cu).
//
// The query heads of all of a group's requests that share a KV head are the rows of one product:
// 4 D flops per row and position against 4 D bytes (16 bits) per position, so that a few hundred rows are
// bound by the tensor cores, a few by HBM.  256 requests of 4 x 8 heads behind 32768 positions, bf16: some 128 us of this
// kernel, 1.6 PFLOP/s with the weights' second part counted; the products keep the tensor cores busy for 70% of the
// cycles under a profiler: the two slots' softmax (one exponential for each score, 16 a cycle) and products do not overlap
// all the time.
//
//  * A unit is a tile of rows (kv head, 128 or 256 of a group's rows); the position tiles of all units,
//    in order, are one list that is cut into equal runs for 152 CTAs, one on an SM (attn_prefix.cu has the rules).  A CTA leaves
//    (m, l, O) of each piece of a unit; pieces are joined in tile order, so that results depend on
//    the sizes alone.
//  * Two softmax warpgroups, a thread for each row, each with its own scores S and value sums O in
//    tensor memory.  With two row tiles in a unit they have 128 rows each and the same K and V (half the
//    reads); with one the same rows, and take the tiles in turn; their sums are joined when the
//    piece ends.  One's softmax runs while the tensor cores work for the other.
//  * The weights P go back to tensor memory over the scores, whose thread has read them; S of the next
//    tile is issued behind the P V that reads them, and one thread's MMAs complete in order.  The P V of a tile's
//    first half runs while the second half's weights are made (with P in one part, 170 us for the case above without, 162 with).
//  * Four warps copy K and V rows with cp.async into a ring of tiles, swizzled as the MMAs want them:
//    16-byte pieces by the block table, so that any page size, layout and stride is the same code (a TMA box
//    cannot cross a page, and pages may have one position).  Over q8_0 four warps have K and four have V: codes
//    and scales land in rings of their own, two or three tiles deep, and become binary16(scale * code) on the way to the
//    tile (33 fp32 requests of 4 x 8 heads behind 32768 positions: 117 us with one set of loaders, 101 so, and 91 since).  A tile's
//    barrier counts the threads whose copies have landed, and each warp's word of the tile's visible positions.
//  * q, scores, sums and l are fp32 or parts: q over its own 16-bit type is exact, a bf16 or fp32 row
//    over binary16 takes the power of two that brings its largest value to 2^14 .. 2^15 and, fp32, a second
//    part (22 bits); fp16 over bf16 is two parts, fp32 over bf16 three, both exact.  P is two parts, 16 (bf16) or 22 bits
//    (binary16), under fp32 queries over bf16 three, as in attn_paged.cuh, so that which of the two kernels attends
//    a position does not show in the result.  (With one part the weights' rounding was as large as a bf16 result's
//    own, 2.3e-3 in the root mean square instead of 1.7e-3; the call for the case above, with rests of 16
//    positions, took 155 us with one part and 187 so.)
//  * The maximum in use is raised, and O rescaled, only when a tile exceeds it by more than kLazy.
//  * Every wait is bounded; a role whose wait ran out stops once its own copies or MMAs have ended.  The block's later pieces
//    are then missing, so that a word says so (blocks that start later have nothing to do) and the join makes all rows
//    behind a prefix NaN.
#pragma once

#include "attn_paged.cuh"
#include "tc_util.cuh"

namespace wsw {
namespace prefix {

using paged::cp16;
using paged::ex2;
using paged::kLazy;
using paged::kLog2e;
using paged::split;
using paged::split3;

constexpr int kCtas = 152;     // runs of the tile list
constexpr int kLoaders = 4;    // warps that share a tile
constexpr int kSeen = 16;      // tiles whose visible positions are kept
constexpr int kControl = 2048, kTileBytes = 227 * 1024 - kControl - 1024;
constexpr uint32_t kTmemCols = 512;
constexpr int kHead = 8;       // floats before a record's O: whole sectors

// What the plan kernel leaves: [groups + 1] each but `run`.
struct Plan {
    const int *begin;  // first request of a group
    const int *off;    // its tiles' place in the list
    const int *used;   // its prefix's positions
    const int *rep;    // the request whose table row holds its pages
    const int *stride; // places that each of its units has in the list, its tiles at least
    int *run;          // [1] places of a CTA; 0 once a wait ran out
    const int2 *start; // [kCtas] group and place in its part where a CTA's run begins; group -1: nothing
};

struct Args {
    const void *q;
    const float *slopes;
    const int32_t *table, *lens;
    int32_t *err;
    Plan plan;
    float *rec;    // [kCtas][2][rows of a unit][D + kHead]: (m - shift, l, - ..., O) of pieces
    float *whole;  // [requests * q_heads][D + kHead]: of units that one CTA has whole
    KvView kv;
    int64_t table_stride;
    float scale2;  // |scale| log2 e
    float cap_in;  // |scale| / softcap, 0: not capped
    float cap_out; // softcap log2 e
    int q_heads, group, groups, max_len;
    int dtype, negative;  // of q; scale < 0
};

// Positions of a tile.  fp32 queries and q8_0 under two row tiles: 64, for room.
constexpr int tile_positions(bool wide, int cache, int row_tiles) {
    return !wide && !(cache == WSW_Q8_0 && row_tiles == 2) ? 128 : 64;
}

// cap tanh(x) of v = 2 log2(e) x.  From |x| = 0.3 on 1 - 2 / (1 + e^2|x|) with x's sign, off by 7 2^-24 at most: the power's
// 2^-22 counts half where 2 / (1 + e^2|x|) moves most, its argument's roundings 2^-24 together, the sum, the reciprocal
// (2^-23) and the difference 2^-24 to 2^-23 each.  Below, where that difference would leave errors of the cap's size, not of the
// score's, Taylor's series x - x^3 / 3 + 2 x^5 / 15 - 17 x^7 / 315 + 62 x^9 / 2835, whose next term is 2^-24 of it at 0.3.
// Either way tanh is off by 24 2^-24 of itself at most.  Chunks of scores that are all below take the series alone.  (256
// requests behind 32768 positions as above, capped: 319 us where all are, 408 where both forms are computed, 153 uncapped; both
// for all: 366.  33 fp32 requests over q8_0: 114, 142 and 90.)
constexpr float kNear = 0.875f;  // of v: |x| = 0.303
__device__ __forceinline__ float capped_near(float v, float cap) {
    constexpr double a = 0.34657359027997264;  // x = a v: ln 2 / 2
    constexpr float c1 = a, c3 = -a * a * a / 3, c5 = 2 * a * a * a * a * a / 15, c7 = -17 * a * a * a * a * a * a * a / 315,
                    c9 = 62 * a * a * a * a * a * a * a * a * a / 2835;
    const float y = v * v;
    return cap * v * fmaf(fmaf(fmaf(fmaf(c9, y, c7), y, c5), y, c3), y, c1);
}
__device__ __forceinline__ float capped(float v, float cap) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(fabsf(v))));
    return fabsf(v) < kNear ? capped_near(v, cap) : copysignf(fmaf(-2.f * cap, r, cap), v);
}

// Shape of one variant: cache type, head_dim, parts of q, row tiles of a unit.
template <int CT, int D_, int QP_, int RT_>
struct Cfg {
    static constexpr int D = D_, QP = QP_, RT = RT_;
    static constexpr bool q8 = CT == WSW_Q8_0, bf16 = CT == WSW_BF16;
    static constexpr bool wide = QP == (bf16 ? 3 : 2);     // fp32 queries
    static constexpr int PP = QP == 3 ? 3 : 2;             // parts of P
    static constexpr int TP = tile_positions(wide, CT, RT);
    static constexpr int stage = TP * D * 2;               // a K or V tile
    static constexpr int q_part = 128 * D * 2;             // of a row tile
    static constexpr int q_bytes = RT * QP * q_part;
    // q8_0 rows land as codes and scales, a few tiles of K and of V deep, and become tiles from there
    static constexpr int raw = q8 ? TP * (D + D / 16) : 0, raw_stages = 2 + (TP == 64);
    static constexpr int fit = (kTileBytes - q_bytes - 2 * raw_stages * raw) / stage;
    static constexpr int stages = fit < 8 ? fit : 8;
    static constexpr int ahead = RT == 1 ? 2 : 1;          // K tiles before their V tiles
    // of a slot: scores, then P's parts.  Two parts of 32 weights take the place of their own scores, side by side; three
    // take more, and all scores' places, which a thread keeps meanwhile.
    static constexpr int s_cols = PP == 3 ? 96 : TP;
    // the column of part k of the weights of 16 positions, of P's first
    static constexpr int p_col(int k, int sixteen) {
        return PP == 3 ? k * (TP / 2) + 8 * sixteen : (sixteen >> 1) * 32 + 16 * k + 8 * (sixteen & 1);
    }
    static constexpr uint32_t o_col = 2 * s_cols;
    static constexpr float shift = bf16 ? -kLazy : 7.f;    // log2 of the weights' scale
    static constexpr int rec = D + kHead;
    // Warpgroups: two of softmax, one or (q8_0, whose codes become values on the way) two of loaders, K's and V's, and
    // the MMAs' warp with three idle ones.
    static constexpr int load_groups = q8 ? 2 : 1;
    static constexpr int mma_warp = 8 + 4 * load_groups, threads = 32 * (mma_warp + 4);
    // registers of a thread, as launched and by role
    static constexpr int regs = q8 ? 96 : 128;
    static constexpr int soft_regs = q8 ? 128 : 144, load_regs = q8 ? 80 : 112, mma_regs = q8 ? 64 : 112;
    static_assert(2 * soft_regs + load_groups * load_regs + mma_regs == (3 + load_groups) * regs && regs * threads <= 65536,
                  "what the block was launched with");
    static_assert(2 * s_cols + 2 * D <= 512 && stages >= 3 && kSeen >= stages + 4 + (q8 ? raw_stages : 0), "room");
    static constexpr int smem = q_bytes + stages * stage + 2 * raw_stages * raw + kControl + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
};

struct Control {
    uint64_t full[8], empty[8];
    uint64_t s_full[2], p_full[2][2];  // of a slot; of each half of its weights
    uint64_t q_full, o_done, stopped;
    uint32_t seen[kSeen][4];
    float unit[256];    // of the rows' scores
    uint32_t tmem;
};
static_assert(sizeof(Control) <= kControl && kTileBytes + kControl + 1024 <= 227 * 1024, "control");

// The pieces of a CTA's run, in order; every role walks them.
template <typename C>
struct Walk {
    const Args &a;
    int pos, end;                 // places in the list
    int g, in;                    // group, place in its part
    int begin, rows, used, rep;   // of the group: first request, query rows per KV head, positions
    int nt, stride, per_head;     // tiles and places of a unit, units of a KV head
    // the piece
    int head, tile, t0, n;        // KV head, unit of the head, first tile, tiles

    __device__ Walk(const Args &a_, int pos_, int end_, int g_, int in_) : a(a_), pos(pos_), end(end_), g(g_), in(in_) {}
    // read again for each piece (from L1): not kept in registers meanwhile
    __device__ void group() {
        begin = a.plan.begin[g];
        rows = (a.plan.begin[g + 1] - begin) * a.group;
        used = a.plan.used[g];
        rep = a.plan.rep[g];
        nt = (used + C::TP - 1) / C::TP;
        stride = a.plan.stride[g];
        per_head = (rows + 128 * C::RT - 1) / (128 * C::RT);
    }
    __device__ bool next() {
        if (pos >= end) return false;
        group();
        for (;;) {
            while (in >= stride * per_head * a.kv.heads) {  // the next group with tiles
                do ++g;
                while (g < a.groups && a.plan.off[g + 1] == a.plan.off[g]);
                if (g >= a.groups) return false;
                in = 0;
                group();
            }
            const int unit = in / stride;
            t0 = in - unit * stride;
            if (t0 < nt) {
                head = unit / per_head;
                tile = unit - head * per_head;
                break;
            }
            pos += stride - t0;  // places without tiles
            in += stride - t0;
            if (pos >= end) return false;
        }
        n = min(nt - t0, end - pos);
        pos += n;
        in += n;
        return true;
    }
    __device__ bool whole() const { return n == nt; }
};

__device__ __forceinline__ void cp16_all(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 32 bytes at a 32-byte boundary: a whole sector
__device__ __forceinline__ void st32(float *p, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
// The two softmax warpgroups' barrier; whether all their threads say yes.
__device__ __forceinline__ bool both_agree(bool yes) {
    uint32_t all;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, 256, p;\n"
                 " selp.u32 %0, 1, 0, q;\n}" : "=r"(all) : "r"(static_cast<uint32_t>(yes)) : "memory");
    return all;
}
// byte address of 16-byte piece c of row r in a swizzled tile of boxes of 64 values
__device__ __forceinline__ uint32_t swizzled(int r, int c, int rows) {
    return static_cast<uint32_t>((c >> 3) * rows * 128 + r * 128 + ((c & 7) ^ (r & 7)) * 16);
}

template <int CT, int D, int QP, int RT>
__global__ void __launch_bounds__(Cfg<CT, D, QP, RT>::threads, 1) attn_prefix_kernel(const __grid_constant__ Args a) {
    using namespace tc;
    using C = Cfg<CT, D, QP, RT>;
    constexpr int TP = C::TP, S = C::stages, PP = C::PP;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *tiles = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                             ~static_cast<uintptr_t>(1023));
    unsigned char *q_sm = tiles, *ring = tiles + C::q_bytes;
    unsigned char *raw_ring = ring + S * C::stage;
    Control &ct = *reinterpret_cast<Control *>(raw_ring + 2 * C::raw_stages * C::raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&ct.full[i], C::q8 ? kLoaders : 33 * kLoaders);
            mbar_init(&ct.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ct.s_full[i], 1);
            mbar_init(&ct.p_full[i][0], 4);
            mbar_init(&ct.p_full[i][1], 4);
        }
        mbar_init(&ct.q_full, 8);
        mbar_init(&ct.o_done, 1);
        mbar_init(&ct.stopped, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::mma_warp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&ct.tmem)),
                     "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_launch_dependents();
    pdl_wait();
    const int2 start = a.plan.start[blockIdx.x];
    const int total = a.plan.off[a.groups], run = *a.plan.run;
    const int pos = start.x < 0 ? total : static_cast<int>(blockIdx.x) * run;
    const int end = start.x < 0 ? total : min(pos + run, total);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ct.tmem;
    bool ok = true;

    if (warp >= 8 && warp < C::mma_warp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::load_regs));
        Walk<C> w(a, pos, end, start.x, start.y);
        // ---- K and V tiles: K_0 .. K_(ahead - 1), then V_j, K_(j + ahead), ...
        const int lw = warp & 3;
        constexpr int RW = TP / kLoaders;                // rows of a warp
        constexpr int kPieces = C::q8 ? D / 16 : D / 8;  // 16-byte pieces of a row
        constexpr int kRows = 32 / kPieces, kSteps = RW / kRows;
        const int c = lane % kPieces, rr = lane / kPieces;
        const int page_mask = (1 << a.kv.page_shift) - 1;
        constexpr int kTurn = 8 / kRows > 1 ? 8 / kRows : 1;  // steps after which the swizzle repeats
        uint32_t to_row[kTurn];
#pragma unroll
        for (int k = 0; k < kTurn; ++k) to_row[k] = swizzled(lw * RW + k * kRows + rr, c, TP);
        int item = 0, k_tiles = 0;                       // of the whole run
        while (ok && w.next()) {
            const int32_t *row = a.table + static_cast<int64_t>(w.rep) * a.table_stride;
            // q8_0: this warpgroup's items are the K tiles, or the V tiles
            const bool only_v = C::q8 && warp >= 12;
            const int items = C::q8 ? w.n : 2 * w.n, lead = min(C::ahead, w.n);
            // tile of the i-th item and whether it is V
            auto tile_of = [&](int i, bool &v) {
                if constexpr (C::q8) {
                    v = only_v;
                    return i;
                }
                if (i < lead) { v = false; return i; }
                i -= lead;
                // V_0, K_lead, V_1, K_(lead + 1), ... and the last V's alone
                const int pairs = w.n - lead;
                if (i < 2 * pairs) { v = (i & 1) == 0; return v ? i >> 1 : lead + (i >> 1); }
                v = true;
                return i - pairs;
            };
            auto page_of = [&](int i) {
                bool v;
                const int p = (w.t0 + tile_of(i, v)) * TP + lw * RW + lane;
                return lane < RW && p < w.used ? row[p >> a.kv.page_shift] : -1;
            };
            int page = page_of(0);
            const bool first_piece = item == 0;
            auto wait_empty = [&](int it) {
                // The first queries come before most of the first tiles: behind a ring full of copies a load takes
                // 4 us.  In the first piece alone: the barrier's next phase needs all of that piece's tiles, so it
                // cannot pass while this waits; behind a first piece of one tile it could.
                if (first_piece && it == 2 && !__all_sync(WSW_FULL_MASK, mbar_wait(&ct.q_full, 0))) return false;
                return it < S || __all_sync(WSW_FULL_MASK, mbar_wait(&ct.empty[it % S], ((it / S) - 1) & 1u));
            };
            // a tile's rows to where they lie: lane's row, for all lanes
            struct Rows {
                const unsigned char *base;  // of K or V, the head's
                int64_t at, dat;
                uint32_t valid;
                bool v;
            };
            auto rows_of = [&](int i) {
                Rows x;
                const int p = (w.t0 + tile_of(i, x.v)) * TP + lw * RW + lane;
                const bool in = lane < RW && p < w.used;
                const bool there = in && static_cast<unsigned>(page) < static_cast<unsigned>(a.kv.num_pages);
                if (in && !there && a.err) atomicOr(a.err, 1);
                x.valid = __ballot_sync(WSW_FULL_MASK, there);
                x.at = there ? page * a.kv.page_stride + (p & page_mask) * a.kv.pos_stride : 0;
                x.dat = C::q8 && there ? page * a.kv.d_page_stride + (p & page_mask) * a.kv.d_pos_stride : 0;
                x.base = (x.v ? a.kv.v : a.kv.k) + w.head * a.kv.head_stride;
                if (i + 1 < items) page = page_of(i + 1);
                if (!x.v) {
                    if (lane == 0) {
                        if constexpr (RW == 32) ct.seen[k_tiles % kSeen][lw] = x.valid;
                        else reinterpret_cast<uint16_t *>(ct.seen[k_tiles % kSeen])[lw] = static_cast<uint16_t>(x.valid);
                    }
                    ++k_tiles;
                }
                return x;
            };
            if constexpr (!C::q8) {
                for (int i = 0; i < items; ++i, ++item) {
                    const int st = item % S;
                    if (!wait_empty(item)) {
                        ok = false;
                        break;
                    }
                    const Rows x = rows_of(i);
                    const uint32_t dst = saddr(ring + st * C::stage);
                    if (x.valid == (RW == 32 ? 0xffffffffu : 0xffffu) && a.kv.page_shift >= 4) {
                        // sixteen rows of a page at a time, pos_stride apart: few instructions, since this warp issues
                        // in between the softmax's (shuffles for each row: the MMAs waited 600 cycles a tile)
                        const int64_t pitch = kRows * a.kv.pos_stride;
#pragma unroll
                        for (int g = 0; g < RW / 16; ++g) {
                            const unsigned char *src = x.base + __shfl_sync(WSW_FULL_MASK, x.at, 16 * g) + rr * a.kv.pos_stride + c * 16;
#pragma unroll
                            for (int k = 0; k < 16 / kRows; ++k) {
                                cp16_all(dst + to_row[k % kTurn] + (16 * g + k / kTurn * 8) * 128, src);
                                src += pitch;
                            }
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            const int r = k * kRows + rr;
                            const int64_t o = __shfl_sync(WSW_FULL_MASK, x.at, r);
                            cp16(dst + swizzled(lw * RW + r, c, TP), x.base + o + c * 16, (x.valid >> r) & 1);
                        }
                    }
                    // this thread arrives once its copies have landed (the MMAs' warp has the proxy fence), and the lane
                    // that wrote the visible positions for that store, which is no copy
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(saddr(&ct.full[st])) : "memory");
                    if (lane == 0) mbar_arrive(&ct.full[st]);
                }
            } else {
                // codes and scales of the warp's own rows on their way, raw_stages - 1 tiles ahead
                constexpr int kScale = D / 16;  // bytes of a row's scales
                // this kind's place in the ring: K_0 .. K_(lead - 1), V_0, K_lead, V_1, ..., the last V's alone
                auto place = [&](int i) {
                    return item + (only_v ? (i < w.n - lead ? lead + 2 * i : w.n + i) : i < lead ? i : 2 * i - lead + 1);
                };
                auto raw_of = [&](int i) { return raw_ring + (only_v * C::raw_stages + i % C::raw_stages) * C::raw; };
                auto issue = [&](int i) {
                    if (i < items) {
                        const Rows x = rows_of(i);
                        unsigned char *to = raw_of(i);
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            const int r = k * kRows + rr;
                            const int64_t o = __shfl_sync(WSW_FULL_MASK, x.at, r);
                            cp16(saddr(to) + (lw * RW + r) * D + c * 16, x.base + o + c * 16, (x.valid >> r) & 1);
                        }
                        if (lane < RW)
                            paged::cp_small<kScale>(saddr(to) + TP * D + (lw * RW + lane) * kScale,
                                                    (x.v ? a.kv.vd : a.kv.kd) + w.head * a.kv.d_head_stride + x.dat,
                                                    (x.valid >> lane) & 1);
                    }
                    paged::cp_commit();  // a group for each turn, empty past the end
                };
                __syncwarp();  // every lane has read the last piece's rows
#pragma unroll
                for (int i = 0; i < C::raw_stages - 1; ++i) issue(i);
                for (int i = 0; i < items; ++i) {
                    __syncwarp();  // every lane has read the place that the next copies reuse
                    issue(i + C::raw_stages - 1);
                    paged::cp_wait<C::raw_stages - 1>();
                    __syncwarp();  // the rows that every lane copied
                    const int at = place(i), st = at % S;
                    if (!wait_empty(at)) {
                        ok = false;
                        break;
                    }
                    const unsigned char *from = raw_of(i);
                    unsigned char *to = ring + st * C::stage;
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        const int r = lw * RW + k * kRows + rr;
                        const uint4 code = *reinterpret_cast<const uint4 *>(from + r * D + c * 16);
                        const __half2 d2 = __half2half2(*reinterpret_cast<const __half *>(from + TP * D + r * kScale + (c >> 1) * 2));
                        const uint32_t u[4] = {code.x ^ 0x80808080u, code.y ^ 0x80808080u, code.z ^ 0x80808080u, code.w ^ 0x80808080u};
                        uint32_t h[8];  // rows that are not there are zeros: codes and scales
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            h[2 * x] = paged::dequant2(u[x], 0x4140, d2);
                            h[2 * x + 1] = paged::dequant2(u[x], 0x4342, d2);
                        }
                        *reinterpret_cast<uint4 *>(to + swizzled(r, 2 * c, TP)) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4 *>(to + swizzled(r, 2 * c + 1, TP)) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ct.full[st]);
                }
                item += 2 * w.n;
            }
        }
        cp_wait_all();
        __syncwarp();
    } else if (warp >= C::mma_warp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::mma_regs));
        if (warp == C::mma_warp) {
            // The whole warp walks, so that addresses and descriptors are uniform values; one elected lane issues.
            // (With one lane walking alone an MMA was issued every 115 cycles.)
            Walk<C> w(a, pos, end, start.x, start.y);
            constexpr uint32_t id_s = instr_desc(128, TP, C::bf16);
            constexpr uint32_t id_pv = instr_desc(128, D, C::bf16) | (1u << 16);  // B (V) MN-major
            int item = 0, piece = 0;
            uint32_t p_phase[2] = {0, 0};
            auto wait = [&](uint64_t *b, uint32_t parity) { return __all_sync(WSW_FULL_MASK, mbar_wait(b, parity)) != 0; };
            auto landed = [&](int i) {
                const bool yes = wait(&ct.full[i % S], (i / S) & 1u);
                fence_async_shared();  // what the copies wrote, for the tensor cores
                return yes;
            };
            auto commit = [&](uint64_t *b) {
                if (elect_one()) mma_commit(b);
            };
            auto scores = [&](int slot, int k) {
                const uint32_t kt = saddr(ring + (k % S) * C::stage), qt = saddr(q_sm + (RT == 2 ? slot : 0) * QP * C::q_part);
                const uint64_t dq = sw128_desc(qt), dk = sw128_desc(kt);
                const uint32_t d = tmem + slot * C::s_cols;
                tc_fence_after();
                // q's last part first: an MMA's sum is cut to fp32's bits, which costs nothing while the sum is small
                if (elect_one()) {
#pragma unroll
                    for (int part = QP - 1; part >= 0; --part)
#pragma unroll
                        for (int b = 0; b < D / 64; ++b)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_bf16(d, dq + ((part * C::q_part + b * 128 * 128) >> 4) + 2 * kk,
                                         dk + ((b * TP * 128) >> 4) + 2 * kk, id_s, part < QP - 1 || (b | kk) != 0);
                }
                __syncwarp();
            };
            // half of a tile's positions: the first half's products run while the other half's weights are made
            auto values = [&](int slot, int v, int half, bool more) {
                const uint64_t dv = sw128_mn_desc(saddr(ring + (v % S) * C::stage), TP * 128) + half * (TP / 32) * 128;
                const uint32_t d = tmem + C::o_col + slot * D, p = tmem + slot * C::s_cols;
                if (elect_one()) {
#pragma unroll
                    for (int part = 0; part < PP; ++part)
#pragma unroll
                        for (int kk = 0; kk < TP / 32; ++kk)
                            mma_ts(d, p + C::p_col(part, half * (TP / 32) + kk), dv + 128 * kk, id_pv, more || (part | kk) != 0);
                }
                __syncwarp();
            };
            while (ok && w.next()) {
                ok = wait(&ct.q_full, piece & 1u);
                ++piece;
                if (!ok) break;
                const int lead = min(C::ahead, w.n);
                for (int j = 0; j < lead; ++j) {
                    if (!(ok = landed(item))) break;
                    for (int s = 0; s < RT; ++s) {
                        const int slot = RT == 2 ? s : j;
                        scores(slot, item);
                        commit(&ct.s_full[slot]);
                    }
                    commit(&ct.empty[item % S]);
                    ++item;
                }
                for (int j = 0; j < w.n && ok; ++j) {
                    const bool more_k = j + lead < w.n;
                    const int v = item++, k = more_k ? item++ : 0;
                    for (int s = 0; s < RT; ++s) {
                        const int slot = RT == 2 ? s : j & 1;
                        if (!(ok = wait(&ct.p_full[slot][0], p_phase[slot]))) break;
                        if (s == 0 && !(ok = landed(v))) break;
                        tc_fence_after();
                        values(slot, v, 0, RT == 2 ? j > 0 : j > 1);
                        if (!(ok = wait(&ct.p_full[slot][1], p_phase[slot]))) break;
                        p_phase[slot] ^= 1u;
                        tc_fence_after();
                        values(slot, v, 1, true);
                        if (s == RT - 1) commit(&ct.empty[v % S]);
                        if (!more_k) continue;
                        if (s == 0 && !(ok = landed(k))) break;
                        scores(slot, k);
                        commit(&ct.s_full[slot]);
                        if (s == RT - 1) commit(&ct.empty[k % S]);
                    }
                }
                if (ok) commit(&ct.o_done);
            }
            if (!ok) {  // what was issued reads shared memory and writes tensor memory
                commit(&ct.stopped);
                wait(&ct.stopped, 0);
            }
        }
    } else {
        // ---- softmax: slot and row of this thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::soft_regs));
        Walk<C> w(a, pos, end, start.x, start.y);
        const int slot = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t s_base = lane_base + slot * C::s_cols, o_base = lane_base + C::o_col + slot * D;
        uint32_t s_phase = 0;
        int piece = 0, k_tiles = 0;
        while (ok && w.next()) {
            const int in_group = (w.tile * RT + (RT == 2 ? slot : 0)) * 128 + r;
            const bool real = in_group < w.rows;
            const int req = w.begin + (real ? in_group : 0) / a.group, gq = (real ? in_group : 0) % a.group;
            const int64_t head = static_cast<int64_t>(req) * a.q_heads + w.head * a.group + gq;
            // ---- q.  A warp has 32 rows of its slot, or 16 of those that both slots share: sixteen (D 64: eight) lanes
            // load a row, eight values each.  (A thread for each row took 4 us with 16-bit rows and 10 with fp32.)
            float unit = a.cap_in != 0.f ? a.cap_in * (2.f * kLog2e) : a.scale2;  // of a score's product sum; capped()'s if capped
            {
                constexpr int kLanes = D / 8, kPer = 32 / kLanes, kRowsOfWarp = RT == 2 ? 32 : 16;
                const int ch = lane % kLanes, r0 = (warp & 3) * 32 + (RT == 2 ? 0 : slot * 16) + lane / kLanes;
                const int first_in_group = (w.tile * RT + (RT == 2 ? slot : 0)) * 128;
                unsigned char *to = q_sm + (RT == 2 ? slot : 0) * QP * C::q_part;
                constexpr int kTurns = kRowsOfWarp / kPer, kAtOnce = 4;
                // the lane's rows in turn, as request and head of the group
                int in = first_in_group + r0, rq = in / a.group, rg = in - rq * a.group;
                auto source = [&](int esize) {
                    return static_cast<const unsigned char *>(a.q) +
                           ((static_cast<int64_t>(w.begin + rq) * a.q_heads + w.head * a.group + rg) * D + 8 * ch) * esize;
                };
                auto step_row = [&] {
                    in += kPer;
                    rg += kPer;
                    while (rg >= a.group) {
                        rg -= a.group;
                        ++rq;
                    }
                };
                // 16-bit rows of the cache's own type as they are
                const bool as_is = QP == 1 && a.dtype == (C::bf16 ? WSW_BF16 : WSW_F16) && !a.negative;
                if (as_is) {
#pragma unroll 1
                    for (int t = 0; t < kTurns; ++t) {
                        const bool there = in < w.rows;
                        cp16(saddr(to) + swizzled(r0 + t * kPer, ch, 128), there ? source(2) : static_cast<const unsigned char *>(a.q),
                             there);
                        step_row();
                    }
                    cp_wait_all();
                }
#pragma unroll 1
                for (int t = 0; t < kTurns && !as_is; t += kAtOnce) {
                    uint4 raw[kAtOnce][C::wide ? 2 : 1];  // fp32 rows are twice as wide
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        const uint4 *src = reinterpret_cast<const uint4 *>(source(C::wide ? 4 : 2));
#pragma unroll
                        for (int k = 0; k < (C::wide ? 2 : 1); ++k)
                            raw[u][k] = in < w.rows ? src[k] : make_uint4(0u, 0u, 0u, 0u);
                        step_row();
                    }
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u) {
                        const int row = r0 + (t + u) * kPer;
                        float x[8];
#pragma unroll
                        for (int k = 0; k < (C::wide ? 2 : 1); ++k) {
                            const uint32_t y[4] = {raw[u][k].x, raw[u][k].y, raw[u][k].z, raw[u][k].w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if constexpr (C::wide) {
                                    x[4 * k + i] = __uint_as_float(y[i]);
                                } else {
                                    const float2 f = a.dtype == WSW_BF16 ? make_float2(bf16lo(y[i]), bf16hi(y[i]))
                                                                         : __half22float2(*reinterpret_cast<const __half2 *>(&y[i]));
                                    x[2 * i] = f.x;
                                    x[2 * i + 1] = f.y;
                                }
                            }
                        }
                        float up = a.negative ? -1.f : 1.f;
                        if constexpr (!C::bf16) {
                            if (a.dtype != WSW_F16) {
                                float top = 0.f;
#pragma unroll
                                for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
                                for (int d = kLanes / 2; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(WSW_FULL_MASK, top, d));
                                const int e = max(static_cast<int>(__float_as_uint(top) >> 23), 15);
                                up *= __uint_as_float((268u - e) << 23);
                                if (ch == 0) ct.unit[(RT == 2 ? slot * 128 : 0) + row] = __uint_as_float((e - 14u) << 23);
                            }
                        }
                        uint32_t part[3][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float x0 = x[2 * i] * up, x1 = x[2 * i + 1] * up;
                            if constexpr (QP == 1) part[0][i] = pack2<C::bf16>(x0, x1);
                            else if constexpr (QP == 2) split<CT>(x0, x1, part[0][i], part[1][i]);
                            else split3(x0, x1, part[0][i], part[1][i], part[2][i]);
                        }
#pragma unroll
                        for (int k = 0; k < QP; ++k)
                            *reinterpret_cast<uint4 *>(to + k * C::q_part + swizzled(row, ch, 128)) =
                                make_uint4(part[k][0], part[k][1], part[k][2], part[k][3]);
                    }
                }
                fence_async_shared();
                tc_fence_before();  // O of the piece before has been read
                __syncwarp();
                if (lane == 0) mbar_arrive(&ct.q_full);
                if constexpr (!C::bf16) {
                    if (a.dtype != WSW_F16) {
                        if (RT == 1) asm volatile("bar.sync 1, 256;" ::: "memory");
                        unit *= ct.unit[(RT == 2 ? slot * 128 : 0) + r];
                    }
                }
            }
            const float slope = a.slopes && real ? a.slopes[w.head * a.group + gq] * kLog2e : 0.f;
            const int last = real && a.slopes ? min(max(a.lens[req], 0), a.max_len) - 1 : 0;
            float m = -INFINITY, l = 0.f;
            const int step = RT == 2 ? 1 : 2;
            for (int j = RT == 2 ? 0 : slot; j < w.n; j += step) {
                if (!__all_sync(WSW_FULL_MASK, mbar_wait(&ct.s_full[slot], s_phase))) {
                    ok = false;
                    break;
                }
                s_phase ^= 1u;
                tc_fence_after();
                const uint32_t *seen = ct.seen[(k_tiles + j) % kSeen];
                const bool all = TP == 128 ? (seen[0] & seen[1] & seen[2] & seen[3]) == 0xffffffffu
                                           : (seen[0] & seen[1]) == 0xffffffffu;
                const bool plain = all && a.cap_in == 0.f && !a.slopes;
                uint64_t l2a = 0ull, l2b = 0ull;  // a tile's sum by itself: l gets one rounding a tile
                auto top = [](const uint32_t (&v)[32], float mx) {
                    float q4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        asm("max.f32 %0, %0, %1, %2;" : "+f"(q4[(i >> 1) & 3]) : "f"(__uint_as_float(v[i])), "f"(__uint_as_float(v[i + 1])));
                    return fmaxf(fmaxf(q4[0], q4[1]), fmaxf(q4[2], q4[3]));
                };
                // the maximum in use, with the tile's mt in mind
                auto raise_to = [&](float mt) {
                    const bool raise = mt > m + kLazy;  // m = -inf: by anything visible
                    if (j >= step && __any_sync(WSW_FULL_MASK, raise)) {
                        // the S that was waited for was issued behind the last P V: O is complete
                        const float al = raise ? ex2(m - mt) : 1.f;
                        l *= al;
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            float o[16];
                            tmem_ld16(o_base + 16 * c, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= al;
                            tmem_st16(o_base + 16 * c, reinterpret_cast<const uint32_t (&)[16]>(o));
                        }
                    }
                    if (raise) m = mt;
                };
                // weights 2^(x mul - ref) of a chunk of 32 scores, into tensor memory
                auto put = [&](const uint32_t (&v)[32], int chunk, float mul, float ref) {
                    const uint64_t mul2 = f2_pack(mul, mul), ref2 = f2_pack(-ref, -ref);
                    uint32_t part[PP][16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        uint64_t t = f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                        asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(t) : "l"(mul2), "l"(ref2));
                        float t0, t1;
                        f2_unpack(t, t0, t1);
                        const float w0 = ex2(t0), w1 = ex2(t1);
                        if (i & 1) asm("add.rn.f32x2 %0, %0, %1;" : "+l"(l2b) : "l"(f2_pack(w0, w1)));
                        else asm("add.rn.f32x2 %0, %0, %1;" : "+l"(l2a) : "l"(f2_pack(w0, w1)));
                        if constexpr (PP == 2) split<CT>(w0, w1, part[0][i], part[1][i]);
                        else split3(w0, w1, part[0][i], part[1][i], part[2][i]);
                    }
#pragma unroll
                    for (int k = 0; k < PP; ++k) tmem_st16(s_base + C::p_col(k, 2 * chunk), part[k]);
                };
                auto ready = [&](int half) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ct.p_full[slot][half]);
                };
                auto ref_of = [&] { return m == -INFINITY ? 0.f : m - C::shift; };  // nothing seen yet: all weights 0
                if (plain) {
                    // Two chunks of scores stay in registers, the others are read twice, a chunk at a time (weights take no
                    // other chunk's place, or both chunks' of 64 positions).  With P in one part, 256 requests behind 32768
                    // positions: 157 us; three chunks 162, four 163, the second half on its way while the first half's
                    // weights are made 163.
                    uint32_t v[2][32];
                    float mx = -INFINITY;
#pragma unroll
                    for (int c = 2; c < TP / 32; ++c) {
                        tmem_ld32(s_base + 32 * c, v[0]);
                        tmem_wait_ld();
                        mx = top(v[0], mx);
                    }
                    tmem_ld32(s_base, v[0]);
                    tmem_ld32(s_base + 32, v[1]);
                    tmem_wait_ld();
                    raise_to(top(v[1], top(v[0], mx)) * unit);
                    const float ref = ref_of();
                    put(v[0], 0, unit, ref);
                    if constexpr (TP == 64) ready(0);
                    put(v[1], 1, unit, ref);
                    if constexpr (TP == 128) ready(0);
#pragma unroll
                    for (int c = 2; c < TP / 32; ++c) {
                        tmem_ld32(s_base + 32 * c, v[0]);
                        tmem_wait_ld();
                        put(v[0], c, unit, ref);
                    }
                } else {
                    const int p0 = (w.t0 + j) * TP;
                    // 32 scores of a chunk in log2 units
                    auto read = [&](uint32_t (&v)[32], int chunk) {
                        tmem_ld32(s_base + 32 * chunk, v);
                        tmem_wait_ld();
                        const uint32_t mask = seen[chunk];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * unit);
                        if (a.cap_in != 0.f) {
                            float far = 0.f;
#pragma unroll
                            for (int i = 0; i < 32; ++i) far = fmaxf(far, fabsf(__uint_as_float(v[i])));
                            if (!__any_sync(WSW_FULL_MASK, far >= kNear)) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(capped_near(__uint_as_float(v[i]), a.cap_out));
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(capped(__uint_as_float(v[i]), a.cap_out));
                            }
                        }
                        if (a.slopes) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = __float_as_uint(fmaf(-slope, static_cast<float>(last - (p0 + 32 * chunk + i)),
                                                            __uint_as_float(v[i])));
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = (mask >> i) & 1 ? v[i] : 0xff800000u;
                    };
                    // the second half's maximum comes first (its scores go back for the weights); weights take their own
                    // scores' places or, in three parts, those of two chunks that have been read
                    float mx = -INFINITY;
                    uint32_t va[32], vb[32];
                    if constexpr (TP == 128) {
#pragma unroll 1
                        for (int c = 2; c < 4; ++c) {
                            read(va, c);
                            mx = top(va, mx);
                            tmem_st32(s_base + 32 * c, va);
                        }
                    }
                    read(va, 0);
                    read(vb, 1);
                    mx = top(vb, top(va, mx));
                    raise_to(mx);
                    const float ref = ref_of();
                    put(va, 0, 1.f, ref);
                    if constexpr (TP == 64) ready(0);
                    put(vb, 1, 1.f, ref);
                    if constexpr (TP == 128) {
                        ready(0);
#pragma unroll 1
                        for (int c = 2; c < 4; ++c) {
                            tmem_ld32(s_base + 32 * c, va);  // as they were left (ready's wait has seen to that)
                            tmem_wait_ld();
                            put(va, c, 1.f, ref);
                        }
                    }
                }
                ready(1);
                float l0, l1, l2, l3;
                f2_unpack(l2a, l0, l1);
                f2_unpack(l2b, l2, l3);
                l += (l0 + l1) + (l2 + l3);
            }
            k_tiles += w.n;
            // ---- the piece's (m, l, O)
            ok = ok && mbar_wait(&ct.o_done, piece & 1u);
            ++piece;
            float2 *ml = reinterpret_cast<float2 *>(q_sm);  // [2][128] of both slots' rows: q has been read
            if (RT == 1) ml[slot * 128 + r] = make_float2(m, l);
            const bool have = both_agree(ok);
            ok = have;
            tc_fence_after();
            float *rec = w.whole() ? a.whole + head * C::rec
                                   : a.rec + ((static_cast<int64_t>(blockIdx.x) * 2 + (w.t0 == 0)) * RT +
                                              (RT == 2 ? slot : 0)) * 128 * C::rec + r * C::rec;
            // both slots' sums of the same rows: a warp reaches its quarter's rows of either, so each warpgroup
            // joins half of the columns
            float f0 = 1.f, f1 = 0.f;
            if (RT == 1 && have) {
                const float2 x = ml[r], y = ml[128 + r];
                m = fmaxf(x.x, y.x);
                f0 = x.x == -INFINITY ? 0.f : ex2(x.x - m);
                f1 = y.x == -INFINITY ? 0.f : ex2(y.x - m);
                l = x.y * f0 + y.y * f1;
            }
            if (real && (RT == 2 || slot == 0)) *reinterpret_cast<float2 *>(rec) = make_float2(m == -INFINITY ? m : m - C::shift, l);
            // (a rolled loop of few instructions: code that runs once a piece is mostly waited for)
            constexpr int kCols = RT == 2 ? D : D / 2;
            const int col0 = RT == 2 ? 0 : slot * kCols;
            const uint32_t from = RT == 2 ? o_base : lane_base + C::o_col + col0;
#pragma unroll 1
            for (int c = 0; c < kCols; c += 8) {
                uint32_t o[8], y[8];
                tmem_ld8(from + c, o);
                if (RT == 1) tmem_ld8(from + D + c, y);
                tmem_wait_ld();
                if (RT == 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // a part without weights holds nothing (0 times what its rows hold may be NaN)
                        const float x = f0 == 0.f ? 0.f : __uint_as_float(o[i]) * f0;
                        o[i] = __float_as_uint(f1 == 0.f ? x : fmaf(__uint_as_float(y[i]), f1, x));
                    }
                }
                if (real) st32(rec + kHead + col0 + c, o);
            }
            // both have read the sums and O before the next piece's
            if (RT == 1) asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        if (!ok && tid == 0) *a.plan.run = 0;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::mma_warp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int CT, int D, int QP, int RT>
cudaError_t launch_one(const Args &a, cudaStream_t s, int ctas) {
    using C = Cfg<CT, D, QP, RT>;
    const auto kernel = attn_prefix_kernel<CT, D, QP, RT>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kernel), C::smem);
    if (e != cudaSuccess) return e;
    // the roles' registers are shared out of what the block is launched with: with less, a role would wait for them
    static const int regs = [kernel] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, reinterpret_cast<const void *>(kernel)) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs < C::regs) return cudaErrorLaunchOutOfResources;
    return launch(kernel, dim3(static_cast<unsigned>(ctas)), dim3(C::threads), C::smem, s, true, a);
}

// Row tiles of a unit: two (the warpgroups share K and V) where a group has more than 128 rows on average
// and q is one part.
template <int CT>
cudaError_t launch_prefix(const Args &a, int row_tiles, cudaStream_t s, int ctas);

#define WSW_PREFIX_ONE(CT, QP, RT)                                                   \
    (a.kv.head_dim == 64 ? launch_one<CT, 64, QP, RT>(a, s, ctas) : launch_one<CT, 128, QP, RT>(a, s, ctas))

}  // namespace prefix
}  // namespace wsw
