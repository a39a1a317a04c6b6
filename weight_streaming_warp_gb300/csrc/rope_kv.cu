// rope_kv.cu -- rotary positions of q and k fused with the write of k and v into the paged
// KV cache (the host table of frequencies: rope_table.cu).
//
// Pair (x0, x1) of a head at position p turns by the angle a = p f:
//   (x0, x1) -> m (x0 cos a - x1 sin a, x1 cos a + x0 sin a)
// ("RoFormer: Enhanced Transformer with Rotary Position Embedding", section 3.4.2), f from
// the table, m its attention factor.
//
// Angles: p f in fp32 is off by p f 2^-24 radians, 0.06 at p = 10^6 and f = 1.  The table
// holds f in fractions of a turn as 64-bit fixed point, so p * turns modulo 2^64 drops the
// whole turns exactly.  Its top 24 bits are an fp32 value for sincospi; the next 32, an angle d below
// 4e-7, turn the result once more by first order (cos d = 1 - 7e-14): all 32 bits in one
// rounded fp32 value were off by 9e-8 radians.  One 64-bit
// integer product replaces an FP64 one, which this part runs at a sixtieth of fp32's rate.
// Each (token, pair) is computed once per CTA and shared by all heads through shared memory.
//
// Work: a thread owns 8 consecutive dimensions of one row (a row: one head of one token);
// for the half layout it loads its 8 partners too, which its own warp's neighbours have
// just brought into L1.  Bytes decide: q, k and v once in, q out, k and v out.  Prompts whose
// rows are aligned take a persistent form that streams tokens through shared memory
// (rope_stream_kernel): 8191 bf16 tokens of 40 query and 4 KV heads of 128 in 40 us (4.9 TB/s, bound by
// instructions), 64 tokens of a decode step in 2.8 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "kv_cache.cuh"
#include "q8_math.cuh"

namespace wsw {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 8;  // tokens per CTA

struct RopeArgs {
    const void *q, *k, *v;
    int64_t qts, qhs, kts, khs, vts, vhs;  // token and head strides, elements
    const uint64_t *turns;
    const int32_t *positions;
    const int64_t *slots;
    void *q_out;
    int32_t *err;
    KvView kv;
    int64_t tokens;
    float mscale;
    int q_heads, rot, interleaved, tile;
    int lane_shift;  // log2(head_dim / 8): threads per row
    bool vec;        // q, k, v rows 16-byte aligned
    bool vec_out;    // q_out 16-byte aligned
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2(x[0], x[1], T()), pack2(x[2], x[3], T()), pack2(x[4], x[5], T()), pack2(x[6], x[7], T()));
}

// the two values of a word
__device__ __forceinline__ float2 two(uint32_t u, __half) { return __half22float2(*reinterpret_cast<const __half2 *>(&u)); }
__device__ __forceinline__ float2 two(uint32_t u, __nv_bfloat16) { return make_float2(bf16lo(u), bf16hi(u)); }

// 8 consecutive values; plain loads, as the call may write q in place
template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec, float (&x)[8]) {
    if (!vec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f(p[i]);
    } else if constexpr (sizeof(T) == 4) {
        const float4 u = reinterpret_cast<const float4 *>(p)[0], v = reinterpret_cast<const float4 *>(p)[1];
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = two(w[i], T());
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// 4 consecutive values of an aligned row
template <typename T>
__device__ __forceinline__ void load4(const T *p, float (&x)[4]) {
    alignas(16) T t[4];
    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(t) = *reinterpret_cast<const uint4 *>(p);
    else *reinterpret_cast<uint2 *>(t) = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = to_f(t[i]);
}

__device__ __forceinline__ void store8(float *p, bool vec, const float (&x)[8]) {
    if (vec) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = x[i];
    }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, bool vec, const float (&x)[8]) {
    const uint4 u = pack8<T>(x);
    if (vec) {
        *reinterpret_cast<uint4 *>(p) = u;
    } else {
        const T *t = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = t[i];
    }
}

// (cos, sin) of a position's angle, `turns` of a pair's 2^-64 turns each
__device__ __forceinline__ float2 cos_sin(int32_t position, uint64_t turns) {
    const uint64_t turn = static_cast<uint64_t>(position < 0 ? 0 : position) * turns;
    const int32_t top = static_cast<int32_t>(turn >> 32) & ~0xff;  // a signed fraction: half turns in [-1, 1)
    const float d = static_cast<float>(static_cast<uint32_t>(turn >> 8)) * 8.7196712e-17f;  // pi 2^-55
    float s, c;
    sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    return make_float2(fmaf(-s, d, c), fmaf(c, d, s));
}

// Where pair p's (cos, sin) sits among a token's: neighbouring lanes read neighbouring places at
// every step of their loops (a plain order is an eight-way bank conflict).
__device__ __forceinline__ int place(int p, int half, int group) {
    return group == 8 ? (p & 7) * (half >> 3) + (p >> 3) : group == 4 ? (p & 3) * ((half + 3) >> 2) + (p >> 2) : p;
}

// One CTA for a few tokens.  It is bound by the loads in flight, so threads count for more
// than registers: 8191 tokens of 48 heads, fp32 into binary16, 66 us with 6 CTAs on an SM and 69
// with 8; bf16 with pairs 20 apart, 56 and 52 us.
template <typename T, int CT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 6 : 8) rope_kv_kernel(const RopeArgs a) {
    __shared__ float2 cs[kMaxTile][128 + 4];  // (m cos, m sin) of each token and pair
    __shared__ int32_t pos_sm[kMaxTile];
    __shared__ int64_t slot_sm[kMaxTile];
    const int tid = threadIdx.x;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile;
    const int tile = static_cast<int>(a.tokens - t0 < a.tile ? a.tokens - t0 : a.tile);
    const int half = a.rot >> 1;
    const int group = a.interleaved ? 4 : (half & 7) == 0 ? 8 : 1;
    pdl_launch_dependents();
    pdl_wait();
    for (int i = tid; i < tile * half; i += kThreads) {
        const int tt = i / half, pair = i - tt * half;
        const float2 z = cos_sin(a.positions[t0 + tt], a.turns[pair]);
        cs[tt][place(pair, half, group)] = make_float2(a.mscale * z.x, a.mscale * z.y);
    }
    if (tid < tile) {
        pos_sm[tid] = a.positions[t0 + tid];
        slot_sm[tid] = a.slots[t0 + tid];
    }
    __syncthreads();

    const int lanes = 1 << a.lane_shift, D = lanes * 8;
    const int rows = a.q_heads + 2 * a.kv.heads;
    const int d0 = (tid & (lanes - 1)) * 8;
    const int step = static_cast<int>(gridDim.y * kThreads) >> a.lane_shift;  // rows per round of the grid's y
    const int step_t = step / rows, step_h = step - step_t * rows;
    int row = static_cast<int>(blockIdx.y * kThreads + tid) >> a.lane_shift;
    int tt = row / rows, h = row - tt * rows;
    const int total = tile * rows;
    const int warp_row = row - ((tid & 31) >> a.lane_shift);  // the warp's first row: a uniform loop
    for (int base = warp_row; base < total; base += step) {
        const bool active = tt < tile;  // a row's lanes are all active or all idle
        const int64_t t = t0 + (active ? tt : 0);
        const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv.heads;
        const int kh = is_v ? h - a.q_heads - a.kv.heads : h - a.q_heads;
        const T *src;
        if (is_q) src = static_cast<const T *>(a.q) + t * a.qts + h * a.qhs;
        else if (is_v) src = static_cast<const T *>(a.v) + t * a.vts + kh * a.vhs;
        else src = static_cast<const T *>(a.k) + t * a.kts + kh * a.khs;
        const int32_t pos = active ? pos_sm[tt] : -1;
        float x[8];
        if (pos >= 0) {
            load8(src + d0, a.vec, x);
            if (!is_v && d0 < a.rot) {
                const float2 *w = cs[tt];
                if (group == 8) {
                    const bool lo = d0 < half;
                    float y[8];
                    load8(src + (lo ? d0 + half : d0 - half), a.vec, y);
                    w += (lo ? d0 : d0 - half) >> 3;
                    const int stride = half >> 3;
                    const float sign = lo ? -1.f : 1.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 z = w[i * stride];
                        x[i] = fmaf(x[i], z.x, y[i] * (sign * z.y));
                    }
                } else if (group == 4) {
                    w += d0 >> 3;
                    const int stride = (half + 3) >> 2;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (d0 + 2 * i >= a.rot) break;
                        const float2 z = w[i * stride];
                        const float x0 = x[2 * i], x1 = x[2 * i + 1];
                        x[2 * i] = fmaf(x0, z.x, -x1 * z.y);
                        x[2 * i + 1] = fmaf(x1, z.x, x0 * z.y);
                    }
                } else if ((half & 3) == 0 && a.vec) {  // partners four by four
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int d = d0 + 4 * c;
                        if (d >= a.rot) break;
                        const bool lo = d < half;
                        float y[4];
                        load4(src + (lo ? d + half : d - half), y);
                        const float2 *z = w + (lo ? d : d - half);
                        const float sign = lo ? -1.f : 1.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[4 * c + i] = fmaf(x[4 * c + i], z[i].x, y[i] * (sign * z[i].y));
                    }
                } else {  // the halves do not meet at a multiple of 4: partners one by one
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const int d = d0 + i;
                        if (d >= a.rot) break;
                        const bool lo = d < half;
                        const float y = to_f(src[lo ? d + half : d - half]), own = to_f(src[d]);
                        const float2 z = w[lo ? d : d - half];
                        const float turned = fmaf(own, z.x, y * (lo ? -z.y : z.y));
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = j == i ? turned : x[j];
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.f;  // padding
        }
        __syncwarp();  // a row in place: its partners are read before it is written
        int64_t where = -1, dwhere = 0;
        if (!is_q && pos >= 0) {
            const int64_t slot = slot_sm[tt];
            const int64_t page = slot >> a.kv.page_shift;
            if (slot >= 0 && page < a.kv.num_pages) {
                const int64_t off = slot & ((int64_t(1) << a.kv.page_shift) - 1);
                where = page * a.kv.page_stride + off * a.kv.pos_stride + kh * a.kv.head_stride;
                dwhere = page * a.kv.d_page_stride + off * a.kv.d_pos_stride + kh * a.kv.d_head_stride;
            } else if (slot >= 0 && a.err) {
                atomicOr(a.err, 1);
            }
        }
        if constexpr (CT == WSW_Q8_0) {
            const float amax = q8m::block_amax<32>(x);  // every lane of the warp
            if (where >= 0) {
                const float d = q8m::scale(amax);
                uint32_t codes[2];
                q8m::codes(x, amax, d, codes);
                *reinterpret_cast<uint2 *>((is_v ? a.kv.v : a.kv.k) + where + d0) = make_uint2(codes[0], codes[1]);
                if ((d0 & 31) == 0)
                    reinterpret_cast<__half *>((is_v ? a.kv.vd : a.kv.kd) + dwhere)[d0 >> 5] = __float2half_rn(d);
            }
        } else if (where >= 0) {
            unsigned char *dst = (is_v ? a.kv.v : a.kv.k) + where + d0 * 2;
            if constexpr (CT == WSW_F16) *reinterpret_cast<uint4 *>(dst) = pack8<__half>(x);
            else *reinterpret_cast<uint4 *>(dst) = pack8<__nv_bfloat16>(x);
        }
        if (active && is_q) store8(static_cast<T *>(a.q_out) + (t * a.q_heads + h) * D + d0, a.vec_out, x);
        tt += step_t;
        h += step_h;
        if (h >= rows) {
            h -= rows;
            ++tt;
        }
    }
}

// Many tokens whose rows are 16-byte aligned: a persistent form.  Each thread keeps the sines
// and cosines of its dimensions in registers for a token's rows, and its rows come through a
// ring of cp.async stages in shared memory, so that loads in flight cost no registers; a
// partner's values are the neighbour's slot.  The next token's angles are computed beside
// this one's rows.
constexpr int kRing = 4;
constexpr int kStreamCtas = 3;  // on an SM: 8191 bf16 tokens of 48 heads 40 us, with 4 and 5 CTAs 45 and 59 us

template <typename T, int CT>
__global__ void __launch_bounds__(kThreads, kStreamCtas) rope_stream_kernel(const RopeArgs a) {
    constexpr int kV = sizeof(T) / 2;  // 16-byte vectors of 8 values
    __shared__ uint4 ring[kRing][kThreads * kV];
    __shared__ float2 cs[2][128 + 4];
    struct Token {
        int64_t where, dwhere;  // its cached row of head 0 (bytes), -1: not cached
        int32_t pos;
    };
    __shared__ Token tok[2];
    const int tid = threadIdx.x;
    const int half = a.rot >> 1;
    const int group = a.interleaved ? 4 : 8;
    const int lanes = 1 << a.lane_shift, D = lanes * 8;
    const int rows = a.q_heads + 2 * a.kv.heads;
    const int d0 = (tid & (lanes - 1)) * 8;
    const int rp = kThreads >> a.lane_shift, rs = tid >> a.lane_shift;  // rows a round, this thread's
    const int stride = gridDim.x;
    const int count = static_cast<int>((a.tokens - blockIdx.x + stride - 1) / stride);  // this CTA's tokens
    const bool turns = d0 < a.rot, lo = d0 < half;
    const int partner = group == 8 && turns ? (lo ? half >> 3 : -(half >> 3)) : 0;  // in lanes
    auto token = [&](int i) { return blockIdx.x + static_cast<int64_t>(i) * stride; };
    pdl_launch_dependents();
    pdl_wait();

    // the next row to copy: tokens left, its row, its slot, and that token's rows
    int p_left = count, ph = rs;
    const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(&ring[0][tid * kV]));
    constexpr uint32_t kSlot = kThreads * kV * 16;
    uint32_t p_slot = ring_s;
    const T *pq = static_cast<const T *>(a.q) + blockIdx.x * a.qts + d0;
    const T *pk = static_cast<const T *>(a.k) + blockIdx.x * a.kts + d0;
    const T *pv = static_cast<const T *>(a.v) + blockIdx.x * a.vts + d0;
    auto issue = [&]() {
        if (p_left > 0) {
            if (ph < rows) {
                const int kh = ph - a.q_heads, vh = kh - a.kv.heads;
                const T *src = kh < 0 ? pq + ph * a.qhs : vh < 0 ? pk + kh * a.khs : pv + vh * a.vhs;
#pragma unroll
                for (int i = 0; i < kV; ++i)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(p_slot + 16 * i),
                                 "l"(reinterpret_cast<const uint4 *>(src) + i) : "memory");
            }
            p_slot = p_slot == ring_s + (kRing - 1) * kSlot ? ring_s : p_slot + kSlot;
            ph += rp;
            if (ph - rs >= rows) {  // the next token
                ph = rs;
                --p_left;
                pq += stride * a.qts;
                pk += stride * a.kts;
                pv += stride * a.vts;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < kRing - 1; ++i) issue();

    const uint64_t turn = tid < half ? a.turns[tid] : 0;
    // positions and slots are read a token ahead of their use
    int32_t p_ahead = a.positions[token(0)];
    int64_t slot_ahead = tid == kThreads - 1 ? a.slots[token(0)] : 0;
    auto prepare = [&](int i) {
        const int32_t p = p_ahead;
        const int64_t slot = slot_ahead;
        if (i + 1 < count) {
            if (tid < half || tid == kThreads - 1) p_ahead = a.positions[token(i + 1)];
            if (tid == kThreads - 1) slot_ahead = a.slots[token(i + 1)];
        }
        if (tid < half) {
            const float2 z = cos_sin(p, turn);
            cs[i & 1][place(tid, half, group)] = make_float2(a.mscale * z.x, a.mscale * z.y);
        }
        if (tid == kThreads - 1) {
            Token w{-1, 0, p};
            const int64_t page = slot >> a.kv.page_shift;
            if (p >= 0 && slot >= 0) {
                if (page < a.kv.num_pages) {
                    const int64_t off = slot & ((int64_t(1) << a.kv.page_shift) - 1);
                    w.where = page * a.kv.page_stride + off * a.kv.pos_stride;
                    w.dwhere = page * a.kv.d_page_stride + off * a.kv.d_pos_stride;
                } else if (a.err) {
                    atomicOr(a.err, 1);
                }
            }
            tok[i & 1] = w;
        }
    };
    prepare(0);
    __syncthreads();

    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        if (i + 1 < count) prepare(i + 1);
        const Token w = tok[i & 1];
        float2 z[8];
        if (turns) {
            const float2 *c = cs[i & 1];
            if (group == 8) {
                const int at = (lo ? d0 : d0 - half) >> 3, st = half >> 3;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    z[k] = c[at + k * st];
                    z[k].y = lo ? -z[k].y : z[k].y;
                }
            } else {
                const int st = (half + 3) >> 2;
#pragma unroll
                for (int k = 0; k < 4; ++k) z[k] = d0 + 2 * k < a.rot ? c[(d0 >> 3) + k * st] : make_float2(1.f, 0.f);
            }
        }
        T *ob = static_cast<T *>(a.q_out) + token(i) * a.q_heads * D + d0;
#pragma unroll 1
        for (int h = rs; h - rs < rows; h += rp) {
            __syncwarp();  // the slot that the next copy takes has been read, by the partners too
            issue();
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            __syncwarp();
            const bool active = h < rows;  // a row's lanes are all active or all idle
            const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv.heads;
            const int kh = is_v ? h - a.q_heads - a.kv.heads : h - a.q_heads;
            float x[8];
            if (active && w.pos >= 0) {
                const T *own = reinterpret_cast<const T *>(&ring[slot][tid * kV]);
                load8(own, true, x);
                if (turns && !is_v) {
                    if (group == 8) {
                        float y[8];
                        load8(own + partner * 8, true, y);
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = fmaf(x[k], z[k].x, y[k] * z[k].y);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float x0 = x[2 * k], x1 = x[2 * k + 1];
                            // past the turned part (1, 0): the values as they are
                            if (d0 + 2 * k >= a.rot) continue;
                            x[2 * k] = fmaf(x0, z[k].x, -x1 * z[k].y);
                            x[2 * k + 1] = fmaf(x1, z[k].x, x0 * z[k].y);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = 0.f;  // padding
            }
            if (++slot == kRing) slot = 0;
            const bool cached = active && !is_q && w.where >= 0;
            if constexpr (CT == WSW_Q8_0) {
                const float amax = q8m::block_amax<32>(x);  // every lane of the warp
                if (cached) {
                    const float d = q8m::scale(amax);
                    uint32_t codes[2];
                    q8m::codes(x, amax, d, codes);
                    *reinterpret_cast<uint2 *>((is_v ? a.kv.v : a.kv.k) + w.where + kh * a.kv.head_stride + d0) =
                        make_uint2(codes[0], codes[1]);
                    if ((d0 & 31) == 0)
                        reinterpret_cast<__half *>((is_v ? a.kv.vd : a.kv.kd) + w.dwhere +
                                                   kh * a.kv.d_head_stride)[d0 >> 5] = __float2half_rn(d);
                }
            } else if (cached) {
                unsigned char *dst = (is_v ? a.kv.v : a.kv.k) + w.where + kh * a.kv.head_stride + d0 * 2;
                if constexpr (CT == WSW_F16) *reinterpret_cast<uint4 *>(dst) = pack8<__half>(x);
                else *reinterpret_cast<uint4 *>(dst) = pack8<__nv_bfloat16>(x);
            }
            if (active && is_q) store8(ob + h * D, true, x);
        }
        __syncthreads();  // the next token's angles are there, this one's have been read
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T>
cudaError_t launch_stream(const RopeArgs &a, int cache_type, dim3 grid, cudaStream_t s, bool pdl) {
    if (cache_type == WSW_F16) return launch(rope_stream_kernel<T, WSW_F16>, grid, dim3(kThreads), 0, s, pdl, a);
    if (cache_type == WSW_BF16) return launch(rope_stream_kernel<T, WSW_BF16>, grid, dim3(kThreads), 0, s, pdl, a);
    return launch(rope_stream_kernel<T, WSW_Q8_0>, grid, dim3(kThreads), 0, s, pdl, a);
}

template <typename T>
cudaError_t launch_rope(const RopeArgs &a, int cache_type, dim3 grid, cudaStream_t s, bool pdl) {
    if (cache_type == WSW_F16) return launch(rope_kv_kernel<T, WSW_F16>, grid, dim3(kThreads), 0, s, pdl, a);
    if (cache_type == WSW_BF16) return launch(rope_kv_kernel<T, WSW_BF16>, grid, dim3(kThreads), 0, s, pdl, a);
    return launch(rope_kv_kernel<T, WSW_Q8_0>, grid, dim3(kThreads), 0, s, pdl, a);
}

}  // namespace
}  // namespace wsw

extern "C" int wsw_rope_kv_write(const void *q, const void *k, const void *v, int32_t dtype, int64_t tokens,
                                 int64_t q_heads, int64_t q_tok_stride, int64_t q_head_stride, int64_t k_tok_stride,
                                 int64_t k_head_stride, int64_t v_tok_stride, int64_t v_head_stride,
                                 const uint64_t *turns, int64_t rot_dim, float mscale, int32_t interleaved,
                                 const int32_t *positions, const int64_t *slots, void *q_out,
                                 const wsw_kv_cache *cache, int32_t *err_flag, void *stream,
                                 const wsw_launch_opts *opts) {
    using namespace wsw;
    Opts o;
    int st = resolve_opts(opts, &o);
    if (st != WSW_OK) return st;
    RopeArgs a;
    st = check_kv_cache(cache, &a.kv);
    if (st != WSW_OK) return st;
    if (dtype != WSW_F32 && dtype != WSW_F16 && dtype != WSW_BF16) return WSW_ERR_UNSUPPORTED;
    if (tokens < 0 || q_heads < 0 || rot_dim < 0 || rot_dim > a.kv.head_dim || (rot_dim & 1) ||
        (interleaved != 0 && interleaved != 1) || !std::isfinite(mscale) || q_tok_stride < 0 || q_head_stride < 0 ||
        k_tok_stride < 0 || k_head_stride < 0 || v_tok_stride < 0 || v_head_stride < 0)
        return WSW_ERR_INVALID_ARG;
    if (tokens >= (int64_t(1) << 31) || q_heads > 65535) return WSW_ERR_UNSUPPORTED;
    if (tokens == 0) return WSW_OK;
    if (!k || !v || !positions || !slots || (q_heads > 0 && (!q || !q_out)) || (rot_dim > 0 && !turns))
        return WSW_ERR_INVALID_ARG;
    const int64_t esize = dtype == WSW_F32 ? 4 : 2;
    const uintptr_t in = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
                         (q_heads > 0 ? reinterpret_cast<uintptr_t>(q) : 0);
    const uintptr_t strides = static_cast<uintptr_t>(k_tok_stride | k_head_stride | v_tok_stride | v_head_stride |
                                                     (q_heads > 0 ? q_tok_stride | q_head_stride : 0)) * esize;
    const uintptr_t qo = q_heads > 0 ? reinterpret_cast<uintptr_t>(q_out) : 0;
    if (((in | qo) & (esize - 1)) || (reinterpret_cast<uintptr_t>(positions) & 3) ||
        (reinterpret_cast<uintptr_t>(slots) & 7) || (reinterpret_cast<uintptr_t>(turns) & 7) ||
        (reinterpret_cast<uintptr_t>(err_flag) & 3))
        return WSW_ERR_MISALIGNED;
    DeviceInfo di;
    if (!device_info(&di, &st)) return st;
    a.q = q; a.k = k; a.v = v;
    a.qts = q_tok_stride; a.qhs = q_head_stride;
    a.kts = k_tok_stride; a.khs = k_head_stride;
    a.vts = v_tok_stride; a.vhs = v_head_stride;
    a.turns = turns;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.err = err_flag;
    a.tokens = tokens;
    a.mscale = mscale;
    a.q_heads = static_cast<int>(q_heads);
    a.rot = static_cast<int>(rot_dim);
    a.interleaved = interleaved;
    a.lane_shift = a.kv.head_dim == 64 ? 3 : a.kv.head_dim == 128 ? 4 : 5;
    a.vec = ((in | strides) & 15) == 0;
    a.vec_out = (qo & 15) == 0;
    const int64_t passes = (((q_heads + 2 * a.kv.heads) << a.lane_shift) + kThreads - 1) / kThreads;  // of one token
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    // The streaming form wants aligned rows, pairs that fall into whole vectors, a few tokens for
    // each CTA and enough of each token for its threads.  8191 tokens of 48 heads, streaming and
    // plain form: bf16 41 and 55 us, fp32 into q8_0 61 and 70 us; fp32 into a 16-bit cache 69 and 66
    // us, so that one stays plain.  bf16 rows of 128: 24 a token 29.1 and 31.8 us, 12 21.2 and
    // 18.3, 3 19.0 and 8.3.  1024 and 1500 tokens of 48 heads: bf16 6.8 and 10.7, 10.3 and 14.5 us, fp32 into
    // q8_0 12.4 and 13.9, 15.4 and 16.3 us; of 24 rows 5.4 and 6.4, 7.0 and 7.7 us.
    const int64_t vectors = (q_heads + 2 * a.kv.heads) << a.lane_shift;  // 8 values, of one token
    const bool heavy = dtype != WSW_F32 || cache->dtype == WSW_Q8_0;
    if (tokens >= 1024 && heavy && vectors >= 384 && a.vec && a.vec_out && (interleaved || (rot_dim & 15) == 0)) {
        const dim3 all(static_cast<unsigned>(tokens < kStreamCtas * di.sm_count ? tokens : kStreamCtas * di.sm_count));
        if (dtype == WSW_F32) e = launch_stream<float>(a, cache->dtype, all, s, o.pdl);
        else if (dtype == WSW_F16) e = launch_stream<__half>(a, cache->dtype, all, s, o.pdl);
        else e = launch_stream<__nv_bfloat16>(a, cache->dtype, all, s, o.pdl);
        return e == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
    }
    // Tokens of a CTA: two, or so many that its threads have three vectors each (8191 bf16 tokens of 3
    // rows: 10.0 us with 2, 8.3 with 8), while there are two CTAs for each of 152 SMs (1024 tokens of
    // 12 rows: 4.4 us with 2, 6.0 with 8).
    int64_t tile = 3 * kThreads / vectors;
    if (tile > tokens / 304) tile = tokens / 304;
    if (tile > kMaxTile) tile = kMaxTile;
    a.tile = tokens < 1024 ? 1 : tile < 2 ? 2 : static_cast<int>(tile);
    const int64_t slabs = tokens >= 1024 ? 1 : passes;
    const dim3 grid(static_cast<unsigned>((tokens + a.tile - 1) / a.tile),
                    static_cast<unsigned>(slabs < 65535 ? slabs : 65535));
    if (dtype == WSW_F32) e = launch_rope<float>(a, cache->dtype, grid, s, o.pdl);
    else if (dtype == WSW_F16) e = launch_rope<__half>(a, cache->dtype, grid, s, o.pdl);
    else e = launch_rope<__nv_bfloat16>(a, cache->dtype, grid, s, o.pdl);
    return e == cudaSuccess ? WSW_OK : WSW_ERR_CUDA;
}
