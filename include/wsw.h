/*
 * wsw.h -- C ABI of libwsw.so, the decode-time weight-streaming hot path for one
 * NVIDIA GB300 (sm_103a).
 *
 * The calls cover the memory-bound mat-vec y = W.x that streams every weight byte
 * once per decoded token, the block quantizer that turns the activation into int8
 * blocks with absmax scales in front of the quantized mat-vec, the grouped MoE
 * form of that mat-vec, the one-pass q8_0 KV-cache dequantizer, the small-batch prefill
 * GEMM, attention, and the operators of a decode step around a paged KV cache.  Each call
 * is one or more hand-written CUDA kernels.
 *
 * Sources (web pages, cited by title and section):
 *   [P1] "vulkan : dequant q8_0 KV once in coopmat1" (llama.cpp pull request)
 *   [P2] "ggml-cuda: pad matmul weight rows to avoid cache-set aliasing"
 *   [P3] "QuantizeQ8KK is thread-per-superblock: 95.5us/call against llama.cpp's
 *        1.6us, and 41% of the ROCm decode gap"
 *   [P4] "perf(vulkan): decode GEMV reads four elements per load, and the row lever
 *        is dead"
 *   [P5] "cuda: prefetch the next PTQ1_0 mat-vec's weights into L2 from the last CTAs"
 *
 * Conventions shared by every call
 *   - Every pointer is a CUDA device pointer owned by the caller.  The library
 *     allocates nothing and keeps no state between calls apart from per-device
 *     kernel attributes set on first use.
 *   - bf16 and binary16 (fp16) data travel as uint16_t bit patterns.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls are
 *     asynchronous and stream-ordered; none synchronizes the host.
 *   - Arguments are validated on the host before anything is launched.  A rejected
 *     call returns a nonzero wsw_status and launches nothing.  A launch failure
 *     returns WSW_ERR_CUDA (the CUDA error is not cleared; query it with
 *     cudaGetLastError).  No kernel traps, asserts or spins without a bound.
 *   - Row strides (ld, ldq, ldx) are in elements.  The elements between the row
 *     length and the stride are padding and are never read ([P2] Overview: the
 *     pad is zero-filled by the uploader, the kernels take the stride as given).
 *   - A pointer or stride that is not aligned for 32-byte loads does not fail:
 *     the weight load width degrades 32 -> 16 -> 8 -> 4 -> 2 bytes until aligned,
 *     and the result is bit-identical to the 32-byte path ([P4] "What shipped": the
 *     load width degrades one step at a time when an offset is misaligned).
 *     The exception is wsw_gemm_bf16, whose TMA tile loads need 16-byte
 *     alignment (WSW_ERR_MISALIGNED otherwise).
 *   - Results do not depend on wsw_launch_opts: any rows_per_warp, load_bytes,
 *     pdl or ctas_per_sm gives bit-identical output ([P4] "What did NOT work":
 *     rows-per-workgroup variants verified bit-identical by full-output hash).
 */
#ifndef WSW_H
#define WSW_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define WSW_ABI_VERSION 7

typedef enum wsw_status {
    WSW_OK = 0,
    WSW_ERR_INVALID_ARG = 1, /* null pointer, bad size, stride or block size */
    WSW_ERR_MISALIGNED = 2,  /* alignment that the call cannot degrade around */
    WSW_ERR_UNSUPPORTED = 3, /* device is not sm_103 / shape beyond a stated limit */
    WSW_ERR_WORKSPACE = 4,   /* a required caller workspace is absent or too small */
    WSW_ERR_CUDA = 5,        /* a CUDA runtime call or launch failed */
    WSW_ERR_TIMEOUT = 6      /* a bounded device-side wait gave up (read on the
                                device: wsw_bounded_wait_check, bit 1 of the MoE
                                error flag) */
} wsw_status;

/* Steps of the next link that a chain link prefetches into L2 by default: 0 = off.
 * Programmatic dependent launch already issues each link's first loads while the one
 * before drains; on GB300 the 257-link 27B-shaped chain ran 0.4% (2 steps) to 3.8%
 * (16 steps) slower with the prefetch on. */
#define WSW_CHAIN_L2_PREFETCH_STEPS 0

/* Launch knobs.  Pass NULL for the defaults.  0 in a field means "choose". */
typedef struct wsw_launch_opts {
    int32_t rows_per_warp; /* output rows one warp reduces together: 1, 2 or 4
                              (the pages' rows per workgroup, [P4] "What did NOT
                              work"); 0 = the library's choice (2; 4 for bf16
                              mat-vecs of at least 16384 rows) */
    int32_t load_bytes;    /* cap on the weight load width: 32, 16, 8, 4 or 2;
                              0 = 32 (one 256-bit load per lane) */
    int32_t pdl;           /* 1 = launch with programmatic dependent launch: the
                              kernel issues its first weight loads before waiting
                              for the previous kernel in the stream ([P5]
                              "Additional information": PDL on sm_90 and newer) */
    int32_t ctas_per_sm;   /* resident CTAs per SM for persistent grids; 0 = auto */
    int32_t l2_prefetch_steps; /* wsw_gemv_bf16_chain only: once done with a link,
                              its warps request into L2 the first this-many 1 KB steps
                              of every warp's first unit of the next link ([P5]
                              Overview); 1..64, -1 = off, 0 = the library's choice
                              (WSW_CHAIN_L2_PREFETCH_STEPS) */
} wsw_launch_opts;

/* Human-readable name of a wsw_status value (static storage, never NULL). */
const char *wsw_status_string(int status);

/* ABI version of the loaded library (WSW_ABI_VERSION it was built with). */
int wsw_abi_version(void);

/*
 * wsw_quantize_q8 -- block quantizer for the activation ([P3] Cause: the amax
 * scan over one superblock; [P3] Scope: quantize, then the quantized mat-vec).
 *
 * For each block of `block` consecutive values of a row:
 *   amax = max |x|;  d = amax / 127 (fp32 division);
 *   q = round_half_away_from_zero(x / d) (fp32 division by the fp32 d), in
 *   [-127, 127];  an all-zero block gives d = +0 and q = 0.
 * One thread per 8 elements and a warp-shuffle reduction of amax; each element is
 * loaded once (the page's second defect, a second load per element, is avoided).
 *
 *   x       fp32 [rows][ldx]; the first n values of each row are quantized.
 *   rows    >= 0;  n >= 0, a multiple of `block`;  ldx >= n.
 *   block   32 (q8_0) or 256 (superblock).
 *   q       int8 [rows][n], packed.
 *   scales  block 32: binary16 [rows][n/32]; block 256: fp32 [rows][n/256].
 * rows == 0 or n == 0 launches nothing and returns WSW_OK.
 */
int wsw_quantize_q8(const float *x, int64_t rows, int64_t n, int64_t ldx, int32_t block,
                    int8_t *q, void *scales, void *stream, const wsw_launch_opts *opts);

/*
 * wsw_gemv_bf16 -- decode mat-vec with bf16 weights ([P4] opening paragraph: the
 * decode GEMV streams ~52 GB of bf16 weights once per token and is bound by DRAM
 * bandwidth; [P2] Overview: the row stride may exceed the row).
 *
 *   y[r] = alpha * sum_{k<K} W[r*ld + k] * x[k],  r < M,
 * with bf16 x fp32 products accumulated in fp32.
 *
 *   W      bf16 [M][ld], row-major;  ld >= K.
 *   x      fp32 [K] (not rounded to bf16).
 *   y      fp32 [M]; must not overlap x.
 * M == 0 launches nothing; K == 0 writes y = 0.
 */
int wsw_gemv_bf16(const uint16_t *W, int64_t M, int64_t K, int64_t ld, const float *x,
                  float alpha, float *y, void *stream, const wsw_launch_opts *opts);

/*
 * One link of a decode chain: y = alpha * W . x, as wsw_gemv_bf16.  x may point
 * into an earlier link's y ([P5] Overview: consecutive mat-vecs of the decode
 * graph, each paying a ramp-up and ramp-down in which DRAM idles).
 */
typedef struct wsw_gemv_link {
    const uint16_t *W;
    int64_t M, K, ld;
    const float *x;
    float alpha;
    float *y;
} wsw_gemv_link;

/*
 * wsw_gemv_bf16_chain -- launch n_links bf16 mat-vecs back to back on one stream,
 * each one programmatically dependent on the one before ([P5] "Additional
 * information": programmatic dependent launch is the sm_90+ tool for the idle
 * window between chained mat-vecs).  Every link is validated before the first
 * launch; the results equal n_links separate wsw_gemv_bf16 calls, bit for bit.
 * opts->pdl = 0 turns the dependency off (plain stream order).
 */
int wsw_gemv_bf16_chain(int64_t n_links, const wsw_gemv_link *links, void *stream,
                        const wsw_launch_opts *opts);

/* The launch that wsw_gemv_bf16 (or one link of wsw_gemv_bf16_chain) makes. */
typedef struct wsw_gemv_plan {
    int32_t load_bytes;    /* bytes per weight load of a lane: 32, 16, 8, 4 or 2 */
    int32_t rows_per_warp; /* 1, 2 or 4 */
    int32_t pdl;           /* 1 = programmatic dependent launch */
    int32_t ctas;          /* CTAs in the grid; 0 = no kernel (M == 0, or K == 0,
                              where y is zero-filled by a memset) */
    int32_t threads;       /* threads per CTA */
    int32_t log2_segments; /* each row's K is cut into 2^log2_segments segments
                              whose sums are combined in a fixed order */
    int32_t x_in_smem;     /* 1 = x is staged in shared memory, 0 = read via L1 */
    int32_t l2_prefetch_steps; /* chain links: steps of the next link's first units
                              requested into L2 (0 = none; the last link has no next) */
} wsw_gemv_plan;

/*
 * wsw_gemv_bf16_plan -- the launch choices of wsw_gemv_bf16 (chain == 0) or of a link
 * of wsw_gemv_bf16_chain (chain == 1) for these arguments, without launching anything
 * or calling CUDA ([P4] "What shipped": the load width follows the alignment of the
 * weight base and row pitch and degrades one step at a time; [P4] "Gates": a
 * variant-selection test pins what the launcher picks).  The launchers take their
 * choices from the same host function.
 *
 *   W          only its address is used (alignment); it is never dereferenced.
 *   M, K, ld   as wsw_gemv_bf16, validated the same way.
 *   sm_count   multiprocessors of the target device (> 0; 152 on GB300).
 *   chain      0 or 1.
 *   opts       as the call (NULL = defaults).
 *   out        host struct, written on WSW_OK.
 */
int wsw_gemv_bf16_plan(const uint16_t *W, int64_t M, int64_t K, int64_t ld, int32_t sm_count,
                       int32_t chain, const wsw_launch_opts *opts, wsw_gemv_plan *out);

/*
 * wsw_gemv_q8_0 -- decode mat-vec with q8_0 weights and a q8_0 activation ([P3]
 * Scope: the quantized mat-vec behind the quantizer).
 *
 *   y[r] = sum_b fp32(Wd[r][b]) * fp32(xd[b]) * (sum_{i<32} Wq[r*ldq + 32b+i] * xq[32b+i])
 * with the block sums in exact int32 and the rest in fp32.
 *
 *   Wq   int8 [M][ldq];  K % 32 == 0, ldq % 32 == 0 and ldq >= K (a quantized
 *        row stride must divide exactly into blocks, [P2] Overview).
 *   Wd   binary16 [M][K/32], packed.
 *   xq   int8 [K];  xd binary16 [K/32]  (as written by wsw_quantize_q8, block 32).
 *   y    fp32 [M].
 */
int wsw_gemv_q8_0(const int8_t *Wq, const uint16_t *Wd, int64_t M, int64_t K, int64_t ldq,
                  const int8_t *xq, const uint16_t *xd, float *y, void *stream,
                  const wsw_launch_opts *opts);

/*
 * wsw_quantize_gemv_q8_0 -- the batch-1 decode step of [P3] Scope (quantize the
 * activation to q8_0, then the quantized mat-vec) in one launch: every CTA quantizes
 * the fp32 x itself while its first weight loads are in flight, so no separate
 * quantizer kernel sits between two chained mat-vecs.
 *
 *   y = wsw_gemv_q8_0(Wq, Wd, M, K, ldq, q(x), d(x))  with (q(x), d(x)) =
 *       wsw_quantize_q8(x, 1, K, K, 32), bit for bit.
 *
 *   Wq, Wd, M, K, ldq, y   as wsw_gemv_q8_0.
 *   x        fp32 [K], 4-byte aligned.
 *   xq_out   int8 [K] and xd_out binary16 [K/32]: both NULL, or both set to receive
 *            the quantized activation (the bytes wsw_quantize_q8 writes).
 */
int wsw_quantize_gemv_q8_0(const int8_t *Wq, const uint16_t *Wd, int64_t M, int64_t K, int64_t ldq,
                           const float *x, int8_t *xq_out, uint16_t *xd_out, float *y, void *stream,
                           const wsw_launch_opts *opts);

/*
 * wsw_moe_workspace_bytes -- bytes of device workspace that wsw_moe_gemv_q8_0 can use
 * for E experts, row length K and R routed rows (0: that call needs none).  With the
 * workspace, calls with more than 256 routed rows run on the tensor cores; without it
 * they run on the CUDA cores.
 */
size_t wsw_moe_workspace_bytes(int64_t E, int64_t K, int64_t R);

/*
 * wsw_moe_gemv_q8_0 -- grouped MoE mat-vec over per-expert q8_0 weights ([P3]
 * Cause and Scope: the MoE path quantizes m = T x top_k rows, then runs a grouped
 * GEMM over the experts).
 *
 * For each row m < R with e = ids[m] in [0, E):
 *   y[m][o] = gemv_q8_0(W_e, x_m)[o],  o < Mo,
 * bit-identical to wsw_gemv_q8_0 on expert e's matrix and row m for R <= 256.
 * Each expert that some row uses is streamed from DRAM once per call; experts no row
 * uses are not read.  (For R <= 16 each routed row streams its own expert's rows; a
 * repeated expert's second pass is served by L2 while the routed experts' weights fit
 * in it, as they do for 16 rows of 128 x 1536 x 2048 experts.)  For R > 256 with a workspace, a prepass sorts
 * and converts the activations into the workspace and the rows of an expert are
 * multiplied on the tensor cores with exact integer block sums; results then agree
 * with the CUDA-core form within fp32 rounding, not bit for bit.
 *
 *   Wq   int8 [E][Mo][K];  Wd binary16 [E][Mo][K/32];  K % 32 == 0.
 *   xq   int8 [R][K];  xd binary16 [R][K/32].
 *   ids  int32 [R] (device).  A row whose id is outside [0, E) is skipped, its y
 *        row is left untouched, and bit 0 of *err_flag (if err_flag != NULL) is
 *        set.  Bit 1 is set if a bounded wait of the tensor-core form gave up (a
 *        WSW_ERR_TIMEOUT condition); the y rows that CTA had not finished are then
 *        NaN.  The library only ORs bits in; it never clears *err_flag.
 *   y    fp32 [R][Mo].
 *   ws   device workspace of ws_bytes >= wsw_moe_workspace_bytes(E, K, R) bytes,
 *        256-byte aligned, owned by the caller and overwritten by the call; NULL (or
 *        too small) keeps every row count on the CUDA cores.  Two calls in flight at
 *        once need two workspaces.
 *   R <= 16384 and E <= 1024, else WSW_ERR_UNSUPPORTED.
 */
int wsw_moe_gemv_q8_0(const int8_t *Wq, const uint16_t *Wd, int64_t E, int64_t Mo, int64_t K,
                      const int8_t *xq, const uint16_t *xd, const int32_t *ids, int64_t R,
                      float *y, int32_t *err_flag, void *ws, size_t ws_bytes, void *stream,
                      const wsw_launch_opts *opts);

/*
 * wsw_moe_gemv_q8_0_noalloc -- wsw_moe_gemv_q8_0 for callers that cannot allocate device
 * memory, such as a plugin or custom-operator interface that receives only its input
 * and output buffers, a runtime that reserves all device memory in its own pool at
 * start-up, or a path that cannot accept cudaMalloc's device synchronisation.  The pages
 * have no counterpart: this is a convenience of this library.
 *
 * Arguments, results and errors are those of wsw_moe_gemv_q8_0, except that there is
 * no ws / ws_bytes.  The workspace is a fixed 8 MiB scratch array inside the library,
 * which every GPU that loads the library holds until the process exits.  Sizes whose
 * wsw_moe_workspace_bytes(E, K, R) exceeds 8 MiB return WSW_ERR_UNSUPPORTED and launch
 * nothing (for example E = 128 takes R up to 1540 routed rows at K = 2048, and up to
 * 4096 at K = 768, the tensor-core limit).  The call
 * performs no cudaMalloc, cudaFree or other allocation.
 *
 *   - The first call on a device looks up the scratch array's device address on that
 *     device (it must be the current device).  Make that first call before any stream
 *     capture.
 *   - Every call on a device shares the one scratch array and leaves its contents
 *     behind.  Nothing in it needs to start at zero, because each call writes what it
 *     reads.  Calls whose executions overlap on the GPU (for example on two streams)
 *     race on the scratch; calls on one stream do not.
 */
int wsw_moe_gemv_q8_0_noalloc(const int8_t *Wq, const uint16_t *Wd, int64_t E, int64_t Mo, int64_t K,
                              const int8_t *xq, const uint16_t *xd, const int32_t *ids, int64_t R,
                              float *y, int32_t *err_flag, void *stream, const wsw_launch_opts *opts);

/*
 * wsw_dequant_q8_0_kv -- dequantize one layer's q8_0 K (or V) cache once into a
 * per-head-contiguous binary16 buffer ([P1] Overview and the stride discussion:
 * the cache walks [dim][position][head] with a position stride of
 * head_dim * heads elements; the scratch puts one head's positions back to back).
 *
 *   out[h][p][i] = f16_rn(fp32(d[p][h][i/32]) * q[p][h][i])
 *
 *   q     int8 [depth][heads][head_dim];  head_dim % 32 == 0.
 *   d     binary16 [depth][heads][head_dim/32].
 *   out   binary16 [heads][depth][head_dim]; must not overlap the inputs.
 * Returns WSW_ERR_INVALID_ARG for negative sizes, head_dim % 32 != 0, depth > 2^32,
 * heads or head_dim > 65536, or more than 2^45 values; WSW_ERR_MISALIGNED for an odd d
 * or out address.  Any size of zero is a no-op.
 */
int wsw_dequant_q8_0_kv(const int8_t *q, const uint16_t *d, int64_t depth, int64_t heads,
                        int64_t head_dim, uint16_t *out, void *stream,
                        const wsw_launch_opts *opts);

/*
 * wsw_attn_decode_f16 -- one decoding step of attention over a binary16 KV cache, the
 * consumer of the dequantized scratch ([P1] Overview: the flash-attention pass reads
 * the f16 K and V; the stride discussion: the cache keeps one head's rows
 * head_dim * n_head_kv elements apart, the scratch back to back).
 *
 *   s_p          = scale * sum_i q[h][g][i] * K(h, p)[i]
 *   out[h][g][i] = sum_p exp(s_p - m) * V(h, p)[i] / sum_p exp(s_p - m),  m = max_p s_p
 * over every position p < depth, for `heads` KV heads with `group` query heads each.
 * K(h, p) is the row of head_dim binary16 values at k + h * k_head_stride +
 * p * k_pos_stride (elements); V likewise.  The per-head-contiguous scratch that
 * wsw_dequant_q8_0_kv writes has (pos, head) strides (head_dim, depth * head_dim), the
 * position-major cache (heads * head_dim, head_dim).  Groups of 1 and 2 compute in fp32;
 * groups of 4 and 8 on the tensor cores, with q and the softmax weights entering as a
 * binary16 high part plus a binary16 residual (about 22 bits) and fp32 accumulation.
 * Either way results agree with fp64 within 1e-4 (normwise per output row) and do not
 * depend on the launch options.
 *
 *   q      fp32 [heads][group][head_dim].
 *   k, v   binary16; 16-byte aligned, strides multiples of 8 elements.
 *   out    fp32 [heads][group][head_dim]; must not overlap the inputs.
 *   ws     device workspace of ws_bytes >= wsw_attn_decode_workspace_bytes(depth,
 *          heads, group) bytes (WSW_ERR_WORKSPACE otherwise), 16-byte aligned.  It
 *          starts with one arrival counter per head, which must be zero before the
 *          first call; every call that completes leaves them zero, so a workspace is
 *          zero-filled once and then reused.  The rest is overwritten.  Two calls in
 *          flight at once need two workspaces.
 *   depth >= 1;  group in {1, 2, 4, 8};  head_dim == 128;  heads <= 65535
 *   (WSW_ERR_UNSUPPORTED otherwise).
 * One launch: chunks of positions in parallel; the last chunk of a head to finish
 * merges that head's chunks.
 */
size_t wsw_attn_decode_workspace_bytes(int64_t depth, int64_t heads, int64_t group);
int wsw_attn_decode_f16(const float *q, const uint16_t *k, const uint16_t *v, int64_t depth,
                        int64_t heads, int64_t group, int64_t head_dim, int64_t k_pos_stride,
                        int64_t k_head_stride, int64_t v_pos_stride, int64_t v_head_stride,
                        float scale, float *out, void *ws, size_t ws_bytes, void *stream,
                        const wsw_launch_opts *opts);

/*
 * wsw_attn_prefill_f16 -- causal prefill attention over a binary16 KV cache on the tensor
 * cores: the flash-attention pass of prompt processing that reads the dequantized
 * scratch ([P1] Overview: pp512 at depth 32768 and 65536 over the binary16 K and V; the
 * stride discussion: the cache keeps one head's rows head_dim * n_head_kv elements
 * apart, the scratch back to back).
 *
 * A batch of nq queries at the end of a cache of `depth` positions: query i of query
 * head (h, g) sits at position depth - nq + i and attends to positions
 * 0 .. depth - nq + i:
 *   s_p          = scale * sum_d q[h][g][i][d] * K(h, p)[d]
 *   out[h][g][i] = sum_p exp(s_p - m) V(h, p) / sum_p exp(s_p - m),  m = max_p s_p
 * K(h, p) is the row of head_dim binary16 values at k + h * k_head_stride +
 * p * k_pos_stride (elements); V likewise (the per-head scratch of
 * wsw_dequant_q8_0_kv: strides (head_dim, depth * head_dim); the position-major cache:
 * (heads * head_dim, head_dim)).  Products of binary16 values (q, K, V and the
 * probabilities P, rounded to binary16) accumulate in fp32; P's rounding bounds an
 * output element's error by about 2^-11 * sum_p w_p |V(h, p)| / sum_p w_p.
 *
 *   q      binary16 [heads][group][nq][head_dim], 16-byte aligned.
 *   k, v   binary16, 16-byte aligned; strides multiples of 8 elements.
 *   out    fp32 [heads][group][nq][head_dim], 16-byte aligned; must not overlap inputs.
 *   scale  finite and > 0.
 *   1 <= nq <= depth < 2^31;  head_dim == 128;  heads * group <= 65535
 *   (WSW_ERR_UNSUPPORTED / WSW_ERR_INVALID_ARG otherwise).  heads == 0 does nothing.
 * One launch; a bounded wait that gives up leaves NaN in the rows of its query tile.
 */
int wsw_attn_prefill_f16(const uint16_t *q, const uint16_t *k, const uint16_t *v, int64_t depth,
                         int64_t heads, int64_t group, int64_t nq, int64_t head_dim, int64_t k_pos_stride,
                         int64_t k_head_stride, int64_t v_pos_stride, int64_t v_head_stride, float scale,
                         float *out, void *stream, const wsw_launch_opts *opts);

/*
 * wsw_attn_prefill_q8_0 -- the same causal prefill attention over a q8_0 KV cache, with a
 * scratch of bounded size: the cache is dequantized and attended one window of
 * positions at a time ([P1] author's reply, "A few directions ... as follow-ups":
 * bounding the scratch with a chunked / streamed scratch that caps the peak, instead of
 * one binary16 layer of K and V for the whole depth; the dequantization is [P1]'s
 * dequant-once pass, wsw_dequant_q8_0_kv, applied to each window).
 *
 * For each window of `window` positions (the last one may be shorter): dequantize the
 * window's K and V rows into the per-head binary16 scratch, then attend over them,
 * carrying every query row's online-softmax state (running maximum, sum and unnormalized
 * output) from window to window.  Three launches per window, PDL-linked with opts->pdl.
 * The result equals wsw_dequant_q8_0_kv of K and V followed by wsw_attn_prefill_f16
 * within that call's stated error bound (not bit for bit: the maximum the
 * probabilities are taken against can differ between the two).
 *
 *   q        binary16 [heads][group][nq][head_dim], 16-byte aligned.
 *   kq, vq   int8 [depth][heads][head_dim];  kd, vd binary16 [depth][heads][head_dim/32]
 *            (the cache layout wsw_dequant_q8_0_kv reads).
 *   window   positions per window: a multiple of 128, at least 128.
 *   ws       device workspace of ws_bytes >= wsw_attn_prefill_q8_0_workspace_bytes(...)
 *            bytes, 256-byte aligned, overwritten (WSW_ERR_WORKSPACE otherwise): the K and
 *            V scratch of one window (2 * heads * min(window, depth) * head_dim * 2 bytes)
 *            and, with more than one window, the state (heads * group * nq * 528 bytes).
 *            Two calls in flight at once need two workspaces.
 *   out      as wsw_attn_prefill_f16.
 * Other limits as wsw_attn_prefill_f16.
 */
size_t wsw_attn_prefill_q8_0_workspace_bytes(int64_t depth, int64_t heads, int64_t group, int64_t nq,
                                             int64_t window);
int wsw_attn_prefill_q8_0(const uint16_t *q, const int8_t *kq, const uint16_t *kd, const int8_t *vq,
                          const uint16_t *vd, int64_t depth, int64_t heads, int64_t group, int64_t nq,
                          int64_t head_dim, float scale, int64_t window, void *ws, size_t ws_bytes, float *out,
                          void *stream, const wsw_launch_opts *opts);

/*
 * wsw_gemm_bf16 -- small-batch prefill product on the tensor cores ([P2] Results:
 * small-batch prefill streams the whole weight matrix for a short run of output
 * rows; the weight's row stride may carry one extra 128-byte line).
 *
 *   Y[n][r] = sum_{k<K} W[r*ld + k] * X[n*ldx + k],  r < M, n < N,
 * bf16 products accumulated in fp32.  Y row stride = M.
 *
 *   W   bf16 [M][ld];  X bf16 [N][ldx];  Y fp32 [N][M].
 *   W and X 16-byte aligned; K, ld and ldx multiples of 8 (WSW_ERR_MISALIGNED
 *   otherwise).
 */
int wsw_gemm_bf16(const uint16_t *W, int64_t M, int64_t K, int64_t ld, const uint16_t *X,
                  int64_t N, int64_t ldx, float *Y, void *stream, const wsw_launch_opts *opts);

/* ------------------------------------------------------------------------------------
 * A decode step around a paged KV cache.  Requests of different lengths share one pool of
 * pages; a block table lists each request's pages in order.  wsw_kv_page_plan gives the
 * step's new tokens their pages, positions and cache slots, wsw_rope_kv_write rotates q
 * and k and writes K and V there, wsw_attn_paged_decode attends, and wsw_token_logprobs
 * reads the lm_head's rows.  Lengths, tables and slots stay on the device, so that a step
 * can be captured in a CUDA graph and replayed while they change.
 */

/* Element types of the calls below. */
typedef enum wsw_dtype {
    WSW_F32 = 0,
    WSW_F16 = 1,  /* IEEE binary16 */
    WSW_BF16 = 2,
    WSW_Q8_0 = 3  /* int8 codes, one binary16 scale per 32 values (caches only) */
} wsw_dtype;

/*
 * A paged KV cache.  Position p of a request lives in its page table[p / page_size] at
 * offset p % page_size; a slot is page * page_size + offset.  The row of KV head h there is
 * the head_dim elements at k + page * page_stride + offset * pos_stride + h * head_stride
 * (v likewise); both orders of positions and heads inside a page, and K and V interleaved
 * in one buffer, are strides.  q8_0 rows are int8 codes with head_dim / 32 binary16 scales
 * at kd (vd) + page * d_page_stride + offset * d_pos_stride + h * d_head_stride, as
 * wsw_quantize_q8 (block 32) writes them.
 *
 *   k, v         16-byte aligned; strides multiples of 16 bytes.
 *   kd, vd       NULL unless dtype is WSW_Q8_0; base and strides multiples of
 *                head_dim / 16 bytes.
 *   page_size    a power of two, at most 65536.
 *   head_dim     64, 128 or 256;  heads <= 65535;  1 <= num_pages < 2^31.
 *   dtype        WSW_F16, WSW_BF16 or WSW_Q8_0.
 * A null pointer, a size below 1 or a negative stride is WSW_ERR_INVALID_ARG, a type or
 * size beyond these limits WSW_ERR_UNSUPPORTED.
 */
typedef struct wsw_kv_cache {
    void *k, *v;
    uint16_t *kd, *vd;
    int64_t num_pages, page_size, heads, head_dim;
    int64_t page_stride, pos_stride, head_stride;       /* elements of k and v */
    int64_t d_page_stride, d_pos_stride, d_head_stride; /* elements of kd and vd */
    int32_t dtype;                                      /* a wsw_dtype */
} wsw_kv_cache;

/*
 * wsw_kv_page_plan -- block table and slot map of a step from the requests' lengths.
 * Request r holds seq_len[r] cached tokens and adds new_len[r] (0 is fine); its new pages
 * come from the list of free pages, in request order:
 *   cu[r]        = sum of new_len before r;  need(r) = ceil((seq_len + new_len) / page_size)
 *                  - ceil(seq_len / page_size);  off(r) = sum of need before r
 *   table[r][j]  = free_pages[head + off(r) + j - ceil(seq_len / page_size)] for each new j
 *   token cu[r] + i:  position = seq_len[r] + i,
 *                     slot = table[r][position / page_size] * page_size + position % page_size
 *   len_out[r]   = seq_len[r] + new_len[r];  head_out = head + pages taken
 * A request that cannot be served keeps its length and takes no page, its tokens get
 * position and slot -1, and a bit of *err_flag is set: 1 (bit 0) a negative length (it
 * has no tokens); 2 more than max_pages pages (or 2^31 positions); 4 tokens beyond `tokens` (cu is cut there);
 * 8 the free list ran out (the requests before it are served, it and those after it that
 * need a page are not).  Tokens from cu[requests] to `tokens` get -1 and -1; a token whose
 * table entry is negative gets slot -1.  Table entries other than the new ones are left
 * as they are.
 *
 *   seq_len, new_len  int32 [requests].
 *   free_pages        int32 [n_free]; head: int32 [1], the next free entry (outside
 *                     [0, n_free]: nothing is free).
 *   table             int32 [requests][table_stride], max_pages entries used of each row.
 *   positions, slots  int32 and int64 [tokens];  cu int32 [requests + 1].
 *   len_out, head_out may be seq_len and head themselves: every length is read before
 *                     one is written.
 *   err_flag          int32 [1] or NULL; bits are ORed in, never cleared.
 *   requests <= 16384, page_size a power of two <= 65536, tokens <= 2^31 - 2^20, n_free <
 *   2^31 - 1, max_pages < 2^31 (WSW_ERR_UNSUPPORTED otherwise).  requests == 0 plans no token.
 */
int wsw_kv_page_plan(const int32_t *seq_len, const int32_t *new_len, int64_t requests, const int32_t *free_pages,
                     int64_t n_free, const int32_t *head, int64_t page_size, int32_t *table, int64_t max_pages,
                     int64_t table_stride, int64_t tokens, int32_t *positions, int64_t *slots, int32_t *cu,
                     int32_t *len_out, int32_t *head_out, int32_t *err_flag, void *stream,
                     const wsw_launch_opts *opts);

/* How wsw_rope_table scales the frequencies f_i = theta^(-2 i / rot_dim) for contexts
 * `factor` times as long as the `original` one. */
typedef enum wsw_rope_scaling {
    WSW_ROPE_PLAIN = 0,
    WSW_ROPE_LINEAR = 1,  /* f_i / factor */
    WSW_ROPE_NTK = 2,     /* theta * factor^(rot_dim / (rot_dim - 2)) in place of theta */
    WSW_ROPE_BY_PARTS = 3 /* between f_i / factor for pairs that turn at most once over
                             `original` positions and f_i for those that turn 32 times or
                             more, linear in the turns (NTK-by-parts of "YaRN: Efficient
                             Context Window Extension of Large Language Models", section
                             3.2); cos and sin times 0.1 ln(factor) + 1 (section 3.3) */
} wsw_rope_scaling;

/*
 * wsw_rope_table -- host: the per-pair frequencies of wsw_rope_kv_write in fractions of a
 * turn, turns[i] = round(2^64 * f_i / (2 pi)) with f_i carried to some 100 bits, and the
 * factor on cos and sin.  A position's angle is then the exact 64-bit product position *
 * turns[i] modulo one turn: the table's rounding makes it wrong by position * 2^-65 turns at
 * most, 7e-10 radians at position 2^31.
 *   freqs    NULL, or rot_dim / 2 radians per position of the caller's own, in [0, 2 pi):
 *            they are taken as given and theta, scaling, factor, original ignored.
 *   turns    host uint64 [rot_dim / 2];  mscale: host float.
 * WSW_ERR_INVALID_ARG: rot_dim not a positive even number (<= 256; > 2 for NTK),
 * theta <= 1, factor < 1, original < 1 (BY_PARTS), or a frequency outside [0, 2 pi).
 */
int wsw_rope_table(int64_t rot_dim, double theta, int32_t scaling, double factor, int64_t original,
                   const double *freqs, uint64_t *turns, float *mscale);

/*
 * wsw_rope_kv_write -- rotary positions of q and k, and the write of k and v into the
 * paged cache, in one pass.  Pair i < rot_dim / 2 of a head is (x[i], x[i + rot_dim / 2]),
 * or (x[2 i], x[2 i + 1]) with interleaved = 1; with angle a = positions[t] * 2 pi *
 * turns[i] / 2^64 it becomes
 *   mscale * (x0 cos a - x1 sin a, x1 cos a + x0 sin a);
 * the dimensions from rot_dim on are copied.  q goes to q_out, k and v to the row of
 * slots[t] in the cache, rounded once to its type (q8_0: by wsw_quantize_q8's rule).
 * A token with a negative position is padding: its q_out row is zero and nothing is
 * cached.  One with a negative slot is rotated and not cached; a slot outside the cache
 * is treated so too and sets bit 0 of *err_flag.  Two tokens of one call must not share
 * a slot.
 *
 *   q         `dtype` [tokens][q_heads][head_dim] with the given token and head strides
 *             (elements), unit stride in head_dim; k and v likewise with cache->heads heads:
 *             views of one fused QKV row or separate tensors.
 *   dtype     WSW_F32, WSW_F16 or WSW_BF16, of q, k, v and q_out.  16-byte aligned bases
 *             and strides give the widest loads; others take narrower ones.
 *   turns     device uint64 [rot_dim / 2] (from wsw_rope_table);  rot_dim even, <= head_dim.
 *   q_out     `dtype` [tokens][q_heads][head_dim], packed; it may be q itself only when q is
 *             packed, too.
 *   positions int32 [tokens];  slots int64 [tokens].
 * q_heads may be 0.  tokens == 0 does nothing.
 */
int wsw_rope_kv_write(const void *q, const void *k, const void *v, int32_t dtype, int64_t tokens, int64_t q_heads,
                      int64_t q_tok_stride, int64_t q_head_stride, int64_t k_tok_stride, int64_t k_head_stride,
                      int64_t v_tok_stride, int64_t v_head_stride, const uint64_t *turns, int64_t rot_dim,
                      float mscale, int32_t interleaved, const int32_t *positions, const int64_t *slots,
                      void *q_out, const wsw_kv_cache *cache, int32_t *err_flag, void *stream,
                      const wsw_launch_opts *opts);

/*
 * wsw_attn_paged_decode -- attention of one new token per request over a paged cache.
 * For request r with n = lens[r] cached tokens (the new one, at position n - 1, among
 * them), query head a = h * group + g of KV head h and every position p that it sees
 * (max(0, n - window) <= p < n; window = 0: all p < n):
 *   x_p  = scale * q[r][a] . K(h, p);  x_p = softcap * tanh(x_p / softcap) if softcap > 0
 *   x_p -= slopes[a] * (n - 1 - p)     if slopes != NULL
 *   out[r][a] = sum_p exp(x_p - m) V(h, p) / sum_p exp(x_p - m);  lse[r][a] = ln sum_p exp(x_p)
 * K(h, p) and V(h, p) are the cached rows; a q8_0 value is binary16(scale * code), the
 * value wsw_dequant_q8_0_kv writes.  A request of length 0 (an unused row of a padded
 * batch) gets out = 0 and lse = -inf, as does one whose seen scores are all -inf.
 * Positions past lens[r] in a page are never used.
 *
 * Scores, the softmax's maximum and sum, and the value sums are fp32.  The products run
 * on tensor cores in the cache's 16-bit type (binary16 for q8_0); q and the softmax
 * weights enter as a high part plus a residual in that type, so that they keep about 22
 * bits (binary16; a query row times a power of two of its own, so any finite row; a weight
 * is off by 2^-22 of itself or 2^-32 of the row's largest) or 16 bits (bf16 under 16-bit
 * queries, which are exact).  Under fp32 queries over bf16 they are three parts, exact.
 *
 *   q, out    `dtype` (WSW_F32, WSW_F16 or WSW_BF16) [requests][q_heads][head_dim], packed,
 *             16-byte aligned; q_heads = group * cache->heads, any group >= 1.
 *   table     int32 [requests][table_stride], max_pages entries of each row used.  An
 *             entry outside [0, num_pages) hides its positions and sets bit 0 of *err_flag.
 *   lens      int32 [requests]; below 0 or above max_pages * page_size is cut to that
 *             range and sets bit 1.
 *   lse       fp32 [requests][q_heads] or NULL;  slopes fp32 [q_heads] or NULL.
 *   scale     scale * log2(e) finite in fp32; softcap finite, >= 0;  0 <= window < 2^31.
 *   ws        device workspace of ws_bytes >= wsw_attn_paged_decode_workspace_bytes(...)
 *             bytes, 16-byte aligned, zero-filled before its first use and then reused:
 *             its arrival counters are zero again after every call.  Two calls in flight
 *             at once need two workspaces.
 *   requests <= 65535, requests * q_heads < 2^31 and q_heads * head_dim / 4 <= 2^31 - 4096;
 *   max_pages * page_size <= 2^31 - 4096;
 *   requests * kv heads * ceil(max_pages * page_size / 16) < 2^31 (with more than 16
 *   query heads per KV head, times ceil(group / 16); with a window, min(window, ...)).
 * One launch; results depend on the arguments alone, not on the launch or the device.
 */
size_t wsw_attn_paged_decode_workspace_bytes(int64_t requests, int64_t q_heads, int64_t kv_heads, int64_t head_dim);
int wsw_attn_paged_decode(const void *q, int32_t dtype, int64_t requests, int64_t q_heads,
                          const wsw_kv_cache *cache, const int32_t *table, int64_t max_pages, int64_t table_stride,
                          const int32_t *lens, float scale, float softcap, int64_t window, const float *slopes,
                          void *out, float *lse, int32_t *err_flag, void *ws, size_t ws_bytes, void *stream,
                          const wsw_launch_opts *opts);

/*
 * wsw_token_logprobs -- what a step answers with, in one pass over its logits: for each row
 * x of `vocab` logits, y = scale * x, and its token t,
 *   lse = ln sum_j exp(y_j);  logprob = y_t - lse;  entropy = -sum_j p_j ln p_j, p = exp(y - lse)
 *   rank = number of j with x_j > x_t, or x_j = x_t and j < t (0: the most likely token)
 *   top_id[i], top_logprob[i], i < top: the i-th largest x_j (ties: the lower j first), y_j - lse
 * -inf logits (forbidden tokens) have probability 0.  A row of nothing but -inf has
 * lse = -inf, entropy = 0 and every log probability -inf.  A NaN or +inf logit makes the
 * row's fp32 results NaN (its ids stay within [-1, vocab)).  A token outside [0, vocab)
 * gets logprob NaN and rank -1.
 *
 *   logits   `dtype` (WSW_F32, WSW_F16 or WSW_BF16) [rows][ld], ld >= vocab, aligned to
 *            its element.
 *   tokens   int32 [rows], or NULL with logprob and rank NULL.
 *   scale    > 0 (1 / temperature), scale * log2(e) finite in fp32.
 *   top      0 .. 32, at most vocab; with 0 top_logprob and top_id may be NULL.
 *   logprob, lse, entropy fp32 [rows];  rank int32 [rows];  top_logprob fp32 and top_id
 *            int32 [rows][top].
 *   ws       device workspace of ws_bytes >= wsw_token_logprobs_workspace_bytes(...) bytes
 *            (0: none needed, ws may be NULL), 16-byte aligned, zero-filled before its
 *            first use and then reused, as the attention's.
 *   1 <= vocab < 2^31 - 65536;  rows < 2^31.  rows == 0 does nothing.
 */
size_t wsw_token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int64_t top);
int wsw_token_logprobs(const void *logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t ld,
                       const int32_t *tokens, float scale, int32_t top, float *logprob, int32_t *rank, float *lse,
                       float *entropy, float *top_logprob, int32_t *top_id, void *ws, size_t ws_bytes, void *stream,
                       const wsw_launch_opts *opts);

/* ------------------------------------------------------------------------------------
 * Rows that continue one prompt (beams, parallel samples, a shared system prompt).  Their
 * block tables list the same pages for what they have in common.
 */

/*
 * wsw_kv_page_fork -- block table rows of a step's children from their parents'.  With
 * n = seq_len[parent[i]], row i of the new table lists the pages of its parent:
 *   table_out[i][j] = table[parent[i]][j] for j < ceil(n / page_size);  len_out[i] = n
 * Full pages are shared.  A partly filled last page (n % page_size > 0) stays with the lowest
 * child of its row; each other child takes a fresh page in its place, the k-th of them in row
 * order free_pages[head + k], and leaves a copy for wsw_kv_page_copy:
 *   src[k] = the parent's last page, dst[k] = the fresh one, fill[k] = n % page_size
 *   *count = number of copies;  *head_out = head + *count
 * Entries of the new rows from their pages on become -1 as far as any row of `table` reaches.
 * A partly filled last page has to be its row's alone, as this call leaves it.  What no row
 * lists any more goes back to the free list by wsw_kv_page_compact.
 *
 *   parent      int32 [children]: a row of `table`, or -1 for an empty row (length 0).
 *   seq_len     int32 [requests], the old rows' lengths; their pages lie in `table`, int32
 *               [requests][table_stride], max_pages entries of each row used.
 *   table_out   int32 [children][out_stride]; table itself (out_stride = table_stride) or
 *               elsewhere (WSW_ERR_INVALID_ARG if they overlap otherwise).
 *   len_out     int32 [children] and head_out int32 [1]; they may be seq_len and head.
 *   src, dst, fill  int32 [children], the first *count entries written; count int32 [1].
 *   free_pages, head  as wsw_kv_page_plan's.
 *   err_flag    int32 [1] or NULL; bits are ORed in: 1 (bit 0) a parent outside [-1, requests),
 *               2 a parent of negative length or more than max_pages pages, 8 the free list
 *               ran out.  The rows concerned are empty.
 *   children, requests <= 8192;  n_free < 2^31 - 1;  max_pages <= 2^31 - 2^20;  page_size a
 *   power of two <= 65536.
 */
int wsw_kv_page_fork(const int32_t *parent, int64_t children, const int32_t *seq_len, int64_t requests,
                     const int32_t *free_pages, int64_t n_free, const int32_t *head, int64_t page_size,
                     const int32_t *table, int64_t max_pages, int64_t table_stride, int32_t *table_out,
                     int64_t out_stride, int32_t *len_out, int32_t *head_out, int32_t *src, int32_t *dst,
                     int32_t *fill, int32_t *count, int32_t *err_flag, void *stream, const wsw_launch_opts *opts);

/*
 * wsw_kv_page_copy -- copy pages within every one of `n_caches` caches (the layers of a
 * model): for e < *count, the first fill[e] positions of page src[e] to page dst[e], K, V and
 * scales.  A copy from or to a page outside a cache is left out there and sets bit 0 of
 * *err_flag.  The other positions of dst[e] stay as they are.
 *
 *   src, dst    int32 [copies];  fill int32 [copies] (cut to [0, page_size]) or NULL: whole
 *               pages.  No page may be the dst of two copies, or the dst of one and the src of
 *               another.
 *   count       int32 [1], cut to [0, copies].
 *   caches      host array of pointers; page_size equal in all, the rest their own.
 *   copies < 2^31;  n_caches <= 65536.  One launch for each 32 caches.
 */
int wsw_kv_page_copy(const int32_t *src, const int32_t *dst, const int32_t *fill, const int32_t *count,
                     int64_t copies, const wsw_kv_cache *const *caches, int64_t n_caches, int32_t *err_flag,
                     void *stream, const wsw_launch_opts *opts);

/*
 * wsw_kv_page_compact -- the free list from what the rows list, and live pages moved together.
 * A page is live if a row lists it (among its first ceil(seq_len / page_size) entries) or
 * held[p] is not 0.  With N live pages, the k-th live page >= N that is not held moves to the
 * k-th page below N that is not live, both counted in ascending order, for k < max_moves:
 *   src[k], dst[k]  that move, for wsw_kv_page_copy (whole pages);  *count = number of moves
 *   table_out       the rows' used entries with the moved pages' new numbers
 *   free_pages      [N .. num_pages - 1]: the pages that are not live then, ascending;
 *   *head = N
 * max_moves = 0 only frees: no table is written, src and dst may be NULL.  Pages that a row
 * of no table lists, but that have to stay (a prefix kept for later), are `held`; they never
 * move.  One call sees all the rows that use the pool.
 *
 *   seq_len     int32 [requests];  table int32 [requests][table_stride].
 *   held        uint8 [num_pages] or NULL.
 *   table_out   int32 [requests][out_stride]; table itself (equal strides) or elsewhere; entries
 *               past a row's pages are not written.
 *   free_pages  int32 [num_pages]; entries before *head are left as they are.
 *   src, dst    int32 [max_moves];  count, head int32 [1].
 *   err_flag    int32 [1] or NULL; bits are ORed in: 1 (bit 0) an entry outside [0, num_pages) (it
 *               lists nothing and stays as it is), 2 a length that is negative or needs more than
 *               max_pages entries (the row lists nothing).
 *   ws          device workspace of ws_bytes >= wsw_kv_page_compact_workspace_bytes(num_pages),
 *               16-byte aligned, overwritten.
 *   requests <= 65535;  num_pages <= 2^22;  max_pages <= 2^31 - 2^20;  page_size a power of two
 *   <= 65536;  max_moves < 2^31.
 */
size_t wsw_kv_page_compact_workspace_bytes(int64_t num_pages);
int wsw_kv_page_compact(const int32_t *seq_len, int64_t requests, const int32_t *table, int64_t max_pages,
                        int64_t table_stride, int64_t page_size, int64_t num_pages, const uint8_t *held,
                        int64_t max_moves, int32_t *table_out, int64_t out_stride, int32_t *free_pages,
                        int32_t *head, int32_t *src, int32_t *dst, int32_t *count, int32_t *err_flag, void *ws,
                        size_t ws_bytes, void *stream, const wsw_launch_opts *opts);

/*
 * wsw_beam_select -- the next beams of every request from the logits of all its beams, in one
 * pass.  With x[b] the row of beam b (row request * beams + b of the logits), y = scale * x,
 *   s[b][j] = scores[b] + y[b][j] - ln sum_i exp(y[b][i])
 * The candidates (b, j) with s finite in fp32 are taken in descending order of s, equal ones by the
 * lower b, then the lower j, until `beams` of them do not end: those are the next beams, in that
 * order.  A candidate ends if its token is one of end_tokens; it is reported as an ended one
 * if fewer than `beams` candidates come before it.
 *   parent[i], token[i], score[i]   of the i-th next beam of a request: the row of the logits that
 *                      it continues, its token, its s rounded to fp32
 *   end_parent, end_token, end_score   the same of the ended ones, in order
 * Places without a candidate hold -1, -1 and -inf.  A forbidden token (logit -inf), a beam whose
 * score is not finite, and every beam whose row holds a NaN or +inf have no candidates.
 * Sums are fp32 within a thread's tile and pairs of fp32 above, scores are compared as pairs: s is off by some
 * 1e-8 as a rule and 2^-18 at most, before its rounding.  Equal rows have equal sums, whatever their
 * alignment.  parent is what wsw_kv_page_fork takes.
 *
 *   logits      `dtype` (WSW_F32, WSW_F16 or WSW_BF16) [requests * beams][ld], ld >= vocab,
 *               aligned to its element.
 *   scores      fp32 [requests][beams]: the beams' log probabilities so far (-inf: no beam).
 *   end_tokens  host int32 [n_ends].
 *   scale       > 0 (1 / temperature), scale * log2(e) finite in fp32.
 *   parent, token int32 and score fp32 [requests][beams];  end_parent, end_token and
 *               end_score likewise (all NULL is fine without end tokens).
 *   ws          device workspace of ws_bytes >= wsw_beam_select_workspace_bytes(...) bytes,
 *               16-byte aligned, zero-filled before its first use and then reused, as
 *               wsw_attn_paged_decode's.
 *   requests <= 16384;  beams <= 32;  n_ends <= 8;  beams * (1 + n_ends) <= 32;
 *   1 <= vocab < 2^31 - 65536.  requests == 0 does nothing.
 */
size_t wsw_beam_select_workspace_bytes(int64_t requests, int64_t beams, int64_t vocab, int64_t n_ends);
int wsw_beam_select(const void *logits, int32_t dtype, int64_t requests, int64_t beams, int64_t vocab, int64_t ld,
                    const float *scores, const int32_t *end_tokens, int64_t n_ends, float scale, int32_t *parent,
                    int32_t *token, float *score, int32_t *end_parent, int32_t *end_token, float *end_score, void *ws,
                    size_t ws_bytes, void *stream, const wsw_launch_opts *opts);

/*
 * wsw_attn_paged_prefix -- wsw_attn_paged_decode for a batch in which groups of requests share a
 * long prefix, whose K and V are read once for all requests of a group.  Group g is the
 * requests cu_groups[g] <= r < cu_groups[g + 1]; the first prefix_len[g] positions of all of them
 * hold the same keys and values (in the same pages, as wsw_kv_page_fork leaves them, or in
 * copies).  Results are those of wsw_attn_paged_decode without a window: each request sees all its
 * lens[r] positions.  The prefix is read through the table row of the group's first request
 * with lens[r] >= prefix_len[g]; a shorter request (or an unused row of length 0), a group of
 * one request, and a request outside all groups are attended as wsw_attn_paged_decode does.
 *
 * A prefix's products run on the tensor cores with fp32 sums.  The softmax weights keep 22 bits over
 * binary16 and q8_0 and 16 over bf16 (under fp32 queries all 24), as there; q keeps 22 bits over binary16 and
 * q8_0 (its own binary16 all of them), and all of them over bf16.  softcap's tanh is off by 24 2^-24 of itself at most.
 *
 *   cu_groups   int32 [groups + 1], ascending within [0, requests];  prefix_len int32 [groups], within
 *               [0, max_pages * page_size].  A bound that is not is moved to the nearest one that is,
 *               and sets bit 2 of *err_flag; bits 0 and 1 as wsw_attn_paged_decode's.
 *   share       1: always in this way.  0: batches whose cached positions have 128 MB at most (requests *
 *               max_pages * page_size of them) are attended as wsw_attn_paged_decode does, in one
 *               launch and without a look at the groups, which is sooner.
 *   head_dim    64 or 128.
 *   ws          device workspace of ws_bytes >= wsw_attn_paged_prefix_workspace_bytes(...) bytes,
 *               256-byte aligned, zero-filled before its first use and then reused, as
 *               wsw_attn_paged_decode's.
 *   1 <= groups <= 16384;  requests * q_heads <= 2^30;
 *   kv heads * (requests * group / 128 + groups) * (max_pages * page_size / 16 + 9) < 2^31 - 65536.
 *   Other arguments and limits as wsw_attn_paged_decode.  Four launches.
 */
size_t wsw_attn_paged_prefix_workspace_bytes(int64_t requests, int64_t groups, int64_t q_heads, int64_t kv_heads,
                                             int64_t head_dim);
int wsw_attn_paged_prefix(const void *q, int32_t dtype, int64_t requests, int64_t q_heads, const wsw_kv_cache *cache,
                          const int32_t *table, int64_t max_pages, int64_t table_stride, const int32_t *lens,
                          const int32_t *cu_groups, int64_t groups, const int32_t *prefix_len, int32_t share,
                          float scale, float softcap, const float *slopes, void *out, float *lse, int32_t *err_flag,
                          void *ws, size_t ws_bytes, void *stream, const wsw_launch_opts *opts);

/*
 * wsw_bounded_wait_check -- run the bounded mbarrier wait of the tensor-core kernels
 * on its own, one thread of one CTA.  The library has no device-side fault injection:
 * this call is how the give-up path of a wait is exercised on a GPU.
 *
 *   arrive = 1   the barrier's phase completes before the wait: *status = WSW_OK.
 *   arrive = 0   nothing completes the phase: the wait gives up after about one
 *                second and *status = WSW_ERR_TIMEOUT.  The kernel then returns
 *                normally and the context stays usable.
 *   status       int32 on the device, written by the kernel.
 */
int wsw_bounded_wait_check(int32_t arrive, int32_t *status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* WSW_H */
