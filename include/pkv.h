/*
 * pkv.h — C ABI of the GB300 paged KV-cache decode library (libpkv.so).
 *
 * What the library computes, and where the reference pages state it:
 *   - "KV Cache는 왜 LLM 서빙의 핵심인가", section "KV Cache: O(T²)를 O(T)로"
 *     (decode-step listing): each step appends the new token's k_t, v_t to the
 *     cache and computes softmax(q_t K^T / sqrt(d)) V over the whole cache.
 *   - "LLM 서빙과 KV Cache, VLLM", section "PagedAttention": the cache is cut
 *     into fixed-size token blocks that live anywhere in one shared pool.
 *   - "KV Cache는 왜 LLM 서빙의 핵심인가", section "메모리 공식과 GQA의 동기",
 *     and "KV 캐시 시스템 (KV Cache System)", section "MQA / GQA": n_h query
 *     heads share n_kv K/V groups; MHA is n_kv = n_h, MQA is n_kv = 1.
 *   - "KV Cache는 왜 LLM 서빙의 핵심인가", section "KVQuant: 마지막 4배": INT4
 *     K per channel, V per token, step size (max - min) / (2^4 - 1).
 *   - "Research Paper Review : CACHE BLEND ...", section "Background": reused
 *     chunks are brought to their real position by one extra RoPE rotation of
 *     their keys by (real start - 0).
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *     allocates no device memory and frees nothing; scratch space is passed in
 *     (`workspace`).  Tensors are dense, row-major, in the layouts stated below.
 *   - bf16 / fp16 tensors are passed as `void*` (2-byte elements).
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every call
 *     only enqueues work on `stream` and returns; the caller orders calls (e.g.
 *     append before attend) by issuing them on one stream.
 *     Kernels are launched ahead of the end of the kernel before them (programmatic dependent
 *     launch) and wait for it on the device.  Rotary calls, the 8-bit and the accounted attention,
 *     the 8-bit append and the eviction read nothing before that wait: whatever earlier work on
 *     the stream wrote, also the kernel directly ahead, is there.  pkv_paged_decode_attn and
 *     pkv_paged_decode_attn_int4 (with their window and noalloc forms) read context_lens, and only
 *     those, before it when batch <= 256: write the lengths ahead of the step's append, or of any
 *     other kernel, not in the kernel directly ahead of these calls; later lengths may be read as
 *     they were before (a wrong result or PKV_DEV_TIMEOUT, never an access out of bounds).
 *   - Argument errors are returned synchronously as a negative pkv_status and
 *     nothing is enqueued.  Errors only the GPU can see (a block-table entry or
 *     slot out of range, a context length out of range, a bounded wait that gave
 *     up) set bits in `*err_flag` (a caller-owned device int32, may be NULL): the
 *     offending item is skipped (its block contributes nothing / the token is
 *     not written) and no access goes out of bounds.  The caller clears the flag.
 *   - Pool layout (bf16): [num_blocks][n_kv][block_size][head_dim]; the tile of
 *     one (block, kv head) is contiguous.
 *   - Supported: head_dim in {64, 128}; block_size in {16, 32, 64};
 *     n_h % n_kv == 0 with group n_h / n_kv <= 64.  Other values give PKV_EINVAL.
 *     q, out, pools, codes and workspace must be 16-byte aligned.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PKV_OK = 0,
  PKV_EINVAL = -1,   /* bad argument: shape, null pointer, alignment, unsupported size */
  PKV_ERANGE = -2,   /* a size beyond a documented maximum */
  PKV_ECUDA = -3,    /* a CUDA call failed (no device, launch error); see pkv_last_cuda_error() */
  PKV_ENOSPC = -4    /* workspace smaller than pkv_decode_workspace_bytes() */
} pkv_status;

/* Bits ORed into *err_flag by the kernels. */
#define PKV_DEV_BAD_BLOCK 1  /* block_tables entry outside [0, num_blocks): block skipped   */
#define PKV_DEV_BAD_SLOT  2  /* slot >= num_blocks * block_size (or bad tail row): skipped  */
#define PKV_DEV_BAD_CTX   4  /* context_lens[s] < 0 or > max_blocks * block_size: clamped  */
#define PKV_DEV_TIMEOUT   8  /* a bounded wait inside a kernel gave up (about 2 s)          */
#define PKV_DEV_BAD_TREE 16  /* q_start out of order or range, more drafted tokens than cached
                                rows, or an accepted path that does not ascend over them     */

/* Output element types of the attention calls. */
#define PKV_OUT_BF16 0
#define PKV_OUT_F32  1

/* Human-readable name of a status. */
const char* pkv_status_str(int status);
/* The last CUDA error code seen by the library on this thread (cudaError_t as int). */
int pkv_last_cuda_error(void);

/*
 * kv_append — write each new token's K and V rows into the pools at its slot.
 * "KV Cache는 왜 LLM 서빙의 핵심인가", section "KV Cache: O(T²)를 O(T)로": the append
 * of the new token's k_t, v_t in each decode step (see file header).
 *   k, v          bf16 [n_tok][n_kv][head_dim]
 *   slot_mapping  int64 [n_tok]; slot = physical block * block_size + row.
 *                 A negative slot is padding and is skipped.  Slots must be distinct.
 *   k_pool,v_pool bf16 [num_blocks][n_kv][block_size][head_dim], updated in place.
 * Bit-exact copy.  A slot >= num_blocks * block_size sets PKV_DEV_BAD_SLOT.
 */
pkv_status pkv_kv_append(const void* k, const void* v, const int64_t* slot_mapping, int n_tok,
                         void* k_pool, void* v_pool, int num_blocks, int block_size, int n_kv,
                         int head_dim, int32_t* err_flag, void* stream);

/*
 * Bytes of workspace pkv_paged_decode_attn (int4 = 0) or pkv_paged_decode_attn_int4
 * (int4 = 1) needs for this shape on the current device.  0 on an invalid shape.
 */
size_t pkv_decode_workspace_bytes(int batch, int n_h, int n_kv, int head_dim, int block_size, int int4);

/*
 * paged_decode_attn — one decode step of attention over a paged bf16 cache.
 * "KV Cache는 왜 LLM 서빙의 핵심인가", section "KV Cache: O(T²)를 O(T)로": the attention
 * of each decode step over the whole cache; PagedAttention blocks; GQA groups (see file
 * header).
 *   q             bf16 [batch][n_h][head_dim]
 *   k_pool,v_pool bf16 [num_blocks][n_kv][block_size][head_dim]
 *   block_tables  int32 [batch][max_blocks]; entry i of row s is the physical block
 *                 holding tokens [i*block_size, (i+1)*block_size) of sequence s.
 *                 Entries past ceil(context_lens[s] / block_size) are not read.
 *   context_lens  int32 [batch]; tokens of sequence s, including the one appended
 *                 this step.  0 gives a zero output row.
 *   scale         multiplies q.k before the softmax (1/sqrt(head_dim) for the usual layer)
 *   out           [batch][n_h][head_dim], bf16 (out_dtype PKV_OUT_BF16, round to
 *                 nearest even) or fp32 (PKV_OUT_F32)
 *   workspace     device scratch of at least pkv_decode_workspace_bytes(..., 0) bytes,
 *                 256-byte aligned; its contents on entry do not matter.
 * Arithmetic: q.k and p.v products in fp32 (tensor-core mma, bf16 inputs, fp32
 * accumulate; p is carried as a bf16 high + low pair), softmax online in fp32.
 * The result depends only on the logical token order, never on which physical
 * blocks hold the tokens.
 * Kernel choice: groups of 17-32 query heads at head_dim 128 run, when the environment
 * variable PKV_ATTN_KERNEL is "tc" at the time of the call, on the fifth-generation tensor
 * cores (tcgen05.mma, 128-token tiles, accumulators in tensor memory, one CTA per SM);
 * otherwise, and for every other shape, on warp-level mma.sync kernels (several CTAs per
 * SM), which measured faster on that shape.  Same arithmetic and bounds either way.
 * The first call of a kernel variant on the device sets its shared-memory attribute and
 * queries occupancy (host-side calls, no stream work); to capture the call into a CUDA
 * graph, make one call of the same shape on the stream before the capture begins.
 */
pkv_status pkv_paged_decode_attn(const void* q, const void* k_pool, const void* v_pool,
                                 const int32_t* block_tables, int max_blocks,
                                 const int32_t* context_lens, float scale, int batch, int n_h,
                                 int n_kv, int head_dim, int block_size, int num_blocks,
                                 void* out, int out_dtype, void* workspace, size_t workspace_bytes,
                                 int32_t* err_flag, void* stream);

/*
 * paged_decode_attn_window — pkv_paged_decode_attn for a layer with a limited
 * attention window.  "KV 캐시 시스템 (KV Cache System)", sections "제한된 어텐션 윈도우
 * 크기 (Limited Attention Window Size)" and "어텐션 윈도우 크기" (max_attention_window).
 *   window        tokens the query attends to: the last `window` tokens of the
 *                 context, [context_lens[s] - window, context_lens[s]); 0 means the
 *                 whole context (the call is then pkv_paged_decode_attn).  Negative:
 *                 PKV_EINVAL.
 *   Table entries of blocks that end before the window are not read (they may hold
 *   released or reused block ids).  Every other argument, the workspace size and the
 *   arithmetic: as pkv_paged_decode_attn.
 */
pkv_status pkv_paged_decode_attn_window(const void* q, const void* k_pool, const void* v_pool,
                                        const int32_t* block_tables, int max_blocks,
                                        const int32_t* context_lens, float scale, int window,
                                        int batch, int n_h, int n_kv, int head_dim, int block_size,
                                        int num_blocks, void* out, int out_dtype, void* workspace,
                                        size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * paged_decode_attn_noalloc — pkv_paged_decode_attn without a caller workspace.
 * The reference pages have no counterpart: this entry point exists for callers that
 * cannot allocate device memory when they decode (an engine that gave all free memory
 * to its KV pool, a host program that only receives device pointers from another
 * runtime, code that must not reach an allocator on its hot path).  Its scratch space
 * is a fixed array of PKV_STATIC_SCRATCH_BYTES inside the library, held on every GPU
 * that loads the library until the process exits; the call allocates nothing.
 *   Arguments, layouts, output and device errors: as pkv_paged_decode_attn, minus the
 *   workspace.  Returns PKV_ERANGE, without launching anything, when this shape needs
 *   more scratch than the array holds (pkv_decode_workspace_bytes(..., 0) >
 *   PKV_STATIC_SCRATCH_BYTES).
 *   The first call with a given device current looks up the array's device address
 *   for that device (and looks it up again when the current context has changed, as
 *   after a device reset); make that call before any stream capture.
 *   All calls share the array: calls whose GPU work can overlap (other streams, other
 *   host threads) race on it and must be serialised by the caller.
 */
#define PKV_STATIC_SCRATCH_BYTES (16u * 1024u * 1024u)
pkv_status pkv_paged_decode_attn_noalloc(const void* q, const void* k_pool, const void* v_pool,
                                         const int32_t* block_tables, int max_blocks,
                                         const int32_t* context_lens, float scale, int batch,
                                         int n_h, int n_kv, int head_dim, int block_size,
                                         int num_blocks, void* out, int out_dtype,
                                         int32_t* err_flag, void* stream);

/*
 * layer_window — the attention window of one layer from a max_attention_window list.
 * "KV 캐시 시스템 (KV Cache System)", section "어텐션 윈도우 크기": the list gives one
 * window per layer and is repeated over the layers when it has fewer entries than the
 * model has layers, so layer l takes windows[l % n].  A window at least as long as a
 * context is full attention for it (pkv_paged_decode_attn_window).
 *   windows  host int32 [n], every entry > 0
 * Returns the window (> 0), or -1 for a NULL list, n <= 0, layer < 0 or an entry <= 0.
 */
int pkv_layer_window(const int32_t* windows, int n, int layer);

/*
 * kv_quant_append_int4 — quantize-on-append into an INT4 paged cache.
 * "KVQuant: 마지막 4배": K per channel, V per token, s = (max - min) / 15.
 * Exact op sequence (codes are bit-exact against it):
 *   lo, hi = fp32 min / max of the group (a zero lo is taken as +0);
 *   s32 = (hi - lo) / 15 (fp32, nearest);
 *   s16 = fp16(s32), m16 = fp16(lo) (nearest even);
 *   code = clamp(rint_half_even((x - m16) / s16), 0, 15) (fp32 subtract / divide; the
 *     kernel takes the quotient from the rounded reciprocal away from ties, which gives the
 *     same codes),
 *   code = 0 when s16 == 0; the dequantized value is x^ = code * s16 + m16, exact.
 * Groups: V = the head_dim channels of one (token, kv head); K = one channel of one
 * (block, kv head) over the block's block_size rows.  K rows of a block that is not
 * yet full stay in bf16 in `k_tail`; when a call appends a block's last row, the
 * whole block is quantized from the rows appended earlier in the same call and the
 * tail rows, and the tail is left as it was.
 *   k, v          bf16 [n_tok][n_kv][head_dim]
 *   slot_mapping  int64 [n_tok] (negative = padding); tail_seq int32 [n_tok]: the
 *                 tail row (batch index) of each token's sequence, in [0, tail_rows).
 *   cache         uint8 [num_blocks][n_kv][R], R = pkv_int4_record_bytes(block_size,
 *                 head_dim): one record per (block, kv head), read by the attention
 *                 kernel as one contiguous copy.  Byte offsets inside a record:
 *                   0              K codes  [block_size][head_dim/2]
 *                   bs*d/2         V codes  [block_size][head_dim/2]
 *                   bs*d           K meta   fp16 [2][head_dim]: scale row, then min row
 *                   bs*d + 4d      V meta   fp16 [block_size][2]: (scale, min) per token
 *                 A code row packs 8 channels per little-endian 32-bit word: nibble n of
 *                 word w holds channel 8w + (0,2,4,6,1,3,5,7)[n] (even channels in the
 *                 low half-word).  The K codes and K meta of a block not yet full are
 *                 not defined.
 *   k_tail        bf16 [tail_rows][n_kv][block_size][head_dim].
 * Caller contract: slots distinct; within one call the tokens of a sequence are
 * consecutive entries in logical order with one tail_seq; a sequence starts at
 * row 0 of its first block.  Values must lie within fp16 range.
 * Enqueues two kernels (quantize, then tail update) on `stream`.
 */
pkv_status pkv_kv_quant_append_int4(const void* k, const void* v, const int64_t* slot_mapping,
                                    const int32_t* tail_seq, int n_tok, uint8_t* cache, void* k_tail,
                                    int tail_rows, int num_blocks, int block_size, int n_kv,
                                    int head_dim, int32_t* err_flag, void* stream);

/*
 * Bytes of one (block, kv head) record of the INT4 cache: block_size * head_dim (codes
 * of K and V) + 4 * head_dim (K scale and min rows) + 4 * block_size (V scale and min per
 * token); a multiple of 16.  0 on a shape the INT4 kernels do not take.
 */
size_t pkv_int4_record_bytes(int block_size, int head_dim);

/*
 * paged_decode_attn_int4 — decode attention over the INT4 cache written by
 * pkv_kv_quant_append_int4, equal to the attention over the exact x^ = code * s + m
 * up to fp32 accumulation: no value is dequantized.  Per block, K's per-channel scale is
 * folded into q (q * s as an fp16 pair, high part + exact residual) against the codes as
 * exact small integers, and the block's sum of q * min is one more product; V's per-token
 * scale is folded into the softmax weights (p * s as a bf16 high + low pair) against the
 * codes, and sum_t p_t * (min_t + 8 s_t) is added per head at the end.  The last,
 * unfinished block of sequence s takes its K rows from k_tail[s] (bf16) and its V rows
 * from the codes.
 * Same arguments and output as pkv_paged_decode_attn, with the INT4 cache and the
 * K tail in place of the pools; the batch index is the tail row.  q.k uses fp16 and p.v
 * bf16 tensor-core mma with fp32 accumulation.  q, the tail and every product q_c * s_c
 * must lie in fp16 range.
 */
pkv_status pkv_paged_decode_attn_int4(const void* q, const uint8_t* cache, const void* k_tail,
                                      const int32_t* block_tables,
                                      int max_blocks, const int32_t* context_lens, float scale,
                                      int batch, int n_h, int n_kv, int head_dim, int block_size,
                                      int num_blocks, void* out, int out_dtype, void* workspace,
                                      size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * paged_decode_attn_int4_window — pkv_paged_decode_attn_int4 over the last `window`
 * tokens of each context (0: the whole context), with the window read as for
 * pkv_paged_decode_attn_window: the records and table entries of blocks that end before
 * the window are not read.
 */
pkv_status pkv_paged_decode_attn_int4_window(const void* q, const uint8_t* cache, const void* k_tail,
                                             const int32_t* block_tables,
                                             int max_blocks, const int32_t* context_lens, float scale,
                                             int window, int batch, int n_h, int n_kv, int head_dim,
                                             int block_size, int num_blocks, void* out, int out_dtype,
                                             void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                             void* stream);

/*
 * rope_shift_k — re-rotate the keys of reused chunks in place.
 * "Research Paper Review : CACHE BLEND ...", section "Background" (full KV reuse).
 * Every row and kv head of block block_ids[i] is rotated by position deltas[i]:
 * channel pairs (j, j + head_dim/2), angle deltas[i] * rope_base^(-2j/head_dim),
 *   x_j' = x_j cos - x_{j+d/2} sin,  x_{j+d/2}' = x_j sin + x_{j+d/2} cos,
 * angle reduced in fp64, rotation in fp32, stored bf16 (nearest even).
 * A delta of 0 leaves the block untouched.  block_ids must be distinct; an id
 * outside [0, num_blocks) sets PKV_DEV_BAD_BLOCK and is skipped.
 *   k_pool   bf16 [num_blocks][n_kv][block_size][head_dim]
 *   block_ids, deltas  int32 [n_blocks]
 */
pkv_status pkv_rope_shift_k(void* k_pool, const int32_t* block_ids, const int32_t* deltas,
                            int n_blocks, int num_blocks, int n_kv, int block_size, int head_dim,
                            double rope_base, int32_t* err_flag, void* stream);

/*
 * Rotary positions of new tokens.
 *
 * rope_init — the angle table of a rotary embedding (host).  Channel pair j < rotary_dim / 2
 * turns by pos * inv_j, inv_j = base^(-2j / rotary_dim) before scaling; channels from
 * rotary_dim on are copied.  Pairs are (j, j + rotary_dim / 2), or (2j, 2j + 1) with
 * interleaved != 0.  Scalings for contexts `factor` times the trained length:
 *   PKV_ROPE_NONE    inv_j as it is (factor ignored)
 *   PKV_ROPE_LINEAR  inv_j / factor
 *   PKV_ROPE_NTK     base * factor^(r / (r - 2)) in place of base, r = rotary_dim
 *   PKV_ROPE_PARTS   w inv_j + (1 - w) inv_j / factor, w = (turns - low) / (high - low) clamped
 *                    to [0, 1], turns = original_len * inv_j / (2 pi): the turns that the pair
 *                    makes over the trained length
 *   PKV_ROPE_YARN    the same blend with w falling linearly with j, from 1 at pair
 *                    floor(c(high)) to 0 at pair ceil(c(low)), c(t) = r ln(original_len /
 *                    (2 pi t)) / (2 ln base), both clamped to [0, r - 1]; cos and sin are
 *                    multiplied by 0.1 ln(factor) + 1
 * amplitude > 0 replaces that multiplier (1 for the other scalings).
 * The table holds turns per position as 64-bit fractions, so pos * inv_j modulo one turn is
 * exact for every int32 position, also negative ones; it is plain data (copy it freely).
 * PKV_EINVAL: head_dim not 64 or 128, rotary_dim not a multiple of 16 in [16, head_dim], base
 * <= 1, factor < 1, and for the last two scalings original_len <= 0 or not 0 < low < high.
 */
#define PKV_ROPE_NONE   0
#define PKV_ROPE_LINEAR 1
#define PKV_ROPE_NTK    2
#define PKV_ROPE_PARTS  3
#define PKV_ROPE_YARN   4
typedef struct {
  int32_t head_dim, rotary_dim, interleaved, scaling;
  double base, factor, original_len, low, high, amplitude;
} pkv_rope_config;
typedef struct {
  int32_t head_dim, rotary_dim, interleaved;
  float amplitude;
  uint64_t turns[64];
} pkv_rope_table;
pkv_status pkv_rope_init(const pkv_rope_config* config, pkv_rope_table* table);

/*
 * rope_append — rotate a step's queries and keys by their positions and append the keys and
 * values to the bf16 cache, in one pass (pkv_kv_append with the rotation in front of it).
 *   q, k, v       bf16 [n_tok][heads][head_dim] with q_stride / k_stride / v_stride elements
 *                 between tokens (multiples of 8, at least heads * head_dim): parts of one
 *                 fused projection output are taken as they lie
 *   positions     int32 [n_tok]
 *   slot_mapping  int64 [n_tok], as for pkv_kv_append.  A negative slot is padding: nothing of
 *                 the token is written, its q_out row neither.
 *   q_out         bf16, q_out_stride elements between tokens; may be q itself (with its stride)
 *   k_pool,v_pool as for pkv_kv_append
 * The rotation runs in fp32 and rounds once, to nearest even; copied channels and V are
 * bit-exact.  A slot >= num_blocks * block_size sets PKV_DEV_BAD_SLOT and skips the token.  n_h and
 * n_kv are at most 1024.
 */
pkv_status pkv_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping, int n_tok,
                           const pkv_rope_table* table, void* q_out, int64_t q_out_stride, void* k_pool,
                           void* v_pool, int num_blocks, int block_size, int n_h, int n_kv, int head_dim,
                           int32_t* err_flag, void* stream);

/*
 * rope_qk — the rotation alone (ahead of a quantizing append): q_out and k_out get the rotated
 * heads, with strides as above; each may be its input.
 */
pkv_status pkv_rope_qk(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const int32_t* positions,
                       int n_tok, const pkv_rope_table* table, void* q_out, int64_t q_out_stride, void* k_out,
                       int64_t k_out_stride, int n_h, int n_kv, int head_dim, void* stream);

/*
 * The 8-bit cache: codes of 8 bits with one fp32 scale per (block, kv head) for K and one for V.
 *
 * kv_quant_append_q8 — quantize-on-append.  Exact op sequence, in fp32, per (block, kv head) and
 * for K and V apart, over the rows that the block holds after the call:
 *   big = max |x|;  scale = big * (1 / M) and inv = (1 / big) * M, each operation rounded to
 *   nearest, M = 448 (PKV_Q8_E4M3) or 127 (PKV_Q8_INT8); both are 0 when big < 2^-110
 *   code = e4m3(x * inv), nearest even, saturating; or rint(x * inv) clamped to +-127
 * and the value held is code * scale.  A block's codes depend on its rows alone, not on the calls
 * that brought them: the bf16 rows of a sequence's unfinished block are kept in k_tail / v_tail,
 * and each append writes the record anew from them and its own tokens.
 *   k, v          bf16 [n_tok][n_kv][head_dim], k_stride / v_stride elements between tokens
 *                 (multiples of 8)
 *   slot_mapping  int64 [n_tok] (negative = padding); tail_seq int32 [n_tok]: the tail row of
 *                 each token's sequence, in [0, tail_rows)
 *   cache         uint8 [num_blocks][n_kv][R], R = pkv_q8_record_bytes(block_size, head_dim) =
 *                 2 bs d + 16: K codes [bs * d], V codes [bs * d], K scale, V scale (fp32), 8
 *                 bytes of zeros.  Codes are stored per 16-token tile in the order in which a
 *                 warp's lanes hold the operands of mma.m16n8k16: lane 4 i + j of a group of 32
 *                 channels has 16 bytes; byte 8 a + 4 b + 2 c + e of it is
 *                   K: token 8 b + i, channel 16 a + 8 c + 2 j + e
 *                   V: token 8 c + 2 j + e, channel 16 a + 8 b + i
 *                 with the groups of a tile and the tiles of a block one after another.  Rows
 *                 not yet appended have codes 0.
 *   k_tail,v_tail bf16 [tail_rows][n_kv][block_size][head_dim], read and written
 * Caller contract: as for pkv_kv_quant_append_int4 (slots distinct; within a call the tokens of a
 * sequence are consecutive entries in logical order with one tail_seq; a sequence starts at row 0
 * of its first block); values finite (a NaN is lost in INT8 and stays NaN in E4M3, an infinity
 * spoils its block); n_tok <= 0x7fff0000.  A sequence may be cut back inside its unfinished block (the tail still holds
 * the rows that remain), not into a finished one.  A slot or tail row out of range sets PKV_DEV_BAD_SLOT and is skipped.
 */
#define PKV_Q8_E4M3 0
#define PKV_Q8_INT8 1
size_t pkv_q8_record_bytes(int block_size, int head_dim);
pkv_status pkv_kv_quant_append_q8(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                  const int64_t* slot_mapping, const int32_t* tail_seq, int n_tok, int format,
                                  uint8_t* cache, void* k_tail, void* v_tail, int tail_rows, int num_blocks,
                                  int block_size, int n_kv, int head_dim, int32_t* err_flag, void* stream);

/*
 * paged_decode_attn_q8 — decode attention over the records written by pkv_kv_quant_append_q8,
 * equal to the attention over the values held (code * scale) up to fp32 accumulation: the scales
 * are taken out of the products, the codes enter the tensor cores exactly (as fp16), q exactly up
 * to 2^-39 of its head's largest value, p as a high + low fp16 pair (22 bits, down to 2^-31); for a
 * bf16 output and groups of over four query heads p is rounded to fp16 once (an error of at most
 * 2^-11 sum p |v|, under the output's own rounding wherever its terms do not cancel).
 * window as for pkv_paged_decode_attn_window (0: the whole context).  Other arguments, output and
 * errors as for pkv_paged_decode_attn; workspace of pkv_q8_workspace_bytes (0: invalid shape).
 * The tails are not read; max_blocks * block_size is at most 0x7fff0000 (PKV_ERANGE).
 */
size_t pkv_q8_workspace_bytes(int batch, int n_h, int n_kv, int head_dim, int block_size, int format);
pkv_status pkv_paged_decode_attn_q8(const void* q, const uint8_t* cache, int format, const int32_t* block_tables,
                                    int max_blocks, const int32_t* context_lens, float scale, int window, int batch,
                                    int n_h, int n_kv, int head_dim, int block_size, int num_blocks, void* out,
                                    int out_dtype, void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                    void* stream);

/*
 * paged_decode_attn_mass — pkv_paged_decode_attn that also adds, for each token t of sequence s
 * and kv head g, the attention weights it got from the group's query heads to an account:
 *   mass[(s * n_kv + g) * mass_stride + t] += sum over h in g of p[s][h][t],  t < context_lens[s]
 * in fp32 and in a fixed order (the same bits on every call).  p is carried with all of its 24 bits
 * as three bf16 parts; for a bf16 output and groups of over eight query heads as a high + low pair
 * (16 bits: an error of at most 2^-17 sum p |v| of the output; the accounts always get all bits).
 * Entries at or behind the context are left as they were.  The accounts are per sequence, also where
 * sequences share blocks.
 *   mass          fp32, mass_stride >= max_blocks * block_size
 *   workspace     pkv_mass_workspace_bytes bytes (it holds the step's scores: 4 n_h bytes per
 *                 token of max_blocks * block_size, so a table no wider than needed is better; 0:
 *                 invalid shape), 256-byte aligned
 * Tokens of a bad block weigh nothing; max_blocks * block_size is at most 0x7fff0000 (PKV_ERANGE).
 * Other arguments and errors as for pkv_paged_decode_attn.
 */
size_t pkv_mass_workspace_bytes(int batch, int n_h, int n_kv, int head_dim, int block_size, int max_blocks);
pkv_status pkv_paged_decode_attn_mass(const void* q, const void* k_pool, const void* v_pool,
                                      const int32_t* block_tables, int max_blocks, const int32_t* context_lens,
                                      float scale, int batch, int n_h, int n_kv, int head_dim, int block_size,
                                      int num_blocks, void* out, int out_dtype, float* mass, int64_t mass_stride,
                                      void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * kv_evict — cut sequences of the bf16 cache to a budget of rows by the accounts above.
 * For each sequence s with n = context_lens[s] > K = max(0, keep[s]), and each kv head g apart,
 * K rows stay: those that hold one of the sequence's last min(recent, K) tokens, then those with
 * the largest mass (equal mass: lowest row first; NaN above +inf, -0 below +0).  Kept rows below K stay in place; the kept rows
 * at or behind K are moved, in ascending order, into the other rows below K, in ascending order
 * (attention does not depend on the order of rows; a limited attention window does, so it has no
 * meaning on a sequence after an eviction).  Sequences with n <= K are left as they are.
 * State, per sequence and kv head (rows of `stride` >= max_blocks * block_size entries):
 *   mass       fp32: moved with the rows; rows [K, n) become 0, so later tokens start at 0
 *   positions  int32: the token each row r < kept[s] holds (counting from the sequence's start);
 *              row r >= kept[s] holds token dropped[s] + r
 *   kept       int32 [batch]: rows that the last eviction left (0 at the start)
 *   dropped    int32 [batch]: tokens evicted so far (0 at the start)
 * The new state goes to the _out pointers: all four equal to the inputs (in place), or none, and then
 * without overlap with them, the lengths or the budgets (PKV_EINVAL).
 * Entries of mass_out behind n, and of positions_out behind the new kept, are left as they were.
 *   new_lens   int32 [batch]: min(n, K); must not overlap context_lens, keep or the old or new kept and
 *              dropped
 *   workspace  pkv_evict_workspace_bytes bytes, 256-byte aligned
 * max_blocks * block_size is at most 0x7fff0000 (PKV_ERANGE); the work is laid out for that many
 * rows, so give a table no wider than the longest sequence needs.
 * The blocks that hold the first K rows are rewritten: they must belong to the sequence alone.
 * Nothing here can tell; pkv_bm_evict does, and is called before this (see there).  Moves from or to a
 * block id outside the pool set PKV_DEV_BAD_BLOCK and are skipped; context lengths out of range are clamped with PKV_DEV_BAD_CTX.
 */
size_t pkv_evict_workspace_bytes(int batch, int n_kv, int block_size, int max_blocks);
pkv_status pkv_kv_evict(void* k_pool, void* v_pool, const int32_t* block_tables, int max_blocks,
                        const int32_t* context_lens, const int32_t* keep, int recent, const float* mass,
                        const int32_t* positions, const int32_t* kept, const int32_t* dropped, float* mass_out,
                        int32_t* positions_out, int32_t* kept_out, int32_t* dropped_out, int64_t stride,
                        int32_t* new_lens, int batch, int n_kv, int head_dim, int block_size, int num_blocks,
                        void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * Several tokens of a sequence in one step: drafted tokens that form a chain or a tree.
 *
 * A step's tokens lie one sequence after another; q_start int32 [batch + 1] gives each sequence's
 * first token, so sequence s has n = q_start[s + 1] - q_start[s] of them (0 is allowed; tokens in
 * front of the first sequence or behind the last one belong to none, and their output rows are left
 * as they were).  q_start NULL: every sequence has n_tok / batch tokens (n_tok a multiple of batch).
 * Their rows are in the cache before the attention: they are its last n rows, and context_lens[s]
 * counts them.  Token i attends to all rows before the n, and of the n to
 *   tree_mask NULL: its own and the earlier ones (a chain)
 *   else          : those j with bit (j & 63) of tree_mask[token * mask_words + (j >> 6)] set (its
 *                   ancestors and itself, for a tree); rows past 64 * mask_words are not attended.
 * A token with nothing to attend to gets a zero output row; so do the tokens of a sequence of
 * context length 0.  Where 0 < context_lens[s] < n the first n - context_lens[s] tokens' rows are taken
 * as missing, with PKV_DEV_BAD_TREE.  A range of q_start that is out of order or outside [0, n_tok] gives
 * its sequence no tokens, with PKV_DEV_BAD_TREE.
 *
 * paged_tree_attn — pkv_paged_decode_attn for such tokens.
 *   q             bf16 [n_tok][n_h][head_dim]
 *   q_start       int32 [batch + 1] or NULL
 *   tree_mask     int64 [n_tok][mask_words] or NULL (mask_words is ignored then)
 *   out           [n_tok][n_h][head_dim]; neither it nor the workspace may overlap the other arguments (PKV_EINVAL)
 *   workspace     pkv_tree_workspace_bytes bytes (0: invalid shape), 256-byte aligned; a call of other
 *                 n_tok or batch may need another size
 * Softmax and sums are fp32 and taken in a fixed order (the same bits on every call).  p is carried in bf16 parts: all
 * of its 24 bits in three for an fp32 output, in two for a bf16 output (an error of at most 2^-16 sum p |v|).  Cached rows
 * that no token of the sequence attends to do not
 * reach any output, whatever they hold; a row that some of its tokens attend to and others mask has to
 * hold finite values (0 times an infinity of V is no number).  A score of minus infinity has weight zero, and a
 * token that has no other a zero output row.  Weights are held as exp(score - c) with a c that may lie
 * 2^32 in weight below the largest until the end, so values of V beyond 2^95 / context_lens[s] may overflow.  Pools, tables, lengths, scale, other
 * errors and the first call of a shape as for pkv_paged_decode_attn; max_blocks * block_size is at most
 * 0x7fff0000 and n_tok * n_h at most 0x7fffffff (PKV_ERANGE).
 */
size_t pkv_tree_workspace_bytes(int batch, int n_tok, int n_h, int n_kv, int head_dim, int block_size);
pkv_status pkv_paged_tree_attn(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                               int max_blocks, const int32_t* context_lens, const int32_t* q_start,
                               const int64_t* tree_mask, int mask_words, float scale, int n_tok, int batch, int n_h,
                               int n_kv, int head_dim, int block_size, int num_blocks, void* out, int out_dtype,
                               void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * kv_tree_accept — keep the accepted path of each sequence's drafted tokens: for i < n_accept[s] the
 * cache row of drafted token path[s][i] becomes row base + i, base = context_lens[s] - n, in every given
 * cache; the rows behind are no longer part of the sequence.  (The drafted keys were rotated by their
 * depth in the tree, which is where an accepted path puts them.)
 *   caches        HOST array of n_caches device pointers to caches of one shape,
 *                 [num_blocks][heads][block_size][row_bytes]: the K and V pools of every layer, or the latent
 *                 caches (heads = 1).  They must not overlap (PKV_EINVAL).  row_bytes is a multiple of 16
 *   q_start, n_tok, batch as above
 *   path          int32 [batch][path_stride]: drafted tokens in ascending order (a tree lists parents before
 *                 children), at least n_accept[s] of them
 *   n_accept      int32 [batch], 0 .. min(n, path_stride)
 *   new_lens      int32 [batch]: base + n_accept[s]; must not overlap context_lens, n_accept, path or q_start
 * An entry that is not larger than the one before it, or not below n, ends the path there, with
 * PKV_DEV_BAD_TREE (so does n_accept out of range, which is clamped); a sequence with more drafted tokens than
 * rows keeps its length, with the same flag (but for a padded one: length 0 and n_accept 0).  The blocks that hold the drafted rows must belong to the sequence alone, and
 * stay so until the path is decided on: pkv_bm_append_drafts and pkv_bm_accept_drafts of pkv_bm.h see to it.  A
 * move from or to a block id outside the pool sets PKV_DEV_BAD_BLOCK and is skipped.
 */
pkv_status pkv_kv_tree_accept(void* const* caches, int n_caches, int row_bytes, int heads, const int32_t* block_tables,
                              int max_blocks, const int32_t* context_lens, const int32_t* q_start, int n_tok,
                              const int32_t* path, int path_stride, const int32_t* n_accept, int32_t* new_lens, int batch,
                              int block_size, int num_blocks, int32_t* err_flag, void* stream);

/*
 * The latent cache: one vector per token for all heads, bf16 [num_blocks][block_size][latent + rope]: the
 * latent part, from which a layer's keys and values are linear maps, and a key part with rotary positions
 * that all heads share.  With the maps taken into the query and the output projection (the absorbed form),
 * attention runs on the vectors themselves.
 * latent is 256 or 512, rope 32 or 64.
 *
 * latent_append — normalise, rotate and write a step's vectors, and rotate the queries' position part.
 *   kv            bf16 [n_tok][latent + rope], kv_stride elements between tokens: part of a projection's output
 *   q             bf16 [n_tok][n_h][rope], q_stride / q_head_stride elements between tokens / heads
 *   table         of pkv_rope_init with rotary_dim = rope
 *   weight        bf16 [latent] or NULL: x * weight / sqrt(mean(x^2) + eps) over the latent part, in
 *                 fp32, rounded once; NULL copies it as it is
 *   q_out         bf16 [n_tok][n_h][rope] with strides (inside the absorbed queries [n_tok][n_h][latent +
 *                 rope], say); may be q itself, with its strides
 *   cache         written at slot_mapping (int64 [n_tok]; negative: padding, nothing of the token is written;
 *                 the others must be distinct)
 * Strides are multiples of 8 elements, a token's heads lie within its stride (q_stride >= (n_h - 1) * q_head_stride + rope),
 * pointers are 16-byte aligned; but for q_out = q, what is written must not overlap what is read.  A slot >= num_blocks * block_size sets
 * PKV_DEV_BAD_SLOT and skips the token.  n_h is at most 1024.
 */
pkv_status pkv_latent_append(const void* kv, int64_t kv_stride, const void* q, int64_t q_stride, int64_t q_head_stride,
                             const int32_t* positions, const int64_t* slot_mapping, int n_tok,
                             const pkv_rope_table* table, const void* weight, float eps, void* q_out,
                             int64_t q_out_stride, int64_t q_out_head_stride, void* cache, int num_blocks, int block_size,
                             int n_h, int latent, int rope, int32_t* err_flag, void* stream);

/*
 * paged_latent_attn — attention of one or several tokens per sequence over the latent cache:
 *   out[token][h] = sum over attended rows t of softmax_t(scale * q[token][h] . cache[t]) cache[t][:latent]
 *   q             bf16 [n_tok][n_h][latent + rope]; n_h at most 1024
 *   out           [n_tok][n_h][latent]
 * q_start, tree_mask and everything else as for pkv_paged_tree_attn (one token per sequence: q_start NULL and
 * n_tok = batch).
 */
size_t pkv_latent_workspace_bytes(int batch, int n_tok, int n_h, int latent, int rope, int block_size);
pkv_status pkv_paged_latent_attn(const void* q, const void* cache, const int32_t* block_tables, int max_blocks,
                                 const int32_t* context_lens, const int32_t* q_start, const int64_t* tree_mask,
                                 int mask_words, float scale, int n_tok, int batch, int n_h, int latent, int rope,
                                 int block_size, int num_blocks, void* out, int out_dtype, void* workspace,
                                 size_t workspace_bytes, int32_t* err_flag, void* stream);

/*
 * CacheBlend's model-free steps ("Research Paper Review : CACHE BLEND ...", sections
 * "Methods" and "System Design"): the KV deviation of candidate tokens, the selection of
 * the tokens with the largest deviation under the recompute ratio, and the fuse of their
 * recomputed K/V into the cache.  Recomputing K/V needs the model and is the caller's.
 */

/*
 * kv_deviation — dev[i] = L2 distance between the cached K and V of the token at
 * slots[i] and its recomputed rows k_new[i], v_new[i], over all kv heads and channels of
 * K and V together (fp32 accumulation of the squared bf16 differences, then sqrt).
 *   k_pool,v_pool bf16 [num_blocks][n_kv][block_size][head_dim]
 *   slots         int64 [n]
 *   k_new,v_new   bf16 [n][n_kv][head_dim]
 *   dev           fp32 [n] (device)
 * A slot outside the pool sets PKV_DEV_BAD_SLOT and gives dev 0.
 */
pkv_status pkv_kv_deviation(const void* k_pool, const void* v_pool, const int64_t* slots, const void* k_new,
                            const void* v_new, int n, int num_blocks, int block_size, int n_kv, int head_dim,
                            float* dev, int32_t* err_flag, void* stream);

/*
 * select_top — for each segment s = [seg_offsets[s], seg_offsets[s+1]) of dev, the
 * counts[s] elements with the largest values (equal values: lowest index first), written
 * as ascending global indices to out, segment after segment (segment s starts at the sum
 * of the earlier segments' counts).  counts are clamped to [0, segment length].  Values
 * are compared in float32 (NaN above +inf, -0 below +0).
 *   dev fp32 [seg_offsets[n_seg]], seg_offsets int32 [n_seg + 1] (non-decreasing),
 *   counts int32 [n_seg], out int32 [sum of counts]; all device memory.
 */
pkv_status pkv_select_top(const float* dev, const int32_t* seg_offsets, const int32_t* counts, int n_seg,
                          int32_t* out, void* stream);

/*
 * kv_fuse — write the recomputed rows of the selected tokens into the cache:
 * pools[row_slots[rows[j]]] = k_new[rows[j]], v_new[rows[j]] for j < n_sel (rows as
 * pkv_select_top returns them, indexing the candidate rows of k_new / v_new).
 *   k_new,v_new bf16 [n_rows][n_kv][head_dim]; row_slots int64 [n_rows] (the cache slot of
 *   each candidate row); rows int32 [n_sel].
 * A row outside [0, n_rows) or a slot outside the pool sets PKV_DEV_BAD_SLOT and is
 * skipped.  The selected rows' slots must be distinct.
 */
pkv_status pkv_kv_fuse(const void* k_new, const void* v_new, const int64_t* row_slots, int n_rows,
                       const int32_t* rows, int n_sel, void* k_pool, void* v_pool, int num_blocks, int block_size,
                       int n_kv, int head_dim, int32_t* err_flag, void* stream);

/*
 * selftest_wait — exercise the bounded wait that guards every shared-memory ring (the
 * pages have no counterpart: this checks the failure detection of this library).  One
 * thread initialises an mbarrier for one arrival, arrives on it (arrive != 0) or not, and
 * waits for the phase at most limit_us microseconds (1 .. 2 000 000).  A wait that runs out
 * sets PKV_DEV_TIMEOUT in *err_flag (device int32) and the kernel returns normally; the
 * context stays usable.  PKV_EINVAL for a limit out of range or a NULL flag.
 */
pkv_status pkv_selftest_wait(int arrive, int limit_us, int32_t* err_flag, void* stream);

/*
 * probe_read / probe_copy — the HBM bandwidth ceilings the decode kernels are measured
 * against (the pages have no counterpart: these measure the denominator of the roofline
 * fractions).  probe_read streams `bytes` from `buf` with 16-byte loads over a persistent
 * grid (every SM's resident blocks, several loads in flight per thread) and folds the
 * words into a value that is stored to *sink only in a case no data in practice gives;
 * probe_copy copies `bytes` from `src` to `dst` with 16-byte loads and stores.  Time them
 * with events on `stream` over buffers many times the L2: read GB/s = bytes / time,
 * copy GB/s = 2 * bytes / time.
 *   buf, src, dst  device memory, 16-byte aligned; src and dst must not overlap
 *   bytes          a multiple of 16, > 0
 *   sink           device uint32 or NULL
 * PKV_EINVAL on a bad pointer, size or overlap.
 */
pkv_status pkv_probe_read(const void* buf, size_t bytes, uint32_t* sink, void* stream);
pkv_status pkv_probe_copy(const void* src, void* dst, size_t bytes, void* stream);

/* The recompute ratio max(15%, load_time / full_recompute_time), at most 1: the ratio at
 * which recomputing the selected tokens takes as long as loading the layer's KV
 * ("System Design"), recompute time taken as proportional to the tokens recomputed. */
double pkv_recompute_ratio(double load_time, double full_recompute_time);
/* Tokens selected out of n at a ratio: ceil(ratio * n), within [0, n]. */
int pkv_select_count(double ratio, int n);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H_ */
