// Attention of several query tokens per sequence over the paged cache, and over the latent cache.
// The simplest form: a CTA per (token, head) whose warps take every eighth row of the cache.
#include <cmath>

#include "drafts.cuh"
#include "nvtx_range.h"

namespace pkv {

struct RowsArgs {
  const __nv_bfloat16 *q, *k, *v;                // latent: v == k
  const int32_t *bt, *ctx, *q_start;
  const int64_t* mask;
  int max_blocks, max_ctx, mask_words, n_tok, batch, n_h, n_kv, G, bs_log2, num_blocks, n_each, w;
  float scale_log2;
  void* out;
  int out_f32;
  int32_t* err;
};

template <int DK, int DV>
__global__ void __launch_bounds__(256) rows_simple_kernel(const RowsArgs a) {
  constexpr int CK = DK / 32, CV = DV / 32;
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tok = blockIdx.x / a.n_h, h = blockIdx.x % a.n_h, g = h / a.G;
  __shared__ float sm[8], sl[8], so[8][DV];
  int s = -1, flags = 0;
  Drafts d = {};
  for (int c = 0; c < a.batch; ++c) {
    const Drafts x = drafts_of(a.ctx, a.q_start, a.n_each, a.n_tok, a.max_ctx, c, flags);
    if (tok >= x.q0 && tok < x.q0 + x.n) {
      s = c;
      d = x;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && flags) set_err(a.err, flags);
  if (s < 0) return;
  const int base = d.ctx - d.n, i = tok - d.q0, bs = 1 << a.bs_log2;
  float q[CK], o[CV], m = -INFINITY, l = 0.f;
  for (int j = 0; j < CK; ++j) {
    const int c = j * 32 + lane;
    q[j] = c < a.w ? __bfloat162float(a.q[((size_t)tok * a.n_h + h) * a.w + c]) : 0.f;
  }
  for (int j = 0; j < CV; ++j) o[j] = 0.f;
  for (int t = warp; t < d.ctx; t += 8) {
    const int j = t - base;
    if (j >= 0) {
      if (!a.mask ? j > i : (j >= 64 * a.mask_words || !((a.mask[(size_t)tok * a.mask_words + (j >> 6)] >> (j & 63)) & 1))) continue;
    }
    const int b = a.bt[(size_t)s * a.max_blocks + (t >> a.bs_log2)];
    if ((unsigned)b >= (unsigned)a.num_blocks) {
      if (lane == 0) set_err(a.err, PKV_DEV_BAD_BLOCK);
      continue;
    }
    const size_t row = (((size_t)b * a.n_kv + g) << a.bs_log2) + (t & (bs - 1));
    float x = 0.f;
    for (int c = 0; c < CK; ++c)
      if (c * 32 + lane < a.w) x += q[c] * __bfloat162float(a.k[row * a.w + c * 32 + lane]);
    for (int z = 16; z; z >>= 1) x += __shfl_xor_sync(FULL_MASK, x, z);
    x *= a.scale_log2;
    const float mn = fmaxf(m, x), al = ex2(m - mn), p = ex2(x - mn);
    m = mn;
    l = l * al + p;
    for (int c = 0; c < CV; ++c) o[c] = o[c] * al + p * __bfloat162float(a.v[row * a.w + c * 32 + lane]);
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int c = 0; c < CV; ++c) so[warp][c * 32 + lane] = o[c];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w]);
  if (M == -INFINITY) M = 0.f;
  for (int w = 0; w < 8; ++w) L += sl[w] * ex2(sm[w] - M);
  for (int c = threadIdx.x; c < DV; c += 256) {
    float x = 0.f;
    for (int w = 0; w < 8; ++w) x += so[w][c] * ex2(sm[w] - M);
    x = L == 0.f ? 0.f : x / L;                                 // a sum that is no number stays one
    const size_t at = ((size_t)tok * a.n_h + h) * DV + c;
    if (a.out_f32) reinterpret_cast<float*>(a.out)[at] = x;
    else reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(x);
  }
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr long long kRowsMaxCtx = 0x7fff0000LL;

// Checks that both calls share; fills what they share.
static pkv_status rows_args(RowsArgs& a, const void* q, const void* k, const void* v, const int32_t* bt, int max_blocks,
                            const int32_t* ctx, const int32_t* q_start, const int64_t* mask, int mask_words, float scale,
                            int n_tok, int batch, int n_h, int n_kv, int w, int block_size, int num_blocks, void* out,
                            int out_dtype, void* ws, size_t ws_bytes, size_t need, int32_t* err) {
  if (!q || !k || !v || !bt || !ctx || !out || !ws) return PKV_EINVAL;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(out) || (reinterpret_cast<uintptr_t>(mask) & 7u) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u))
    return PKV_EINVAL;
  if ((long long)max_blocks * block_size > kRowsMaxCtx || (long long)n_tok * n_h > 0x7fffffffLL) return PKV_ERANGE;
  if (ws_bytes < need) return PKV_ENOSPC;
  a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.bt = bt; a.ctx = ctx; a.q_start = q_start; a.mask = mask; a.mask_words = mask_words;
  a.max_blocks = max_blocks;
  a.max_ctx = max_blocks * block_size;
  a.n_tok = n_tok; a.batch = batch; a.n_h = n_h; a.n_kv = n_kv; a.G = n_h / n_kv; a.w = w;
  a.bs_log2 = block_size == 16 ? 4 : (block_size == 32 ? 5 : 6);
  a.num_blocks = num_blocks;
  a.n_each = q_start ? 0 : n_tok / batch;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = out;
  a.out_f32 = out_dtype == PKV_OUT_F32;
  a.err = err;
  return PKV_OK;
}
static bool valid_step(int n_tok, int batch, const int32_t* q_start, const int64_t* mask, int mask_words, int out_dtype,
                       int max_blocks, int num_blocks) {
  if (n_tok < 0 || batch < 0 || max_blocks < 0 || num_blocks < 0) return false;
  if (out_dtype != PKV_OUT_BF16 && out_dtype != PKV_OUT_F32) return false;
  if (mask && mask_words < 1) return false;
  return q_start || batch == 0 ? true : n_tok % batch == 0;
}
static bool valid_block(int bs) { return bs == 16 || bs == 32 || bs == 64; }
static bool valid_heads(int n_h, int n_kv, int d, int bs) {
  return n_h > 0 && n_kv > 0 && n_h % n_kv == 0 && n_h / n_kv <= 64 && (d == 64 || d == 128) && valid_block(bs);
}
static bool valid_latent(int n_h, int latent, int rope, int bs) {
  return n_h > 0 && n_h <= 1024 && (latent == 256 || latent == 512) && (rope == 32 || rope == 64) && valid_block(bs);
}
static pkv_status launched(cudaError_t e) {
  if (e == cudaSuccess) return PKV_OK;
  record_cuda_error(e);
  return PKV_ECUDA;
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_tree_workspace_bytes(int batch, int n_tok, int n_h, int n_kv, int head_dim, int block_size) {
  return batch < 0 || n_tok < 0 || !valid_heads(n_h, n_kv, head_dim, block_size) ? 0 : 256;
}

extern "C" pkv_status pkv_paged_tree_attn(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                                          int max_blocks, const int32_t* context_lens, const int32_t* q_start,
                                          const int64_t* tree_mask, int mask_words, float scale, int n_tok, int batch,
                                          int n_h, int n_kv, int head_dim, int block_size, int num_blocks, void* out,
                                          int out_dtype, void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                          void* stream) {
  PKV_NVTX("pkv_paged_tree_attn");
  if (!valid_heads(n_h, n_kv, head_dim, block_size) ||
      !valid_step(n_tok, batch, q_start, tree_mask, mask_words, out_dtype, max_blocks, num_blocks))
    return PKV_EINVAL;
  if (n_tok == 0 || batch == 0) return PKV_OK;
  RowsArgs a;
  const pkv_status st = rows_args(a, q, k_pool, v_pool, block_tables, max_blocks, context_lens, q_start, tree_mask, mask_words,
                                  scale, n_tok, batch, n_h, n_kv, head_dim, block_size, num_blocks, out, out_dtype, workspace,
                                  workspace_bytes, pkv_tree_workspace_bytes(batch, n_tok, n_h, n_kv, head_dim, block_size), err_flag);
  if (st != PKV_OK) return st;
  void* kargs[] = {&a};
  return launched(launch_pdl(head_dim == 128 ? (const void*)rows_simple_kernel<128, 128> : (const void*)rows_simple_kernel<64, 64>,
                             dim3(n_tok * n_h), dim3(256), 0, static_cast<cudaStream_t>(stream), kargs));
}

extern "C" size_t pkv_latent_workspace_bytes(int batch, int n_tok, int n_h, int latent, int rope, int block_size) {
  return batch < 0 || n_tok < 0 || !valid_latent(n_h, latent, rope, block_size) ? 0 : 256;
}

extern "C" pkv_status pkv_paged_latent_attn(const void* q, const void* cache, const int32_t* block_tables, int max_blocks,
                                            const int32_t* context_lens, const int32_t* q_start, const int64_t* tree_mask,
                                            int mask_words, float scale, int n_tok, int batch, int n_h, int latent, int rope,
                                            int block_size, int num_blocks, void* out, int out_dtype, void* workspace,
                                            size_t workspace_bytes, int32_t* err_flag, void* stream) {
  PKV_NVTX("pkv_paged_latent_attn");
  if (!valid_latent(n_h, latent, rope, block_size) ||
      !valid_step(n_tok, batch, q_start, tree_mask, mask_words, out_dtype, max_blocks, num_blocks))
    return PKV_EINVAL;
  if (n_tok == 0 || batch == 0) return PKV_OK;
  RowsArgs a;
  const pkv_status st = rows_args(a, q, cache, cache, block_tables, max_blocks, context_lens, q_start, tree_mask, mask_words,
                                  scale, n_tok, batch, n_h, 1, latent + rope, block_size, num_blocks, out, out_dtype, workspace,
                                  workspace_bytes, pkv_latent_workspace_bytes(batch, n_tok, n_h, latent, rope, block_size), err_flag);
  if (st != PKV_OK) return st;
  void* kargs[] = {&a};
  return launched(launch_pdl(latent == 512 ? (const void*)rows_simple_kernel<576, 512> : (const void*)rows_simple_kernel<320, 256>,
                             dim3(n_tok * n_h), dim3(256), 0, static_cast<cudaStream_t>(stream), kargs));
}
