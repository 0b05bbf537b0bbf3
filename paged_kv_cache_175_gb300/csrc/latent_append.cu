// Append to the latent cache: the latent part of each token normalised, the shared key part and the
// queries' part rotated by the token's position, the token's vector written at its slot.
//
// Mathematics: y = x w / sqrt(mean(x^2) + eps) in fp32 with one rounding; the rotation and its angles as in
// rope_append.cu (the position times a 64-bit fraction of a turn, exact for every int32 position).
//
// What bounds it: every element is read once and written once.  Long calls of many heads are at HBM (4001 tokens of 128 heads,
// 140 MB: 24.4 us, 5.8 TB/s), of few heads at issue (54% busy: angles, shuffles, conversions) and latency with 32 warps per SM
// (16001 of 16, 103 MB: 20.8 us, 4.9 TB/s), short ones at the launch and two dependent memory round trips
// (position and slot beside the rows, then the stores): 64 tokens of 128 heads 2.3 us.
// Split: a warp per (token, part).  Part 0 is the token's vector: 16 or 8 channels of the latent part
// per lane, whose squares meet in five shuffles, and the key part.  The other parts are runs of
// 32 * NI items of the token's query heads, an item being two 16-byte vectors (eight channel pairs): one item per lane
// while that does not fill the GPU, more where it does, so that a warp's fixed work (position, angles) goes round more
// bytes (16 heads: 24.5 us with one item, 20.8 with two, 21.9 with four; 128 heads: 32.0, 24.8 and 24.4).
// A lane computes the angle of pair `lane`; the eight that an item needs come by shuffles, and are the same
// for all of a lane's items.  All loads are issued before the first use.
#include <cmath>

#include "decode_common.cuh"
#include "nvtx_range.h"

namespace pkv {

struct LatentAppendArgs {
  const __nv_bfloat16 *kv, *q, *weight;
  long long kv_stride, q_stride, qh_stride, qo_stride, qoh_stride;
  __nv_bfloat16 *q_out, *cache;
  const int32_t* positions;
  const int64_t* slots;
  long long n_slots;
  int n_tok, n_h;
  float eps;
  int32_t* err;
  pkv_rope_table t;
};

constexpr int kLatentThreads = 128;

template <int LATENT, int ROPE, int NI>
__global__ void __launch_bounds__(kLatentThreads) latent_append_kernel(const __grid_constant__ LatentAppendArgs a) {
  constexpr int IPH = ROPE / 16, VL = LATENT / 256;           // items per head; latent vectors per lane
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const long long group = (long long)blockIdx.z * gridDim.y + blockIdx.y, t = group * (kLatentThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.n_tok) return;
  const int tok = (int)t, part = blockIdx.x;
  const bool inter = a.t.interleaved != 0;
  const int p = lane % IPH;                                   // this lane's group of eight pairs
  const int va = inter ? 2 * p : p, vb = inter ? 2 * p + 1 : p + IPH;   // its two vectors
  int64_t slot = a.slots[tok];
  const int pos = a.positions[tok];
  uint4 x[NI], y[NI], z[VL], w[VL];
  const int items = a.n_h * IPH, first = (part - 1) * 32 * NI + lane;
  if (part == 0) {
    const uint4* row = reinterpret_cast<const uint4*>(a.kv + tok * a.kv_stride);
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      z[i] = row[lane + 32 * i];
      if (a.weight) w[i] = reinterpret_cast<const uint4*>(a.weight)[lane + 32 * i];
    }
    if (lane < IPH) x[0] = row[LATENT / 8 + va], y[0] = row[LATENT / 8 + vb];
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = first + 32 * i;
      if (it >= items) continue;
      const uint4* row = reinterpret_cast<const uint4*>(a.q + tok * a.q_stride + (it / IPH) * a.qh_stride);
      x[i] = row[va];
      y[i] = row[vb];
    }
  }
  // angle of pair `lane` (the table holds zeros past the last pair)
  float sv, cv, cs[8], sn[8];
  sincospif((float)(int32_t)(((uint64_t)(int64_t)pos * a.t.turns[lane]) >> 32) * 4.656612873077393e-10f, &sv, &cv);   // half turns
  cv *= a.t.amplitude;
  sv *= a.t.amplitude;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cs[j] = __shfl_sync(FULL_MASK, cv, 8 * p + j);
    sn[j] = __shfl_sync(FULL_MASK, sv, 8 * p + j);
  }
  if (slot >= a.n_slots) {
    if (part == 0 && lane == 0) set_err(a.err, PKV_DEV_BAD_SLOT);
    slot = -1;
  }
  if (slot < 0) return;
  // u c - v s and u s + v c with the contraction spelled out, as in rope_append.cu
  auto turn2 = [&](float u, float v, int j, float& ou, float& ov) {
    ou = __fmaf_rn(u, cs[j], -__fmul_rn(v, sn[j]));
    ov = __fmaf_rn(u, sn[j], __fmul_rn(v, cs[j]));
  };
  auto turn = [&](uint4& s, uint4& t) {
    uint32_t* u = reinterpret_cast<uint32_t*>(&s);
    uint32_t* v = reinterpret_cast<uint32_t*>(&t);
    float a0, b0, a1, b1;
    if (inter) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        turn2(bf16_lo(u[j]), bf16_hi(u[j]), j, a0, b0);
        u[j] = pack_bf16(a0, b0);
        turn2(bf16_lo(v[j]), bf16_hi(v[j]), 4 + j, a0, b0);
        v[j] = pack_bf16(a0, b0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        turn2(bf16_lo(u[j]), bf16_lo(v[j]), 2 * j, a0, b0);
        turn2(bf16_hi(u[j]), bf16_hi(v[j]), 2 * j + 1, a1, b1);
        u[j] = pack_bf16(a0, a1);
        v[j] = pack_bf16(b0, b1);
      }
    }
  };
  if (part == 0) {
    uint4* row = reinterpret_cast<uint4*>(a.cache + slot * (LATENT + ROPE));
    if (a.weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const uint32_t* v = reinterpret_cast<const uint32_t*>(&z[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) ss += bf16_lo(v[j]) * bf16_lo(v[j]) + bf16_hi(v[j]) * bf16_hi(v[j]);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(FULL_MASK, ss, o);
      const float inv = 1.f / sqrtf(ss * (1.f / LATENT) + a.eps);
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        uint32_t* v = reinterpret_cast<uint32_t*>(&z[i]);
        const uint32_t* g = reinterpret_cast<const uint32_t*>(&w[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = pack_bf16(bf16_lo(v[j]) * inv * bf16_lo(g[j]), bf16_hi(v[j]) * inv * bf16_hi(g[j]));
      }
    }
#pragma unroll
    for (int i = 0; i < VL; ++i) row[lane + 32 * i] = z[i];
    if (lane < IPH) {
      turn(x[0], y[0]);
      row[LATENT / 8 + va] = x[0];
      row[LATENT / 8 + vb] = y[0];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = first + 32 * i;
      if (it >= items) continue;
      turn(x[i], y[i]);
      uint4* row = reinterpret_cast<uint4*>(a.q_out + tok * a.qo_stride + (it / IPH) * a.qoh_stride);
      row[va] = x[i];
      row[vb] = y[i];
    }
  }
}

template <int NI>
static const void* latent_append_fn(int latent, int rope) {
  if (latent == 512) return rope == 64 ? (const void*)latent_append_kernel<512, 64, NI> : (const void*)latent_append_kernel<512, 32, NI>;
  return rope == 64 ? (const void*)latent_append_kernel<256, 64, NI> : (const void*)latent_append_kernel<256, 32, NI>;
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_latent_append(const void* kv, int64_t kv_stride, const void* q, int64_t q_stride, int64_t q_head_stride,
                                        const int32_t* positions, const int64_t* slot_mapping, int n_tok,
                                        const pkv_rope_table* table, const void* weight, float eps, void* q_out,
                                        int64_t q_out_stride, int64_t q_out_head_stride, void* cache, int num_blocks,
                                        int block_size, int n_h, int latent, int rope, int32_t* err_flag, void* stream) {
  PKV_NVTX("pkv_latent_append");
  if (n_tok < 0 || num_blocks < 0 || n_h <= 0 || n_h > 1024) return PKV_EINVAL;
  if ((latent != 256 && latent != 512) || (rope != 32 && rope != 64)) return PKV_EINVAL;
  if (block_size != 16 && block_size != 32 && block_size != 64) return PKV_EINVAL;
  if (!table || table->rotary_dim != rope || !std::isfinite(table->amplitude)) return PKV_EINVAL;
  if (weight && !(eps >= 0.f && std::isfinite(eps))) return PKV_EINVAL;
  if (n_tok == 0) return PKV_OK;
  if (!kv || !q || !positions || !slot_mapping || !q_out || !cache) return PKV_EINVAL;
  for (const void* p : {kv, q, (const void*)q_out, (const void*)cache, weight})
    if (!al16(p)) return PKV_EINVAL;
  for (int64_t s : {kv_stride, q_stride, q_head_stride, q_out_stride, q_out_head_stride})
    if (s < 0 || s % 8) return PKV_EINVAL;
  if (kv_stride < latent + rope || q_head_stride < rope || q_out_head_stride < rope ||
      q_stride < (n_h - 1) * q_head_stride + rope || q_out_stride < (n_h - 1) * q_out_head_stride + rope)
    return PKV_EINVAL;
  LatentAppendArgs a = {};
  a.kv = static_cast<const __nv_bfloat16*>(kv);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.weight = static_cast<const __nv_bfloat16*>(weight);
  a.kv_stride = kv_stride; a.q_stride = q_stride; a.qh_stride = q_head_stride;
  a.qo_stride = q_out_stride; a.qoh_stride = q_out_head_stride;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.cache = static_cast<__nv_bfloat16*>(cache);
  a.positions = positions;
  a.slots = slot_mapping;
  a.n_slots = (long long)num_blocks * block_size;
  a.n_tok = n_tok; a.n_h = n_h;
  a.eps = eps;
  a.err = err_flag;
  a.t = *table;
  const int items = n_h * (rope / 16), sms = device_sm_count() > 0 ? device_sm_count() : 128;
  const bool wide = (long long)n_tok * items >= (long long)sms * 32 * 64;
  const int ni = !wide ? 1 : (items <= 64 ? 2 : 4);
  // the parts of a few tokens run side by side, near one another in memory (4001 tokens of 128 heads: 26.3 us the other way about)
  const unsigned groups = (n_tok - 1) / (kLatentThreads / 32) + 1, rows = groups < 32768u ? groups : 32768u;
  const dim3 grid(1 + (items + 32 * ni - 1) / (32 * ni), rows, (groups + rows - 1) / rows);
  void* kargs[] = {&a};
  const void* fn = ni == 1 ? latent_append_fn<1>(latent, rope) : (ni == 2 ? latent_append_fn<2>(latent, rope) : latent_append_fn<4>(latent, rope));
  const cudaError_t e = launch_pdl(fn, grid, dim3(kLatentThreads), 0, static_cast<cudaStream_t>(stream), kargs);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return PKV_ECUDA;
  }
  return PKV_OK;
}
