// Rotary positions of new tokens: rotate the query and key heads of each token by its
// position and write them out, with the K / V rows going straight to their cache slots.
//
// Mathematics: channel pair j of the rotary part turns by theta_j * pos; theta_j is held as a
// fraction of a turn in 64-bit fixed point (pkv_rope_init), so pos * theta_j modulo one turn is
// one wrapping 64-bit integer product, exact to 2^-64 turn times pos for any int32 position
// (fp64 would do the same at a fraction of the rate: this GPU has few fp64 units).  The top 32
// bits of the product, as a signed fraction of half a turn, go to sincospif; cos and sin are
// scaled by the table's amplitude; the rotation runs in fp32 and rounds once to bf16.
//
// What bounds it: every element is read once and written once, so HBM for long calls and the
// launch plus two dependent memory round trips (position and slot, row) for short ones.
// Split: the tokens' rows are cut into items of two 16-byte vectors (the two halves of eight
// channel pairs in the half layout; 16 neighbouring channels in the interleaved one, and for
// channels that are only copied).  A CTA takes NI * 256 consecutive items of the flat (token,
// row, vector) order, issues all its loads first and builds the angle table of its tokens
// (shared by all their heads) while they are in flight.  What an item needs besides its data is
// worked out again for the store: held over the barrier it cost the registers of two CTAs per SM
// (16384 tokens of 32 + 8 + 8 heads of 128: 80 us instead of 63).
#include <cmath>

#include "decode_common.cuh"
#include "nvtx_range.h"

namespace pkv {

struct RopeArgs {
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;        // elements between tokens
  __nv_bfloat16 *q_out, *k_out;                  // k_out: rows of [n_tok][n_kv][d] (no append)
  long long qo_stride, ko_stride;
  __nv_bfloat16 *k_pool, *v_pool;                // append: [num_blocks][n_kv][block_size][d]
  const int32_t* positions;
  const int64_t* slots;
  long long n_slots;
  int n_tok, n_h, n_kv, bs_log2;
  int items_per_tok;                             // (n_h + n_kv (+ n_kv)) * d / 16, at most 24576
  uint32_t token_magic;                          // ceil(2^32 / items_per_tok): exact for numerators below 2^17
  int32_t* err;
  pkv_rope_table t;
};

constexpr int kRopeThreads = 256;
constexpr int kRopeItems = 3;              // per thread in long calls

// u c - v s and u s + v c, the contraction spelled out so that every variant of the kernel
// rounds alike (a token's result does not depend on the size of the call).
__device__ __forceinline__ float turn_a(float u, float v, float2 c) { return __fmaf_rn(u, c.x, -__fmul_rn(v, c.y)); }
__device__ __forceinline__ float turn_b(float u, float v, float2 c) { return __fmaf_rn(u, c.y, __fmul_rn(v, c.x)); }

template <int D, int NI, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, 5) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int VP = D / 16;                                  // items per row
  extern __shared__ float2 angles[];                         // [tokens][rotary_dim / 2]: cos, sin; then [tokens] slots
  // Launched while the kernel before may still run; nothing is read or written before the wait, and the
  // next kernel is let in only behind it (so its setup, too, finds that kernel's results).
  grid_dep_wait();
  grid_dep_launch();                       // the attention's launch may overlap this kernel
  const int H = a.t.rotary_dim >> 1, RP = a.t.rotary_dim >> 4;
  const bool inter = a.t.interleaved != 0;
  const long long total = (long long)a.n_tok * a.items_per_tok;
  const long long i0 = (long long)blockIdx.x * (NI * kRopeThreads);
  const int tok0 = (int)(i0 / a.items_per_tok);
  const int off0 = (int)(i0 - (long long)tok0 * a.items_per_tok);
  const int n_here = (int)(total - i0 < NI * kRopeThreads ? total - i0 : NI * kRopeThreads);
  const int tokens = (int)__umulhi((uint32_t)(off0 + n_here - 1), a.token_magic) + 1;
  int64_t* slots_s = reinterpret_cast<int64_t*>(angles + tokens * H);

  // item: its token of the CTA, its row (q heads, k heads, v heads) and its vectors within the row
  struct Item {
    int tl, row, p, vec, gap;
    bool turns;
  };
  auto item = [&](int idx) {
    Item it;
    const int flat = off0 + idx;
    it.tl = (int)__umulhi((uint32_t)flat, a.token_magic);
    const int rem = flat - it.tl * a.items_per_tok;
    it.row = rem / VP;
    it.p = rem % VP;
    it.turns = it.row < a.n_h + a.n_kv && it.p < RP;
    it.vec = it.turns && !inter ? it.p : 2 * it.p;
    it.gap = it.turns && !inter ? RP : 1;
    return it;
  };
  uint4 x[NI], y[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int idx = threadIdx.x + i * kRopeThreads;
    if (idx >= n_here) continue;
    const Item it = item(idx);
    const long long tok = tok0 + it.tl;
    const __nv_bfloat16* src;
    if (it.row < a.n_h) src = a.q + tok * a.q_stride + it.row * D;
    else if (it.row < a.n_h + a.n_kv) src = a.k + tok * a.k_stride + (it.row - a.n_h) * D;
    else src = a.v + tok * a.v_stride + (it.row - a.n_h - a.n_kv) * D;
    const uint4* s4 = reinterpret_cast<const uint4*>(src) + it.vec;
    x[i] = s4[0];
    y[i] = s4[it.gap];
  }
  if (APPEND)
    for (int e = threadIdx.x; e < tokens; e += kRopeThreads) {
      int64_t slot = a.slots[tok0 + e];
      if (slot >= a.n_slots) {
        if (e > 0 || off0 == 0) set_err(a.err, PKV_DEV_BAD_SLOT);   // by the CTA in which the token begins
        slot = -1;
      }
      slots_s[e] = slot;
    }
  for (int e = threadIdx.x; e < tokens * H; e += kRopeThreads) {
    const int tl = e / H, j = e - tl * H;
    const uint64_t turn = (uint64_t)(int64_t)a.positions[tok0 + tl] * a.t.turns[j];
    float sv, cv;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &sv, &cv);   // 2^-31: half turns
    angles[e] = make_float2(cv * a.t.amplitude, sv * a.t.amplitude);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int idx = threadIdx.x + i * kRopeThreads;
    if (idx >= n_here) continue;
    const Item it = item(idx);
    if (it.turns) {
      const float2* cs = angles + it.tl * H + 8 * it.p;       // eight pairs of the table, both layouts
      if (inter) {
        auto turn = [&](uint32_t& w, float2 c) {
          const float u = bf16_lo(w), v = bf16_hi(w);
          w = pack_bf16(turn_a(u, v, c), turn_b(u, v, c));
        };
        turn(x[i].x, cs[0]); turn(x[i].y, cs[1]); turn(x[i].z, cs[2]); turn(x[i].w, cs[3]);
        turn(y[i].x, cs[4]); turn(y[i].y, cs[5]); turn(y[i].z, cs[6]); turn(y[i].w, cs[7]);
      } else {
        auto turn = [&](uint32_t& wa, uint32_t& wb, float2 c0, float2 c1) {
          const float u0 = bf16_lo(wa), v0 = bf16_lo(wb), u1 = bf16_hi(wa), v1 = bf16_hi(wb);
          wa = pack_bf16(turn_a(u0, v0, c0), turn_a(u1, v1, c1));
          wb = pack_bf16(turn_b(u0, v0, c0), turn_b(u1, v1, c1));
        };
        turn(x[i].x, y[i].x, cs[0], cs[1]); turn(x[i].y, y[i].y, cs[2], cs[3]);
        turn(x[i].z, y[i].z, cs[4], cs[5]); turn(x[i].w, y[i].w, cs[6], cs[7]);
      }
    }
    const long long tok = tok0 + it.tl;
    const int64_t slot = APPEND ? slots_s[it.tl] : 0;
    if (slot < 0) continue;                // padding or flagged: nothing of this token is written
    __nv_bfloat16* dst;
    if (it.row < a.n_h) {
      dst = a.q_out + tok * a.qo_stride + it.row * D;
    } else {
      const bool is_k = it.row < a.n_h + a.n_kv;
      const int g = it.row - a.n_h - (is_k ? 0 : a.n_kv);
      if (APPEND) {
        const long long blk = slot >> a.bs_log2;
        const int r = (int)slot & ((1 << a.bs_log2) - 1);
        dst = (is_k ? a.k_pool : a.v_pool) + (((blk * a.n_kv + g) << a.bs_log2) + r) * D;
      } else {
        dst = a.k_out + tok * a.ko_stride + g * D;
      }
    }
    uint4* d4 = reinterpret_cast<uint4*>(dst) + it.vec;
    d4[0] = x[i];
    d4[it.gap] = y[i];
  }
}

template <int NI, bool APPEND>
static cudaError_t launch_rope(const RopeArgs& a, int head_dim, cudaStream_t st) {
  const long long total = (long long)a.n_tok * a.items_per_tok;
  const long long grid = (total + NI * kRopeThreads - 1) / (NI * kRopeThreads);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  // a range of NI * 256 items starts inside a token, so it can touch one more than it fills
  int tokens = (NI * kRopeThreads - 1) / a.items_per_tok + 2;
  if (tokens > a.n_tok) tokens = a.n_tok;
  const size_t smem = (size_t)tokens * (a.t.rotary_dim / 2 * sizeof(float2) + sizeof(int64_t));
  void* kargs[] = {const_cast<RopeArgs*>(&a)};
  return launch_pdl(head_dim == 128 ? (const void*)rope_append_kernel<128, NI, APPEND> : (const void*)rope_append_kernel<64, NI, APPEND>,
                    dim3((unsigned)grid), dim3(kRopeThreads), smem, st, kargs);
}

template <bool APPEND>
static cudaError_t launch_rope_any(const RopeArgs& a, int head_dim, cudaStream_t st) {
  // Three items per thread, five CTAs of them per SM, hide the memory latency of long calls: 16384
  // tokens of 32 + 8 + 8 heads of 128 in 63.0 us (6.4 TB/s, 94% of the measured copy rate); two items
  // 64.5 (six CTAs) and 69.5 (five), four 66.1 (four CTAs).  A call too small to give every SM two
  // CTAs of those takes one item per thread and three times the CTAs: 64 tokens in 2.3 us.
  const long long total = (long long)a.n_tok * a.items_per_tok;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 128;
  if (total >= (long long)sms * 2 * kRopeItems * kRopeThreads) return launch_rope<kRopeItems, APPEND>(a, head_dim, st);
  return launch_rope<1, APPEND>(a, head_dim, st);
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool good_stride(long long s, int heads, int d) { return s >= (long long)heads * d && s % 8 == 0; }

static bool valid_table(const pkv_rope_table* t, int head_dim) {
  return t && t->head_dim == head_dim && t->rotary_dim >= 16 && t->rotary_dim <= head_dim && t->rotary_dim % 16 == 0 &&
         std::isfinite(t->amplitude);
}

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_rope_init(const pkv_rope_config* c, pkv_rope_table* t) {
  if (!c || !t) return PKV_EINVAL;
  const int r = c->rotary_dim;
  if ((c->head_dim != 64 && c->head_dim != 128) || r < 16 || r > c->head_dim || r % 16) return PKV_EINVAL;
  if (!(c->base > 1.0) || !std::isfinite(c->base)) return PKV_EINVAL;
  if (c->scaling < PKV_ROPE_NONE || c->scaling > PKV_ROPE_YARN) return PKV_EINVAL;
  const double two_pi = 6.283185307179586476925286766559;
  const bool scaled = c->scaling != PKV_ROPE_NONE;
  if (scaled && (!(c->factor >= 1.0) || !std::isfinite(c->factor))) return PKV_EINVAL;
  const bool parts = c->scaling == PKV_ROPE_PARTS || c->scaling == PKV_ROPE_YARN;
  if (parts && (!(c->original_len > 0.0) || !std::isfinite(c->original_len) || !(c->low > 0.0) || !(c->high > c->low) ||
                !std::isfinite(c->high)))
    return PKV_EINVAL;
  const double s = scaled ? c->factor : 1.0;
  double base = c->base, amp = 1.0, first = 0.0, last = 0.0;
  if (c->scaling == PKV_ROPE_NTK) base *= std::pow(s, r / (r - 2.0));
  if (c->scaling == PKV_ROPE_YARN) {
    // the pair that makes `turns` turns over the original length
    auto place = [&](double turns) { return r * std::log(c->original_len / (turns * two_pi)) / (2.0 * std::log(base)); };
    first = std::fmax(std::floor(place(c->high)), 0.0);
    last = std::fmin(std::ceil(place(c->low)), r - 1.0);
    amp = 0.1 * std::log(s) + 1.0;
  }
  t->head_dim = c->head_dim;
  t->rotary_dim = r;
  t->interleaved = c->interleaved ? 1 : 0;
  t->amplitude = (float)(c->amplitude > 0.0 ? c->amplitude : amp);
  if (!std::isfinite(t->amplitude)) return PKV_EINVAL;
  for (int j = 0; j < 64; ++j) {
    t->turns[j] = 0;
    if (j >= r / 2) continue;
    double inv = std::pow(base, -2.0 * j / r);
    double w = 1.0;                                            // share of the unscaled frequency
    if (c->scaling == PKV_ROPE_LINEAR) w = 0.0;
    if (c->scaling == PKV_ROPE_PARTS) w = (c->original_len * inv / two_pi - c->low) / (c->high - c->low);
    if (c->scaling == PKV_ROPE_YARN) w = 1.0 - (j - first) / std::fmax(last - first, 0.001);
    if (c->scaling == PKV_ROPE_NTK) w = 1.0;
    w = std::fmin(std::fmax(w, 0.0), 1.0);
    inv = w * inv + (1.0 - w) * inv / s;
    const double turn = inv / two_pi;                          // turns per position, < 1
    t->turns[j] = (uint64_t)((turn - std::floor(turn)) * 18446744073709551616.0);
  }
  return PKV_OK;
}

extern "C" pkv_status pkv_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                      int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                                      int n_tok, const pkv_rope_table* table, void* q_out, int64_t q_out_stride,
                                      void* k_pool, void* v_pool, int num_blocks, int block_size, int n_h, int n_kv,
                                      int head_dim, int32_t* err_flag, void* stream) {
  PKV_NVTX("pkv_rope_append");
  if (n_tok < 0 || num_blocks < 0 || n_h <= 0 || n_kv <= 0 || n_h > 1024 || n_kv > 1024) return PKV_EINVAL;
  if (head_dim != 64 && head_dim != 128) return PKV_EINVAL;
  if (block_size != 16 && block_size != 32 && block_size != 64) return PKV_EINVAL;
  if (!valid_table(table, head_dim)) return PKV_EINVAL;
  if (n_tok == 0) return PKV_OK;
  if (!q || !k || !v || !positions || !slot_mapping || !q_out || !k_pool || !v_pool) return PKV_EINVAL;
  for (const void* p : {q, k, v, (const void*)q_out, (const void*)k_pool, (const void*)v_pool})
    if (!al16(p)) return PKV_EINVAL;
  if (!good_stride(q_stride, n_h, head_dim) || !good_stride(q_out_stride, n_h, head_dim) ||
      !good_stride(k_stride, n_kv, head_dim) || !good_stride(v_stride, n_kv, head_dim))
    return PKV_EINVAL;
  RopeArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.qo_stride = q_out_stride;
  a.k_pool = static_cast<__nv_bfloat16*>(k_pool);
  a.v_pool = static_cast<__nv_bfloat16*>(v_pool);
  a.positions = positions;
  a.slots = slot_mapping;
  a.n_slots = (long long)num_blocks * block_size;
  a.n_tok = n_tok; a.n_h = n_h; a.n_kv = n_kv;
  a.bs_log2 = block_size == 16 ? 4 : (block_size == 32 ? 5 : 6);
  a.items_per_tok = (n_h + 2 * n_kv) * (head_dim / 16);
  a.token_magic = (uint32_t)((0x100000000ull + a.items_per_tok - 1) / a.items_per_tok);
  a.err = err_flag;
  a.t = *table;
  const cudaError_t e = launch_rope_any<true>(a, head_dim, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return PKV_ECUDA;
  }
  return PKV_OK;
}

extern "C" pkv_status pkv_rope_qk(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                  const int32_t* positions, int n_tok, const pkv_rope_table* table, void* q_out,
                                  int64_t q_out_stride, void* k_out, int64_t k_out_stride, int n_h, int n_kv,
                                  int head_dim, void* stream) {
  PKV_NVTX("pkv_rope_qk");
  if (n_tok < 0 || n_h <= 0 || n_kv <= 0 || n_h > 1024 || n_kv > 1024) return PKV_EINVAL;
  if (head_dim != 64 && head_dim != 128) return PKV_EINVAL;
  if (!valid_table(table, head_dim)) return PKV_EINVAL;
  if (n_tok == 0) return PKV_OK;
  if (!q || !k || !positions || !q_out || !k_out) return PKV_EINVAL;
  for (const void* p : {q, k, (const void*)q_out, (const void*)k_out})
    if (!al16(p)) return PKV_EINVAL;
  if (!good_stride(q_stride, n_h, head_dim) || !good_stride(q_out_stride, n_h, head_dim) ||
      !good_stride(k_stride, n_kv, head_dim) || !good_stride(k_out_stride, n_kv, head_dim))
    return PKV_EINVAL;
  RopeArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.q_stride = q_stride; a.k_stride = k_stride;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.qo_stride = q_out_stride; a.ko_stride = k_out_stride;
  a.positions = positions;
  a.n_tok = n_tok; a.n_h = n_h; a.n_kv = n_kv;
  a.items_per_tok = (n_h + n_kv) * (head_dim / 16);
  a.token_magic = (uint32_t)((0x100000000ull + a.items_per_tok - 1) / a.items_per_tok);
  a.t = *table;
  const cudaError_t e = launch_rope_any<false>(a, head_dim, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return PKV_ECUDA;
  }
  return PKV_OK;
}
