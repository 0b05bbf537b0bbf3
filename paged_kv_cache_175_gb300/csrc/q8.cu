// Quantize-on-append into the 8-bit paged cache (record layout: q8_common.cuh).
//
// Mathematics, per (block, kv head) and for K and V apart: big = max |x| over the rows that the
// block holds; scale = big / M, code = round_to_nearest_even(x * (M / big)), M = 448 (e4m3) or
// 127 (int8), every operation in fp32.  The result is a function of the rows alone, not of how
// many calls brought them: the bf16 rows of a sequence's unfinished block are kept in its tail
// and the record is written anew from them at each append, so the attention reads records only
// and a finished block was rounded once.
//
// What bounds it: long calls read 4 d bytes and write 2 d per token and kv head (HBM).  A decode
// step reads the open rows and writes one record per (sequence, kv head): a few hundred KB, so
// the launch and three dependent round trips (slots, rows, stores).
// Split: one CTA per kv head and span of tokens takes each run of tokens that lands in one
// block.  A span is one token for small calls (every run its own CTA, for latency) and
// block_size tokens above kSpanTokens (one or two runs per CTA, so that the CTAs whose tokens
// all continue a run do not cost a launch slot each).
#include <cuda_fp8.h>

#include <cmath>

#include "nvtx_range.h"
#include "q8_common.cuh"

namespace pkv {

struct Q8AppendArgs {
  const __nv_bfloat16 *k, *v;                    // [n_tok][n_kv][d], strides between tokens
  long long k_stride, v_stride;
  const int64_t* slots;
  const int32_t* tail_seq;
  uint8_t* records;
  __nv_bfloat16 *k_tail, *v_tail;                // [tail_rows][n_kv][bs][d]
  long long n_slots;
  int n_tok, n_kv, tail_rows, span;
  int32_t* err;
};

constexpr int kQ8Threads = 256;
constexpr int kSpanTokens = 2048;

__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, bool e4m3) {
  if (e4m3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
  auto one = [](float x) { return (uint32_t)(int)fminf(fmaxf(rintf(x), -127.f), 127.f) & 255u; };
  return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
}

// Whether token i belongs to sequence seq (padding belongs to none).
__device__ __forceinline__ bool of_seq(const Q8AppendArgs& a, int i, int seq) {
  return a.slots[i] >= 0 && a.tail_seq[i] == seq;
}
// First token past i (dir = 1), or last before it (dir = -1), that is not of seq: the tokens of
// a sequence are consecutive, so a whole warp narrows the range 32-fold per step.
__device__ int seq_edge(const Q8AppendArgs& a, int i, int seq, int dir) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = dir > 0 ? a.n_tok - i : i + 1;             // offset lo is of seq; offset hi is not (or outside)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int o = lo + (lane + 1) * step;
    const bool in = o < hi && of_seq(a, i + dir * o, seq);
    const unsigned out = ~__ballot_sync(FULL_MASK, in);
    const int f = out ? __ffs(out) - 1 : 32;                  // first probe that is not of seq
    const int nlo = lo + f * step, nhi = lo + (f + 1) * step;
    lo = nlo;
    hi = nhi < hi ? nhi : hi;
  }
  return i + dir * hi;
}

template <int D, int BS>
__global__ void __launch_bounds__(kQ8Threads) q8_append_kernel(const Q8AppendArgs a, const int e4m3) {
  constexpr int ROW = D + 8;                                  // padded row: the gathers below hit distinct banks
  constexpr int VPR = D / 8;                                  // 16-byte vectors per row
  constexpr int CHUNKS = BS * D / 16;                         // 16-byte chunks of codes per K (or V)
  extern __shared__ __align__(16) __nv_bfloat16 rows_s[];    // K rows, then V rows
  __shared__ float big_s[2][kQ8Threads / 32];
  __shared__ int run_s, edge_s;
  const int g = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i1 = min(a.n_tok, ((int)blockIdx.x + 1) * a.span);
  for (int i = blockIdx.x * a.span; i < i1;) {
    const int64_t slot = a.slots[i];
    if (slot < 0) { ++i; continue; }
    const int seq = a.tail_seq[i];
    if (slot >= a.n_slots || (unsigned)seq >= (unsigned)a.tail_rows) {
      if (g == 0 && threadIdx.x == 0) set_err(a.err, PKV_DEV_BAD_SLOT);
      ++i;
      continue;
    }
    const int row0 = (int)(slot % BS);
    // tokens i, i + 1, ... in consecutive rows of this block
    if (threadIdx.x == 0) run_s = BS - row0;
    __syncthreads();
    if (threadIdx.x < BS - row0) {
      const int j = i + threadIdx.x;
      if (j >= a.n_tok || a.slots[j] != slot + (int)threadIdx.x || a.tail_seq[j] != seq) atomicMin(&run_s, (int)threadIdx.x);
    }
    __syncthreads();
    const int m = run_s, end = row0 + m;
    // a run that began before this span is its predecessor's
    const bool leads = i == 0 || row0 == 0 || a.slots[i - 1] != slot - 1 || a.tail_seq[i - 1] != seq;
    if (leads) {
      const long long phys = slot / BS;
      const size_t tail0 = ((size_t)seq * a.n_kv + g) * BS * D;
      // rows into shared memory, with the largest magnitudes on the way
      float big[2] = {0.f, 0.f};
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const __nv_bfloat16* x = (kv ? a.v + (long long)i * a.v_stride : a.k + (long long)i * a.k_stride) + (size_t)g * D;
        const long long stride = kv ? a.v_stride : a.k_stride;
        const __nv_bfloat16* tail = (kv ? a.v_tail : a.k_tail) + tail0;
#pragma unroll 4
        for (int e = threadIdx.x; e < BS * VPR; e += kQ8Threads) {
          const int r = e / VPR, c = e - r * VPR;
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (r < end) w = *(reinterpret_cast<const uint4*>(r < row0 ? tail + (size_t)r * D : x + (r - row0) * stride) + c);
          *reinterpret_cast<uint4*>(rows_s + (kv * BS + r) * ROW + 8 * c) = w;
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) big[kv] = fmaxf(big[kv], fmaxf(fabsf(bf16_lo(ws[q])), fabsf(bf16_hi(ws[q]))));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) big[kv] = fmaxf(big[kv], __shfl_xor_sync(FULL_MASK, big[kv], o));
        if (lane == 0) big_s[kv][warp] = big[kv];
      }
      __syncthreads();
      uint8_t* rec = a.records + ((size_t)phys * a.n_kv + g) * q8_record_bytes(BS, D);
      const float most = e4m3 ? 448.f : 127.f;
      float inv[2], scale[2];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        float b = 0.f;
#pragma unroll
        for (int w = 0; w < kQ8Threads / 32; ++w) b = fmaxf(b, big_s[kv][w]);
        const bool some = b >= kQ8Tiny;
        scale[kv] = some ? __fdiv_rn(b, most) : 0.f;
        inv[kv] = some ? __fdiv_rn(most, b) : 0.f;
      }
      for (int e = threadIdx.x; e < 2 * CHUNKS; e += kQ8Threads) {
        const int kv = e / CHUNKS, c = e - kv * CHUNKS;
        const int ln = c & 31, gid = ln >> 2, tig = ln & 3, j = (c >> 5) % (D / 32), tt = (c >> 5) / (D / 32);
        uint32_t w[4];
        if (kv == 0) {
          const __nv_bfloat16* p = rows_s + (16 * tt + gid) * ROW + 32 * j + 2 * tig;
#pragma unroll
          for (int q = 0; q < 4; ++q) {                       // q = 2 ks + hi
            const __nv_bfloat16* s = p + (q & 1) * 8 * ROW + (q >> 1) * 16;
            const uint32_t x0 = *reinterpret_cast<const uint32_t*>(s), x1 = *reinterpret_cast<const uint32_t*>(s + 8);
            w[q] = code4(bf16_lo(x0) * inv[0], bf16_hi(x0) * inv[0], bf16_lo(x1) * inv[0], bf16_hi(x1) * inv[0], e4m3);
          }
        } else {
          const __nv_bfloat16* p = rows_s + (BS + 16 * tt + 2 * tig) * ROW + 32 * j + gid;
#pragma unroll
          for (int q = 0; q < 4; ++q) {                       // q = 2 md + hi
            const __nv_bfloat16* s = p + (q >> 1) * 16 + (q & 1) * 8;
            w[q] = code4(__bfloat162float(s[0]) * inv[1], __bfloat162float(s[ROW]) * inv[1],
                         __bfloat162float(s[8 * ROW]) * inv[1], __bfloat162float(s[9 * ROW]) * inv[1], e4m3);
          }
        }
        *reinterpret_cast<uint4*>(rec + (size_t)e * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (threadIdx.x == 0)
        *reinterpret_cast<uint4*>(rec + 2 * BS * D) = make_uint4(__float_as_uint(scale[0]), __float_as_uint(scale[1]), 0u, 0u);

      // ---- the sequence's tail ----
      // The CTA that read old rows from the tail (a run continuing a block) is the only one
      // that may then overwrite them, also with the rows of a later block of the same call.
      if (end < BS) {
        bool mine = true;
        if (row0 == 0 && i > 0 && of_seq(a, i - 1, seq)) {    // a later block: did the sequence start inside one?
          if (warp == 0) {
            const int first = seq_edge(a, i, seq, -1) + 1;
            if (lane == 0) edge_s = first;
          }
          __syncthreads();
          mine = a.slots[edge_s] % BS == 0;
        }
        if (mine) {
          for (int e = threadIdx.x; e < 2 * m * VPR; e += kQ8Threads) {
            const int kv = e / (m * VPR), f = e - kv * m * VPR, r = row0 + f / VPR, c = f % VPR;
            *(reinterpret_cast<uint4*>((kv ? a.v_tail : a.k_tail) + tail0 + (size_t)r * D) + c) =
                *reinterpret_cast<const uint4*>(rows_s + (kv * BS + r) * ROW + 8 * c);
          }
        }
      } else if (row0 > 0 && i + m < a.n_tok && of_seq(a, i + m, seq)) {
        // the block is full and the sequence goes on: the open rows behind it are this CTA's
        if (warp == 0) {
          const int last = seq_edge(a, i, seq, 1);
          if (lane == 0) edge_s = last;
        }
        __syncthreads();
        const int stop = edge_s, n = (int)(a.slots[stop - 1] % BS) + 1;   // rows of the last block
        if (n < BS && n <= stop - i - m) {
          for (int e = threadIdx.x; e < 2 * n * VPR; e += kQ8Threads) {
            const int kv = e / (n * VPR), f = e - kv * n * VPR, r = f / VPR, c = f % VPR;
            const __nv_bfloat16* x = (kv ? a.v + (long long)(stop - n + r) * a.v_stride
                                         : a.k + (long long)(stop - n + r) * a.k_stride) + (size_t)g * D;
            *(reinterpret_cast<uint4*>((kv ? a.v_tail : a.k_tail) + tail0 + (size_t)r * D) + c) =
                *(reinterpret_cast<const uint4*>(x) + c);
          }
        }
      }
      __syncthreads();                                        // rows_s, big_s and edge_s are reused
    }
    i += m;
  }
}

template <int D, int BS>
static cudaError_t launch_q8(const Q8AppendArgs& a, bool e4m3, cudaStream_t st) {
  const size_t smem = 2 * BS * (D + 8) * sizeof(__nv_bfloat16);
  const unsigned gx = (unsigned)((a.n_tok + a.span - 1) / a.span);
  q8_append_kernel<D, BS><<<dim3(gx, (unsigned)a.n_kv), kQ8Threads, smem, st>>>(a, e4m3 ? 1 : 0);
  return cudaGetLastError();
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_q8_record_bytes(int block_size, int head_dim) {
  if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32 && block_size != 64)) return 0;
  return (size_t)q8_record_bytes(block_size, head_dim);
}

extern "C" pkv_status pkv_kv_quant_append_q8(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                             const int64_t* slot_mapping, const int32_t* tail_seq, int n_tok, int format,
                                             uint8_t* cache, void* k_tail, void* v_tail, int tail_rows, int num_blocks,
                                             int block_size, int n_kv, int head_dim, int32_t* err_flag, void* stream) {
  PKV_NVTX("pkv_kv_quant_append_q8");
  if (n_tok < 0 || num_blocks < 0 || tail_rows < 0 || n_kv <= 0 || n_kv > 65535) return PKV_EINVAL;
  if (pkv_q8_record_bytes(block_size, head_dim) == 0) return PKV_EINVAL;
  if (format != PKV_Q8_E4M3 && format != PKV_Q8_INT8) return PKV_EINVAL;
  if (n_tok == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !tail_seq || !cache || !k_tail || !v_tail) return PKV_EINVAL;
  if (!al16(k) || !al16(v) || !al16(cache) || !al16(k_tail) || !al16(v_tail)) return PKV_EINVAL;
  const long long row = (long long)n_kv * head_dim;
  if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return PKV_EINVAL;
  Q8AppendArgs a = {};
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.k_stride = k_stride; a.v_stride = v_stride;
  a.slots = slot_mapping;
  a.tail_seq = tail_seq;
  a.records = cache;
  a.k_tail = static_cast<__nv_bfloat16*>(k_tail);
  a.v_tail = static_cast<__nv_bfloat16*>(v_tail);
  a.n_slots = (long long)num_blocks * block_size;
  a.n_tok = n_tok; a.n_kv = n_kv; a.tail_rows = tail_rows;
  a.span = n_tok <= kSpanTokens ? 1 : block_size;
  a.err = err_flag;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f = format == PKV_Q8_E4M3;
  cudaError_t e;
  if (head_dim == 128)
    e = block_size == 16 ? launch_q8<128, 16>(a, f, st) : (block_size == 32 ? launch_q8<128, 32>(a, f, st) : launch_q8<128, 64>(a, f, st));
  else
    e = block_size == 16 ? launch_q8<64, 16>(a, f, st) : (block_size == 32 ? launch_q8<64, 32>(a, f, st) : launch_q8<64, 64>(a, f, st));
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return PKV_ECUDA;
  }
  return PKV_OK;
}
