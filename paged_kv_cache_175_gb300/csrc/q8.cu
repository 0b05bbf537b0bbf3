// Quantize-on-append into the 8-bit paged cache (record layout: q8_common.cuh).
//
// Mathematics, per (block, kv head) and for K and V apart: big = max |x| over the rows that the
// block holds; scale = big * (1 / M), code = round_to_nearest_even(x * ((1 / big) * M)), M = 448
// (e4m3) or 127 (int8), every operation rounded to fp32.  The result is a function of the rows alone, not of how
// many calls brought them: the bf16 rows of a sequence's unfinished block are kept in its tail
// and the record is written anew from them at each append, so the attention reads records only
// and a finished block was rounded once.
//
// What bounds it: long calls read 4 d bytes and write 2 d per token and kv head (HBM).  A decode
// step reads the open rows and writes one record per (sequence, kv head): a few hundred KB, so
// the launch and three dependent round trips (slots, rows, stores).
// Split: one CTA per kv head, K or V, and span of tokens takes each run of tokens that lands in
// one block.  A span is one token for small calls (every run its own CTA, for latency) and
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

constexpr int kSpanTokens = 2048;

// Four codes.  INT8: |x| <= 127 (1 + 2^-22), so adding 1.5 * 2^23 rounds x to the nearest integer
// (ties to even) and leaves it in the low byte; no conversion instruction, no clamp.  (The caller's
// products are __fmul_rn: fused with this addition they would skip the rounding to fp32 between.)
template <bool E4M3>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
  if constexpr (E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
  constexpr float kRound = 12582912.f;
  const uint32_t x = __byte_perm(__float_as_uint(a + kRound), __float_as_uint(b + kRound), 0x0040);
  const uint32_t y = __byte_perm(__float_as_uint(c + kRound), __float_as_uint(d + kRound), 0x0040);
  return __byte_perm(x, y, 0x5410);
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
struct Q8Shape {
  static constexpr int VECS = BS * D / 8;                     // 16-byte vectors of a block's rows
  static constexpr int NT = VECS < 256 ? VECS : 256;
  static constexpr int NV = VECS / NT;
};

template <int D, int BS, bool E4M3>
__global__ void __launch_bounds__(Q8Shape<D, BS>::NT) q8_append_kernel(const Q8AppendArgs a) {
  constexpr int NT = Q8Shape<D, BS>::NT, NV = Q8Shape<D, BS>::NV;
  constexpr int ROW = D + 8;                                  // padded row: the gathers below spread over the banks
  constexpr int VPR = D / 8;                                  // 16-byte vectors per row
  constexpr int CHUNKS = BS * D / 16;                         // 16-byte chunks of codes
  __shared__ __align__(16) __nv_bfloat16 rows_s[BS * ROW];
  __shared__ float big_s[NT / 32];
  // the span's tokens and the block_size behind them, which the last run may reach
  constexpr int WIN = 2 * BS;
  __shared__ int64_t slot_s[WIN];
  __shared__ int seq_s[WIN];
  __shared__ uint32_t lead_s[WIN / 32], cont_s[WIN / 32 + 1];  // bit t: token t starts / continues a run
  __shared__ int edge_s;
  const int g = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const bool values = blockIdx.z != 0;                        // this CTA's half of the record: V or K
  const __nv_bfloat16* x = (values ? a.v : a.k) + (size_t)g * D;
  const long long stride = values ? a.v_stride : a.k_stride;
  __nv_bfloat16* tails = values ? a.v_tail : a.k_tail;
  const int i0 = blockIdx.x * a.span;
  if (tid < WIN) {
    const int i = i0 + tid;
    const bool in = i < a.n_tok && tid < a.span + BS;
    const int64_t slot = in ? a.slots[i] : -1;
    const int seq = in ? a.tail_seq[i] : -1;
    const int64_t slot_before = in && i > 0 ? a.slots[i - 1] : -1;
    const int seq_before = in && i > 0 ? a.tail_seq[i - 1] : -1;
    const bool good = slot >= 0 && slot < a.n_slots && (unsigned)seq < (unsigned)a.tail_rows;
    if (slot >= 0 && !good && tid < a.span && g == 0 && blockIdx.z == 0) set_err(a.err, PKV_DEV_BAD_SLOT);
    // a run: consecutive rows of one block, of one sequence
    const bool goes_on = good && (slot & (BS - 1)) != 0 && slot_before == slot - 1 && seq_before == seq;
    slot_s[tid] = slot;
    seq_s[tid] = seq;
    const unsigned c = __ballot_sync(FULL_MASK, goes_on), l = __ballot_sync(FULL_MASK, good && !goes_on && tid < a.span);
    if (lane == 0) {
      cont_s[warp] = c;
      lead_s[warp] = l;
    }
  }
  if (tid == 0) cont_s[WIN / 32] = 0u;
  __syncthreads();
  for (int t = 0;;) {
    // next run that starts in the span
    {
      uint32_t bits = 0;
      int wd = t >> 5;
      if (wd < WIN / 32) bits = lead_s[wd] & (0xffffffffu << (t & 31));
      while (!bits && ++wd < WIN / 32) bits = lead_s[wd];
      if (!bits) break;
      t = 32 * wd + __ffs(bits) - 1;
    }
    const int i = i0 + t, seq = seq_s[t];
    const int64_t slot = slot_s[t];
    const int row0 = (int)(slot & (BS - 1));
    int m = 1;                                                // its length: the tokens that go on from it
    {
      int p = t + 1, wd = p >> 5;
      uint32_t stop = wd < WIN / 32 ? ~cont_s[wd] & (0xffffffffu << (p & 31)) : 0xffffffffu;
      while (!stop) stop = ~cont_s[++wd];
      m = 32 * wd + __ffs(stop) - 1 - t;
      if (wd >= WIN / 32) m = WIN - t;
    }
    m = min(m, BS - row0);
    const int end = row0 + m;
    {
      const long long phys = slot / BS;
      const size_t tail0 = ((size_t)seq * a.n_kv + g) * BS * D;
      // rows into shared memory, with the largest magnitude on the way
      uint4 w[NV];
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int e = tid + u * NT, r = e / VPR, c = e % VPR;
        w[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r < end)
          w[u] = *(reinterpret_cast<const uint4*>(r < row0 ? tails + tail0 + (size_t)r * D : x + (long long)(i + r - row0) * stride) + c);
      }
      __nv_bfloat162 big2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int e = tid + u * NT, r = e / VPR, c = e % VPR;
        *reinterpret_cast<uint4*>(rows_s + r * ROW + 8 * c) = w[u];
        const uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) big2 = __hmax2(big2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&ws[q])));
      }
      // magnitudes are not negative: their bits order as integers
      const float mine = fmaxf(__low2float(big2), __high2float(big2));
      const uint32_t wb = __reduce_max_sync(FULL_MASK, __float_as_uint(mine));
      if (lane == 0) big_s[warp] = __uint_as_float(wb);
      __syncthreads();
      uint8_t* rec = a.records + ((size_t)phys * a.n_kv + g) * q8_record_bytes(BS, D);
      const float most = E4M3 ? 448.f : 127.f;
      float big = 0.f;
#pragma unroll
      for (int k = 0; k < NT / 32; ++k) big = fmaxf(big, big_s[k]);
      const bool some = big >= kQ8Tiny;
      const float scale = some ? __fmul_rn(big, __fdiv_rn(1.f, most)) : 0.f, inv = some ? __fmul_rn(__fdiv_rn(1.f, big), most) : 0.f;
      uint8_t* codes = rec + (values ? BS * D : 0);
      if (!values) {
#pragma unroll
        for (int e = tid; e < CHUNKS; e += NT) {
          const int ln = e & 31, gid = ln >> 2, tig = ln & 3, j = (e >> 5) % (D / 32), tt = (e >> 5) / (D / 32);
          const __nv_bfloat16* p = rows_s + (16 * tt + gid) * ROW + 32 * j + 2 * tig;
          uint32_t o[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {                       // q = 2 ks + hi
            const __nv_bfloat16* s = p + (q & 1) * 8 * ROW + (q >> 1) * 16;
            const uint32_t x0 = *reinterpret_cast<const uint32_t*>(s), x1 = *reinterpret_cast<const uint32_t*>(s + 8);
            o[q] = code4<E4M3>(__fmul_rn(bf16_lo(x0), inv), __fmul_rn(bf16_hi(x0), inv), __fmul_rn(bf16_lo(x1), inv), __fmul_rn(bf16_hi(x1), inv));
          }
          *reinterpret_cast<uint4*>(codes + (size_t)e * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      } else {
        // the chunks of two neighbouring channels (gid = 2 gp, 2 gp + 1) from one set of loads
#pragma unroll
        for (int e = tid; e < CHUNKS / 2; e += NT) {
          const int ln = e & 15, gp = ln >> 2, tig = ln & 3, j = (e >> 4) % (D / 32), tt = (e >> 4) / (D / 32);
          const __nv_bfloat16* p = rows_s + (16 * tt + 2 * tig) * ROW + 32 * j + 2 * gp;
          uint32_t o[2][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {                       // q = 2 md + hi
            const __nv_bfloat16* s = p + (q >> 1) * 16 + (q & 1) * 8;
            const uint32_t t0 = *reinterpret_cast<const uint32_t*>(s), t1 = *reinterpret_cast<const uint32_t*>(s + ROW);
            const uint32_t t2 = *reinterpret_cast<const uint32_t*>(s + 8 * ROW), t3 = *reinterpret_cast<const uint32_t*>(s + 9 * ROW);
            o[0][q] = code4<E4M3>(__fmul_rn(bf16_lo(t0), inv), __fmul_rn(bf16_lo(t1), inv), __fmul_rn(bf16_lo(t2), inv), __fmul_rn(bf16_lo(t3), inv));
            o[1][q] = code4<E4M3>(__fmul_rn(bf16_hi(t0), inv), __fmul_rn(bf16_hi(t1), inv), __fmul_rn(bf16_hi(t2), inv), __fmul_rn(bf16_hi(t3), inv));
          }
          uint8_t* d = codes + (size_t)(((e >> 4) << 5) + 8 * gp + tig) * 16;
          *reinterpret_cast<uint4*>(d) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
          *reinterpret_cast<uint4*>(d + 64) = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
        }
      }
      if (tid == 0) {
        float* sc = reinterpret_cast<float*>(rec + 2 * BS * D);
        sc[values ? 1 : 0] = scale;
        sc[values ? 3 : 2] = 0.f;
      }

      // ---- the sequence's tail ----
      // The CTA that read old rows from the tail (a run continuing a block) is the only one
      // that may then overwrite them, also with the rows of a later block of the same call.
      if (end < BS) {
        bool own = true;
        if (row0 == 0 && i > 0 && of_seq(a, i - 1, seq)) {    // a later block: did the sequence start inside one?
          if (warp == 0) {
            const int first = seq_edge(a, i, seq, -1) + 1;
            if (lane == 0) edge_s = first;
          }
          __syncthreads();
          own = a.slots[edge_s] % BS == 0;
        }
        if (own) {
          for (int e = tid; e < m * VPR; e += NT) {
            const int r = row0 + e / VPR, c = e % VPR;
            *(reinterpret_cast<uint4*>(tails + tail0 + (size_t)r * D) + c) = *reinterpret_cast<const uint4*>(rows_s + r * ROW + 8 * c);
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
          for (int e = tid; e < n * VPR; e += NT) {
            const int r = e / VPR, c = e % VPR;
            *(reinterpret_cast<uint4*>(tails + tail0 + (size_t)r * D) + c) =
                *(reinterpret_cast<const uint4*>(x + (long long)(stop - n + r) * stride) + c);
          }
        }
      }
    }
    t += m;
    if (t >= a.span) break;
    __syncthreads();                                          // the shared arrays are reused
  }
}

template <int D, int BS>
static cudaError_t launch_q8(const Q8AppendArgs& a, bool e4m3, cudaStream_t st) {
  const unsigned gx = (unsigned)((a.n_tok + a.span - 1) / a.span);
  const dim3 grid(gx, (unsigned)a.n_kv, 2), block(Q8Shape<D, BS>::NT);
  if (e4m3) q8_append_kernel<D, BS, true><<<grid, block, 0, st>>>(a);
  else q8_append_kernel<D, BS, false><<<grid, block, 0, st>>>(a);
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
