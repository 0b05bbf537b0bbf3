// Quantize-on-append into the 8-bit paged cache (record layout: q8_common.cuh).
//
// Mathematics, per (block, kv head) and for K and V apart: big = max |x| over the rows that the
// block holds; scale = big * (1 / M), code = round_to_nearest_even(x * ((1 / big) * M)), M = 448
// (e4m3) or 127 (int8), every operation rounded to fp32.  (Products with reciprocals are how elementary
// torch operations on the GPU divide a tensor by a number and a number by a tensor, so the codes equal
// theirs; divisions rounded once would be as repeatable and differ in a last place now and then.)
// The result is a function of the rows alone, not of how many calls brought them: the bf16 rows of a
// sequence's unfinished block are kept in its tail and the record is written anew from them at each
// append, so the attention reads records only and a finished block was rounded once.
//
// What bounds it: long calls read 4 d bytes and write 2 d per token and kv head (HBM).  A decode
// step reads the open rows and writes one record per (sequence, kv head): a few hundred KB, so
// the launch and three dependent round trips (slots, rows, stores).
// Split: one CTA per kv head, K or V, and span of tokens takes each run of tokens that lands in
// one block, 64 / block_size runs side by side (64 rows in shared memory at a time).  A span is 64
// tokens in long calls and as many tokens as there are places for runs in short ones, where every
// token of a decode step is a run (kSpanTokens says what that costs a prompt chunk).  The runs of a span
// are found in one round trip; the search for a sequence's end, which few runs need, goes on while the
// rows arrive.
// Measured (8 kv heads of 128): 8000 tokens of one prompt in blocks of 16 in 15.1 us (3.3 TB/s), one
// run at a time 21.7, four CTAs per SM instead of six 17.3; 23 ragged prompts of 234-701 tokens in
// blocks of 64 in 23.8 us (3.1 TB/s; the CTAs with two or three runs end last; asking for the next
// run's rows ahead cost the registers of a CTA per SM and was level); 64 single tokens in 3.0 us.
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

// Calls of up to this many tokens are taken for decode steps.  Single tokens of as many sequences, 8 kv heads
// of 128, spans of 64 / block_size tokens against spans of 64: 64 tokens 3.3 us against 26 (blocks of 64: 6.0
// and 86), 2048 tokens 37 against 64 (128 and 224).  One prompt is the other way round from 100-500 tokens on, since
// only one token in block_size starts a run and the other CTAs find nothing to do: 256 tokens in blocks of 16
// 4.4 against 5.2, 2048 13 against 7.6; in blocks of 64 256 tokens 7.0 against 5.2, 2048 36 against 7.6, with 32
// kv heads 135 against 13.  A rule that knows the runs would serve both.
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

constexpr int kQ8Rows = 64;              // rows that a CTA quantizes at a time: 64 / BS runs

template <int D, int BS>
struct Q8Shape {
  static constexpr int NT = 256, GROUPS = kQ8Rows / BS, GT = NT / GROUPS;   // threads per run
  static constexpr int NV = BS * D / 8 / GT;                  // 16-byte vectors of a run per thread
  static constexpr int WIN = kQ8Rows + BS;                    // tokens of a span, and behind it
};

template <int D, int BS, bool E4M3>
__global__ void __launch_bounds__(256, 6) q8_append_kernel(const Q8AppendArgs a) {
  using S = Q8Shape<D, BS>;
  constexpr int NT = S::NT, GROUPS = S::GROUPS, GT = S::GT, NV = S::NV, WIN = S::WIN, WORDS = (WIN + 31) / 32;
  constexpr int ROW = D + 8;                                  // padded row: the gathers below spread over the banks
  constexpr int VPR = D / 8;                                  // 16-byte vectors per row
  __shared__ __align__(16) __nv_bfloat16 rows_s[kQ8Rows * ROW];
  __shared__ float big_s[NT / 32];
  // the span's tokens and the block_size behind them, which the last run may reach
  __shared__ int64_t slot_s[WIN];
  __shared__ int seq_s[WIN];
  __shared__ uint32_t lead_s[WORDS], cont_s[WORDS + 1];       // bit t: token t starts / continues a run
  __shared__ int tail_from_s[GROUPS], tail_rows_s[GROUPS];    // see below
  const int g = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const int group = tid / GT, gtid = tid % GT;
  const bool values = blockIdx.z != 0;                        // this CTA's half of the records: V or K
  const __nv_bfloat16* x = (values ? a.v : a.k) + (size_t)g * D;
  const long long stride = values ? a.v_stride : a.k_stride;
  __nv_bfloat16* tails = values ? a.v_tail : a.k_tail;
  __nv_bfloat16* rows = rows_s + group * BS * ROW;
  const int i0 = blockIdx.x * a.span;
  grid_dep_wait();                         // launched while the kernel before may still run
  grid_dep_launch();
  if (tid < WORDS * 32) {
    const int i = i0 + tid;
    const bool in = i < a.n_tok && tid < a.span + BS && tid < WIN;
    const int64_t slot = in ? a.slots[i] : -1;
    const int seq = in ? a.tail_seq[i] : -1;
    const int64_t slot_before = in && i > 0 ? a.slots[i - 1] : -1;
    const int seq_before = in && i > 0 ? a.tail_seq[i - 1] : -1;
    const bool good = slot >= 0 && slot < a.n_slots && (unsigned)seq < (unsigned)a.tail_rows;
    if (slot >= 0 && !good && tid < a.span && g == 0 && !values) set_err(a.err, PKV_DEV_BAD_SLOT);
    // a run: consecutive rows of one block, of one sequence
    const bool goes_on = good && (slot & (BS - 1)) != 0 && slot_before == slot - 1 && seq_before == seq;
    if (tid < WIN) {
      slot_s[tid] = slot;
      seq_s[tid] = seq;
    }
    const unsigned c = __ballot_sync(FULL_MASK, goes_on), l = __ballot_sync(FULL_MASK, good && !goes_on && tid < a.span);
    if (lane == 0) {
      cont_s[warp] = c;
      lead_s[warp] = l;
    }
  }
  if (tid == 0) cont_s[WORDS] = 0u;
  __syncthreads();
  int n_runs = 0;
#pragma unroll
  for (int w = 0; w < WORDS; ++w) n_runs += __popc(lead_s[w]);
  struct Run {
    int t, m, seq, row0, end;              // first token of the span, tokens, sequence, rows [row0, end) of the block
    int64_t slot;
  };
  // the k-th run that starts in the span (end = 0: there is none)
  auto find = [&](int k) {
    Run r = {0, 0, 0, 0, 0, 0};
    if (k >= n_runs) return r;
    int left = k, wd = 0;
    while (left >= __popc(lead_s[wd])) left -= __popc(lead_s[wd++]);
    uint32_t bits = lead_s[wd];
    for (; left > 0; --left) bits &= bits - 1;
    r.t = 32 * wd + __ffs(bits) - 1;
    r.slot = slot_s[r.t];
    r.seq = seq_s[r.t];
    r.row0 = (int)(r.slot & (BS - 1));
    const int p = r.t + 1;                                    // its length: the tokens that go on from it
    wd = p >> 5;
    uint32_t stop = wd < WORDS ? ~cont_s[wd] & (0xffffffffu << (p & 31)) : 0xffffffffu;
    while (!stop) stop = ~cont_s[++wd];
    r.m = min(32 * wd + __ffs(stop) - 1 - r.t, BS - r.row0);
    r.end = r.row0 + r.m;
    return r;
  };
  uint4 w[NV];
  auto load = [&](const Run& r) {
    const __nv_bfloat16* old = tails + ((size_t)r.seq * a.n_kv + g) * BS * D;
    const __nv_bfloat16* now = x + (long long)(i0 + r.t - r.row0) * stride;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int e = gtid + u * GT, row = e / VPR, c = e % VPR;
      w[u] = make_uint4(0u, 0u, 0u, 0u);
      if (row < r.end) w[u] = *(reinterpret_cast<const uint4*>(row < r.row0 ? old + (size_t)row * D : now + row * stride) + c);
    }
  };
  for (int first = 0; first < n_runs; first += GROUPS) {
    const Run run = find(first + group);
    load(run);
    const bool busy = run.end > 0;
    const int m = run.m, seq = run.seq, row0 = run.row0, end = run.end, i = i0 + run.t;
    const size_t tail0 = ((size_t)seq * a.n_kv + g) * BS * D;
    // The sequence's tail, while the rows arrive.  Rows of an unfinished block go to the tail; but the
    // CTA that read old rows from it (a run continuing a block) is the only one that may then
    // overwrite them, also with the rows of a later block of the same call.
    //   tail_from < 0: the run's own m rows;  >= 0: rows 0 .. tail_rows of the tokens from there on
    if (busy && gtid < 32) {
      int from = -1, count = 0;
      if (end < BS) {
        count = m;
        if (row0 == 0 && i > 0 && of_seq(a, i - 1, seq)) {    // a later block: did the sequence start inside one?
          const int begin = seq_edge(a, i, seq, -1) + 1;
          if ((a.slots[begin] & (BS - 1)) != 0) count = 0;
        }
      } else if (row0 > 0 && i + m < a.n_tok && of_seq(a, i + m, seq)) {
        // the block is full and the sequence goes on: the open rows behind it are this CTA's
        const int stop = seq_edge(a, i, seq, 1), n = (int)(a.slots[stop - 1] & (BS - 1)) + 1;
        if (n < BS && n <= stop - i - m) {
          from = stop - n;
          count = n;
        }
      }
      if (lane == 0) {
        tail_from_s[group] = from;
        tail_rows_s[group] = count;
      }
    }
    __nv_bfloat162 big2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int e = gtid + u * GT, r = e / VPR, c = e % VPR;
      *reinterpret_cast<uint4*>(rows + r * ROW + 8 * c) = w[u];
      const uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) big2 = __hmax2(big2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&ws[q])));
    }
    // magnitudes are not negative: their bits order as integers
    const float mine = fmaxf(__low2float(big2), __high2float(big2));
    const uint32_t wb = __reduce_max_sync(FULL_MASK, __float_as_uint(mine));
    if (lane == 0) big_s[warp] = __uint_as_float(wb);
    __syncthreads();
    if (busy) {
      uint8_t* rec = a.records + ((size_t)(run.slot / BS) * a.n_kv + g) * q8_record_bytes(BS, D);
      const float most = E4M3 ? 448.f : 127.f;
      float big = 0.f;
#pragma unroll
      for (int k = 0; k < GT / 32; ++k) big = fmaxf(big, big_s[group * (GT / 32) + k]);
      const bool some = big >= kQ8Tiny;
      const float scale = some ? __fmul_rn(big, __fdiv_rn(1.f, most)) : 0.f, inv = some ? __fmul_rn(__fdiv_rn(1.f, big), most) : 0.f;
      uint8_t* codes = rec + (values ? BS * D : 0);
      if (!values) {
#pragma unroll
        for (int e = gtid; e < BS * D / 16; e += GT) {        // 16-byte chunks of codes
          const int ln = e & 31, gid = ln >> 2, tig = ln & 3, j = (e >> 5) % (D / 32), tt = (e >> 5) / (D / 32);
          const __nv_bfloat16* p = rows + (16 * tt + gid) * ROW + 32 * j + 2 * tig;
          uint32_t o[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {                       // q = 2 ks + hi
            const __nv_bfloat16* sp = p + (q & 1) * 8 * ROW + (q >> 1) * 16;
            const uint32_t x0 = *reinterpret_cast<const uint32_t*>(sp), x1 = *reinterpret_cast<const uint32_t*>(sp + 8);
            o[q] = code4<E4M3>(__fmul_rn(bf16_lo(x0), inv), __fmul_rn(bf16_hi(x0), inv), __fmul_rn(bf16_lo(x1), inv), __fmul_rn(bf16_hi(x1), inv));
          }
          *reinterpret_cast<uint4*>(codes + (size_t)e * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      } else {
        // the chunks of two neighbouring channels (gid = 2 gp, 2 gp + 1) from one set of loads
#pragma unroll
        for (int e = gtid; e < BS * D / 32; e += GT) {
          const int ln = e & 15, gp = ln >> 2, tig = ln & 3, j = (e >> 4) % (D / 32), tt = (e >> 4) / (D / 32);
          const __nv_bfloat16* p = rows + (16 * tt + 2 * tig) * ROW + 32 * j + 2 * gp;
          uint32_t o[2][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {                       // q = 2 md + hi
            const __nv_bfloat16* sp = p + (q >> 1) * 16 + (q & 1) * 8;
            const uint32_t t0 = *reinterpret_cast<const uint32_t*>(sp), t1 = *reinterpret_cast<const uint32_t*>(sp + ROW);
            const uint32_t t2 = *reinterpret_cast<const uint32_t*>(sp + 8 * ROW), t3 = *reinterpret_cast<const uint32_t*>(sp + 9 * ROW);
            o[0][q] = code4<E4M3>(__fmul_rn(bf16_lo(t0), inv), __fmul_rn(bf16_lo(t1), inv), __fmul_rn(bf16_lo(t2), inv), __fmul_rn(bf16_lo(t3), inv));
            o[1][q] = code4<E4M3>(__fmul_rn(bf16_hi(t0), inv), __fmul_rn(bf16_hi(t1), inv), __fmul_rn(bf16_hi(t2), inv), __fmul_rn(bf16_hi(t3), inv));
          }
          uint8_t* d = codes + (size_t)(((e >> 4) << 5) + 8 * gp + tig) * 16;
          *reinterpret_cast<uint4*>(d) = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
          *reinterpret_cast<uint4*>(d + 64) = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
        }
      }
      if (gtid == 0) {
        float* sc = reinterpret_cast<float*>(rec + 2 * BS * D);
        sc[values ? 1 : 0] = scale;
        sc[values ? 3 : 2] = 0.f;
      }
      const int from = tail_from_s[group], count = tail_rows_s[group];
      for (int e = gtid; e < count * VPR; e += GT) {
        const int k = e / VPR, c = e % VPR, r = from < 0 ? row0 + k : k;
        *(reinterpret_cast<uint4*>(tails + tail0 + (size_t)r * D) + c) =
            from < 0 ? *reinterpret_cast<const uint4*>(rows + r * ROW + 8 * c)
                     : *(reinterpret_cast<const uint4*>(x + (long long)(from + k) * stride) + c);
      }
    }
    __syncthreads();                                          // the shared arrays are reused
  }
}

template <int D, int BS>
static cudaError_t launch_q8(const Q8AppendArgs& a, bool e4m3, cudaStream_t st) {
  const unsigned gx = (unsigned)((a.n_tok + a.span - 1) / a.span);
  const dim3 grid(gx, (unsigned)a.n_kv, 2), block(256);
  void* kargs[] = {const_cast<Q8AppendArgs*>(&a)};
  return launch_pdl(e4m3 ? (const void*)q8_append_kernel<D, BS, true> : (const void*)q8_append_kernel<D, BS, false>, grid, block, 0, st,
                    kargs);
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
  if (n_tok > 0x7fff0000) return PKV_ERANGE;                  // token numbers of a span stay in 32 bits
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
  // long calls: 64 tokens; short ones (decode steps): as many tokens as the CTA has places for runs
  a.span = n_tok <= kSpanTokens ? kQ8Rows / block_size : kQ8Rows;
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
