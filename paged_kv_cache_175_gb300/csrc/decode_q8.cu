// Paged decode attention over the 8-bit cache (GQA / MHA / MQA; record layout: q8_common.cuh).
//
// Mathematics: with K^ = s_k * c_k and V^ = s_v * c_v per (block, kv head), the scores of a
// block are (s_k * scale) * (c_k . q) and its output is s_v * sum_t p_t c_v,t: both scales stay
// outside the products, so the codes enter the tensor cores as they are.  Codes become fp16
// exactly (e4m3 and small integers are fp16 values).  q is bf16; each head's q is multiplied by
// a power of two that puts its largest value at 2^14, so that every value above 2^-31 of the
// largest is exact in fp16 (and the rest is off by 2^-39 of the largest at most); the power is
// taken out of the scores again.  p enters as fp16 of 128 p (128: p <= 2^8 by the lazy offset, so
// 2^15 at most, and the smallest step is 2^-31 of p = 1): as a high + low pair, 22 bits, for fp32
// outputs and for groups of up to four heads, where the pair is free; rounded once (2^-11 of p at
// most, against the 2^-8 of the output's own rounding) for bf16 outputs of larger groups, whose
// kernels are bound by the products: 32 heads on one kv head 54.8 -> 38.1 us, 64 heads 97.8 -> 62.0
// (64 x 2-8K tokens).  Softmax, sums and outputs are fp32.
//
// Structure: the persistent grid and the line of blocks of decode_common.cuh, NW streams per CTA
// (piece_streams.cuh).  A stage is 32 tokens: two records of 16 tokens, one of 32, or half of a
// 64-token record (its K half, V half and scales as three copies that land in the layout of a
// 32-token record), so one kernel serves every block size.  Per 16-token tile, S^T = C_k Q^T and
// O^T += C_v^T P^T with mma.m16n8k16; the A fragments of both are one 16-byte load per lane and 32
// channels, since the records hold the codes in fragment order.
#include <cmath>
#include <cstdlib>
#include <mutex>


#include "nvtx_range.h"
#include "piece_streams.cuh"
#include "q8_common.cuh"
#include "stream_plan.cuh"

namespace pkv {

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Four codes (bytes 0..3) as two fp16 pairs, exact.
template <bool E4M3>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // code + 128 as the low byte of 1024 + (code + 128), minus 1152
    const uint32_t b = w ^ 0x80808080u;
    const uint32_t x = prmt(b, 0x64646464u, 0x4140), y = prmt(b, 0x64646464u, 0x4342);
    const __half2 c = __float2half2_rn(1152.f);
    const __half2 u = __hsub2(*reinterpret_cast<const __half2*>(&x), c), v = __hsub2(*reinterpret_cast<const __half2*>(&y), c);
    lo = *reinterpret_cast<const uint32_t*>(&u);
    hi = *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 lds_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ float h2_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float h2_hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }
// Keep the halves of a pair of rows (t, t + 1) that lie in [lead, ntok); zero the others.
__device__ __forceinline__ uint32_t keep_pair(uint32_t b, int t, int lead, int ntok) {
  return b & ((t < ntok && t >= lead ? 0x0000ffffu : 0u) | (t + 1 < ntok && t + 1 >= lead ? 0xffff0000u : 0u));
}

// p enters the products times 2^7: the exponent is taken against the running offset minus 7.
constexpr float kPBits = 7.f;
constexpr int kQ8Rows = 32;           // tokens per stage

__host__ __device__ constexpr size_t q8_smem_bytes(int streams, int stages, int stage_bytes) {
  return 128 + (size_t)streams * stages * (stage_bytes + 16 + 16);
}

// NH n-tiles of 8 heads per consumer warp, MT consumer warps per stream, NW streams.
// COMB (groups of up to 4 heads): column n of the n-tile holds head n % 4; columns 0-3 carry the
// high parts of p and columns 4-7 the low parts, so the pair costs one product.
template <int D, int NH, int MT, int NW, bool E4M3, bool COMB, bool PAIR>
__global__ void __launch_bounds__((NW * MT + 1) * 32, NH == 2 ? 2 : 4) decode_q8_kernel(const DecodeArgs a, const int sub) {
  constexpr int KS = D / 16, MD = D / 16, HW = 8 * NH, TT = kQ8Rows / 16;
  static_assert(!COMB || (NH == 1 && MT == 1), "one n-tile holds the whole group");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t ring0 = (smem_u32(smem_raw) + 127u) & ~127u;
  const int S = a.stages, BS = a.block_size, NB = kQ8Rows / BS;   // BS: 16 or 32 (units of the line)
  const int REC = q8_record_bytes(BS, D), STAGE = NB * REC;
  uint8_t* smem = smem_raw + (ring0 - smem_u32(smem_raw));
  int4* meta = reinterpret_cast<int4*>(smem + (size_t)NW * S * STAGE);
  uint64_t* full = reinterpret_cast<uint64_t*>(meta + NW * S);
  uint64_t* empty = full + NW * S;
  __shared__ volatile int abort_flag;
  __shared__ StreamStart starts[NW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tig = lane & 3, gid = lane >> 2;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < NW * S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], MT);
    }
    fence_barrier_init();
  }
  // Every thread waits for the kernel before this one (the append, or whatever wrote the context lengths)
  // ahead of its first read and, also without work, so that no later launch on the stream can pass it.  The
  // merge is let in behind the wait: its setup reads the lengths, too.
  grid_dep_wait();
  grid_dep_launch();
  if (warp < NW * MT && warp % MT == 0)
    stream_setup(a, blockIdx.x * NW + warp / MT, gridDim.x * NW, &starts[warp / MT]);
  __syncthreads();

  if (warp == NW * MT) {
    const uint64_t pol = policy_evict_first();
    const int big = q8_record_bytes(BS << sub, D);             // bytes of a record of the cache
    produce_streams(a, starts, NW, S, NB, sub, (uint32_t)REC, 2 * D, meta, full, empty, &abort_flag,
                    [&](int w, int slot, int k, int phys, int u, int kvh) {
                      const uint32_t dst = ring0 + (uint32_t)((w * S + slot) * STAGE + k * REC);
                      const uint32_t bar = smem_u32(&full[w * S + slot]);
                      const uint8_t* src = a.cache + ((size_t)phys * a.n_kv + kvh) * big;
                      if (sub == 0) {
                        bulk_g2s_u32(dst, src, REC, bar, pol);
                      } else {
                        const uint32_t half = (uint32_t)(BS * D);
                        src += (u & 1) * half;
                        bulk_g2s_u32(dst, src, half, bar, pol);
                        bulk_g2s_u32(dst + half, src + 2 * half, half, bar, pol);
                        bulk_g2s_u32(dst + 2 * half, src + (4 - (u & 1)) * half, 16, bar, pol);
                      }
                    });
    return;
  }

  // ---------------- consumer warp: local heads [warp % MT * HW, + HW) of its stream ----------------
  const int w = warp / MT;
  if (starts[w].len <= 0) return;
  const int p = blockIdx.x * NW + w;
  const uint32_t ring = ring0 + (uint32_t)(w * S * STAGE);
  meta += w * S;
  full += w * S;
  empty += w * S;
  uint32_t qb[KS][NH][2];
  float o[MD][NH][4];
  float m[NH][2], l[NH][2], qs[NH][2];          // m: running offset - 7; qs: what a head's scores are multiplied by
  const int hw0 = warp % MT * HW;
  int slot = 0;
  uint32_t phase = 0;
  // plain loads: the kernel before (a rotary append) may write q while this grid is already resident
  auto load_q = [&](size_t qrow0) {
#pragma unroll
    for (int nh = 0; nh < NH; ++nh) {
      const int hl = COMB ? gid & 3 : hw0 + nh * 8 + gid;      // B-fragment column n = gid
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(a.q) + (qrow0 + hl) * (D / 2);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int r = 0; r < 2; ++r) qb[ks][nh][r] = hl < a.G ? qp[ks * 8 + 4 * r + tig] : 0u;
    }
  };
  // the first segment's queries, while its first stage is on the way
  bool have_q = true;
  load_q((size_t)starts[w].cur.s * a.n_h + (size_t)starts[w].cur.g * a.G);
  for (;;) {
    if (!mbar_wait(&full[slot], phase) || abort_flag) {
      set_err(a.err, PKV_DEV_TIMEOUT);
      abort_flag = 1;
      break;
    }
    const int4 mt = meta[slot];
    const int s = mt.x, g = mt.y, ntok = mt.w & 255, flags = (mt.w >> 8) & 255, lead = mt.w >> 16;
    const size_t qrow0 = (size_t)s * a.n_h + (size_t)g * a.G;

    if (flags & F_FIRST) {
      if (!have_q) load_q(qrow0);
      have_q = false;
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        float big = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t x = qb[ks][nh][r];
            big = fmaxf(big, fmaxf(fabsf(bf16_lo(x)), fabsf(bf16_hi(x))));
          }
        big = fmaxf(big, __shfl_xor_sync(FULL_MASK, big, 1));
        big = fmaxf(big, __shfl_xor_sync(FULL_MASK, big, 2));
        // 2^k with k = 14 - floor(log2(big)), at most 2^126 (also for zeros)
        const int k = min(126, 14 + 127 - (int)(__float_as_uint(big) >> 23));
        const float up = __uint_as_float((uint32_t)(k + 127) << 23);
        const float down = a.scale_log2 * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int r = 0; r < 2; ++r) qb[ks][nh][r] = pack_f16(bf16_lo(qb[ks][nh][r]) * up, bf16_hi(qb[ks][nh][r]) * up);
        qs[nh][0] = __shfl_sync(FULL_MASK, down, 8 * tig);     // accumulator columns 2 tig, 2 tig + 1
        qs[nh][1] = __shfl_sync(FULL_MASK, down, 8 * tig + 4);
        m[nh][0] = m[nh][1] = -INFINITY;
        l[nh][0] = l[nh][1] = 0.f;
#pragma unroll
        for (int md = 0; md < MD; ++md) o[md][nh][0] = o[md][nh][1] = o[md][nh][2] = o[md][nh][3] = 0.f;
      }
    }

    if (flags & F_VALID) {
      const uint32_t st = ring + (uint32_t)(slot * STAGE);
      // tile t: in one record of 32 tokens, or the first tile of the t-th of two
      const uint32_t rec1 = st + (uint32_t)((NB - 1) * REC);
      const uint32_t kb1 = NB == 2 ? rec1 : st + 16 * D;
      const bool partial = ntok < kQ8Rows || lead > 0;         // rows [lead, ntok) count
      // ---- S^T = C_k Q^T ----
      float sc[TT][NH][4];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t kb = (t ? kb1 : st) + lane * 16;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[t][nh][i] = 0.f;
        if (t && ntok <= 16) continue;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 x = lds128(kb + j * 512);
          uint32_t ka[4];
          codes_f16<E4M3>(x.x, ka[0], ka[2]);
          codes_f16<E4M3>(x.y, ka[1], ka[3]);
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma_f16(sc[t][nh], ka, qb[2 * j][nh][0], qb[2 * j][nh][1]);
          codes_f16<E4M3>(x.z, ka[0], ka[2]);
          codes_f16<E4M3>(x.w, ka[1], ka[3]);
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma_f16(sc[t][nh], ka, qb[2 * j + 1][nh][0], qb[2 * j + 1][nh][1]);
        }
      }
      float sv[TT];
      {
        const float2 s0 = lds_f32x2(st + 2 * BS * D), s1 = lds_f32x2(rec1 + 2 * BS * D);
        sv[0] = s0.y;
        sv[1] = s1.y;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[0][nh][i] *= s0.x * qs[nh][i & 1];
            sc[1][nh][i] *= s1.x * qs[nh][i & 1];
          }
      }
      if (partial) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int tok = t * 16 + gid + 8 * r;
            if (tok >= ntok || tok < lead)
#pragma unroll
              for (int nh = 0; nh < NH; ++nh) sc[t][nh][2 * r] = sc[t][nh][2 * r + 1] = -INFINITY;
          }
      }
      // ---- online softmax over tokens: the offset is raised (to the exact running maximum) only
      // when a score exceeds it by more than kLazyMax, so p <= 2^8 ----
      {
        bool over = false;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(fmaxf(sc[0][nh][e], sc[0][nh][2 + e]), fmaxf(sc[1][nh][e], sc[1][nh][2 + e]));
            over |= mx > m[nh][e] + (kLazyMax + kPBits);
          }
        if (__any_sync(FULL_MASK, over)) {
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) {
            float al[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(fmaxf(sc[0][nh][e], sc[0][nh][2 + e]), fmaxf(sc[1][nh][e], sc[1][nh][2 + e]));
              mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 16));
              const float mn = fmaxf(m[nh][e], mx - kPBits);
              al[e] = ex2(m[nh][e] - mn);
              m[nh][e] = mn;
              l[nh][e] *= al[e];
            }
#pragma unroll
            for (int md = 0; md < MD; ++md) {
              o[md][nh][0] *= al[0]; o[md][nh][1] *= al[1];
              o[md][nh][2] *= al[0]; o[md][nh][3] *= al[1];
            }
          }
        }
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float rs = 0.f;
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float pv = ex2(sc[t][nh][2 * r + e] - m[nh][e]);
                sc[t][nh][2 * r + e] = pv;
                rs += pv;
              }
            l[nh][e] += rs;
          }
      }
      // ---- O^T += s_v C_v^T P^T ----
      uint32_t bh[TT][NH][2], bl[PAIR && !COMB ? TT : 1][NH][2];
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float x = sc[t][nh][2 * r], y = sc[t][nh][2 * r + 1];
            const uint32_t hi = pack_f16(x, y);
            const uint32_t lo = PAIR ? pack_f16(x - h2_lo(hi), y - h2_hi(hi)) : 0u;
            bh[t][nh][r] = movmatrix_t(COMB && tig >= 2 ? lo : hi);
            if constexpr (PAIR && !COMB) bl[t][nh][r] = movmatrix_t(lo);
          }
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (t && ntok <= 16) continue;
        const uint32_t vb = (t ? kb1 : st) + BS * D + lane * 16;
        const int t0 = t * 16 + 2 * tig;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 x = lds128(vb + j * 512);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t va[4];
            codes_f16<E4M3>(h ? x.z : x.x, va[0], va[2]);
            codes_f16<E4M3>(h ? x.w : x.y, va[1], va[3]);
            if (partial) {
              va[0] = keep_pair(va[0], t0, lead, ntok);
              va[1] = keep_pair(va[1], t0, lead, ntok);
              va[2] = keep_pair(va[2], t0 + 8, lead, ntok);
              va[3] = keep_pair(va[3], t0 + 8, lead, ntok);
            }
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
              float acc[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(acc, va, bh[t][nh][0], bh[t][nh][1]);
              if constexpr (PAIR && !COMB) mma_f16(acc, va, bl[t][nh][0], bl[t][nh][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[2 * j + h][nh][i] = fmaf(sv[t], acc[i], o[2 * j + h][nh][i]);
            }
          }
        }
      }
    }

    if (flags & F_LAST) {
      const bool whole = flags & F_WHOLE;
      const long long part = (long long)s * a.n_kv + g + p;
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        if constexpr (COMB) {                                  // the low parts' columns lie two lanes on
#pragma unroll
          for (int md = 0; md < MD; ++md)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[md][nh][i] += __shfl_down_sync(FULL_MASK, o[md][nh][i], 2, 4);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float L = l[nh][e];
          L += __shfl_xor_sync(FULL_MASK, L, 4);
          L += __shfl_xor_sync(FULL_MASK, L, 8);
          L += __shfl_xor_sync(FULL_MASK, L, 16);
          const int hl = hw0 + nh * 8 + 2 * tig + e;           // this thread's head columns
          if (hl >= a.G) continue;
          if (whole) {
            const float inv = L > 0.f ? 1.f / L : 0.f;
            const size_t base = (qrow0 + hl) * D;
            if (a.out_f32) {
              float* out = reinterpret_cast<float*>(a.out) + base;
#pragma unroll
              for (int md = 0; md < MD; ++md) {
                out[md * 16 + gid] = o[md][nh][e] * inv;
                out[md * 16 + gid + 8] = o[md][nh][2 + e] * inv;
              }
            } else {
              __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + base;
#pragma unroll
              for (int md = 0; md < MD; ++md) {
                out[md * 16 + gid] = __float2bfloat16_rn(o[md][nh][e] * inv);
                out[md * 16 + gid + 8] = __float2bfloat16_rn(o[md][nh][2 + e] * inv);
              }
            }
          } else {
            float* wo = a.ws_o + ((size_t)part * a.G + hl) * D;
#pragma unroll
            for (int md = 0; md < MD; ++md) {
              wo[md * 16 + gid] = o[md][nh][e];
              wo[md * 16 + gid + 8] = o[md][nh][2 + e];
            }
            if (gid == 0)
              *reinterpret_cast<float2*>(a.ws_ml + ((size_t)part * a.G + hl) * 2) = make_float2(m[nh][e], L);
          }
        }
      }
    }

    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
    if (flags & F_END) break;
  }
}

// ---------------------------------------------------------------------------------------------
struct Q8Variant {
  const void* fn;
  int stages, warps, streams, P;
  size_t smem;
};

constexpr size_t kQ8MaxSmem = 200 * 1024;

// Three streams and their producer warp fill an SM's registers at four CTAs of 128 registers: 12
// consumer warps.  32/8 heads of 128, 64 sequences of 512-4096 tokens in e4m3 / 32 of 8-32K in int8:
// 54 / 203 us (83% / 97% of the measured copy rate), with four streams 55.3 / 208, with six 56.4 /
// 218, at three CTAs 55 / 215; a producer warp per consumer warp and 64-token stages (six consumers
// per SM) took 72.7 / 324.  A third ring stage costs consumers their shared memory: 55.7 / 212.
// Larger groups: 16 heads per consumer warp (two n-tiles share the converted codes), 32/2 heads 26.3
// us against 32.7 with two warps of 8; two CTAs per SM (three were slower: fewer registers, spills).
template <int D, bool E4M3, bool PAIR>
static void q8_pick(int G, Q8Variant& v) {
  auto set = [&](const void* fn, int mt, int nw) {
    v.fn = fn;
    v.streams = nw;
    v.warps = nw * mt + 1;
  };
  if (G <= 4) set((const void*)decode_q8_kernel<D, 1, 1, 3, E4M3, true, true>, 1, 3);
  else if (G <= 8) set((const void*)decode_q8_kernel<D, 1, 1, 3, E4M3, false, PAIR>, 1, 3);
  else if (G <= 16) set((const void*)decode_q8_kernel<D, 2, 1, 3, E4M3, false, PAIR>, 1, 3);
  else if (G <= 32) set((const void*)decode_q8_kernel<D, 2, 2, 2, E4M3, false, PAIR>, 2, 2);
  else set((const void*)decode_q8_kernel<D, 2, 4, 1, E4M3, false, PAIR>, 4, 1);
}
static int q8_variant_index(int G) { return G <= 4 ? 0 : head_tiling(G) + 1; }

static Q8Variant* lookup_q8(int D, int BS, int G, bool e4m3, bool pair) {
  // One table per process; the library drives one device per process.
  static std::mutex mu;
  static Q8Variant table[2][2][5][2][2];
  static bool ready[2][2][5][2][2] = {};
  const int di = D == 128 ? 1 : 0, bi = BS == 16 ? 0 : 1, vi = q8_variant_index(G), fi = e4m3 ? 1 : 0;
  std::lock_guard<std::mutex> lock(mu);
  const int pi = pair || G <= 4 ? 1 : 0;
  Q8Variant& v = table[di][bi][vi][fi][pi];
  if (!ready[di][bi][vi][fi][pi]) {
    if (D == 128) {
      if (e4m3) pi ? q8_pick<128, true, true>(G, v) : q8_pick<128, true, false>(G, v);
      else pi ? q8_pick<128, false, true>(G, v) : q8_pick<128, false, false>(G, v);
    } else {
      if (e4m3) pi ? q8_pick<64, true, true>(G, v) : q8_pick<64, true, false>(G, v);
      else pi ? q8_pick<64, false, true>(G, v) : q8_pick<64, false, false>(G, v);
    }
    const int unit = BS == 16 ? 16 : 32, stage = kQ8Rows / unit * q8_record_bytes(unit, D);
    // Stages of a ring: two for groups of up to eight heads at d = 128 (four heads, 64 x 0.5-4K tokens:
    // 55.0 us, three 56.6; 205 against 212 on long contexts); three where a stage is half as long
    // (d = 64: 36.3 -> 33.5 us) or takes longer to consume (16 heads: 68.7 -> 64.5 us).
    v.stages = ring_stages(stage, (D == 128 && G <= 8 ? 2 : 3) * stage, "PKV_STAGES_Q8");
    v.smem = q8_smem_bytes(v.streams, v.stages, stage);
    // one function serves all block sizes, whose rings differ a little: one limit for all
    if (v.smem > kQ8MaxSmem ||
        cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kQ8MaxSmem) != cudaSuccess)
      return nullptr;
    int occ = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, v.fn, v.warps * 32, v.smem) != cudaSuccess || occ < 1)
      return nullptr;
    v.P = device_sm_count() * occ * v.streams;
    ready[di][bi][vi][fi][pi] = true;
  }
  return &v;
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static bool valid_shape(int n_h, int n_kv, int head_dim, int block_size) {
  if (pkv_q8_record_bytes(block_size, head_dim) == 0) return false;
  if (n_kv <= 0 || n_h <= 0 || n_h % n_kv) return false;
  return n_h / n_kv <= 64;
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_q8_workspace_bytes(int batch, int n_h, int n_kv, int head_dim, int block_size, int format) {
  if (batch < 0 || !valid_shape(n_h, n_kv, head_dim, block_size)) return 0;
  if (format != PKV_Q8_E4M3 && format != PKV_Q8_INT8) return 0;
  const int G = n_h / n_kv;
  size_t most = 0;                                             // for either output type
  for (int pair = 0; pair < 2; ++pair) {
    Q8Variant* v = lookup_q8(head_dim, block_size, G, format == PKV_Q8_E4M3, pair != 0);
    if (!v) return 0;
    const size_t n = workspace_layout(batch, n_kv, G, head_dim, v->P).total;
    most = n > most ? n : most;
  }
  return most;
}

extern "C" pkv_status pkv_paged_decode_attn_q8(const void* q, const uint8_t* cache, int format, const int32_t* block_tables,
                                               int max_blocks, const int32_t* context_lens, float scale, int window,
                                               int batch, int n_h, int n_kv, int head_dim, int block_size, int num_blocks,
                                               void* out, int out_dtype, void* workspace, size_t workspace_bytes,
                                               int32_t* err_flag, void* stream) {
  PKV_NVTX("pkv_paged_decode_attn_q8");
  if (batch < 0 || !valid_shape(n_h, n_kv, head_dim, block_size) || max_blocks < 0 || num_blocks < 0 || window < 0)
    return PKV_EINVAL;
  if (format != PKV_Q8_E4M3 && format != PKV_Q8_INT8) return PKV_EINVAL;
  if (out_dtype != PKV_OUT_BF16 && out_dtype != PKV_OUT_F32) return PKV_EINVAL;
  if (batch == 0) return PKV_OK;
  if (!q || !cache || !block_tables || !context_lens || !out || !workspace) return PKV_EINVAL;
  if (!al16(q) || !al16(cache) || !al16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return PKV_EINVAL;
  if ((long long)max_blocks * block_size > kStreamMaxCtx) return PKV_ERANGE;
  const int G = n_h / n_kv;
  Q8Variant* v = lookup_q8(head_dim, block_size, G, format == PKV_Q8_E4M3, out_dtype == PKV_OUT_F32);
  if (!v) {
    record_cuda_error(cudaGetLastError());
    return PKV_ECUDA;
  }
  const WorkspaceLayout wl = workspace_layout(batch, n_kv, G, head_dim, v->P);
  if (workspace_bytes < wl.total) return PKV_ENOSPC;
  char* ws = static_cast<char*>(workspace);
  DecodeArgs a = {};
  a.q = q;
  a.bt = block_tables;
  a.max_blocks = max_blocks;
  a.cum = reinterpret_cast<int32_t*>(ws + wl.cum);
  a.ctx_eff = reinterpret_cast<int32_t*>(ws + wl.ctx);
  a.ctx_raw = context_lens;
  a.max_ctx = max_blocks * block_size;
  const int unit = block_size == 16 ? 16 : 32;                // blocks of 64 tokens count as two units of 32
  a.block_size = unit;
  a.inline_plan = batch <= kInlinePlanSeqs;
  a.pieces = reinterpret_cast<int4*>(ws + wl.pieces);
  a.P_launch = v->P;
  a.batch = batch;
  a.n_h = n_h;
  a.n_kv = n_kv;
  a.G = G;
  a.num_blocks = num_blocks;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = out;
  a.out_f32 = out_dtype == PKV_OUT_F32;
  a.ws_ml = reinterpret_cast<float*>(ws + wl.ml);
  a.ws_o = reinterpret_cast<float*>(ws + wl.o);
  a.err = err_flag;
  a.stages = v->stages;
  a.window = window;
  a.cache = cache;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int sub = block_size == 64 ? 1 : 0;
  cudaError_t e = a.inline_plan ? cudaSuccess
                                : launch_plan_streams(context_lens, batch, max_blocks * block_size, unit, a, v->P, st);
  if (e == cudaSuccess) {
    void* kargs[] = {&a, &sub};
    e = launch_pdl(v->fn, dim3(v->P / v->streams), dim3(v->warps * 32), v->smem, st, kargs);
  }
  if (e == cudaSuccess) e = launch_reduce_streams(head_dim, a, v->P, nullptr, st);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return PKV_ECUDA;
  }
  return PKV_OK;
}
