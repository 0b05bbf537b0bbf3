// Paged decode attention over the bf16 cache that also adds each cached token's attention
// weight, summed over the query heads of its kv group, to a per-sequence account:
//   out[s][h] = sum_t p[h][t] v_t,   mass[s][g][t] += sum_{h in g} p[h][t],   p = softmax(scale q k).
//
// Mathematics: a token's weight needs the final softmax state (M, L) of its row, which is known
// only after the whole context was read.  Reading K a second time would add half of the
// attention's traffic; the scores themselves are 4 G bytes per token and kv head against the
// 4 d bytes of its K and V.  So the attention kernel stores the scaled scores (base-2 units,
// fp32, as they entered the softmax) in the workspace, each row's (M, 1 / L) is stored by
// whoever finishes the row, and a second kernel adds sum_h 2^(x_h - M_h) / L_h to the account.
// Every token's sum is taken by one thread group in a fixed order: no atomics, the same bits on
// every call.
//
// What bounds it: HBM for K and V; the scores of a step mostly stay in L2 between the two
// kernels.  Structure of the attention kernel: the persistent grid of decode_common.cuh with the
// streams of piece_streams.cuh, in units of 16 tokens whatever the block size: a TMA box of 16 rows
// starts inside a larger block as well.  K and V land in 128-byte swizzled boxes and are read by
// ldmatrix.
// Measured: 64 x 0.5-4K tokens, 32 heads on 8 of 128, 110 us (83% of the copy rate; the attention 97,
// merge and addition in series behind it); 8 x 20-40K tokens, 32 heads on one, 42.2 us (30 the
// attention, bound by each consumer warp's chain of products and softmax); small calls 8-11 us.
#include <cmath>
#include <cstdlib>
#include <mutex>
#include <type_traits>

#include "nvtx_range.h"
#include "piece_streams.cuh"
#include "stream_plan.cuh"

namespace pkv {

struct MassArgs {
  float* scores;                 // workspace: [batch][n_kv][max_ctx][G], base-2 units
  float2* fin;                   // workspace: [batch][n_h] (offset, 1 / sum)
};

__host__ __device__ constexpr size_t mass_smem_bytes(int streams, int stages, int stage_bytes) {
  return 1024 + (size_t)streams * stages * (stage_bytes + 16 + 16);
}

// Keep the halves of a pair of rows (t, t + 1) below ntok; zero the others.
__device__ __forceinline__ uint32_t keep_rows(uint32_t b, int t, int ntok) {
  return b & ((t < ntok ? 0x0000ffffu : 0u) | (t + 1 < ntok ? 0xffff0000u : 0u));
}

// TT: 16-token units per stage; NH n-tiles of 8 heads per consumer warp, MT consumer warps per
// stream, NW streams.  sub: log2 of the units per table block.  PARTS: bf16 parts of p (8 bits each).
// COMB (groups of up to 4 heads): column n of the n-tile holds head n % 4, so that two products carry
// three parts.
template <int D, int TT, int NH, int MT, int NW, int PARTS, bool COMB>
__global__ void __launch_bounds__((NW * MT + 1) * 32, MT == 4 && NH == 1 ? 3 : (NH == 2 ? 2 : 1))
    decode_mass_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                       const DecodeArgs a, const MassArgs ms, const int sub) {
  constexpr int KS = D / 16, MD = D / 16, HW = 8 * NH, NBOX = D / 64;
  constexpr int PROD = COMB ? 2 : PARTS;
  constexpr int BS = 16, BOX = BS * 128, TILE = BS * D * 2, STAGE = TT * 2 * TILE;
  static_assert(!COMB || (NH == 1 && MT == 1 && PARTS == 3), "one n-tile holds the whole group");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int S = a.stages;
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
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
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
    produce_streams(a, starts, NW, S, TT, sub, (uint32_t)(2 * TILE), 2 * D, meta, full, empty, &abort_flag,
                    [&](int w, int slot, int k, int phys, int u, int kvh) {
                      uint8_t* st = smem + (size_t)(w * S + slot) * STAGE + k * 2 * TILE;
                      const int row = (kvh << sub | (u & ((1 << sub) - 1))) * BS;
#pragma unroll
                      for (int b = 0; b < NBOX; ++b) {
                        tma_load_3d(st + b * BOX, &tmk, b * 64, row, phys, &full[w * S + slot], pol);
                        tma_load_3d(st + TILE + b * BOX, &tmv, b * 64, row, phys, &full[w * S + slot], pol);
                      }
                    });
    return;
  }

  // ---------------- consumer warp: local heads [warp % MT * HW, + HW) of its stream ----------------
  const int w = warp / MT;
  if (starts[w].len <= 0) return;
  const int p = blockIdx.x * NW + w;
  smem += (size_t)w * S * STAGE;
  meta += w * S;
  full += w * S;
  empty += w * S;
  uint32_t qb[KS][NH][2];
  float o[MD][NH][4];
  float m[NH][2], l[NH][2];
  const int hw0 = warp % MT * HW;
  const bool even = (a.G & 1) == 0;
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
    const int s = mt.x, g = mt.y, ntok = mt.w & 255, flags = (mt.w >> 8) & 255;
    const size_t qrow0 = (size_t)s * a.n_h + (size_t)g * a.G;
    // this thread's score of token t of the stage and its head column n: at sp[t * G + n]
    float* sp = ms.scores + (((size_t)s * a.n_kv + g) * a.max_ctx + (size_t)mt.z * BS) * a.G + hw0 + 2 * tig;

    if (flags & F_FIRST) {
      if (!have_q) load_q(qrow0);
      have_q = false;
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        m[nh][0] = m[nh][1] = -INFINITY;
        l[nh][0] = l[nh][1] = 0.f;
#pragma unroll
        for (int md = 0; md < MD; ++md) o[md][nh][0] = o[md][nh][1] = o[md][nh][2] = o[md][nh][3] = 0.f;
      }
    }

    if (flags & F_VALID) {
      const uint32_t st = smem_u32(smem + (size_t)slot * STAGE);
      const int tiles = (ntok + 15) >> 4, mi = lane >> 3;
      // ---- S^T = K Q^T ----
      float sc[TT][NH][4];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[t][nh][i] = 0.f;
        if (t >= tiles) continue;
        const uint32_t kb = st + (uint32_t)(t * 2 * TILE);
        const int tok = ((mi & 1) << 3) + (lane & 7);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int ch = 2 * ks + (mi >> 1);
          uint32_t ka[4];
          ldsm_x4(ka[0], ka[1], ka[2], ka[3], kb + (ch >> 3) * BOX + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma_bf16(sc[t][nh], ka, qb[ks][nh][0], qb[ks][nh][1]);
        }
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            sc[t][nh][2 * r] *= a.scale_log2;
            sc[t][nh][2 * r + 1] *= a.scale_log2;
            const int tk = t * 16 + gid + 8 * r, n = hw0 + nh * 8 + 2 * tig;
            if (tk < ntok && n < a.G) {
              float* d = sp + (size_t)tk * a.G + nh * 8;
              if (even) {
                *reinterpret_cast<float2*>(d) = make_float2(sc[t][nh][2 * r], sc[t][nh][2 * r + 1]);
              } else {
                d[0] = sc[t][nh][2 * r];
                if (n + 1 < a.G) d[1] = sc[t][nh][2 * r + 1];
              }
            }
          }
      }
      softmax_tile<TT, NH, MD>(sc, m, l, o, gid, ntok, 0, 1.f);
      // ---- O^T += V^T P^T, a product per part of P; COMB: the high parts in columns 0-3 with the middle
      // ones in columns 4-7, then the low parts ----
      const bool partial = ntok < TT * 16;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (t >= tiles) continue;
        const uint32_t vb = st + (uint32_t)(t * 2 * TILE + TILE);
        const int tok = ((mi >> 1) << 3) + (lane & 7);
        uint32_t bp[PROD][NH][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float x = sc[t][nh][2 * r], y = sc[t][nh][2 * r + 1];
            const uint32_t hi = pack_bf16(x, y);
            const float x1 = x - bf16_lo(hi), y1 = y - bf16_hi(hi);
            const uint32_t mid = pack_bf16(x1, y1);
            const uint32_t lo = pack_bf16(x1 - bf16_lo(mid), y1 - bf16_hi(mid));
            bp[0][nh][r] = movmatrix_t(COMB && tig >= 2 ? mid : hi);
            bp[1][nh][r] = movmatrix_t(COMB ? (tig >= 2 ? 0u : lo) : mid);
            if constexpr (PROD == 3) bp[2][nh][r] = movmatrix_t(lo);
          }
        const int t0 = t * 16 + 2 * tig;
#pragma unroll
        for (int md = 0; md < MD; ++md) {
          const int ch = 2 * md + (mi & 1);
          uint32_t va[4];
          ldsm_x4_t(va[0], va[1], va[2], va[3], vb + (ch >> 3) * BOX + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
          if (partial) {
            va[0] = keep_rows(va[0], t0, ntok);
            va[1] = keep_rows(va[1], t0, ntok);
            va[2] = keep_rows(va[2], t0 + 8, ntok);
            va[3] = keep_rows(va[3], t0 + 8, ntok);
          }
#pragma unroll
          for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int i = 0; i < PROD; ++i) mma_bf16(o[md][nh], va, bp[i][nh][0], bp[i][nh][1]);
        }
      }
    } else {
      // a block outside the pool: its tokens weigh nothing
      for (int t = gid; t < ntok; t += 8)
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (hw0 + nh * 8 + 2 * tig + e < a.G) sp[(size_t)t * a.G + nh * 8 + e] = -INFINITY;
    }

    if (flags & F_LAST) {
      const bool whole = flags & F_WHOLE;
      const long long part = (long long)s * a.n_kv + g + p;
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        if constexpr (COMB) {                                  // the middle parts' columns lie two lanes on
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
            if (gid == 0) ms.fin[qrow0 + hl] = make_float2(m[nh][e] == -INFINITY ? 0.f : m[nh][e], inv);
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

// mass[s][g][t] += sum over the group's heads of 2^(x - M) / L.  LT lanes share a token's G scores
// (vectors of four where G allows), so a warp reads whole lines, and add their parts by a fixed
// tree; a lane has the loads of U tokens in flight (one at a time left the kernel at 2.2 TB/s of
// scores on 32-head groups).  CTA (c, s, g) takes 256 / LT * U tokens of the table's width; those behind
// the context leave at once, which a table far wider than the contexts still feels (64 x 0.5-4K tokens,
// 8 kv heads: 100 us with a table of 4096 tokens, 111 with 32768, 145 with 131072).
template <bool V4> struct ScoreVec { using type = float4; };
template <> struct ScoreVec<false> { using type = float; };

template <int LT, bool V4, int U>
__global__ void __launch_bounds__(256) mass_add_kernel(const float* scores, const float2* fin, const int32_t* ctx, int max_ctx,
                                                       int n_kv, int G, float* mass, long long mass_stride, int chunks) {
  constexpr int STEP = 256 / LT;
  __shared__ float2 f[64];
  const int chunk = blockIdx.x % chunks, sg = blockIdx.x / chunks, s = sg / n_kv;
  grid_dep_wait();                                            // every thread: see decode_plan.cu's reduce
  const int n = clamp_ctx(ctx[s], max_ctx);
  if (chunk * STEP * U >= n) return;
  const int sub = threadIdx.x % LT, t0 = chunk * STEP * U + threadIdx.x / LT;
  const float* x = scores + ((size_t)sg * max_ctx) * G;
  float* mrow = mass + (size_t)sg * mass_stride;
  // the first scores are asked for together with the states
  using Vec = typename ScoreVec<V4>::type;
  const int vecs = V4 ? G / 4 : G;
  auto score = [&](int u, int i) {
    Vec v = {};
    if (t0 + u * STEP < n && i < vecs) v = __ldcs(reinterpret_cast<const Vec*>(x + (size_t)(t0 + u * STEP) * G) + i);
    return v;
  };
  float before[U], w[U];
  Vec v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = score(u, sub);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    w[u] = 0.f;
    before[u] = sub == 0 && t0 + u * STEP < n ? mrow[t0 + u * STEP] : 0.f;
  }
  if (threadIdx.x < G) f[threadIdx.x] = fin[(size_t)sg * G + threadIdx.x];
  __syncthreads();
  for (int i = sub; i < vecs; i += LT) {
    if constexpr (V4) {
      const float2 f0 = f[4 * i], f1 = f[4 * i + 1], f2 = f[4 * i + 2], f3 = f[4 * i + 3];
#pragma unroll
      for (int u = 0; u < U; ++u)
        w[u] += ex2(v[u].x - f0.x) * f0.y + ex2(v[u].y - f1.x) * f1.y + ex2(v[u].z - f2.x) * f2.y + ex2(v[u].w - f3.x) * f3.y;
    } else {
      const float2 fi = f[i];
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] += ex2(v[u] - fi.x) * fi.y;
    }
    if (i + LT < vecs) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = score(u, i + LT);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int o = LT / 2; o; o >>= 1) w[u] += __shfl_xor_sync(FULL_MASK, w[u], o);
    if (sub == 0 && t0 + u * STEP < n) mrow[t0 + u * STEP] = before[u] + w[u];
  }
}

struct MassAdd {
  const void* fn;
  int tokens;                    // per CTA
};
static MassAdd mass_add(int G) {
  if (G % 4 && G >= 8) return {(const void*)mass_add_kernel<4, false, 8>, 512};
  if (G % 4) return {(const void*)mass_add_kernel<1, false, 4>, 1024};
  if (G >= 32) return {(const void*)mass_add_kernel<8, true, 8>, 256};
  if (G >= 16) return {(const void*)mass_add_kernel<4, true, 8>, 512};
  if (G >= 8) return {(const void*)mass_add_kernel<2, true, 4>, 512};
  return {(const void*)mass_add_kernel<1, true, 4>, 1024};
}

// ---------------------------------------------------------------------------------------------
struct MassVariant {
  const void* fn;
  int stages, warps, streams, P;
  size_t smem;
};

// Streams, consumer warps and heads per warp by group.  One kv head, 17-32 heads, d = 128: four warps
// of 8 heads, three CTAs per SM, 42.4 us for 8 x 20-40K tokens (64 x 2-8K: 54.6) against 43.8 (55.8)
// with two warps of 16; at d = 64, 43.2 against 42.0 the other way.
// Parts of p: three, all of its 24 bits, for groups of up to eight heads, where they cost nothing (64 x
// 0.5-4K tokens, four heads: 101.7 us with two and with three; 32 x 2-8K, eight heads: 122.6 and 122.1),
// and for fp32 outputs.  For bf16 outputs of larger groups two, 16 bits: an error of at most 2^-17 sum p |v|
// ahead of the output's own rounding of 2^-8 (64 x 2-8K tokens, 16 / 32 / 64 heads on one: 43.1 / 53.7 /
// 85.7 us; with three parts 45.3 / 57.9 / 95.9).
template <int D>
static void mass_pick(int tiling, int G, bool all_bits, MassVariant& v) {
  constexpr int T1 = D == 128 ? 1 : 2;                         // stages of 8 KB
  auto set = [&](const void* fn, int mt, int nw) {
    v.fn = fn;
    v.streams = nw;
    v.warps = nw * mt + 1;
  };
  auto pick = [&](auto parts) {
    constexpr int N = decltype(parts)::value;
    if (tiling == 1) set((const void*)decode_mass_kernel<D, 2, 2, 1, 3, N, false>, 1, 3);
    else if (tiling == 3) set((const void*)decode_mass_kernel<D, 2, 2, 4, 1, N, false>, 4, 1);
    else if constexpr (D == 128) set((const void*)decode_mass_kernel<D, 2, 1, 4, 1, N, false>, 4, 1);
    else set((const void*)decode_mass_kernel<D, 2, 2, 2, 2, N, false>, 2, 2);
  };
  if (G <= 4) set((const void*)decode_mass_kernel<D, T1, 1, 1, 3, 3, true>, 1, 3);
  else if (tiling == 0) set((const void*)decode_mass_kernel<D, T1, 1, 1, 3, 3, false>, 1, 3);
  else if (all_bits) pick(std::integral_constant<int, 3>{});
  else pick(std::integral_constant<int, 2>{});
}

static MassVariant* lookup_mass(int D, int G, bool all_bits) {
  // One table per process; the library drives one device per process.
  static std::mutex mu;
  static MassVariant table[2][5][2];
  static bool ready[2][5][2] = {};
  const int di = D == 128 ? 1 : 0, tiling = head_tiling(G), vi = G <= 4 ? 0 : tiling + 1, pi = all_bits || G <= 8 ? 1 : 0;
  std::lock_guard<std::mutex> lock(mu);
  MassVariant& v = table[di][vi][pi];
  if (!ready[di][vi][pi]) {
    const int stage = D == 128 && tiling >= 1 ? 16384 : 8192;
    if (D == 128) mass_pick<128>(tiling, G, all_bits, v);
    else mass_pick<64>(tiling, G, all_bits, v);
    // Stages of a ring: groups of up to eight heads stream with two (three: 110.8 -> 114.9 us for 64 x
    // 0.5-4K tokens, 32 heads on 8); larger groups, whose stages take longer to consume, with three
    // (16 heads 47.7 -> 44.2 us, 32 heads at d = 64 45.0 -> 42.0).
    v.stages = ring_stages(stage, (tiling == 0 ? 2 : 3) * stage, "PKV_STAGES_MASS");
    v.smem = mass_smem_bytes(v.streams, v.stages, stage);
    if (cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)v.smem) != cudaSuccess) return nullptr;
    int occ = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, v.fn, v.warps * 32, v.smem) != cudaSuccess || occ < 1)
      return nullptr;
    v.P = device_sm_count() * occ * v.streams;
    ready[di][vi][pi] = true;
  }
  return &v;
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static bool valid_shape(int n_h, int n_kv, int head_dim, int block_size) {
  if (head_dim != 64 && head_dim != 128) return false;
  if (block_size != 16 && block_size != 32 && block_size != 64) return false;
  if (n_kv <= 0 || n_h <= 0 || n_h % n_kv) return false;
  return n_h / n_kv <= 64;
}

struct MassLayout {
  WorkspaceLayout w;
  size_t fin, scores, total;
};
static MassLayout mass_layout(int B, int n_h, int n_kv, int D, long long max_ctx, int P) {
  MassLayout x;
  x.w = workspace_layout(B, n_kv, n_h / n_kv, D, P);
  x.fin = x.w.total;
  x.scores = align_up(x.fin + sizeof(float2) * (size_t)B * n_h, 256);
  x.total = align_up(x.scores + sizeof(float) * (size_t)B * n_h * (size_t)max_ctx, 256);
  return x;
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_mass_workspace_bytes(int batch, int n_h, int n_kv, int head_dim, int block_size, int max_blocks) {
  if (batch < 0 || max_blocks < 0 || !valid_shape(n_h, n_kv, head_dim, block_size)) return 0;
  if ((long long)max_blocks * block_size > kStreamMaxCtx) return 0;
  size_t most = 0;                                             // for either output type
  for (int all_bits = 0; all_bits < 2; ++all_bits) {
    MassVariant* v = lookup_mass(head_dim, n_h / n_kv, all_bits != 0);
    if (!v) return 0;
    const size_t n = mass_layout(batch, n_h, n_kv, head_dim, (long long)max_blocks * block_size, v->P).total;
    most = n > most ? n : most;
  }
  return most;
}

extern "C" pkv_status pkv_paged_decode_attn_mass(const void* q, const void* k_pool, const void* v_pool,
                                                 const int32_t* block_tables, int max_blocks, const int32_t* context_lens,
                                                 float scale, int batch, int n_h, int n_kv, int head_dim, int block_size,
                                                 int num_blocks, void* out, int out_dtype, float* mass, int64_t mass_stride,
                                                 void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream) {
  PKV_NVTX("pkv_paged_decode_attn_mass");
  if (batch < 0 || !valid_shape(n_h, n_kv, head_dim, block_size) || max_blocks < 0 || num_blocks < 0) return PKV_EINVAL;
  if (out_dtype != PKV_OUT_BF16 && out_dtype != PKV_OUT_F32) return PKV_EINVAL;
  if (batch == 0) return PKV_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !context_lens || !out || !mass || !workspace) return PKV_EINVAL;
  if (!al16(q) || !al16(k_pool) || !al16(v_pool) || !al16(out) || (reinterpret_cast<uintptr_t>(mass) & 3u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return PKV_EINVAL;
  const long long max_ctx = (long long)max_blocks * block_size;
  if (max_ctx > kStreamMaxCtx) return PKV_ERANGE;
  if (mass_stride < max_ctx) return PKV_EINVAL;
  const int G = n_h / n_kv;
  const MassAdd add = mass_add(G);
  const long long chunks = (max_ctx + add.tokens - 1) / add.tokens;
  if (chunks * batch * n_kv > 0x7fffffffLL) return PKV_ERANGE;
  MassVariant* v = lookup_mass(head_dim, G, out_dtype == PKV_OUT_F32);
  if (!v) {
    record_cuda_error(cudaGetLastError());
    return PKV_ECUDA;
  }
  const MassLayout ml = mass_layout(batch, n_h, n_kv, head_dim, max_ctx, v->P);
  if (workspace_bytes < ml.total) return PKV_ENOSPC;

  CUtensorMap tmk, tmv;
  const uint64_t rows = (uint64_t)n_kv * block_size;
  const uint64_t row_bytes = (uint64_t)head_dim * 2, block_bytes = rows * row_bytes;
  const uint64_t nblk = num_blocks > 0 ? (uint64_t)num_blocks : 1;
  if (encode_tensor_map_3d(&tmk, k_pool, head_dim, rows, nblk, row_bytes, block_bytes, 64, 16) ||
      encode_tensor_map_3d(&tmv, v_pool, head_dim, rows, nblk, row_bytes, block_bytes, 64, 16))
    return PKV_ECUDA;

  char* ws = static_cast<char*>(workspace);
  DecodeArgs a = {};
  a.q = q;
  a.bt = block_tables;
  a.max_blocks = max_blocks;
  a.cum = reinterpret_cast<int32_t*>(ws + ml.w.cum);
  a.ctx_eff = reinterpret_cast<int32_t*>(ws + ml.w.ctx);
  a.ctx_raw = context_lens;
  a.max_ctx = (int)max_ctx;
  a.block_size = 16;                                          // the line is in units of 16 tokens
  a.inline_plan = batch <= kInlinePlanSeqs;
  a.pieces = reinterpret_cast<int4*>(ws + ml.w.pieces);
  a.P_launch = v->P;
  a.batch = batch;
  a.n_h = n_h;
  a.n_kv = n_kv;
  a.G = G;
  a.num_blocks = num_blocks;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = out;
  a.out_f32 = out_dtype == PKV_OUT_F32;
  a.ws_ml = reinterpret_cast<float*>(ws + ml.w.ml);
  a.ws_o = reinterpret_cast<float*>(ws + ml.w.o);
  a.err = err_flag;
  a.stages = v->stages;
  MassArgs ma = {reinterpret_cast<float*>(ws + ml.scores), reinterpret_cast<float2*>(ws + ml.fin)};
  int sub = block_size == 16 ? 0 : (block_size == 32 ? 1 : 2);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = a.inline_plan ? cudaSuccess : launch_plan_streams(context_lens, batch, (int)max_ctx, 16, a, v->P, st);
  if (e == cudaSuccess) {
    void* kargs[] = {&tmk, &tmv, &a, &ma, &sub};
    e = launch_pdl(v->fn, dim3(v->P / v->streams), dim3(v->warps * 32), v->smem, st, kargs);
  }
  if (e == cudaSuccess) e = launch_reduce_streams(head_dim, a, v->P, ma.fin, st);
  if (e == cudaSuccess && chunks > 0) {
    const float* scores = ma.scores;
    const float2* fin = ma.fin;
    int mc = (int)max_ctx, nk = n_kv, gg = G, nc = (int)chunks;
    long long stride = mass_stride;
    void* kargs[] = {&scores, &fin, (void*)&context_lens, &mc, &nk, &gg, &mass, &stride, &nc};
    e = launch_pdl(add.fn, dim3((unsigned)(chunks * batch * n_kv)), dim3(256), 0, st, kargs);
  }
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return PKV_ECUDA;
  }
  return PKV_OK;
}
