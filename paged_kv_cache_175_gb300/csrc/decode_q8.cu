// Paged decode attention over the 8-bit cache (GQA / MHA / MQA; record layout: q8_common.cuh).
//
// Mathematics: with K^ = s_k * c_k and V^ = s_v * c_v per (block, kv head), the scores of a
// block are (s_k * scale) * (c_k . q) and its output is s_v * sum_t p_t c_v,t: both scales stay
// outside the products, so the codes enter the tensor cores as they are.  Codes become fp16
// exactly (e4m3 and small integers are fp16 values).  q is bf16; each head's q is multiplied by
// a power of two that puts its largest value at 2^14, so that every value above 2^-31 of the
// largest is exact in fp16 (and the rest is off by 2^-39 of the largest at most); the power is
// taken out of the scores again.  p enters as a high + low pair of fp16 of 128 p (128: p <= 2^8
// by the lazy offset, so 2^15 at most, and the smallest step is 2^-31 of p = 1), which carries
// 22 bits.  Softmax, sums and outputs are fp32.
//
// Structure: the persistent grid and the line of blocks of decode_common.cuh.  A producer warp
// walks the CTA's piece and brings the records of up to TT / (bs / 16) consecutive blocks per
// stage into a ring, one contiguous bulk copy per record, issued by one lane each; consumer
// warps take 8 or 16 heads each.  Per 16-token tile, S^T = C_k Q^T and O^T += C_v^T P^T with
// mma.m16n8k16; the A fragments of both are one 16-byte load per lane and 32 channels, since the
// records hold the codes in fragment order.
#include <cmath>
#include <cstdlib>
#include <mutex>

#include "nvtx_range.h"
#include "piece_producer.cuh"
#include "q8_common.cuh"

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
__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float h2_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float h2_hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }
// Keep the halves of a pair of rows (t, t + 1) that lie in [lead, ntok); zero the others.
__device__ __forceinline__ uint32_t keep_pair(uint32_t b, int t, int lead, int ntok) {
  return b & ((t < ntok && t >= lead ? 0x0000ffffu : 0u) | (t + 1 < ntok && t + 1 >= lead ? 0xffff0000u : 0u));
}

constexpr float kPScale = 128.f;      // p enters the products times this

__host__ __device__ constexpr size_t q8_smem_bytes(int stages, int stage_bytes) {
  return 128 + (size_t)stages * (stage_bytes + 16 + 16);
}

// BSL: log2 of the block size is a runtime value (bs16l = log2(bs / 16)); TT: 16-token tiles per
// stage; NH n-tiles of 8 heads per consumer warp, MT consumer warps.
template <int D, int TT, int NH, int MT, bool E4M3>
__global__ void __launch_bounds__((MT + 1) * 32) decode_q8_kernel(const DecodeArgs a, const int bs16l) {
  constexpr int KS = D / 16, MD = D / 16, HW = 8 * NH;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t ring = (smem_u32(smem_raw) + 127u) & ~127u;
  const int S = a.stages, BS = 16 << bs16l, TPB = 1 << bs16l, NB = TT >> bs16l;
  const int REC = q8_record_bytes(BS, D), STAGE = NB * REC;
  uint8_t* smem = smem_raw + (ring - smem_u32(smem_raw));
  int4* meta = reinterpret_cast<int4*>(smem + (size_t)S * STAGE);
  uint64_t* full = reinterpret_cast<uint64_t*>(meta + S);
  uint64_t* empty = full + S;
  __shared__ volatile int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tig = lane & 3, gid = lane >> 2;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], MT);
    }
    fence_barrier_init();
  }
  __syncthreads();
  if (!a.inline_plan) grid_dep_wait();   // the plan kernel's cum / ctx_eff / cursors
  grid_dep_launch();

  Cursor cur;
  PieceInfo pi;
  piece_setup(a, blockIdx.x, gridDim.x, warp == MT, cur, pi);
  const int p = blockIdx.x;
  const int len = p < pi.P ? (int)(pi.pend - pi.pstart) : 0;
  // Every thread waits for the kernel before this one (the append), also those without work,
  // so that no later launch on the stream can pass it.
  if (len > 0 && warp == MT && lane == 0) prefetch_l2(a.bt + (size_t)cur.s * a.max_blocks + cur.b0 + cur.blk);
  if (a.inline_plan) grid_dep_wait();
  if (len <= 0) return;

  if (warp == MT) {
    const uint64_t pol = policy_evict_first();
    produce_piece(a, cur, pi, len, bs16l, NB, S, (uint32_t)REC, 2 * D, meta, full, empty, &abort_flag,
                  [&](int slot, int k, int phys, int kvh) {
                    bulk_g2s_u32(ring + (uint32_t)(slot * STAGE + k * REC),
                                 a.cache + ((size_t)phys * a.n_kv + kvh) * REC, REC, smem_u32(&full[slot]), pol);
                  });
    return;
  }

  // ---------------- consumer warp: local heads [warp * HW, warp * HW + HW) ----------------
  uint32_t qb[KS][NH][2];
  float o[MD][NH][4];
  float m[NH][2], l[NH][2], qs[NH][2];          // qs: what a head's scores are multiplied by
  const int hw0 = warp * HW;
  int slot = 0;
  uint32_t phase = 0;
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
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        const int hl = hw0 + nh * 8 + gid;                     // B-fragment column n = gid
        const uint32_t* qp = reinterpret_cast<const uint32_t*>(a.q) + (qrow0 + hl) * (D / 2);
        float big = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t w = hl < a.G ? __ldg(qp + ks * 8 + 4 * r + tig) : 0u;
            qb[ks][nh][r] = w;
            big = fmaxf(big, fmaxf(fabsf(bf16_lo(w)), fabsf(bf16_hi(w))));
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
      const int tiles = (ntok + 15) >> 4;
      // ---- S^T = C_k Q^T ----
      float sc[TT][NH][4];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[t][nh][i] = 0.f;
        if (t >= tiles) continue;
        const uint32_t rec = st + (uint32_t)((t >> bs16l) * REC);
        const uint32_t kb = rec + (uint32_t)((t & (TPB - 1)) * 16 * D) + lane * 16;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 w = lds128(kb + j * 512);
          uint32_t ka[4];
          codes_f16<E4M3>(w.x, ka[0], ka[2]);
          codes_f16<E4M3>(w.y, ka[1], ka[3]);
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma_f16(sc[t][nh], ka, qb[2 * j][nh][0], qb[2 * j][nh][1]);
          codes_f16<E4M3>(w.z, ka[0], ka[2]);
          codes_f16<E4M3>(w.w, ka[1], ka[3]);
#pragma unroll
          for (int nh = 0; nh < NH; ++nh) mma_f16(sc[t][nh], ka, qb[2 * j + 1][nh][0], qb[2 * j + 1][nh][1]);
        }
        const float sk = lds_f32(rec + 2 * BS * D);
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
          sc[t][nh][0] *= sk * qs[nh][0];
          sc[t][nh][1] *= sk * qs[nh][1];
          sc[t][nh][2] *= sk * qs[nh][0];
          sc[t][nh][3] *= sk * qs[nh][1];
        }
      }
      softmax_tile<TT, NH, MD>(sc, m, l, o, gid, ntok, lead, 1.f);
      // ---- O^T += s_v C_v^T P^T ----
      const bool partial = ntok < TT * 16 || lead > 0;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (t >= tiles) continue;
        const uint32_t rec = st + (uint32_t)((t >> bs16l) * REC);
        const uint32_t vb = rec + (uint32_t)(BS * D + (t & (TPB - 1)) * 16 * D) + lane * 16;
        const float sv = lds_f32(rec + 2 * BS * D + 4);
        uint32_t bh[NH][2], bl[NH][2];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float x = sc[t][nh][2 * r] * kPScale, y = sc[t][nh][2 * r + 1] * kPScale;
            const uint32_t hi = pack_f16(x, y);
            const uint32_t lo = pack_f16(x - h2_lo(hi), y - h2_hi(hi));
            bh[nh][r] = movmatrix_t(hi);
            bl[nh][r] = movmatrix_t(lo);
          }
        const int t0 = t * 16 + 2 * tig;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 w = lds128(vb + j * 512);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t va[4];
            codes_f16<E4M3>(h ? w.z : w.x, va[0], va[2]);
            codes_f16<E4M3>(h ? w.w : w.y, va[1], va[3]);
            if (partial) {
              va[0] = keep_pair(va[0], t0, lead, ntok);
              va[1] = keep_pair(va[1], t0, lead, ntok);
              va[2] = keep_pair(va[2], t0 + 8, lead, ntok);
              va[3] = keep_pair(va[3], t0 + 8, lead, ntok);
            }
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
              float acc[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(acc, va, bh[nh][0], bh[nh][1]);
              mma_f16(acc, va, bl[nh][0], bl[nh][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[2 * j + h][nh][i] = fmaf(sv, acc[i], o[2 * j + h][nh][i]);
            }
          }
        }
      }
    }

    if (flags & F_LAST) {
      const bool whole = flags & F_WHOLE;
      const long long part = (long long)s * a.n_kv + g + p;
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float L = l[nh][e];
          L += __shfl_xor_sync(FULL_MASK, L, 4);
          L += __shfl_xor_sync(FULL_MASK, L, 8);
          L += __shfl_xor_sync(FULL_MASK, L, 16);
          const int hl = hw0 + nh * 8 + 2 * tig + e;           // this thread's head columns
          if (hl >= a.G) continue;
          const float inv = (whole ? (L > 0.f ? 1.f / L : 0.f) : 1.f) * (1.f / kPScale);
          if (whole) {
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
              wo[md * 16 + gid] = o[md][nh][e] * inv;
              wo[md * 16 + gid + 8] = o[md][nh][2 + e] * inv;
            }
            if (gid == 0)
              *reinterpret_cast<float2*>(a.ws_ml + ((size_t)part * a.G + hl) * 2) = make_float2(m[nh][e], L);
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
  int stages, warps, P;
  size_t smem;
};

constexpr int kQ8Tiles = 4;           // 64 tokens per stage, whatever the block size

constexpr size_t kQ8MaxSmem = 200 * 1024;

template <int D, int NH, int MT, bool E4M3>
static const void* q8_fn() {
  return (const void*)decode_q8_kernel<D, kQ8Tiles, NH, MT, E4M3>;
}

static Q8Variant* lookup_q8(int D, int BS, int tiling, bool e4m3) {
  // One table per process; the library drives one device per process.
  static std::mutex mu;
  static Q8Variant table[2][3][4][2];
  static bool ready[2][3][4][2] = {};
  const int di = D == 128 ? 1 : 0, bi = BS == 16 ? 0 : (BS == 32 ? 1 : 2), fi = e4m3 ? 1 : 0;
  std::lock_guard<std::mutex> lock(mu);
  Q8Variant& v = table[di][bi][tiling][fi];
  if (!ready[di][bi][tiling][fi]) {
#define PKV_V(d, f)                                                                                        \
  if (D == d && e4m3 == f)                                                                                 \
    v.fn = tiling == 0 ? q8_fn<d, 1, 1, f>()                                                               \
                       : (tiling == 1 ? q8_fn<d, 1, 2, f>() : (tiling == 2 ? q8_fn<d, 2, 2, f>() : q8_fn<d, 2, 4, f>()));
    PKV_V(64, true) PKV_V(64, false) PKV_V(128, true) PKV_V(128, false)
#undef PKV_V
    v.warps = (tiling == 0 ? 1 : (tiling == 3 ? 4 : 2)) + 1;
    const int stage = (kQ8Tiles * 16 / BS) * q8_record_bytes(BS, D);
    v.stages = ring_stages(stage, 32768, "PKV_STAGES_Q8");
    v.smem = q8_smem_bytes(v.stages, stage);
    // one function serves several block sizes, whose rings differ a little: one limit for all
    if (v.smem > kQ8MaxSmem ||
        cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kQ8MaxSmem) != cudaSuccess)
      return nullptr;
    int occ = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, v.fn, v.warps * 32, v.smem) != cudaSuccess || occ < 1)
      return nullptr;
    v.P = device_sm_count() * occ;
    ready[di][bi][tiling][fi] = true;
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
  Q8Variant* v = lookup_q8(head_dim, block_size, head_tiling(G), format == PKV_Q8_E4M3);
  return v ? workspace_layout(batch, n_kv, G, head_dim, v->P).total : 0;
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
  if ((long long)max_blocks * block_size > 0x7fffffffLL) return PKV_ERANGE;
  const int G = n_h / n_kv;
  Q8Variant* v = lookup_q8(head_dim, block_size, head_tiling(G), format == PKV_Q8_E4M3);
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
  a.block_size = block_size;
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
  int bs16l = block_size == 16 ? 0 : (block_size == 32 ? 1 : 2);
  cudaError_t e = a.inline_plan ? cudaSuccess
                                : launch_plan(context_lens, batch, max_blocks * block_size, block_size, a, v->P, st);
  if (e == cudaSuccess) {
    void* kargs[] = {&a, &bs16l};
    e = launch_pdl(v->fn, dim3(v->P), dim3(v->warps * 32), v->smem, st, kargs);
  }
  if (e == cudaSuccess) e = launch_reduce(head_dim, a, v->P, st);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return PKV_ECUDA;
  }
  return PKV_OK;
}
