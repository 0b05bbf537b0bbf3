// A step's tokens by sequence (q_start of pkv.h): what the calls for drafted tokens share.
#pragma once

#include "decode_common.cuh"

namespace pkv {

// Sequence s of a step: its cached rows, its first token and its number of tokens.
struct Drafts {
  int ctx, q0, n;
};
// Reads lengths and starts that earlier kernels may have written: called behind the grid-dependency wait.
__device__ __forceinline__ Drafts drafts_of(const int32_t* ctx, const int32_t* q_start, int n_each, int n_tok, int max_ctx,
                                            int s, int& flags) {
  Drafts d;
  const int c = ctx[s];
  d.ctx = clamp_ctx(c, max_ctx);
  if (c != d.ctx) flags |= PKV_DEV_BAD_CTX;
  d.q0 = s * n_each;
  d.n = n_each;
  if (q_start) {
    const int a = q_start[s], b = q_start[s + 1];
    const bool good = a >= 0 && b >= a && b <= n_tok;
    if (!good) flags |= PKV_DEV_BAD_TREE;
    d.q0 = good ? a : 0;
    d.n = good ? b - a : 0;
  }
  if (d.ctx > 0 && d.ctx < d.n) flags |= PKV_DEV_BAD_TREE;
  return d;
}

// Whether two ranges of bytes share any (null: an argument that is not given).
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

}  // namespace pkv
