// Interface between the attention kernels with streams (piece_streams.cuh: decode_q8.cu,
// decode_mass.cu) and the plan and split-reduce kernels (decode_plan.cu).
#pragma once

#include "decode_common.cuh"

namespace pkv {

// Pieces of a line of W positions in `segments` segments on a grid of P streams.  Short contexts are
// cut finely, down to one position per piece: a stream takes about 1 us per segment in series, whatever
// is in it (one sequence of up to 66 tokens, 8 kv heads: 14.3 us with 8 positions per piece, 6.6 with
// one).  From 64 positions per segment on the pieces grow, to 8 positions, since a segment cut into
// more than about a hundred parts is merged slowly (1 x 11.7K tokens, 4 kv heads: 10.6 us with 8
// positions, 12.2 with two, 15.2 with one).
__host__ __device__ __forceinline__ int stream_pieces(long long W, long long segments, int P) {
  const int min_log2 = (W >= segments * 64) + (W >= segments * 128) + (W >= segments * 256);
  const long long q = (W + (1 << min_log2) - 1) >> min_log2;
  return (int)(q < 1 ? 1 : (q < P ? q : P));
}
// streams: whether the grid has streams (stream_pieces), else effective_pieces.
__host__ __device__ __forceinline__ int pieces_of(long long W, long long segments, int P, bool streams) {
  return streams ? stream_pieces(W, segments, P) : effective_pieces(W, P);
}

// launch_plan and launch_reduce for the kernels with streams; the reduce stores each merged row's final
// softmax state, (running offset in base-2 units, 1 / sum), at fin[row] unless fin is null.
cudaError_t launch_plan_streams(const int32_t* context_lens, int batch, int max_ctx, int block_size, const DecodeArgs& a,
                                int P, cudaStream_t stream);
cudaError_t launch_reduce_streams(int head_dim, const DecodeArgs& a, int P, float2* fin, cudaStream_t stream);

}  // namespace pkv
