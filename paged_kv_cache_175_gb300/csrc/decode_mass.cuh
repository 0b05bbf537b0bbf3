// Interface between the accounted attention (decode_mass.cu) and the split reduce (decode_plan.cu).
#pragma once

#include "decode_common.cuh"

namespace pkv {

// launch_reduce that also stores each merged row's final softmax state, (running offset in
// base-2 units, 1 / sum), at fin[row].
cudaError_t launch_reduce_fin(int head_dim, const DecodeArgs& a, int P, float2* fin, cudaStream_t stream);

}  // namespace pkv
