// Layout of the 8-bit cache's records, shared by the quantizer and the attention kernel.
//
// One record per (block, kv head): K codes [bs * d], V codes [bs * d], the K and the V scale
// (fp32), 8 bytes of zeros.  The codes of a 16-token tile are stored in the order in which the
// lanes of a warp hold the operands of mma.m16n8k16, 16 bytes a lane for 32 channels, so the
// attention kernel takes its A fragments with one conflict-free 16-byte shared-memory load per
// lane and no transpose:
//   tile tt of 16 tokens -> group j of 32 channels -> lane (gid = lane / 4, tig = lane % 4)
//   K, byte 8 ks + 4 hi + 2 half + b:  token 16 tt + 8 hi + gid, channel 32 j + 16 ks + 8 half + 2 tig + b
//   V, byte 8 md + 4 hi + 2 half + b:  token 16 tt + 8 half + 2 tig + b, channel 32 j + 16 md + 8 hi + gid
#pragma once

#include "decode_common.cuh"

namespace pkv {

__host__ __device__ __forceinline__ int q8_record_bytes(int bs, int d) { return 2 * bs * d + 16; }

// Groups whose largest magnitude is below this count as zero (scale 0, codes 0): the
// reciprocal of a smaller one could overflow fp32.
constexpr float kQ8Tiny = 7.7037198e-34f;         // 2^-110

}  // namespace pkv
