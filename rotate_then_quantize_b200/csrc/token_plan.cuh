// How token ranges are cut into chunks and parts. Positions go up to 2^31 -
// 65536 and a chunk may be nearly as long, so a sum of the two can pass 32 bits:
// every function here stays within them, and none needs the GPU.
#pragma once

#include <cstdint>

namespace srftq {

// No sequence is longer, so a chunk of this length holds any.
constexpr int32_t kMaxChunk = INT32_MAX / 128 * 128;

// Tokens per chunk, a multiple of 128, for `total` own tokens of a batch and a
// goal of `goal` chunks: sum ceil(own / chunk) <= goal + sequences.
__host__ __device__ inline int32_t chunk_tokens(int64_t total, int32_t goal) {
  const int64_t per = (total + goal - 1) / goal;
  return per >= kMaxChunk ? kMaxChunk : per <= 128 ? 128 : int32_t((per + 127) / 128 * 128);
}

// Chunks of a sequence with `own` tokens.
__host__ __device__ inline int32_t chunks_of(int32_t own, int32_t chunk) {
  return own > 0 ? (own - 1) / chunk + 1 : 0;
}

// End of the range of at most `length` tokens that starts at t0, in tokens that
// end at `end` (t0 itself or less when none are left).
__host__ __device__ inline int32_t range_end(int32_t t0, int32_t length, int32_t end) {
  return end - t0 > length ? t0 + length : end;
}

}  // namespace srftq
