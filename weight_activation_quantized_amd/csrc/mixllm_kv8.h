// Layout of the paged key/value cache held in 8 bits (one layer's cache), shared by the
// kernels that write it and the kernels that read it.  The layout is part of the C ABI
// (include/mixllm.h, "The cache in 8 bits").
//
// One block per (page, key/value head) of P tokens x D channels:
//   K codes   P * D          runs of 16 tokens, 16 D bytes each
//   V codes   P * D          the same
//   scales    8 * P / 16     fp32 pairs (of keys, of values) of the runs, padded to whole 128s
// and in a run, token t, channel ch:
//   keys      ch/64 * 1024 + ch/16%4 * 256 + t * 16 + ch%16
//   values    ch/64 * 1024 + t/4 * 256 + ch%16 * 16 + ch/16%4 * 4 + t%4
//
// Why this order: 1024 bytes of a run are one wide load of a wave, 16 bytes per lane and lane
// after lane, and what lane (n, c) = (lane % 16, lane / 16) gets is what the matrix
// instruction wants of it: for the scores 16 channels of token n, for the weighted sum
// tokens 4c .. 4c+3 of the four channels 16 j + n, whose probabilities the scores' result
// layout leaves in that lane.  Nothing moves between lanes and no LDS is needed on the way.
#ifndef MIXLLM_KV8_H_
#define MIXLLM_KV8_H_

#include "mixllm_kv4.h"

namespace mixllm {

constexpr int kKv8Run = 16;    // tokens that share a scale
constexpr int kKv8Zero = 128;  // the byte of code 0

__host__ __device__ constexpr int32_t kv8_scale_offset(int32_t page, int32_t dim) { return 2 * page * dim; }

// Bytes of one (page, head) block.
__host__ __device__ constexpr int32_t kv8_block_bytes(int32_t page, int32_t dim) {
  return 2 * page * dim + (page / 2 + 127) / 128 * 128;
}

inline int kv8_check_cache(const void *cache, size_t cache_bytes, int32_t pages, int32_t page, int32_t heads,
                           int32_t dim) {
  if (!kv4_dim_ok(dim) || !kv4_page_ok(page) || heads <= 0 || pages <= 0) return MIXLLM_E_SHAPE;
  if ((int64_t)pages * page > 0x7FFFFFFF) return MIXLLM_E_SHAPE;  // slots are int32
  if (!cache) return MIXLLM_E_NULL;
  if (!is_aligned16(cache)) return MIXLLM_E_SHAPE;
  if (cache_bytes / ((size_t)heads * kv8_block_bytes(page, dim)) < (size_t)pages) return MIXLLM_E_SPACE;
  return MIXLLM_OK;
}

}  // namespace mixllm

#endif  // MIXLLM_KV8_H_
