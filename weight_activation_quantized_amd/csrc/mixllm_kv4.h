// Layout of the paged key/value cache held in 4 bits (one layer's cache), shared by the
// kernels that write it and the kernels that read it.  The layout is part of the C ABI
// (include/mixllm.h, "The cache").
//
// One block per (page, key/value head) of P tokens x D channels, D * P * 9 / 8 bytes:
//   K codes   P * D / 2      token t, quarter c (0..3), step s (0..D/32-1): one dword at
//                            t * D/2 + c * D/8 + 4 s with channels 32 s + 8 c + j, nibble j
//   V codes   P * D / 2      word (t / 4 * 16 + n) * 4 + t % 4 of D/32 bytes: column n
//                            (0..15), channels 16 j + n, nibble j (0..D/16-1)
//   K params  P * D / 16     token t: fp16 scales of its D/64 groups, then their minima
//   V params  P * D / 16     the same
//
// Why this order: the matrix instruction's operands hold 8 consecutive contraction indices
// per lane.  For the scores a lane (token n, quarter c) then reads its D/4 channels of one
// token with one wide load (16 bytes at D = 128) and each dword is one instruction's
// operand, all of one group of 64 channels, so a group's scale multiplies a whole partial
// product.  For the weighted sum of the values a lane (column n, quarter c) holds 4
// consecutive tokens of its column with one wide load, and the four tokens are the four
// that the scores' result layout leaves in that lane: the probabilities never move between
// lanes.
#ifndef MIXLLM_KV4_H_
#define MIXLLM_KV4_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm.h"

namespace mixllm {

bool is_aligned16(const void *p);

inline bool is_aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

inline bool kv4_dim_ok(int32_t dim) { return dim == 64 || dim == 128 || dim == 256; }

inline bool kv4_page_ok(int32_t page) { return page >= 16 && page <= 1024 && (page & (page - 1)) == 0; }

inline int32_t log2_of(int32_t power) {
  int32_t n = 0;
  while ((1 << n) < power) ++n;
  return n;
}

// Bytes of one (page, head) block.
__host__ __device__ constexpr int32_t kv4_block_bytes(int32_t page, int32_t dim) { return page * dim / 8 * 9; }

// Checks shared by every call that takes a cache.
inline int kv4_check_cache(const void *cache, size_t cache_bytes, int32_t pages, int32_t page, int32_t heads,
                           int32_t dim) {
  if (!kv4_dim_ok(dim) || !kv4_page_ok(page) || heads <= 0 || pages <= 0) return MIXLLM_E_SHAPE;
  if ((int64_t)pages * page > 0x7FFFFFFF) return MIXLLM_E_SHAPE;  // slots are int32
  if (!cache) return MIXLLM_E_NULL;
  if (!is_aligned16(cache)) return MIXLLM_E_SHAPE;
  if (cache_bytes / ((size_t)heads * kv4_block_bytes(page, dim)) < (size_t)pages) return MIXLLM_E_SPACE;
  return MIXLLM_OK;
}

inline int launch_status() { return hipGetLastError() == hipSuccess ? MIXLLM_OK : MIXLLM_E_HIP; }

}  // namespace mixllm

#endif  // MIXLLM_KV4_H_
