// Moves between the lanes of a wave and conversions of 16-bit values that the kernels share.
#ifndef MIXLLM_LANES_H_
#define MIXLLM_LANES_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mixllm {

// Lane moves inside a row of 16 lanes.  Swapping neighbours, swapping pairs and mirroring each
// 8-lane half and the row leaves, after the four steps of a reduction, the combination of all
// 16 lanes in every lane, without LDS.
constexpr int kDppXor1 = 0xB1;        // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;        // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;
constexpr int kDppMirror = 0x140;

// The 32-bit value v of the lane that the move names.
template <int CTRL, typename T>
__device__ __forceinline__ T moved(T v) {
  static_assert(sizeof(T) == 4, "one register");
  return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

// The value of the low 16 bits, fp16 or bf16, and the bits of a value rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ float up(uint32_t bits) {
  if (BF16) return __uint_as_float(bits << 16);
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

template <bool BF16>
__device__ __forceinline__ uint32_t down(float v) {
  if (BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

}  // namespace mixllm

#endif  // MIXLLM_LANES_H_
