// Quantization of one (token, group) pair of activations by a 16-lane quarter of a wave,
// shared by the kernels that write the GEMM's row operands (mixllm_quant_act.hip has the
// arithmetic's definition, mixllm_norm.hip the norms fused with it).
#ifndef MIXLLM_QUANT_PAIR_H_
#define MIXLLM_QUANT_PAIR_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm.h"
#include "mixllm_lanes.h"

#ifndef MIXLLM_QA_DIV
#define MIXLLM_QA_DIV 0
#endif

namespace mixllm {

__device__ __forceinline__ float h2f(uint32_t bits16) { return up<false>(bits16); }

// Reductions over the 16 lanes of a quarter (a DPP row).
__device__ __forceinline__ float quarter_max(float v) {
  v = fmaxf(v, moved<kDppXor1>(v));
  v = fmaxf(v, moved<kDppXor2>(v));
  v = fmaxf(v, moved<kDppHalfMirror>(v));
  v = fmaxf(v, moved<kDppMirror>(v));
  return v;
}

__device__ __forceinline__ int quarter_sum(int v) {
  v += moved<kDppXor1>(v);
  v += moved<kDppXor2>(v);
  v += moved<kDppHalfMirror>(v);
  v += moved<kDppMirror>(v);
  return v;
}

// x = p0 + p1 + p2 exactly, each a bf16 (returned as p | p << 16 words).
__device__ __forceinline__ void split3(float x, uint32_t w[3]) {
  const uint32_t b0 = __float_as_uint(x) & 0xFFFF0000u;
  const float r1 = x - __uint_as_float(b0);
  const uint32_t b1 = __float_as_uint(r1) & 0xFFFF0000u;
  const uint32_t b2 = __float_as_uint(r1 - __uint_as_float(b1)) & 0xFFFF0000u;
  w[0] = b0 | (b0 >> 16);
  w[1] = b1 | (b1 >> 16);
  w[2] = b2 | (b2 >> 16);
}

// The 8 values of lane `sub` of one (token, group) pair, held by a 16-lane quarter: reduce,
// quantize, store.
__device__ __forceinline__ void quant_values(const float x[8], bool live, int64_t m, int g, int sub, int32_t M,
                                             int32_t K, int8_t *__restrict__ aq, float *__restrict__ sa,
                                             int32_t *__restrict__ asum, uint4 *__restrict__ rowop) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = quarter_max(amax);
  const float s = amax / 127.0f;

  int q[8];
  int qsum = 0;
#if MIXLLM_QA_DIV
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v = amax > 0.0f ? __builtin_rintf(x[i] / s) : 0.0f;
    v = fminf(fmaxf(v, -127.0f), 127.0f);
    q[i] = (int)v;
    qsum += q[i];
  }
#else
  // rne(x / s) without a division per code: t = x * rcp(s) differs from the correctly
  // rounded quotient by less than 6e-5 (|x / s| <= 127, v_rcp_f32 within 1 ulp, one more
  // rounding in the product), so rne(t) is rne(x / s) unless t lies within 2^-12 of a
  // half-integer; those codes take the IEEE division.
  const float r = __builtin_amdgcn_rcpf(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = x[i] * r;
    float v = __builtin_rintf(t);
    if (fabsf(t - v) > 0.5f - 0x1p-12f) v = __builtin_rintf(x[i] / s);
    v = amax > 0.0f ? fminf(fmaxf(v, -127.0f), 127.0f) : 0.0f;
    q[i] = (int)v;
    qsum += q[i];
  }
#endif
  qsum = quarter_sum(qsum);
  if (!live) return;

  uint2 packed;
  packed.x = (uint32_t)(q[0] & 0xFF) | ((uint32_t)(q[1] & 0xFF) << 8) | ((uint32_t)(q[2] & 0xFF) << 16) |
             ((uint32_t)(q[3] & 0xFF) << 24);
  packed.y = (uint32_t)(q[4] & 0xFF) | ((uint32_t)(q[5] & 0xFF) << 8) | ((uint32_t)(q[6] & 0xFF) << 16) |
             ((uint32_t)(q[7] & 0xFF) << 24);
  *reinterpret_cast<uint2 *>(aq + m * K + (int64_t)g * MIXLLM_GROUP + sub * 8) = packed;
  if (sub == 0) {
    sa[(int64_t)g * M + m] = s;
    if (asum) asum[(int64_t)g * M + m] = qsum;
  }
  if (rowop && sub < 2) {
    uint32_t ws[3], wu[3];
    split3(s, ws);
    split3((float)qsum * s, wu);
    rowop[((int64_t)g * M + m) * 2 + sub] =
        sub == 0 ? make_uint4(ws[0], ws[1], ws[2], 0u) : make_uint4(wu[0], wu[1], wu[2], 0u);
  }
}

// The same from 8 packed fp16 values.
__device__ __forceinline__ void quant_pair(uint4 raw, bool live, int64_t m, int g, int sub, int32_t M, int32_t K,
                                           int8_t *__restrict__ aq, float *__restrict__ sa,
                                           int32_t *__restrict__ asum, uint4 *__restrict__ rowop) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = h2f(w[i] & 0xFFFFu);
    x[2 * i + 1] = h2f(w[i] >> 16);
  }
  quant_values(x, live, m, g, sub, M, K, aq, sa, asum, rowop);
}

}  // namespace mixllm

#endif  // MIXLLM_QUANT_PAIR_H_
