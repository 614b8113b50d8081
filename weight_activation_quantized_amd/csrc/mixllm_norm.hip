// The norms around a block, fused with its gate, the residual sum and the quantization of
// the next layer's activations.
//
//   u  = x / rms(x) * w_post           (or x, without a post norm)
//   h' = alpha * h + beta * gate * u   (written in the residual's type)
//   y  = h' / rms(h') * w_pre          (from the unrounded h'; written in 16 bits, and/or
//                                       quantized to int8 as mixllm_quant_act quantizes
//                                       the 16-bit y)
//   rms(v) = sqrt(mean(v^2) + eps)
//
// One pass over the data: a workgroup owns a row and holds it in registers (fp32) between
// the two reductions, so every input is read once and every output written once; separate
// kernels would write and read back u, h' and y.  Bound by HBM bandwidth for prompts (2047 rows
// of 8192, fp32 residual, to int8: 190 MB in 46.5 us, 4.1 TB/s; a large copy reaches 5.15) and by
// the latency of one load, two reductions and one store for single tokens (4 rows of 4096:
// 4.4 us, of which a launch is most).  Rows of more than 32768 hold 64 values a thread, some of
// which spill to scratch memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm.h"
#include "mixllm_kv4.h"
#include "mixllm_lanes.h"
#include "mixllm_quant_pair.h"

namespace {

using mixllm::down;
using mixllm::up;

struct NormArgs {
  const uint16_t *x, *post, *gate, *pre;
  const void *res;
  void *res_out;
  uint16_t *y;
  int8_t *aq;
  float *sa;
  int32_t *asum;
  uint4 *rowop;
  int64_t ldx, ldgate, ldr, ldro, ldy;
  int32_t M, N;
  float eps, alpha, beta;
  int32_t wide;  // rows can be read and written 8 elements at a time
};

// A thread's elements of a row: with wide accesses chunks of 8 neighbours, chunk c of
// thread t at (c * THREADS + t) * 8; else single elements, element c * 8 + j of thread t at
// (c * 8 + j) * THREADS + t.  Either way a wave's accesses are contiguous.
template <int THREADS, int CHUNKS>
struct Row {
  static __device__ __forceinline__ int32_t chunk(int c) { return (c * THREADS + (int)threadIdx.x) * 8; }
  static __device__ __forceinline__ int32_t single(int c, int j) { return (c * 8 + j) * THREADS + (int)threadIdx.x; }

  template <bool BF16>
  static __device__ __forceinline__ void load16(const uint16_t *p, int32_t n, bool wide, float (&v)[CHUNKS][8]) {
    if (wide) {
      uint4 raw[CHUNKS];
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        raw[c] = make_uint4(0, 0, 0, 0);
        if (chunk(c) < n) raw[c] = *reinterpret_cast<const uint4 *>(p + chunk(c));
      }
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[c][2 * j] = up<BF16>(w[j] & 0xFFFFu);
          v[c][2 * j + 1] = up<BF16>(w[j] >> 16);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = single(c, j) < n ? up<BF16>(p[single(c, j)]) : 0.0f;
    }
  }

  static __device__ __forceinline__ void load32(const float *p, int32_t n, bool wide, float (&v)[CHUNKS][8]) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      if (wide) {
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (chunk(c) < n) {
          a = *reinterpret_cast<const float4 *>(p + chunk(c));
          b = *reinterpret_cast<const float4 *>(p + chunk(c) + 4);
        }
        v[c][0] = a.x, v[c][1] = a.y, v[c][2] = a.z, v[c][3] = a.w;
        v[c][4] = b.x, v[c][5] = b.y, v[c][6] = b.z, v[c][7] = b.w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = single(c, j) < n ? p[single(c, j)] : 0.0f;
      }
    }
  }

  template <bool BF16>
  static __device__ __forceinline__ void store16(uint16_t *p, int32_t n, bool wide, const float (&v)[CHUNKS][8]) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      if (wide) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = down<BF16>(v[c][2 * j]) | down<BF16>(v[c][2 * j + 1]) << 16;
        if (chunk(c) < n) *reinterpret_cast<uint4 *>(p + chunk(c)) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (single(c, j) < n) p[single(c, j)] = (uint16_t)down<BF16>(v[c][j]);
      }
    }
  }

  static __device__ __forceinline__ void store32(float *p, int32_t n, bool wide, const float (&v)[CHUNKS][8]) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      if (wide) {
        if (chunk(c) < n) {
          *reinterpret_cast<float4 *>(p + chunk(c)) = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
          *reinterpret_cast<float4 *>(p + chunk(c) + 4) = make_float4(v[c][4], v[c][5], v[c][6], v[c][7]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (single(c, j) < n) p[single(c, j)] = v[c][j];
      }
    }
  }

  // 1 / sqrt(mean(v^2) + eps) of the row, sums in fp32; elements past the row are zero.
  static __device__ __forceinline__ float scale(const float (&v)[CHUNKS][8], int32_t n, float eps, float *tmp) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(v[c][j], v[c][j], s);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    if (THREADS > 64) {
      if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = s;
      __syncthreads();
      s = 0.0f;
#pragma unroll
      for (int w = 0; w < THREADS / 64; ++w) s += tmp[w];
    }
    return 1.0f / sqrtf(s / (float)n + eps);
  }
};

template <int THREADS, int CHUNKS, bool BF16, bool RES32>
__global__ __launch_bounds__(THREADS) void norm_kernel(NormArgs a) {
  using R = Row<THREADS, CHUNKS>;
  __shared__ float tmp[2][THREADS / 64];
  const int64_t m = blockIdx.x;
  const int32_t n = a.N;
  const bool wide = a.wide;
  float h[CHUNKS][8];
  if (RES32) R::load32(static_cast<const float *>(a.res) + m * a.ldr, n, wide, h);
  else R::template load16<BF16>(static_cast<const uint16_t *>(a.res) + m * a.ldr, n, wide, h);
  if (a.x) {
    float u[CHUNKS][8], w[CHUNKS][8];
    R::template load16<BF16>(a.x + m * a.ldx, n, wide, u);
    if (a.post) {
      R::template load16<BF16>(a.post, n, wide, w);
      const float r = R::scale(u, n, a.eps, tmp[0]);
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) u[c][j] *= r * w[c][j];
    }
    if (a.gate) {
      R::template load16<BF16>(a.gate + m * a.ldgate, n, wide, w);
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) u[c][j] *= w[c][j];
    }
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = fmaf(a.beta, u[c][j], a.alpha * h[c][j]);
  } else {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] *= a.alpha;
  }
  if (a.res_out) {
    if (RES32) R::store32(static_cast<float *>(a.res_out) + m * a.ldro, n, wide, h);
    else R::template store16<BF16>(static_cast<uint16_t *>(a.res_out) + m * a.ldro, n, wide, h);
  }
  if (!a.pre) return;
  float w[CHUNKS][8];
  R::template load16<BF16>(a.pre, n, wide, w);
  const float r = R::scale(h, n, a.eps, tmp[1]);
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) h[c][j] *= r * w[c][j];
  if (a.y) R::template store16<BF16>(a.y + m * a.ldy, n, wide, h);
  if (!a.aq) return;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {  // wide holds: chunks of 8, groups of 16 neighbouring lanes
    const int32_t e = R::chunk(c);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[c][j] = up<BF16>(down<BF16>(h[c][j]));
    mixllm::quant_values(h[c], e < n, m, e / MIXLLM_GROUP, threadIdx.x & 15, a.M, n, a.aq, a.sa, a.asum, a.rowop);
  }
}

template <int THREADS, int CHUNKS>
void launch(const NormArgs &a, int32_t dtype, int32_t res_dtype, hipStream_t s) {
  const dim3 grid((unsigned)a.M), block(THREADS);
  if (dtype == MIXLLM_BF16) {
    if (res_dtype == MIXLLM_FP32) hipLaunchKernelGGL((norm_kernel<THREADS, CHUNKS, true, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((norm_kernel<THREADS, CHUNKS, true, false>), grid, block, 0, s, a);
  } else {
    if (res_dtype == MIXLLM_FP32) hipLaunchKernelGGL((norm_kernel<THREADS, CHUNKS, false, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((norm_kernel<THREADS, CHUNKS, false, false>), grid, block, 0, s, a);
  }
}

constexpr int32_t kMaxN = 65536;

}  // namespace

extern "C" int mixllm_residual_norm(const void *x, int64_t ldx, const void *post, const void *gate, int64_t ldgate,
                                    const void *res, int64_t ldr, void *res_out, int64_t ldro, const void *pre,
                                    void *y, int64_t ldy, int8_t *aq, float *sa, int32_t *asum, uint32_t *rowop,
                                    int32_t M, int32_t N, int32_t group, int32_t dtype, int32_t res_dtype, float eps,
                                    float alpha, float beta, void *stream) {
  if (group != MIXLLM_GROUP) return MIXLLM_E_GROUP;
  // a launch has fewer than 2^32 threads; so many rows take 64, 256, 512 or 1024 each
  if (M >= (N <= 512 ? 1 << 26 : N <= 4096 ? 1 << 24 : N <= 16384 ? 1 << 23 : 1 << 22)) return MIXLLM_E_SHAPE;
  if (M < 0 || N <= 0 || N > kMaxN || (dtype != MIXLLM_FP16 && dtype != MIXLLM_BF16) ||
      (res_dtype != dtype && res_dtype != MIXLLM_FP32) || !(eps >= 0.0f))
    return MIXLLM_E_SHAPE;
  if (M == 0) return MIXLLM_OK;
  if (!res || (!x && (post || gate)) || (pre ? !y && !aq : y || aq || !res_out) || (aq ? !sa : sa || asum || rowop))
    return MIXLLM_E_NULL;
  if (ldr < N || (res_out && ldro < N) || (x && ldx < N) || (y && ldy < N) || (gate && ldgate != 0 && ldgate < N))
    return MIXLLM_E_SHAPE;
  const void *all[] = {x, post, gate, res, res_out, pre, y, aq, sa, asum, rowop};
  bool wide = N % 8 == 0 && (!x || ldx % 8 == 0) && (!gate || ldgate % 8 == 0) && ldr % 8 == 0 &&
              (!res_out || ldro % 8 == 0) && (!y || ldy % 8 == 0);
  for (const void *p : all) {
    wide = wide && mixllm::is_aligned16(p);
    if (reinterpret_cast<uintptr_t>(p) & 1) return MIXLLM_E_SHAPE;
  }
  if (res_dtype == MIXLLM_FP32 && (!mixllm::is_aligned4(res) || !mixllm::is_aligned4(res_out))) return MIXLLM_E_SHAPE;
  if (aq && (!wide || N % MIXLLM_GROUP != 0)) return MIXLLM_E_SHAPE;
  const NormArgs a = {static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(post),
                      static_cast<const uint16_t *>(gate), static_cast<const uint16_t *>(pre), res, res_out,
                      static_cast<uint16_t *>(y), aq, sa, asum, reinterpret_cast<uint4 *>(rowop), ldx, ldgate, ldr,
                      ldro, ldy, M, N, eps, alpha, beta, wide};
  const hipStream_t s = (hipStream_t)stream;
  // Threads and chunks of 8 per thread, measured on fp16 rows (us at M = 1 / 256 / 2048):
  // N = 4096: 512 x 1 3.4 / 5.4 / 17.9, 256 x 2 3.7 / 5.8 / 16.4; 8192: 512 x 2 3.9 / 7.1 / 25.3,
  // 256 x 4 4.6 / 7.6 / 25.8, 1024 x 1 4.0 / 7.2 / 28.0 (2047 rows with an fp32 residual, to int8:
  // 46.9, 51.2, 52.9); 14336: 512 x 4 5.1 / 10.3 / 52.0, 1024 x 2 4.9 / 10.4 / 58.2.
  if (N <= 512) launch<64, 1>(a, dtype, res_dtype, s);
  else if (N <= 2048) launch<256, 1>(a, dtype, res_dtype, s);
  else if (N <= 4096 && M <= 512) launch<512, 1>(a, dtype, res_dtype, s);
  else if (N <= 4096) launch<256, 2>(a, dtype, res_dtype, s);
  else if (N <= 8192) launch<512, 2>(a, dtype, res_dtype, s);
  else if (N <= 16384) launch<512, 4>(a, dtype, res_dtype, s);
  else if (N <= 32768) launch<1024, 4>(a, dtype, res_dtype, s);
  else launch<1024, 8>(a, dtype, res_dtype, s);
  return mixllm::launch_status();
}
