// The linear layer in 8 bits with one scale per token and one per output channel:
//   s_a = max |a| / 127, a_q = clamp(rne(a / s_a), -127, 127)     per row of the activations
//   y[m][n] = (sum_k a_q[m][k] w[n][k]) * (s_a[m] * s_w[n])
// The sum is exact in int32 (K <= 131072), so no split of it changes a result.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm_kv4.h"
#include "mixllm_lanes.h"

namespace {

using mixllm::down;
using mixllm::up;

typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int16v __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------------------- the quantizer

struct RowsArgs {
  const uint16_t *a;
  int8_t *q;
  float *s;
  int64_t lda, ldq;
  int32_t M, K;
};

// A workgroup takes a row, 16 values a thread and chunk, held in registers between the maximum
// and the codes.
template <int THREADS, int CHUNKS, bool BF16>
__global__ __launch_bounds__(THREADS) void quant_rows_kernel(RowsArgs a) {
  __shared__ float tops[THREADS / 64];
  const int64_t m = blockIdx.x;
  const uint16_t *src = a.a + m * a.lda;
  uint4 raw[CHUNKS][2];
  float top = 0.0f;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int32_t e = (c * THREADS + (int)threadIdx.x) * 16;
    raw[c][0] = raw[c][1] = make_uint4(0, 0, 0, 0);
    if (e < a.K) {
      raw[c][0] = *reinterpret_cast<const uint4 *>(src + e);
      raw[c][1] = *reinterpret_cast<const uint4 *>(src + e + 8);
    }
  }
  auto value = [&](int c, int j) {
    const uint4 &r = raw[c][j / 8];
    const uint32_t w = j % 8 / 2 == 0 ? r.x : j % 8 / 2 == 1 ? r.y : j % 8 / 2 == 2 ? r.z : r.w;
    return up<BF16>(w >> (16 * (j % 2)) & 0xFFFFu);
  };
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
    for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(value(c, j)));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  if (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) top = fmaxf(top, tops[w]);
  }
  const float s = top / 127.0f;
  if (threadIdx.x == 0) a.s[m] = s;
  int8_t *dst = a.q + m * a.ldq;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int32_t e = (c * THREADS + (int)threadIdx.x) * 16;
    if (e >= a.K) continue;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float q = s > 0.0f ? fminf(fmaxf(__builtin_rintf(value(c, j) / s), -127.0f), 127.0f) : 0.0f;
      w[j / 4] |= ((uint32_t)(int)q & 0xFFu) << (8 * (j % 4));
    }
    *reinterpret_cast<uint4 *>(dst + e) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

constexpr int32_t kMaxK = 131072;

template <bool BF16>
void launch_rows(const RowsArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)a.M);
  if (a.K <= 1024) hipLaunchKernelGGL((quant_rows_kernel<64, 1, BF16>), grid, dim3(64), 0, s, a);
  else if (a.K <= 4096) hipLaunchKernelGGL((quant_rows_kernel<256, 1, BF16>), grid, dim3(256), 0, s, a);
  else if (a.K <= 8192) hipLaunchKernelGGL((quant_rows_kernel<512, 1, BF16>), grid, dim3(512), 0, s, a);
  else if (a.K <= 16384) hipLaunchKernelGGL((quant_rows_kernel<512, 2, BF16>), grid, dim3(512), 0, s, a);
  else if (a.K <= 32768) hipLaunchKernelGGL((quant_rows_kernel<1024, 2, BF16>), grid, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((quant_rows_kernel<1024, 8, BF16>), grid, dim3(1024), 0, s, a);
}

// --------------------------------------------------------------------------- the product

struct Gemm8Args {
  const int8_t *a, *w;
  const float *sa, *sw;
  uint16_t *y;
  int64_t lda, ldw, ldy;
  int32_t M, N, K;
};

// One wave takes 32 tokens x 32 channels.
template <bool BF16>
__global__ __launch_bounds__(256) void gemm8_kernel(Gemm8Args a) {
  const int lane = threadIdx.x & 63, r = lane & 31, half = lane >> 5;
  const int64_t tiles_n = (a.N + 31) / 32, id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int32_t m0 = (int32_t)(id / tiles_n) * 32, n0 = (int32_t)(id % tiles_n) * 32;
  if (m0 >= a.M) return;
  const int32_t m = m0 + r < a.M ? m0 + r : a.M - 1, n = n0 + r < a.N ? n0 + r : a.N - 1;
  const int8_t *pa = a.a + (int64_t)m * a.lda + half * 16, *pw = a.w + (int64_t)n * a.ldw + half * 16;
  int16v acc = {};
  for (int32_t k = 0; k < a.K; k += 32) {
    int4v x = {0, 0, 0, 0}, w = x;
    if (k + half * 16 < a.K) {
      x = *reinterpret_cast<const int4v *>(pa + k);
      w = *reinterpret_cast<const int4v *>(pw + k);
    }
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(x, w, acc, 0, 0, 0);
  }
  if (n0 + r >= a.N) return;
  const float sw = a.sw[n0 + r];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int32_t row = m0 + i / 4 * 8 + half * 4 + i % 4;
    if (row < a.M) a.y[(int64_t)row * a.ldy + n0 + r] = (uint16_t)down<BF16>((float)acc[i] * (a.sa[row] * sw));
  }
}

}  // namespace

extern "C" int mixllm_quant_rows(const void *a, int64_t lda, int32_t dtype, int32_t M, int32_t K, int8_t *q, int64_t ldq,
                                 float *s, void *stream) {
  if (M < 0 || M >= 1 << 22 || K <= 0 || K > kMaxK || K % 16 != 0 || (dtype != MIXLLM_FP16 && dtype != MIXLLM_BF16) ||
      lda < K || lda % 8 != 0 || ldq < K || ldq % 16 != 0)
    return MIXLLM_E_SHAPE;
  if (M == 0) return MIXLLM_OK;
  if (!a || !q || !s) return MIXLLM_E_NULL;
  if (!mixllm::is_aligned16(a) || !mixllm::is_aligned16(q) || !mixllm::is_aligned4(s)) return MIXLLM_E_SHAPE;
  const RowsArgs r = {static_cast<const uint16_t *>(a), q, s, lda, ldq, M, K};
  if (dtype == MIXLLM_BF16) launch_rows<true>(r, (hipStream_t)stream);
  else launch_rows<false>(r, (hipStream_t)stream);
  return mixllm::launch_status();
}

extern "C" int mixllm_gemm_w8a8(const int8_t *aq, int64_t lda, const float *sa, const int8_t *w, int64_t ldw,
                                const float *sw, int32_t M, int32_t N, int32_t K, void *y, int64_t ldy, int32_t dtype,
                                void *stream) {
  if (M < 0 || N <= 0 || K <= 0 || K > kMaxK || K % 16 != 0 || (dtype != MIXLLM_FP16 && dtype != MIXLLM_BF16) ||
      lda < K || lda % 16 != 0 || ldw < K || ldw % 16 != 0 || ldy < N)
    return MIXLLM_E_SHAPE;
  if (M == 0) return MIXLLM_OK;
  if (!aq || !sa || !w || !sw || !y) return MIXLLM_E_NULL;
  if (!mixllm::is_aligned16(aq) || !mixllm::is_aligned16(w) || !mixllm::is_aligned4(sa) || !mixllm::is_aligned4(sw) ||
      (reinterpret_cast<uintptr_t>(y) & 1))
    return MIXLLM_E_SHAPE;
  // a launch has fewer than 2^32 threads, and a wave at least takes 32 x 32 outputs
  if (((int64_t)M + 31) / 32 * (((int64_t)N + 31) / 32) >= 1 << 26) return MIXLLM_E_SHAPE;
  const Gemm8Args g = {aq, w, sa, sw, static_cast<uint16_t *>(y), lda, ldw, ldy, M, N, K};
  const int64_t tiles = ((int64_t)M + 31) / 32 * (((int64_t)N + 31) / 32);
  const dim3 grid((unsigned)((tiles + 3) / 4));
  if (dtype == MIXLLM_BF16) hipLaunchKernelGGL((gemm8_kernel<true>), grid, dim3(256), 0, (hipStream_t)stream, g);
  else hipLaunchKernelGGL((gemm8_kernel<false>), grid, dim3(256), 0, (hipStream_t)stream, g);
  return mixllm::launch_status();
}
