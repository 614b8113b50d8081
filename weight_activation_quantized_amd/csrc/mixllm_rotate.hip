// The norms of queries and keys per head and the rotation by position, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w        per head (y = x without a norm)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = pos * inv_freq[i]
//
// for the pairs i < rot / 2 of a head, channels (i, i + rot / 2) or (2 i, 2 i + 1); channels
// from rot on are only normed.  All in fp32 from one read, rounded once.  The angle is formed
// in fp64 and reduced to (-pi, pi] there: in fp32 a position of 10^6 would leave it 0.03 off.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm_kv4.h"
#include "mixllm_lanes.h"

namespace {

using mixllm::down;
using mixllm::moved;
using mixllm::up;

struct RotateArgs {
  const uint16_t *q, *k;
  uint16_t *qo, *ko;
  const int32_t *pos;
  const float *freq;
  const uint16_t *qn, *kn;
  int64_t ldq, ldk, ldqo, ldko;
  int32_t T, hq, heads, dim, rot;  // heads: of queries and keys
  float eps;
};

// cos and sin of pos * freq.  The product and its share of a turn are formed with what their
// roundings leave, so that 2^31 radians and more lose nothing either.
__device__ __forceinline__ void turn_of(int32_t pos, float freq, float &c, float &s) {
  constexpr double kTurn = 0.15915494309189535, kTurnRest = -9.839338337591243e-18;  // 1 / 2 pi
  const double p = (double)pos * (double)freq, p_rest = fma((double)pos, (double)freq, -p);
  const double t = p * kTurn, t_rest = fma(p, kTurn, -t) + fma(p, kTurnRest, p_rest * kTurn);
  sincospif((float)(2.0 * ((t - rint(t)) + t_rest)), &s, &c);
}

// The sum over groups of L neighbouring lanes, in all of them.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v += moved<mixllm::kDppXor1>(v);
  v += moved<mixllm::kDppXor2>(v);
  if (L >= 8) v += moved<mixllm::kDppHalfMirror>(v);
  if (L >= 16) v += moved<mixllm::kDppMirror>(v);
  typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
  if (L >= 32) {
    const uint2v a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a.x) + __uint_as_float(a.y);
  }
  if (L >= 64) {
    const uint2v a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a.x) + __uint_as_float(a.y);
  }
  return v;
}

template <bool BF16>
__device__ __forceinline__ void unpack4(uint2 w, float *x) {
  x[0] = up<BF16>(w.x & 0xFFFFu), x[1] = up<BF16>(w.x >> 16);
  x[2] = up<BF16>(w.y & 0xFFFFu), x[3] = up<BF16>(w.y >> 16);
}

template <bool BF16>
__device__ __forceinline__ uint2 pack4(const float *x) {
  return make_uint2(down<BF16>(x[0]) | down<BF16>(x[1]) << 16, down<BF16>(x[2]) | down<BF16>(x[3]) << 16);
}

// A wave takes one token and 64 / L of its heads at a time; L lanes hold a head, 8 channels
// each, so that a lane has both channels of its four pairs and nothing but the norm's sum
// crosses lanes.  A lane's cosines and sines are those of all heads: formed once.
template <int L, bool BF16, bool NEXT>
__global__ void rotate_kernel(RotateArgs a) {
  const int lane = threadIdx.x & 63, u = lane & (L - 1);
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t t = blockIdx.x;
  const bool live = u < a.dim / 8, turned = u < a.rot / 8;
  const int e0 = !NEXT && turned ? 4 * u : 8 * u, e1 = !NEXT && turned ? a.rot / 2 + 4 * u : 8 * u + 4;
  const int step = waves * (64 / L);
  int32_t h = wave * (64 / L) + lane / L;
  uint2 raw0 = make_uint2(0, 0), raw1 = raw0;
  auto load = [&](int32_t head) {
    if (head >= a.heads || !live) return;
    const uint16_t *src = head < a.hq ? a.q + t * a.ldq + (int64_t)head * a.dim
                                      : a.k + t * a.ldk + (int64_t)(head - a.hq) * a.dim;
    raw0 = *reinterpret_cast<const uint2 *>(src + e0);
    raw1 = *reinterpret_cast<const uint2 *>(src + e1);
  };
  load(h);
  float cs[4], sn[4], w[2][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[0][j] = w[1][j] = 1.0f;
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const uint16_t *src = z ? a.kn : a.qn;
    if (src && live) {
      unpack4<BF16>(*reinterpret_cast<const uint2 *>(src + e0), w[z]);
      unpack4<BF16>(*reinterpret_cast<const uint2 *>(src + e1), w[z] + 4);
    }
  }
  const int32_t pos = a.rot ? a.pos[t] : 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    cs[j] = 1.0f, sn[j] = 0.0f;
    if (turned) turn_of(pos, a.freq[4 * u + j], cs[j], sn[j]);
  }
  for (; h - lane / L < a.heads; h += step) {
    const bool there = h < a.heads && live;
    float x[8];
    unpack4<BF16>(raw0, x);
    unpack4<BF16>(raw1, x + 4);
    load(h + step);
    const bool key = h >= a.hq;
    if (a.qn || a.kn) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
      ss = lanes_sum<L>(there ? ss : 0.0f);
      const float r = 1.0f / sqrtf(ss / (float)a.dim + a.eps);
      if (key ? a.kn != nullptr : a.qn != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= r * (key ? w[1][j] : w[0][j]);
      }
    }
    if (turned) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float &p = NEXT ? x[2 * j] : x[j], &q = NEXT ? x[2 * j + 1] : x[4 + j];
        const float first = p * cs[j] - q * sn[j], second = fmaf(p, sn[j], q * cs[j]);
        p = first, q = second;
      }
    }
    if (there) {
      uint16_t *dst = key ? a.ko + t * a.ldko + (int64_t)(h - a.hq) * a.dim : a.qo + t * a.ldqo + (int64_t)h * a.dim;
      *reinterpret_cast<uint2 *>(dst + e0) = pack4<BF16>(x);
      *reinterpret_cast<uint2 *>(dst + e1) = pack4<BF16>(x + 4);
    }
  }
}

constexpr int32_t kMaxDim = 512;

// Any even number of channels and element-aligned rows: a wave takes one head, a lane single
// pairs of it.
template <bool BF16, bool NEXT>
__global__ __launch_bounds__(256) void rotate_any_kernel(RotateArgs a) {
  constexpr int kPairs = kMaxDim / 2 / 64;
  const int lane = threadIdx.x & 63;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = id / a.heads;
  if (t >= a.T) return;
  const int32_t h = (int32_t)(id - t * a.heads);
  const bool key = h >= a.hq;
  const uint16_t *src = key ? a.k + t * a.ldk + (int64_t)(h - a.hq) * a.dim : a.q + t * a.ldq + (int64_t)h * a.dim;
  uint16_t *dst = key ? a.ko + t * a.ldko + (int64_t)(h - a.hq) * a.dim : a.qo + t * a.ldqo + (int64_t)h * a.dim;
  const uint16_t *norm = key ? a.kn : a.qn;
  const int32_t pos = a.rot ? a.pos[t] : 0;
  float x[kPairs], y[kPairs], ss = 0.0f;
  // channels of this lane's pair i: neighbours, but for turned pairs of halves
  auto first = [&](int p) { return !NEXT && p < a.rot / 2 ? p : 2 * p; };
  auto second = [&](int p) { return !NEXT && p < a.rot / 2 ? p + a.rot / 2 : 2 * p + 1; };
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int p = lane + 64 * i;
    x[i] = y[i] = 0.0f;
    if (p < a.dim / 2) x[i] = up<BF16>(src[first(p)]), y[i] = up<BF16>(src[second(p)]);
    ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
  }
  if (norm) {
    const float r = 1.0f / sqrtf(lanes_sum<64>(ss) / (float)a.dim + a.eps);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int p = lane + 64 * i;
      if (p < a.dim / 2) x[i] *= r * up<BF16>(norm[first(p)]), y[i] *= r * up<BF16>(norm[second(p)]);
    }
  }
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int p = lane + 64 * i;
    if (p >= a.dim / 2) continue;
    if (p < a.rot / 2) {
      float c, s;
      turn_of(pos, a.freq[p], c, s);
      const float v = x[i] * c - y[i] * s;
      y[i] = fmaf(x[i], s, y[i] * c);
      x[i] = v;
    }
    dst[first(p)] = (uint16_t)down<BF16>(x[i]);
    dst[second(p)] = (uint16_t)down<BF16>(y[i]);
  }
}

template <int L, bool BF16>
void launch(const RotateArgs &a, bool next, hipStream_t s) {
  const int heads_a_wave = 64 / L, all = (a.heads + heads_a_wave - 1) / heads_a_wave;
  int waves = a.T >= 1024 ? 4 : 16;
  waves = waves < all ? waves : all;
  const dim3 grid((unsigned)a.T), block((unsigned)(64 * waves));
  if (next) hipLaunchKernelGGL((rotate_kernel<L, BF16, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((rotate_kernel<L, BF16, false>), grid, block, 0, s, a);
}

template <bool BF16>
void launch(const RotateArgs &a, bool next, bool wide, hipStream_t s) {
  if (!wide) {
    const dim3 grid((unsigned)(((int64_t)a.T * a.heads + 3) / 4));
    if (next) hipLaunchKernelGGL((rotate_any_kernel<BF16, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((rotate_any_kernel<BF16, false>), grid, dim3(256), 0, s, a);
  } else if (a.dim <= 64) {
    launch<8, BF16>(a, next, s);
  } else if (a.dim <= 128) {
    launch<16, BF16>(a, next, s);
  } else if (a.dim <= 256) {
    launch<32, BF16>(a, next, s);
  } else {
    launch<64, BF16>(a, next, s);
  }
}

}  // namespace

extern "C" int mixllm_head_norm_rotate(const void *q, int64_t ldq, const void *k, int64_t ldk, void *q_out,
                                       int64_t ldqo, void *k_out, int64_t ldko, const int32_t *pos,
                                       const float *inv_freq, const void *q_norm, const void *k_norm, int32_t T,
                                       int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t rot, int32_t neighbours,
                                       int32_t dtype, float eps, void *stream) {
  if (T < 0 || q_heads < 0 || kv_heads < 0 || dim <= 0 || dim > kMaxDim || dim % 2 != 0 || rot < 0 || rot > dim ||
      rot % 2 != 0 || (neighbours != 0 && neighbours != 1) || (dtype != MIXLLM_FP16 && dtype != MIXLLM_BF16) ||
      !(eps >= 0.0f) || q_heads > 65535 || kv_heads > 65535)
    return MIXLLM_E_SHAPE;
  const int32_t heads = q_heads + kv_heads;
  // a launch has fewer than 2^32 threads: 64 for a head, or 256 or fewer for each of so many tokens
  if (T >= 1 << 24 || (int64_t)T * heads >= 1 << 26) return MIXLLM_E_SHAPE;
  if (T == 0 || heads == 0) return MIXLLM_OK;
  if ((q_heads && (!q || !q_out)) || (kv_heads && (!k || !k_out)) || (rot && (!pos || !inv_freq)) ||
      (!q_heads && q_norm) || (!kv_heads && k_norm))
    return MIXLLM_E_NULL;
  const int64_t qw = (int64_t)q_heads * dim, kw = (int64_t)kv_heads * dim;
  if (ldq < qw || ldqo < qw || ldk < kw || ldko < kw) return MIXLLM_E_SHAPE;
  const void *all[] = {q, k, q_out, k_out, q_norm, k_norm};
  bool wide = dim % 8 == 0 && rot % 8 == 0;
  for (const void *p : all) {
    if (reinterpret_cast<uintptr_t>(p) & 1) return MIXLLM_E_SHAPE;
    wide = wide && (reinterpret_cast<uintptr_t>(p) & 7) == 0;
  }
  wide = wide && (ldq | ldqo) % 4 == 0 && (ldk | ldko) % 4 == 0;
  if (!mixllm::is_aligned4(pos) || !mixllm::is_aligned4(inv_freq)) return MIXLLM_E_SHAPE;
  const RotateArgs a = {static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k),
                        static_cast<uint16_t *>(q_out), static_cast<uint16_t *>(k_out), pos, inv_freq,
                        static_cast<const uint16_t *>(q_norm), static_cast<const uint16_t *>(k_norm),
                        ldq, ldk, ldqo, ldko, T, q_heads, heads, dim, rot, eps};
  if (dtype == MIXLLM_BF16) launch<true>(a, neighbours != 0, wide, (hipStream_t)stream);
  else launch<false>(a, neighbours != 0, wide, (hipStream_t)stream);
  return mixllm::launch_status();
}
