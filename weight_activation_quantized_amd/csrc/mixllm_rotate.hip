// The norms of queries and keys per head and the rotation by position, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w        per head (y = x without a norm)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = pos * inv_freq[i]
//
// for the pairs i < rot / 2 of a head, channels (i, i + rot / 2) or (2 i, 2 i + 1); channels
// from rot on are only normed.  All in fp32 from one read, rounded once.  The angle is formed
// in fp64 and reduced to (-pi, pi] there: in fp32 a position of 10^6 would leave it 0.03 off.
//
// Bound by the memory for prompts (8191 tokens x 72 heads of 128: 302 MB in 62 us, 4.9 TB/s, a large
// copy's rate) and by latency for single tokens (32 tokens x 40 heads: 3.5 us, a launch and little
// more).  Both needed the angles of a token formed once and not once for every head (153 us with each
// lane's own), and 16 bytes a load.
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
  int32_t parts;                   // waves that share a token
  float eps, inv_dim;
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

// The 8 values of 16 bytes, and back.
template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 v, float *x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) x[2 * j] = up<BF16>(w[j] & 0xFFFFu), x[2 * j + 1] = up<BF16>(w[j] >> 16);
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = down<BF16>(x[2 * j]) | down<BF16>(x[2 * j + 1]) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 either(bool first, uint4 a, uint4 b) {
  return make_uint4(first ? a.x : b.x, first ? a.y : b.y, first ? a.z : b.z, first ? a.w : b.w);
}

constexpr int kWavesOfBlock = 4;

// A wave takes a token, or one of `parts` shares of its heads, and 64 / L heads at a time; L lanes
// hold a head, 16 channels each, so that a lane has both channels of its eight pairs and nothing
// but the norm's sum crosses lanes.  The cosines and sines of a token are formed once, a pair a
// lane, and dealt out through LDS.
template <int L, bool BF16, bool NEXT>
__global__ __launch_bounds__(64 * kWavesOfBlock) void rotate_kernel(RotateArgs a) {
  constexpr int kPairs = 8 * L;  // of the longest head, room for
  __shared__ float2 turns[kWavesOfBlock][kPairs];
  const int lane = threadIdx.x & 63, u = lane & (L - 1), wave = threadIdx.x >> 6;
  const int64_t id = (int64_t)blockIdx.x * kWavesOfBlock + wave, t = id / a.parts;
  if (t >= a.T) return;  // whole waves: none waits for another
  const bool live = u < a.dim / 16, turned = u < a.rot / 16;
  const int e0 = !NEXT && turned ? 8 * u : 16 * u, e1 = !NEXT && turned ? a.rot / 2 + 8 * u : 16 * u + 8;
  const int step = a.parts * (64 / L);
  int32_t h = (int32_t)(id - t * a.parts) * (64 / L) + lane / L;
  auto place = [&](int32_t head, bool key, const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk) {
    return key ? k + t * ldk + (int64_t)(head - a.hq) * a.dim : q + t * ldq + (int64_t)head * a.dim;
  };
  uint4 raw0[2], raw1[2];
  auto load = [&](uint4 (&to)[2], int32_t head) __attribute__((always_inline)) {
    to[0] = to[1] = make_uint4(0, 0, 0, 0);
    if (head >= a.heads || !live) return;
    const uint16_t *src = place(head, head >= a.hq, a.q, a.ldq, a.k, a.ldk);
    to[0] = *reinterpret_cast<const uint4 *>(src + e0);
    to[1] = *reinterpret_cast<const uint4 *>(src + e1);
  };
  load(raw0, h);
  load(raw1, h + step);
  uint4 w[2][2];
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const uint16_t *src = z ? a.kn : a.qn;
    w[z][0] = w[z][1] = make_uint4(0, 0, 0, 0);
    if (src && live) {
      w[z][0] = *reinterpret_cast<const uint4 *>(src + e0);
      w[z][1] = *reinterpret_cast<const uint4 *>(src + e1);
    }
  }
  float cs[8], sn[8];
  if (a.rot) {
    const int32_t pos = a.pos[t];
    for (int p = lane; p < a.rot / 2; p += 64) {
      float c, s;
      turn_of(pos, a.freq[p], c, s);
      turns[wave][p] = make_float2(c, s);
    }
    // a wave's LDS operations are done in order, so only the compiler has to be held
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = turns[wave][8 * u + j];
      cs[j] = v.x, sn[j] = v.y;
    }
  }
  auto one = [&](uint4 (&now)[2]) __attribute__((always_inline)) {
    const bool there = h < a.heads && live, key = h >= a.hq;
    float x[16];
    unpack8<BF16>(now[0], x);
    unpack8<BF16>(now[1], x + 8);
    load(now, h + 2 * step);
    if (a.qn || a.kn) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) ss = fmaf(x[j], x[j], ss);
      ss = lanes_sum<L>(ss);
      if (key ? a.kn != nullptr : a.qn != nullptr) {
        const float r = __builtin_amdgcn_rsqf(ss * a.inv_dim + a.eps);  // within 1 ulp
        float g[16];
        unpack8<BF16>(either(key, w[1][0], w[0][0]), g);
        unpack8<BF16>(either(key, w[1][1], w[0][1]), g + 8);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= r * g[j];
      }
    }
    if (turned) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float &p = NEXT ? x[2 * j] : x[j], &q = NEXT ? x[2 * j + 1] : x[8 + j];
        const float first = fmaf(p, cs[j], -(q * sn[j])), second = fmaf(p, sn[j], q * cs[j]);
        p = first, q = second;
      }
    }
    if (there) {
      uint16_t *dst = const_cast<uint16_t *>(place(h, key, a.qo, a.ldqo, a.ko, a.ldko));
      *reinterpret_cast<uint4 *>(dst + e0) = pack8<BF16>(x);
      *reinterpret_cast<uint4 *>(dst + e1) = pack8<BF16>(x + 8);
    }
    h += step;
  };
  const int32_t end = a.heads + lane / L;  // the wave's first head is past the last one
  while (h < end) {
    one(raw0);
    if (h >= end) break;
    one(raw1);
  }
}

constexpr int32_t kMaxDim = 512;
constexpr int32_t kEnoughWaves = 4096;

// Any even number of channels and element-aligned rows: a wave takes one head, a lane single
// pairs of it, whose angles it forms for every head again: 8191 tokens x 72 heads of 128 take 237 us with
// 40 channels turned, where the kernel above takes 53 with all.  For shapes that no model here has.
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

// Few tokens are shared by waves until each has one head group, or there are about 4096.
template <int L, bool BF16>
void launch(RotateArgs a, bool next, hipStream_t s) {
  const int all = (a.heads + 64 / L - 1) / (64 / L), want = (kEnoughWaves + a.T - 1) / a.T;
  a.parts = want < all ? want : all;
  const dim3 grid((unsigned)(((int64_t)a.T * a.parts + kWavesOfBlock - 1) / kWavesOfBlock)), block(64 * kWavesOfBlock);
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
    launch<4, BF16>(a, next, s);
  } else if (a.dim <= 128) {
    launch<8, BF16>(a, next, s);
  } else if (a.dim <= 256) {
    launch<16, BF16>(a, next, s);
  } else {
    launch<32, BF16>(a, next, s);
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
  // a launch has fewer than 2^32 threads: 64 at most for a head of a token, in whole workgroups of 4
  if (T >= 1 << 24 || (int64_t)T * heads > (1 << 26) - 4) return MIXLLM_E_SHAPE;
  if (T == 0 || heads == 0) return MIXLLM_OK;
  if ((q_heads && (!q || !q_out)) || (kv_heads && (!k || !k_out)) || (rot && (!pos || !inv_freq)) ||
      (!q_heads && q_norm) || (!kv_heads && k_norm))
    return MIXLLM_E_NULL;
  const int64_t qw = (int64_t)q_heads * dim, kw = (int64_t)kv_heads * dim;
  if (ldq < qw || ldqo < qw || ldk < kw || ldko < kw) return MIXLLM_E_SHAPE;
  const void *all[] = {q, k, q_out, k_out, q_norm, k_norm};
  bool wide = dim % 16 == 0 && rot % 16 == 0;
  for (const void *p : all) {
    if (reinterpret_cast<uintptr_t>(p) & 1) return MIXLLM_E_SHAPE;
    wide = wide && mixllm::is_aligned16(p);
  }
  wide = wide && (ldq | ldqo) % 8 == 0 && (ldk | ldko) % 8 == 0;
  if (!mixllm::is_aligned4(pos) || !mixllm::is_aligned4(inv_freq)) return MIXLLM_E_SHAPE;
  const RotateArgs a = {static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k),
                        static_cast<uint16_t *>(q_out), static_cast<uint16_t *>(k_out), pos, inv_freq,
                        static_cast<const uint16_t *>(q_norm), static_cast<const uint16_t *>(k_norm),
                        ldq, ldk, ldqo, ldko, T, q_heads, heads, dim, rot, 1, eps, 1.0f / (float)dim};
  if (dtype == MIXLLM_BF16) launch<true>(a, neighbours != 0, wide, (hipStream_t)stream);
  else launch<false>(a, neighbours != 0, wide, (hipStream_t)stream);
  return mixllm::launch_status();
}
