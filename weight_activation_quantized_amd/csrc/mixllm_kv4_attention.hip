// Attention over the paged key/value cache held in 4 bits, for decoded tokens and for the
// rows of prompts.
//
// For one query row with position p of a request, over the keys t in (p - window, p]:
//   S_t = scale * sum_g (s_g,t (q_g . c_g,t) + m_g,t sum(q_g))      (K = m + s c per group g)
//   O   = sum_t P_t (m_t + s_t c_t) / sum_t P_t,  P_t = exp(S_t - max S)
// so the codes enter the matrix instructions as they are (exact in fp16) and the scales
// multiply whole partial products (keys) or the probabilities (values); the minima enter
// through sum(q_g), known before the loop, and through one sum of P_t m_t per row.
//
// A 16 x 16 x 32 fp16 matrix instruction takes 8 consecutive contraction indices per lane.
// Both products are computed transposed: S^T = K Q^T leaves in lane (n, c) the scores of
// query row n with tokens 4c .. 4c+3, and O^T = V^T P^T takes from lane (n, c) the
// probabilities of row n for the tokens that quarter c holds, which are the same: the
// softmax statistics, the probabilities and the output's scale factors of a row stay in its
// lanes, and only the row maximum crosses quarters.
//
// Codes become fp16 without arithmetic: a nibble masked in place is a subnormal fp16,
// c 2^-24 (or 16 c 2^-24 where it sits 4 bits higher), which the matrix instruction takes
// exactly; the power of two goes into the row's factor (keys: the query's odd nibbles are
// pre-divided by 16).  5 integer operations make 8 operands.
//
// The query is scaled by a power of two per row so that it fits fp16 (bf16 inputs lose
// nothing but values 2^-38 below the row's largest); the probability times the value's
// scale is rounded once to fp16 (relative 2^-11), scaled by a power of two that follows the
// largest value scale seen so that it stays clear of fp16's subnormals.  Statistics, sums
// and outputs are fp32.
//
// A decode step is bound by reading the cache: D * 9 / 8 bytes per token and head.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm_kv4.h"

namespace {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;         // tokens of one step of a wave
constexpr int kRows = 16;         // query rows of a tile (token, head of the group)
constexpr float kLow = -1e38f;    // a running maximum before any score
constexpr float kLazy = 6.0f;     // the maximum moves once a score is this far above it (log2)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Args {
  const uint16_t *q;
  const uint8_t *cache;
  const int32_t *table, *lens, *cu;
  uint16_t *out;
  float *lse, *ws_o, *ws_ml;
  int64_t ldq, ldo, ldt;
  float scale;
  int32_t T, hq, hkv, group, pages, page_log2, width, B, max_rows, max_len, window;
  int32_t tiles, rows_tile;  // row tiles of a request and head, rows of a tile
  int32_t splits, chunk;     // workgroups along the tokens, tokens of each
  int32_t bf16;
};

__device__ __forceinline__ float up(uint32_t bits, bool bf16) {
  return bf16 ? __uint_as_float(bits << 16)
              : static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

__device__ __forceinline__ uint32_t down(float v, bool bf16) {
  return bf16 ? (uint32_t)__builtin_bit_cast(uint16_t, static_cast<__bf16>(v))
              : (uint32_t)__builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

// Maximum and sum over the four lanes n, n + 16, n + 32, n + 48 of a query row.
__device__ __forceinline__ float quarters_max(float v) {
  uint2v a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
}

__device__ __forceinline__ uint32_t quarters_max(uint32_t v) {
  uint2v a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = a.x > a.y ? a.x : a.y;
  a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return __builtin_amdgcn_readfirstlane(a.x > a.y ? a.x : a.y);
}

__device__ __forceinline__ float quarters_sum(float v) {
  uint2v a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a.x) + __uint_as_float(a.y);
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a.x) + __uint_as_float(a.y);
}

// 8 codes of a dword as fp16 operands in the nibble order 0 4 1 5 2 6 3 7; nibbles 1, 3, 5
// and 7 come out 16 times larger.
__device__ __forceinline__ half8 codes8(uint32_t w) {
  const uint32_t v = w >> 8;
  const uint4v r = {w & 0x000F000Fu, w & 0x00F000F0u, v & 0x000F000Fu, v & 0x00F000F0u};
  return __builtin_bit_cast(half8, r);
}

__device__ __forceinline__ uint32_t nibble_pair(uint32_t w, int nib) {
  return (nib >= 2 ? w >> 8 : w) & (nib & 1 ? 0x00F000F0u : 0x000F000Fu);
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
  if (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if (N == 2) {
    const uint2v v = *reinterpret_cast<const uint2v *>(p);
    w[0] = v.x, w[N - 1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4v v = *reinterpret_cast<const uint4v *>(p + 16 * i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

// What a lane holds of 32 tokens: its part of the codes, and one token's parameters of
// keys (lanes 0..31) or values (lanes 32..63).
template <int D>
struct Step {
  uint32_t k[2][D / 32], v[2][D / 32], par[D / 64];
  bool ok[2];  // wave-uniform: the 16 tokens are in the cache
};

// The request, rows and tokens of a workgroup.
struct Tile {
  int32_t b, h, row0, rows, nq, len, q0;  // rows: query rows of this tile
  int32_t lo, hi;                         // tokens that any of its rows sees
};

__device__ __forceinline__ Tile tile_of(const Args &a, int32_t b, int32_t h, int32_t rt) {
  Tile t;
  t.b = b, t.h = h, t.row0 = rt * kRows;
  t.q0 = a.cu[b];
  int32_t end = a.cu[b + 1];
  end = end < a.T ? end : a.T;
  t.q0 = t.q0 < 0 ? 0 : t.q0;
  t.nq = end - t.q0;
  t.nq = t.nq < a.max_rows ? t.nq : a.max_rows;
  const int64_t cap = (int64_t)a.width << a.page_log2;
  const int32_t most = cap < a.max_len ? (int32_t)cap : a.max_len, len = a.lens[b];
  t.len = len < 0 ? 0 : len < most ? len : most;
  const int64_t all = (int64_t)t.nq * a.group;
  const int64_t left = all - t.row0;
  t.rows = left <= 0 ? 0 : left < kRows ? (int32_t)left : kRows;
  if (t.rows > 0) {
    const int32_t first = t.len - t.nq + t.row0 / a.group, last = t.len - t.nq + (t.row0 + t.rows - 1) / a.group;
    t.hi = last + 1 > 0 ? last + 1 : 0;
    t.lo = a.window && first - a.window + 1 > 0 ? first - a.window + 1 : 0;
    t.lo = t.lo < t.hi ? t.lo : t.hi;
  } else {
    t.lo = t.hi = 0;
  }
  return t;
}

// The chunks of a tile start at its first token, rounded down to whole steps.
__device__ __forceinline__ int32_t base_of(const Tile &t) { return t.lo & ~(kStep - 1); }
__device__ __forceinline__ int32_t chunks_of(const Args &a, const Tile &t) {
  return (t.hi - base_of(t) + a.chunk - 1) / a.chunk;
}

template <int D>
__global__ __launch_bounds__(kThreads) void kv4_attention_kernel(Args a) {
  constexpr int G = D / 64, W = D / 32, J = D / 16;
  constexpr int kStride = D + 4;  // floats of a row of partial outputs in LDS
  __shared__ __attribute__((aligned(16))) uint32_t s_par[kWaves][64 * G];
  __shared__ __attribute__((aligned(16))) float s_o[kWaves][kRows * kStride];
  __shared__ float s_m[kWaves][kRows], s_l[kWaves][kRows];

  const int lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int32_t id = blockIdx.x;
  const int32_t split = id % a.splits;
  id /= a.splits;
  const int32_t h = id % a.hkv;
  id /= a.hkv;
  const int32_t rt = id % a.tiles, b = id / a.tiles;
  const Tile t = tile_of(a, b, h, rt);
  if (t.rows <= 0) return;
  const int32_t nchunks = chunks_of(a, t);
  if (split >= nchunks && !(split == 0 && a.splits == 1)) return;
  const int32_t begin = base_of(t) + split * a.chunk;
  const int32_t from = begin > t.lo ? begin : t.lo;
  const int32_t to = t.hi - begin > a.chunk ? begin + a.chunk : t.hi;

  // The query row of this lane, as operands and as sums per group.
  const int32_t r = t.row0 + (n < t.rows ? n : t.rows - 1);
  const int32_t i = r / a.group, head = h * a.group + r % a.group;
  const uint16_t *qp = a.q + (int64_t)(t.q0 + i) * a.ldq + (int64_t)head * D + 8 * c;
  half8 q[W];
  float row_scale, qsum[G];
  {
    uint4v raw[W];
    float top = 0.0f;
#pragma unroll
    for (int s = 0; s < W; ++s) {
      raw[s] = *reinterpret_cast<const uint4v *>(qp + 32 * s);
#pragma unroll
      for (int w = 0; w < 4; ++w)
        top = fmaxf(top, fmaxf(fabsf(up(raw[s][w] & 0xFFFFu, a.bf16)), fabsf(up(raw[s][w] >> 16, a.bf16))));
    }
    top = quarters_max(top);
    int e = top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : 0;  // top in [2^(e-1), 2^e)
    e = e < -100 ? -100 : e;
    const float mul = ldexpf(1.0f, 14 - e), factor = a.scale * kLog2e;
    row_scale = factor * ldexpf(1.0f, e - 14 + 24);
#pragma unroll
    for (int g = 0; g < G; ++g) qsum[g] = 0.0f;
#pragma unroll
    for (int s = 0; s < W; ++s) {
      float x[8];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        x[2 * w] = up(raw[s][w] & 0xFFFFu, a.bf16);
        x[2 * w + 1] = up(raw[s][w] >> 16, a.bf16);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) qsum[s / 2] += x[j];
#pragma unroll
      for (int p = 0; p < 4; ++p) {  // nibbles p and p + 4
        const float f = p & 1 ? mul * 0.0625f : mul;
        q[s][2 * p] = (_Float16)(x[p] * f);
        q[s][2 * p + 1] = (_Float16)(x[p + 4] * f);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) qsum[g] = quarters_sum(qsum[g]) * factor;
  }
  const int32_t pos = t.len - t.nq + i;                       // this lane's row sees tokens
  const int32_t row_hi = pos + 1, row_lo = a.window ? pos - a.window + 1 : 0;  // [row_lo, row_hi)
  // [all_lo, all_hi): tokens that every row of the tile sees
  const int32_t all_hi = t.len - t.nq + t.row0 / a.group + 1;
  const int32_t all_lo = a.window ? t.len - t.nq + (t.row0 + t.rows - 1) / a.group - a.window + 1 : 0;

  float4v o[J];
#pragma unroll
  for (int j = 0; j < J; ++j) o[j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
  float m = kLow, l = 0.0f, bias[G], vs = 1.0f;
#pragma unroll
  for (int g = 0; g < G; ++g) bias[g] = 0.0f;
  uint32_t vbits = 0;  // value scales up to this fp16 pattern fit the power of two vs

  const int32_t P = 1 << a.page_log2;
  const int32_t block = mixllm::kv4_block_bytes(P, D);
  const int32_t *table = a.table + b * a.ldt;
  const int32_t koff = n * (D / 2) + c * (D / 8), voff = P * (D / 2) + (c * 16 + n) * 4 * (D / 32);
  const int32_t poff = P * D + (lane >> 5) * (P * (D / 16)) + (lane & 15) * (4 * G);
  uint32_t *par = s_par[wave];

  auto load = [&](Step<D> &st, int32_t t0) {
    const uint8_t *base[2];
    int32_t in[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int32_t tx = t0 + 16 * x;
      int32_t pg = tx < to ? table[tx >> a.page_log2] : -1;
      st.ok[x] = (uint32_t)pg < (uint32_t)a.pages;
      pg = st.ok[x] ? pg : 0;
      in[x] = tx & (P - 1);
      base[x] = a.cache + ((int64_t)pg * a.hkv + h) * block + in[x] * (D / 2);
      load_words(base[x] + koff, st.k[x]);
      load_words(base[x] + voff, st.v[x]);
    }
    // parameters of this lane's token, nothing for one that is not there
    const int x = (lane >> 4) & 1;
    const uint8_t *bp = x ? base[1] - in[1] * (D / 2) + in[1] * (4 * G) : base[0] - in[0] * (D / 2) + in[0] * (4 * G);
    load_words(bp + poff, st.par);
    const bool there = (x ? st.ok[1] : st.ok[0]) && t0 + (lane & 31) < to;
#pragma unroll
    for (int g = 0; g < G; ++g) st.par[g] = there ? st.par[g] : 0u;
  };

  auto compute = [&](const Step<D> &st, int32_t t0) {
    // Every lane needs the parameters of the 8 tokens of its quarter: through LDS.
#pragma unroll
    for (int g = 0; g < G; ++g) par[lane * G + g] = st.par[g];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    half2v kp[2][4][G], vp[2][4][G];  // [16 tokens][token][scales, then minima]
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          kp[x][u][g] = __builtin_bit_cast(half2v, par[(16 * x + 4 * c + u) * G + g]);
          vp[x][u][g] = __builtin_bit_cast(half2v, par[(32 + 16 * x + 4 * c + u) * G + g]);
        }
    __builtin_amdgcn_wave_barrier();
    auto at = [](const half2v (&p)[G], int e) { return (float)p[e / 2][e % 2]; };

    float s[8];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float4v acc[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        acc[g] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
        acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes8(st.k[x][2 * g]), q[2 * g], acc[g], 0, 0, 0);
        acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes8(st.k[x][2 * g + 1]), q[2 * g + 1], acc[g], 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float dot = 0.0f, add = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          dot = fmaf(at(kp[x][u], g), acc[g][u], dot);
          add = fmaf(at(kp[x][u], G + g), qsum[g], add);
        }
        s[4 * x + u] = fmaf(row_scale, dot, add);
      }
    }
    if (!(t0 >= all_lo && t0 >= from && t0 + kStep <= all_hi && t0 + kStep <= to && st.ok[0] && st.ok[1])) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int32_t tok = t0 + 16 * (e / 4) + 4 * c + e % 4;
        const bool seen = tok < row_hi && tok >= row_lo && tok < to && tok >= from && st.ok[e / 4];
        s[e] = seen ? s[e] : -INFINITY;
      }
    }
    float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
    top = quarters_max(top);
    uint32_t big = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t v = __builtin_bit_cast(uint16_t, vp[e / 4][e % 4][g / 2][g % 2]);
        big = v > big ? v : big;
      }
    if (__any(top > m + kLazy || big > vbits)) {
      float ratio = 1.0f;
      if (__any(big > vbits)) {
        big = quarters_max(big);
        const uint32_t e = big >> 10 ? big >> 10 : 1;
        vbits = e << 10 | 0x3FF;
        const float to_scale = __uint_as_float((127 + 23 - e) << 23);  // a scale below 2^(e-14) times this is below 2^9
        ratio = to_scale / vs;
        vs = to_scale;
      }
      const float next = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
#pragma unroll
      for (int g = 0; g < G; ++g) bias[g] *= f;
#pragma unroll
      for (int j = 0; j < J; ++j) o[j] *= f * ratio;
    }
    half8 p[G];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float w = __builtin_amdgcn_exp2f(s[e] - m);
      l += w;
      const float wv = w * vs;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        bias[g] = fmaf(at(vp[e / 4][e % 4], G + g), w, bias[g]);
        p[g][e] = (_Float16)(wv * at(vp[e / 4][e % 4], g));
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      uint32_t w[4];  // pairs of tokens, the 4 nibbles of group g's channels in each half
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        if (D == 64) {
          w[z] = st.v[z / 2][z % 2];
        } else {
          const int per = D / 128;  // dwords of one token
          const int d0 = (z % 2) * 2 * per + g / 2;
          w[z] = __builtin_amdgcn_perm(st.v[z / 2][d0 + per], st.v[z / 2][d0], g % 2 ? 0x07060302u : 0x05040100u);
        }
      }
#pragma unroll
      for (int nib = 0; nib < 4; ++nib) {
        const uint4v v = {nibble_pair(w[0], nib), nibble_pair(w[1], nib), nibble_pair(w[2], nib), nibble_pair(w[3], nib)};
        o[4 * g + nib] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, v), p[g], o[4 * g + nib], 0, 0, 0);
      }
    }
  };

  {
    int32_t t0 = (from & ~(kStep - 1)) + wave * kStep;
    Step<D> st[2];
    if (t0 < to) load(st[0], t0);
    while (t0 < to) {
      int32_t t1 = t0 + kWaves * kStep;
      if (t1 < to) load(st[1], t1);
      compute(st[0], t0);
      if (t1 >= to) break;
      t0 = t1 + kWaves * kStep;
      if (t0 < to) load(st[0], t0);
      compute(st[1], t1);
    }
  }

  // The four waves' statistics and outputs, over the largest maximum.
  l = quarters_sum(l);
#pragma unroll
  for (int g = 0; g < G; ++g) bias[g] = quarters_sum(bias[g]);
  if (c == 0) {
    s_m[wave][n] = m;
    s_l[wave][n] = l;
  }
  __syncthreads();
  const float best = fmaxf(fmaxf(s_m[0][n], s_m[1][n]), fmaxf(s_m[2][n], s_m[3][n]));
  const float f = __builtin_amdgcn_exp2f(m - best);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float fo = f * (j & 1 ? 0x1p20f : 0x1p24f) / vs, fb = f * bias[j / 4];
    float4v v;
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = fmaf(o[j][u], fo, fb);
    *reinterpret_cast<float4v *>(&s_o[wave][n * kStride + 16 * j + 4 * c]) = v;
  }
  __syncthreads();
  const int64_t part = ((int64_t)(b * a.tiles + rt) * a.hkv + h) * a.splits + split;
  for (int e = threadIdx.x; e < t.rows * (D / 8); e += kThreads) {
    const int row = e / (D / 8), ch = e % (D / 8) * 8;
    float top = s_m[0][row], sum = 0.0f;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, s_m[w][row]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum = fmaf(s_l[w][row], __builtin_amdgcn_exp2f(s_m[w][row] - top), sum);
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] += s_o[w][row * kStride + ch + u];
    if (a.splits > 1) {
      float *dst = a.ws_o + (part * a.rows_tile + row) * D + ch;
      *reinterpret_cast<float4v *>(dst) = float4v{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<float4v *>(dst + 4) = float4v{v[4], v[5], v[6], v[7]};
      if (ch == 0) *reinterpret_cast<float2v *>(a.ws_ml + (part * a.rows_tile + row) * 2) = float2v{top, sum};
    } else {
      const int32_t rr = t.row0 + row, ii = t.q0 + rr / a.group, hh = h * a.group + rr % a.group;
      const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // NaN stays NaN
      uint32_t w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = down(v[2 * u] * inv, a.bf16) | down(v[2 * u + 1] * inv, a.bf16) << 16;
      *reinterpret_cast<uint4v *>(a.out + (int64_t)ii * a.ldo + (int64_t)hh * D + ch) = uint4v{w[0], w[1], w[2], w[3]};
      if (ch == 0 && a.lse) a.lse[(int64_t)ii * a.hq + hh] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
  }
}

// Joins the chunks of a row: out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.  WAVES
// waves share a row and head, wave w takes the chunks w, w + WAVES, ..
template <int D, int WAVES>
__global__ __launch_bounds__(kThreads) void kv4_join_kernel(Args a) {
  constexpr int C = D / 64;  // channels of a lane
  __shared__ float s_m[kWaves], s_l[kWaves], s_o[kWaves][D];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t id = (int64_t)blockIdx.x * (kWaves / WAVES) + wave / WAVES;
  const int64_t all = (int64_t)a.B * a.max_rows * a.hq;
  const bool live = id < all;
  id = live ? id : all - 1;
  const int32_t head = (int32_t)(id % a.hq);
  id /= a.hq;
  const int32_t i = (int32_t)(id % a.max_rows), b = (int32_t)(id / a.max_rows);
  const int32_t h = head / a.group, r = i * a.group + head % a.group, rt = r / kRows, row = r % kRows;
  const Tile t = tile_of(a, b, h, rt);
  const bool there = live && i < t.nq;
  const int32_t nchunks = there ? chunks_of(a, t) : 0;
  const int64_t part0 = ((int64_t)(b * a.tiles + rt) * a.hkv + h) * a.splits;
  const float *ml = a.ws_ml + (part0 * a.rows_tile + row) * 2;
  const float *po = a.ws_o + (part0 * a.rows_tile + row) * D + lane * C;
  float m = kLow, l = 0.0f, o[C] = {};
  for (int32_t s = wave % WAVES; s < nchunks; s += WAVES) {
    const float ms = ml[(int64_t)s * a.rows_tile * 2], ls = ml[(int64_t)s * a.rows_tile * 2 + 1];
    const float next = fmaxf(m, ms), f = __builtin_amdgcn_exp2f(m - next), fs = __builtin_amdgcn_exp2f(ms - next);
    m = next;
    l = fmaf(l, f, ls * fs);
#pragma unroll
    for (int e = 0; e < C; ++e) o[e] = fmaf(o[e], f, po[(int64_t)s * a.rows_tile * D + e] * fs);
  }
  if (WAVES > 1) {
    if (lane == 0) {
      s_m[wave] = m;
      s_l[wave] = l;
    }
#pragma unroll
    for (int e = 0; e < C; ++e) s_o[wave][lane * C + e] = o[e];
    __syncthreads();
    if (wave % WAVES != 0) return;
    float top = m;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) top = fmaxf(top, s_m[w]);
    float f = __builtin_amdgcn_exp2f(m - top);
    l *= f;
#pragma unroll
    for (int e = 0; e < C; ++e) o[e] *= f;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      f = __builtin_amdgcn_exp2f(s_m[w] - top);
      l = fmaf(s_l[w], f, l);
#pragma unroll
      for (int e = 0; e < C; ++e) o[e] = fmaf(s_o[w][lane * C + e], f, o[e]);
    }
    m = top;
  }
  if (!there) return;
  const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
  uint16_t *dst = a.out + (int64_t)(t.q0 + i) * a.ldo + (int64_t)head * D + lane * C;
#pragma unroll
  for (int e = 0; e < C; ++e) dst[e] = (uint16_t)down(o[e] * inv, a.bf16);
  if (lane == 0 && a.lse) a.lse[(int64_t)(t.q0 + i) * a.hq + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// How the work of a call is cut.  Rows: tiles of 16 (row, head) pairs of one key/value head.
// Tokens: chunks of a multiple of 128 (one step of each wave) so that about kTarget
// workgroups run; 256 CUs hold 4 of them each.
constexpr int64_t kTarget = 2048;
constexpr int32_t kMaxChunk = 2048;

struct Cut {
  int32_t tiles, rows_tile, splits, chunk;
};

Cut cut_of(int32_t B, int32_t hq, int32_t hkv, int32_t max_rows, int32_t max_len, int32_t window) {
  Cut k;
  const int64_t rows = (int64_t)max_rows * (hq / hkv);
  k.tiles = (int32_t)((rows + kRows - 1) / kRows);
  k.rows_tile = rows < kRows ? (int32_t)rows : kRows;
  int64_t span = max_len;
  // a tile's rows are at most 16 positions, its first chunk starts at a whole step
  if (window && (int64_t)window + kRows + kStep < span) span = (int64_t)window + kRows + kStep;
  const int64_t groups = (int64_t)B * hkv * k.tiles;
  int64_t chunk = (span * groups + kTarget - 1) / kTarget;
  chunk = (chunk + 127) / 128 * 128;
  chunk = chunk < 128 ? 128 : chunk > kMaxChunk ? kMaxChunk : chunk;
  if (groups >= kTarget) chunk = span < 128 ? 128 : (span + 127) / 128 * 128;
  k.chunk = (int32_t)chunk;
  k.splits = span <= chunk ? 1 : (int32_t)((span + chunk - 1) / chunk);
  return k;
}

bool shape_ok(int64_t T, int32_t B, int32_t hq, int32_t hkv, int32_t dim, int32_t max_rows, int32_t max_len,
              int32_t window) {
  if (T < 0 || B < 0 || hkv <= 0 || hq <= 0 || hq % hkv != 0 || !mixllm::kv4_dim_ok(dim) || max_rows < 0 ||
      max_len < 0 || window < 0)
    return false;
  // 32-bit row and token arithmetic: rows of a request and head, positions plus a window
  return (int64_t)max_rows * (hq / hkv) < (1 << 30) && max_len < (1 << 30) && window < (1 << 30) && hq < (1 << 20);
}

template <int D>
void launch(const Args &a, int64_t blocks, hipStream_t s) {
  hipLaunchKernelGGL((kv4_attention_kernel<D>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
  if (a.splits == 1 || hipPeekAtLastError() != hipSuccess) return;
  const int64_t rows = (int64_t)a.B * a.max_rows * a.hq;
  if (a.splits > 16) hipLaunchKernelGGL((kv4_join_kernel<D, 4>), dim3((unsigned)rows), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((kv4_join_kernel<D, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(kThreads), 0, s, a);
}

}  // namespace

extern "C" size_t mixllm_kv4_attention_workspace_bytes(int32_t T, int32_t B, int32_t q_heads, int32_t kv_heads,
                                                       int32_t dim, int32_t max_rows, int32_t max_len,
                                                       int32_t window) {
  if (!shape_ok(T, B, q_heads, kv_heads, dim, max_rows, max_len, window) || T == 0 || B == 0 || max_rows == 0) return 0;
  const Cut k = cut_of(B, q_heads, kv_heads, max_rows, max_len, window);
  if (k.splits == 1) return 0;
  return (size_t)B * k.tiles * kv_heads * k.splits * k.rows_tile * (dim + 2) * sizeof(float);
}

extern "C" int mixllm_kv4_attention(const void *q, int64_t ldq, int32_t dtype, int32_t T, int32_t q_heads,
                                    const void *cache, size_t cache_bytes, int32_t pages, int32_t page,
                                    int32_t kv_heads, int32_t dim, const int32_t *table, int64_t ldt, int32_t width,
                                    const int32_t *lens, const int32_t *cu, int32_t B, int32_t max_rows,
                                    int32_t max_len, float scale, int32_t window, void *out, int64_t ldo, float *lse,
                                    void *workspace, size_t workspace_bytes, void *stream) {
  if (!shape_ok(T, B, q_heads, kv_heads, dim, max_rows, max_len, window) ||
      (dtype != MIXLLM_FP16 && dtype != MIXLLM_BF16))
    return MIXLLM_E_SHAPE;
  if (T == 0 || B == 0 || max_rows == 0) return MIXLLM_OK;
  const int st = mixllm::kv4_check_cache(cache, cache_bytes, pages, page, kv_heads, dim);
  if (st != MIXLLM_OK) return st;
  const int64_t qw = (int64_t)q_heads * dim;
  if (width <= 0 || ldt < width || ldq < qw || ldo < qw || ldq % 8 != 0 || ldo % 8 != 0) return MIXLLM_E_SHAPE;
  if (!q || !table || !lens || !cu || !out) return MIXLLM_E_NULL;
  if (!mixllm::is_aligned16(q) || !mixllm::is_aligned16(out) || !mixllm::is_aligned4(table) ||
      !mixllm::is_aligned4(lens) || !mixllm::is_aligned4(cu) || !mixllm::is_aligned4(lse) ||
      !mixllm::is_aligned16(workspace))
    return MIXLLM_E_SHAPE;
  const Cut k = cut_of(B, q_heads, kv_heads, max_rows, max_len, window);
  const int64_t parts = (int64_t)B * k.tiles * kv_heads * k.splits;
  if (parts > 0x7FFFFFFF || (int64_t)B * k.tiles > 0x7FFFFFFF || (int64_t)B * max_rows * q_heads > 0x7FFFFFFF)
    return MIXLLM_E_SHAPE;
  float *ws = static_cast<float *>(workspace);
  if (k.splits > 1) {
    if (workspace_bytes < (size_t)parts * k.rows_tile * (dim + 2) * sizeof(float)) return MIXLLM_E_SPACE;
    if (!ws) return MIXLLM_E_NULL;
  }
  const Args a = {static_cast<const uint16_t *>(q), static_cast<const uint8_t *>(cache), table, lens, cu,
                  static_cast<uint16_t *>(out), lse, ws, ws ? ws + parts * k.rows_tile * dim : nullptr,
                  ldq, ldo, ldt, scale, T, q_heads, kv_heads, q_heads / kv_heads, pages,
                  mixllm::log2_of(page), width, B, max_rows,
                  max_len, window, k.tiles, k.rows_tile, k.splits, k.chunk, dtype == MIXLLM_BF16};
  if (dim == 64) launch<64>(a, parts, (hipStream_t)stream);
  else if (dim == 128) launch<128>(a, parts, (hipStream_t)stream);
  else launch<256>(a, parts, (hipStream_t)stream);
  return mixllm::launch_status();
}
