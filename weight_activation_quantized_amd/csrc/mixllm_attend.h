// What the attention kernels over the paged caches share, whatever the cache holds: which rows
// and tokens a workgroup takes, moves between the lanes of a row, the join of the chunks that
// workgroups leave of a row, and the checks of a call.
#ifndef MIXLLM_ATTEND_H_
#define MIXLLM_ATTEND_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm_kv4.h"
#include "mixllm_lanes.h"

namespace {  // each source compiles its own kernels

using mixllm::down;
using mixllm::up;

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRun = 16;          // tokens of a run: a page holds it whole
constexpr int kCols = 16;         // columns of a matrix operand
constexpr int32_t kMinChunk = 256;  // tokens: one step of each wave
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
  int32_t tiles, tile_rows;  // row tiles of a request and head, rows of a full tile
  int32_t splits;            // workgroups along the tokens of a tile
};

// Maximum and sum over the four lanes n, n + 16, n + 32, n + 48 of a query row.
__device__ __forceinline__ float quarters_max(float v) {
  uint2v a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
}

__device__ __forceinline__ float quarters_sum(float v) {
  uint2v a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a.x) + __uint_as_float(a.y);
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a.x) + __uint_as_float(a.y);
}

// The request, rows and tokens of a workgroup.  Row i of the request has the position
// pos0 + i; how many of its rows are computed does not move them.
struct Tile {
  int32_t b, h, row0, rows, n, q0, pos0;  // rows: query rows of this tile; n: of the request, computed ones
  int32_t lo, hi;                         // tokens that any of its rows sees
};

__device__ __forceinline__ Tile tile_of(const Args &a, int32_t b, int32_t h, int32_t rt) {
  Tile t;
  t.b = b, t.h = h, t.row0 = rt * a.tile_rows;
  const int32_t first_row = a.cu[b], end = a.cu[b + 1];
  t.q0 = first_row > 0 ? first_row : 0;
  const int32_t nq = end > t.q0 ? end - t.q0 : 0;  // rows behind T count: they are the request's last ones
  const int32_t room = t.q0 < a.T ? a.T - t.q0 : 0;
  t.n = nq < a.max_rows ? nq : a.max_rows;
  t.n = t.n < room ? t.n : room;
  const int64_t cap = (int64_t)a.width << a.page_log2;
  const int32_t most = cap < a.max_len ? (int32_t)cap : a.max_len, held = a.lens[b];
  const int32_t len = held < 0 ? 0 : held < most ? held : most;
  // the host keeps max_rows below 2^30: from there down no row sees anything
  t.pos0 = len - nq > -(1 << 30) ? len - nq : -(1 << 30);
  const int64_t all = (int64_t)t.n * a.group;
  const int64_t left = all - t.row0;
  t.rows = left <= 0 ? 0 : left < a.tile_rows ? (int32_t)left : a.tile_rows;
  if (t.rows > 0) {
    const int32_t first = t.pos0 + t.row0 / a.group, last = t.pos0 + (t.row0 + t.rows - 1) / a.group;
    t.hi = last + 1 > 0 ? last + 1 : 0;
    t.lo = a.window && first - a.window + 1 > 0 ? first - a.window + 1 : 0;
    t.lo = t.lo < t.hi ? t.lo : t.hi;
  } else {
    t.lo = t.hi = 0;
  }
  return t;
}

// The chunks of a tile start at its first token, rounded down to whole runs.
__device__ __forceinline__ int32_t base_of(const Tile &t) { return t.lo & ~(kRun - 1); }
// Each of the `splits` workgroups takes an equal chunk, a multiple of 64 tokens, 256 or more.
__device__ __forceinline__ int32_t chunk_of(const Args &a, const Tile &t) {
  const int32_t each = (int32_t)(((uint32_t)(t.hi - base_of(t)) + a.splits - 1) / (uint32_t)a.splits);
  return each <= kMinChunk ? kMinChunk : (each + 63) & ~63;
}
__device__ __forceinline__ int32_t chunks_of(const Tile &t, int32_t chunk) {
  return (int32_t)(((uint32_t)(t.hi - base_of(t)) + chunk - 1) / (uint32_t)chunk);
}

// Joins the chunks of a row: out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.  WAVES
// waves share a row and head, wave w takes the chunks w, w + WAVES, ..; a workgroup has 4 waves
// or as many as share.  Up to 16 chunks a wave does alone (4 us, of which a launch is most);
// 64 chunks take 5.7 us with 16 waves, 8.0 with 4.  A: Args, or what a cache adds to them.
template <int D, int WAVES, bool BF16, class A>
__global__ __launch_bounds__(64 * (WAVES > kWaves ? WAVES : kWaves)) void join_kernel(A a) {
  constexpr int C = D / 64;  // channels of a lane
  constexpr int kAll = WAVES > kWaves ? WAVES : kWaves;
  __shared__ float s_m[kAll], s_l[kAll], s_o[kAll][D];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t id = (int64_t)blockIdx.x * (kAll / WAVES) + wave / WAVES;
  const int64_t all = (int64_t)a.B * a.max_rows * a.hq;
  const bool live = id < all;
  id = live ? id : all - 1;
  const int32_t head = (int32_t)(id % a.hq);
  id /= a.hq;
  const int32_t i = (int32_t)(id % a.max_rows), b = (int32_t)(id / a.max_rows);
  const int32_t h = head / a.group, r = i * a.group + head % a.group, rt = r / a.tile_rows, row = r % a.tile_rows;
  const Tile t = tile_of(a, b, h, rt);
  const bool there = live && i < t.n;
  const int32_t nchunks = there ? chunks_of(t, chunk_of(a, t)) : 0;
  const int64_t part0 = ((int64_t)(b * a.tiles + rt) * a.hkv + h) * a.splits;
  const float *ml = a.ws_ml + (part0 * a.tile_rows + row) * 2;
  const float *po = a.ws_o + (part0 * a.tile_rows + row) * D + lane * C;
  float m = 2.0f * kLow, l = 0.0f, o[C] = {};
  const int32_t mine = (nchunks - wave % WAVES + WAVES - 1) / WAVES;  // chunks of this wave
  for (int32_t j0 = 0; j0 < mine; j0 += 64) {
    // 64 chunks' statistics at once, one per lane; then their outputs, whose loads do not wait
    // for one another
    const int32_t many = mine - j0 < 64 ? mine - j0 : 64;
    float2v st = {2.0f * kLow, 0.0f};
    if (lane < many)
      st = *reinterpret_cast<const float2v *>(ml + (int64_t)(wave % WAVES + (j0 + lane) * WAVES) * a.tile_rows * 2);
    float top = st.x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float next = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - next);
    const float weight = __builtin_amdgcn_exp2f(st.x - next);
    m = next;
    float sum = st.y * weight;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    l = fmaf(l, f, sum);
#pragma unroll
    for (int e = 0; e < C; ++e) o[e] *= f;
#pragma unroll 8
    for (int32_t j = 0; j < many; ++j) {
      const float *src = po + (int64_t)(wave % WAVES + (j0 + j) * WAVES) * a.tile_rows * D;
      const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), j));
#pragma unroll
      for (int e = 0; e < C; ++e) o[e] = fmaf(src[e], w, o[e]);
    }
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
  for (int e = 0; e < C; ++e) dst[e] = (uint16_t)down<BF16>(o[e] * inv);
  if (lane == 0 && a.lse) a.lse[(int64_t)(t.q0 + i) * a.hq + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// The second launch of a call whose tokens are split.
template <int D, bool BF16, class A>
void launch_join(const A &a, hipStream_t s) {
  const int64_t rows = (int64_t)a.B * a.max_rows * a.hq;
  if (a.splits > 16) hipLaunchKernelGGL((join_kernel<D, 16, BF16, A>), dim3((unsigned)rows), dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((join_kernel<D, 1, BF16, A>), dim3((unsigned)((rows + 3) / 4)), dim3(kThreads), 0, s, a);
}

struct Cut {
  int32_t tiles, tile_rows, splits;
};

bool shape_ok(int64_t T, int32_t B, int32_t hq, int32_t hkv, int32_t dim, int32_t max_rows, int32_t max_len,
              int32_t window) {
  if (T < 0 || T >= (1 << 30) || B < 0 || hkv <= 0 || hq <= 0 || hq % hkv != 0 || !mixllm::kv4_dim_ok(dim) || max_rows < 0 ||
      max_len < 0 || window < 0)
    return false;
  // 32-bit row and token arithmetic: rows of a request and head, positions plus a window
  return (int64_t)max_rows * (hq / hkv) < (1 << 30) && max_len < (1 << 30) && window < (1 << 30) && hq < (1 << 20);
}

// The checks of a call's arrays but for its cache.
int check_call(const void *q, int64_t ldq, int32_t hq, int32_t dim,
               const int32_t *table, int64_t ldt, int32_t width, const int32_t *lens, const int32_t *cu,
               const void *out, int64_t ldo, const float *lse, const void *workspace) {
  const int64_t qw = (int64_t)hq * dim;
  if (width <= 0 || ldt < width || ldq < qw || ldo < qw || ldq % 8 != 0 || ldo % 8 != 0) return MIXLLM_E_SHAPE;
  if (!q || !table || !lens || !cu || !out) return MIXLLM_E_NULL;
  if (!mixllm::is_aligned16(q) || !mixllm::is_aligned16(out) || !mixllm::is_aligned4(table) ||
      !mixllm::is_aligned4(lens) || !mixllm::is_aligned4(cu) || !mixllm::is_aligned4(lse) ||
      !mixllm::is_aligned16(workspace))
    return MIXLLM_E_SHAPE;
  return MIXLLM_OK;
}

}  // namespace

#endif  // MIXLLM_ATTEND_H_
