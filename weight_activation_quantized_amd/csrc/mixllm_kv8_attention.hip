// Attention over the paged key/value cache held in 8 bits (layout: mixllm_kv8.h), for decoded
// tokens and for the rows of prompts.
//
// For one query row with position p of a request, over the keys t in (p - window, p], with one
// scale for the keys (k) and one for the values (v) of each run r of 16 tokens:
//   S_t = scale * k_r (q . c_t);   O = sum_t P_t v_r c'_t / sum_t P_t,  P_t = exp(S_t - max S)
// so codes enter the 16 x 16 x 32 fp16 matrix instruction as they are (whole numbers of 8 bits
// are exact in fp16) and a run's scale multiplies 16 x 16 scores or weights at once.
//
// Both products are computed transposed: S^T = K Q^T leaves in lane (n, c) the scores of query
// row n with tokens 4c .. 4c+3 of a run, and O^T = V^T P^T takes from lane (n, c) the weights of
// row n for the tokens that quarter c holds, which are the same.  The cache's order makes both
// operands of codes 16-byte loads of the lane that needs them, straight from memory.
//
// A byte b of a code c = b - 128 becomes fp16 by placing it under the exponent of 1024, 1024 + b,
// and taking 1152 away, exactly: two operations for two codes.
//
// Weights 2^(S - ref) times a run's scale v are rounded to fp16 for the product, after a power of
// two per row that follows the largest such product (`shift`), so that rows whose large
// values hardly count lose nothing; what the rounding leaves is a second operand (error of fp16
// outputs 1.0 times that of their own rounding; bf16 prompts, whose rounding is 8 times coarser, go
// without: 145 us for 2 x 1024 rows, where fp16 takes 183 - 190).  Statistics, sums and outputs are fp32.
//
// What bounds it, at 128 channels.  Decodes: the cache's bytes, 128 requests of up to 8192 tokens 1.68 GB
// in 312 us, 5.4 TB/s (a large read reaches 5.9), one of 131071 tokens 269 MB in 45.7 us and 6 for the
// join; small ones latency (77 tokens 5.8 us).  Prompts (2 x 1024 rows over 4096 tokens: 590 TFLOP/s in
// fp16, 750 in bf16, where a large library product reaches 1176): the softmax, whose 250 vector
// operations a step one wave of a SIMD issues at about 7 cycles each while the other multiplies:
// 1800 - 2350 cycles of the weighing phase to 1000 - 1500 of matrix instructions.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm_attend.h"
#include "mixllm_kv8.h"
#include "mixllm_lanes.h"

namespace {

// A launch takes the requests whose (row, head) pairs of a key/value head are `least` to `most`.
struct Args8 : Args {
  int32_t least, most;
  int32_t units;  // tiles of all requests one after another (find_tile); 0: `tiles` for each request
};

__device__ __forceinline__ Tile tile_of(const Args8 &a, int32_t b, int32_t h, int32_t rt) {
  Tile t = tile_of(static_cast<const Args &>(a), b, h, rt);
  const int64_t all = (int64_t)t.n * a.group;
  if (all < a.least || all > a.most) t.n = t.rows = t.lo = t.hi = 0;
  return t;
}

// Tile rt of request b as number `unit` from the last: request b's begin at number cu[b] group / ROWS + b,
// which leaves each request the numbers that its tiles need.  The wave looks for the last request
// that begins at or before it, 64 at a time.  False: there is none, or it has no such tile.
template <int ROWS>
__device__ __forceinline__ bool find_tile(const Args8 &a, int64_t unit, int32_t &b, int32_t &rt) {
  unit = a.units - 1 - unit;
  auto begin = [&](int32_t i) {
    const int32_t row = a.cu[i] < 0 ? 0 : a.cu[i] < a.T ? a.cu[i] : a.T;
    return (int64_t)((uint64_t)((int64_t)row * a.group) / ROWS) + i;
  };
  const int32_t lane = threadIdx.x & 63;
  b = 0;
  for (int32_t left = a.B;;) {
    const int32_t step = (left + 63) / 64, off = lane * step;
    const int32_t before = __popcll(__ballot(off < left && begin(b + (off < left ? off : 0)) <= unit));
    if (before == 0) return false;
    b += (before - 1) * step;
    if (step == 1) break;
    left = left - (before - 1) * step < step ? left - (before - 1) * step : step;
  }
  b = __builtin_amdgcn_readfirstlane(b);
  const int64_t tile = unit - begin(b);
  rt = (int32_t)tile;
  return tile >= 0 && tile < a.tiles;
}

// 8 codes as fp16, exactly.
__device__ __forceinline__ half8 codes8(uint32_t lo, uint32_t hi) {
  constexpr uint32_t k1024 = 0x64646464u;
  const uint4v b = {__builtin_amdgcn_perm(k1024, lo, 0x04010400u), __builtin_amdgcn_perm(k1024, lo, 0x04030402u),
                    __builtin_amdgcn_perm(k1024, hi, 0x04010400u), __builtin_amdgcn_perm(k1024, hi, 0x04030402u)};
  return __builtin_bit_cast(half8, b) - (_Float16)(1024 + mixllm::kKv8Zero);
}

template <int N>
struct Const {
  static constexpr int value = N;
};

constexpr int kTokens = 2 * kRun;  // of a step: two runs fill an operand of the second product
constexpr float kTop = 14.0f;      // weights times scales stay below 2^kTop, fp16 ends at 2^16
constexpr float kRoom = 5.0f;      // and are moved there or kRoom below

// One step's codes, as loaded.
template <int D>
struct Stage {
  uint4v k[2][D / 64], v[2][D / 64];
};

// CT: column blocks of 16 rows that share the operands made of codes.  ONCE: one tile holds all rows of
// a request and head, so a code is read once and its line need not stay in the caches (us, one
// tile: 128 requests of up to 8192 tokens 346 -> 312, 32 of up to 4001 50.3 -> 44.3; two tiles that
// read the same codes 34.6 -> 37.2, so not there; requests whose tables name the same pages read them
// past the caches too, 128 over the same 8192 tokens 166.5 -> 167).
template <int D, int CT, bool ONCE, bool BF16>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void kv8_attention_kernel(Args8 a) {
  constexpr int U = D / 64, E = D / 32, J = D / 16;
  constexpr int kStride = D + 4;  // floats of a row of partial outputs in LDS
  constexpr int kAll = CT * kCols;
  __shared__ __attribute__((aligned(16))) float s_o[kWaves * kAll * kStride];
  __shared__ float s_m[kWaves][kAll], s_l[kWaves][kAll];

  const int lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t h = blockIdx.x / a.splits, split = blockIdx.x - h * a.splits, b = blockIdx.z;
  const int32_t rt = a.tiles - 1 - (int32_t)blockIdx.y;  // a request's last rows see most tokens: their tiles first
  const Tile t = tile_of(a, b, h, rt);
  if (t.rows <= 0) return;
  const int32_t chunk = chunk_of(a, t), nchunks = chunks_of(t, chunk);
  if (split >= nchunks && !(split == 0 && a.splits == 1)) return;
  const int32_t begin = base_of(t) + split * chunk;
  const int32_t from = begin > t.lo ? begin : t.lo;
  const int32_t to = t.hi - begin > chunk ? begin + chunk : t.hi;

  const int32_t P = 1 << a.page_log2, block = mixllm::kv8_block_bytes(P, D);
  const int32_t *table = a.table + b * a.ldt;

  // This wave takes every fourth step, in batches whose pages and scales one load each fetches:
  // lane 2 j + x has those of run x of the batch's step j; page -1 for none.
  constexpr int32_t kStride4 = kWaves * kTokens, kBatch = 32;
  int32_t tb = (from & ~(kRun - 1)) + wave * kTokens, steps = 0, pages = -1;
  float k_scale = 0.0f, v_scale = 0.0f;
  uint64_t there = 0;
  auto load = [&](Stage<D> &st, int32_t j) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int32_t pg = __builtin_amdgcn_readlane(pages, 2 * j + x);
      const int32_t in = (tb + j * kStride4 + kRun * x) & (P - 1);
      // an absent run reads any memory of the cache; its scores are masked
      const uint8_t *src = a.cache + ((int64_t)(pg < 0 ? 0 : pg) * a.hkv + h) * block + (int64_t)in * D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint4v *k = reinterpret_cast<const uint4v *>(src + u * 1024 + lane * 16);
        const uint4v *v = reinterpret_cast<const uint4v *>(src + P * D + u * 1024 + lane * 16);
        st.k[x][u] = ONCE ? __builtin_nontemporal_load(k) : *k;
        st.v[x][u] = ONCE ? __builtin_nontemporal_load(v) : *v;
      }
    }
  };
  auto fetch = [&]() {  // for the batch at tb < to
    const int32_t tok = tb + lane / 2 * kStride4 + lane % 2 * kRun;
    pages = tok < to ? table[tok >> a.page_log2] : -1;
    pages = (uint32_t)pages < (uint32_t)a.pages ? pages : -1;
    there = __ballot(pages >= 0);
    const int32_t left = (to - tb + kStride4 - 1) / kStride4;
    steps = left < kBatch ? left : kBatch;
    k_scale = v_scale = 0.0f;
    if (pages >= 0) {
      const float2v s = *reinterpret_cast<const float2v *>(a.cache + ((int64_t)pages * a.hkv + h) * block +
                                                           mixllm::kv8_scale_offset(P, D) + (tok & (P - 1)) / kRun * 8);
      k_scale = s.x, v_scale = s.y;
    }
  };
  Stage<D> st0, st1;
  if (tb < to) {
    fetch();
    load(st0, 0);
  }

  // The query rows of this lane, as operands: step e has the channels 64 (e/2) + 16 c + 8 (e%2) on.
  half8 q[CT][E];
  float row_scale[CT];
  int32_t row_hi[CT], row_lo[CT];  // the row sees tokens [row_lo, row_hi)
#pragma unroll
  for (int z = 0; z < CT; ++z) {
    const int32_t row = kCols * z + n, r = t.row0 + (row < t.rows ? row : t.rows - 1);
    const int32_t i = r / a.group, head = h * a.group + r % a.group;
    const uint16_t *qp = a.q + (int64_t)(t.q0 + i) * a.ldq + (int64_t)head * D + 16 * c;
    uint4v raw[E];
#pragma unroll
    for (int e = 0; e < E; ++e) raw[e] = *reinterpret_cast<const uint4v *>(qp + e / 2 * 64 + e % 2 * 8);
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        top = fmaxf(top, fmaxf(fabsf(up<BF16>(raw[e][w] & 0xFFFFu)), fabsf(up<BF16>(raw[e][w] >> 16))));
    top = quarters_max(top);
    // a power of two brings the row below 2^14: bf16 fits fp16 but for values 2^-38 below the largest
    int p = top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : 0;  // top in [2^(p-1), 2^p)
    p = p < -100 ? -100 : p;
    const float mul = ldexpf(1.0f, 14 - p);
    row_scale[z] = ldexpf(a.scale * kLog2e, p - 14);
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        q[z][e][2 * w] = (_Float16)(up<BF16>(raw[e][w] & 0xFFFFu) * mul);
        q[z][e][2 * w + 1] = (_Float16)(up<BF16>(raw[e][w] >> 16) * mul);
      }
    const int32_t pos = t.pos0 + i;
    row_hi[z] = pos + 1;
    row_lo[z] = a.window ? pos - a.window + 1 : 0;
  }
  // [all_lo, all_hi): tokens that every row of the tile sees
  const int32_t all_hi = t.pos0 + t.row0 / a.group + 1;
  const int32_t all_lo = a.window ? t.pos0 + (t.row0 + t.rows - 1) / a.group - a.window + 1 : 0;

  // l = sum 2^(s - ref) and o = sum 2^(s - ref) v c 2^-shift of the tokens so far.  `ref` is the
  // largest score seen, up to kLazy, `peak` the largest s - ref + log2 v, up to kRoom.
  float4v o[CT][J];
  float ref[CT], l[CT], limit[CT], peak[CT];
  int32_t shift[CT];
#pragma unroll
  for (int z = 0; z < CT; ++z) {
#pragma unroll
    for (int j = 0; j < J; ++j) o[z][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    ref[z] = limit[z] = kLow;
    l[z] = 0.0f;
    shift[z] = -200;
    peak[z] = -1000.0f;
  }

  auto compute = [&](const Stage<D> &st, int32_t j) __attribute__((always_inline)) {
    const int32_t t0 = tb + j * kStride4;
    const uint32_t here = (uint32_t)(there >> (2 * j)) & 3u;
    float ks[2], vs[2];
    int32_t ve[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      ks[x] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(k_scale), 2 * j + x));
      vs[x] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v_scale), 2 * j + x));
      ve[x] = vs[x] > 0.0f ? __builtin_amdgcn_frexp_expf(vs[x]) : -1000;  // v < 2^ve
    }
    float s[CT][2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float4v acc[CT];
#pragma unroll
      for (int z = 0; z < CT; ++z) acc[z] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const half8 w = codes8(st.k[x][e / 2][e % 2 * 2], st.k[x][e / 2][e % 2 * 2 + 1]);
#pragma unroll
        for (int z = 0; z < CT; ++z) acc[z] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, q[z][e], acc[z], 0, 0, 0);
      }
#pragma unroll
      for (int z = 0; z < CT; ++z) {
        const float f = row_scale[z] * ks[x];
#pragma unroll
        for (int u = 0; u < 4; ++u) s[z][x][u] = acc[z][u] * f;
      }
    }
    if (!(t0 >= all_lo && t0 >= from && t0 + kTokens <= all_hi && t0 + kTokens <= to && here == 3u)) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int32_t tok = t0 + kRun * x + 4 * c + u;
          const bool seen = tok < to && tok >= from && (here >> x & 1);
#pragma unroll
          for (int z = 0; z < CT; ++z)
            s[z][x][u] = seen && tok < row_hi[z] && tok >= row_lo[z] ? s[z][x][u] : -INFINITY;
        }
    }
    float top[CT], m[CT][2];
    bool over = false;
#pragma unroll
    for (int z = 0; z < CT; ++z) {
#pragma unroll
      for (int x = 0; x < 2; ++x) m[z][x] = fmaxf(fmaxf(s[z][x][0], s[z][x][1]), fmaxf(s[z][x][2], s[z][x][3]));
      top[z] = fmaxf(m[z][0], m[z][1]);
      over = over || top[z] > limit[z] ||
             fmaxf(m[z][0] - ref[z] + (float)ve[0], m[z][1] - ref[z] + (float)ve[1]) > (float)shift[z] + kTop;
    }
    if (__any(over)) {
#pragma unroll
      for (int z = 0; z < CT; ++z) {
        const float high = quarters_max(top[z]), next = high > limit[z] ? high : ref[z];
        const float back = ref[z] - next;  // kLow stands for no score so far
        peak[z] = fmaxf(peak[z] + back, quarters_max(fmaxf(m[z][0] - next + (float)ve[0], m[z][1] - next + (float)ve[1])));
        const int32_t to_shift = (int32_t)fminf(fmaxf(ceilf(peak[z]), -180.0f), 180.0f) - (int32_t)(kTop - kRoom);
        const float fl = __builtin_amdgcn_exp2f(back), fo = __builtin_amdgcn_exp2f(back + (float)(shift[z] - to_shift));
        ref[z] = next;
        limit[z] = next + kLazy;
        shift[z] = to_shift;
        l[z] *= fl;
#pragma unroll
        for (int jj = 0; jj < J; ++jj) o[z][jj] *= fo;
      }
    }
    uint4v ph[CT], pl[CT];
#pragma unroll
    for (int z = 0; z < CT; ++z)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float g = fminf(ldexpf(vs[x], -shift[z]), 0x1p120f);  // where it ends, weights are 0
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
          half2v hi, lo;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float w = __builtin_amdgcn_exp2f(s[z][x][u + e] - ref[z]);
            l[z] += w;
            const float p = w * g;
            hi[e] = (_Float16)p;
            lo[e] = (_Float16)(p - (float)hi[e]);
          }
          ph[z][2 * x + u / 2] = __builtin_bit_cast(uint32_t, hi);
          pl[z][2 * x + u / 2] = __builtin_bit_cast(uint32_t, lo);
        }
      }
#pragma unroll
    for (int jj = 0; jj < J; ++jj) {
      const half8 w = codes8(st.v[0][jj / 4][jj % 4], st.v[1][jj / 4][jj % 4]);
#pragma unroll
      for (int z = 0; z < CT; ++z) {
        o[z][jj] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, __builtin_bit_cast(half8, ph[z]), o[z][jj], 0, 0, 0);
        o[z][jj] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w, __builtin_bit_cast(half8, pl[z]), o[z][jj], 0, 0, 0);
      }
    }
  };

  while (tb < to) {
    for (int32_t j = 0;;) {
      if (j + 1 < steps) load(st1, j + 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(st0, j);
      if (++j == steps) break;
      if (j + 1 < steps) load(st0, j + 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(st1, j);
      if (++j == steps) break;
    }
    tb += kBatch * kStride4;
    if (tb < to) {
      fetch();
      load(st0, 0);
    }
  }

  // The waves' statistics and outputs of each row, joined.
#pragma unroll
  for (int z = 0; z < CT; ++z) {
    l[z] = quarters_sum(l[z]);
    if (c == 0) {
      s_m[wave][kCols * z + n] = ref[z];
      s_l[wave][kCols * z + n] = l[z];
    }
  }
  __syncthreads();
#pragma unroll
  for (int z = 0; z < CT; ++z) {
    float best = ref[z];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) best = fmaxf(best, s_m[w][kCols * z + n]);
    const float f = __builtin_amdgcn_exp2f(ref[z] - best);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float4v v;
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = ldexpf(o[z][j][u], shift[z]) * f;
      *reinterpret_cast<float4v *>(s_o + (wave * kAll + kCols * z + n) * kStride + 16 * j + 4 * c) = v;
    }
  }
  __syncthreads();
  const int64_t place = ((int64_t)(b * a.tiles + rt) * a.hkv + h) * a.splits + split;
  for (int e = threadIdx.x; e < t.rows * (D / 8); e += kThreads) {
    const int rr = e / (D / 8), ch = e % (D / 8) * 8;
    float top = kLow * 2.0f, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_m[w][rr]);
    float4v v0 = {0.0f, 0.0f, 0.0f, 0.0f}, v1 = v0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      sum = fmaf(s_l[w][rr], __builtin_amdgcn_exp2f(s_m[w][rr] - top), sum);
      const float *src = s_o + (w * kAll + rr) * kStride + ch;
      v0 += *reinterpret_cast<const float4v *>(src);
      v1 += *reinterpret_cast<const float4v *>(src + 4);
    }
    if (a.splits > 1) {
      float *dst = a.ws_o + (place * a.tile_rows + rr) * D + ch;
      *reinterpret_cast<float4v *>(dst) = v0;
      *reinterpret_cast<float4v *>(dst + 4) = v1;
      if (ch == 0) *reinterpret_cast<float2v *>(a.ws_ml + (place * a.tile_rows + rr) * 2) = float2v{top, sum};
    } else {
      const int32_t rg = t.row0 + rr, ii = t.q0 + rg / a.group, hh = h * a.group + rg % a.group;
      const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // NaN stays NaN
      uint4v w;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        w[u] = down<BF16>(v0[2 * u] * inv) | down<BF16>(v0[2 * u + 1] * inv) << 16;
        w[2 + u] = down<BF16>(v1[2 * u] * inv) | down<BF16>(v1[2 * u + 1] * inv) << 16;
      }
      *reinterpret_cast<uint4v *>(a.out + (int64_t)ii * a.ldo + (int64_t)hh * D + ch) = w;
      if (ch == 0 && a.lse) a.lse[(int64_t)ii * a.hq + hh] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
  }
}

// Many rows (prompts): a wave takes 32 rows over all tokens of the workgroup's chunk, and the
// workgroup's waves share the codes, made fp16 once and kept in LDS, 64 or 32 tokens at a time,
// keys in two stages, values, which are needed later, in three.  32 x 32 x 16 instructions: S^T leaves in lane (n, c), c = 0 or 1, row n's scores of the
// tokens 8 (i / 4) + 4 c + i % 4 of 32, so the eight of a run are the operand of one step of the
// second product, if the values lie in LDS in that order.  Rows of both stages' arrays are turned
// by 16-byte units so that 16 lanes read 16 different banks' worth.
template <int D>
struct Many {
  static constexpr int kWaves = D == 256 ? 4 : 8, kThreads = 64 * kWaves, kRows = 32 * kWaves;
  static constexpr int kStep = D == 256 ? 32 : 64, kRuns = kStep / kRun, kBatch = 64 / kRuns;
  static constexpr int U = D / 64, kBlocks = 2 * kRuns * U / kWaves;  // 1024-byte units of a step for each wave
  static constexpr int kStage = kStep * D * 2;                        // bytes of a step's keys, or values
  static constexpr bool kTurns = kWaves == 8;                         // two waves a SIMD, which take turns
  static constexpr int kKeyUnits = D / 8;                             // 16-byte units of a token's keys
  static __device__ __forceinline__ int key_turn(int token) { return D == 64 ? (token >> 1) & 7 : token & 15; }
  static constexpr int kValueUnits = 2 * kRuns;                       // of a channel's values
  static __device__ __forceinline__ int value_turn(int ch) { return kRuns == 4 ? (ch >> 1) & 7 : (ch >> 2) & 3; }
};

__device__ __forceinline__ float halves_max(float v) {
  const uint2v a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
}

typedef float float16v __attribute__((ext_vector_type(16)));

template <int D, bool BF16>
__global__ __launch_bounds__(Many<D>::kThreads, Many<D>::kWaves / 4) void kv8_many_kernel(Args8 a) {
  using M = Many<D>;
  constexpr int U = M::U, E = D / 16, J = D / 32, R = M::kRuns;
  constexpr int kParts = BF16 ? 1 : 2;
  __shared__ __attribute__((aligned(16))) uint8_t all_keys[2 * M::kStage], all_values[3 * M::kStage];

  const int lane = threadIdx.x & 63, n = lane & 31, c = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t h = blockIdx.x / a.splits, split = blockIdx.x - h * a.splits;
  int32_t b = blockIdx.z, rt = a.tiles - 1 - (int32_t)blockIdx.y;
  if (a.units && !find_tile<M::kRows>(a, (int64_t)blockIdx.z * gridDim.y + blockIdx.y, b, rt)) return;
  const Tile t = tile_of(a, b, h, rt);
  if (t.rows <= 0) return;
  const int32_t chunk = chunk_of(a, t), nchunks = chunks_of(t, chunk);
  if (split >= nchunks && !(split == 0 && a.splits == 1)) return;
  const int32_t begin = base_of(t) + split * chunk;
  const int32_t from = begin > t.lo ? begin : t.lo;
  const int32_t to = t.hi - begin > chunk ? begin + chunk : t.hi;
  const int32_t start = from & ~(kRun - 1), steps = to > start ? (to - start + M::kStep - 1) / M::kStep : 0;

  const int32_t P = 1 << a.page_log2, block = mixllm::kv8_block_bytes(P, D);
  const int32_t *table = a.table + b * a.ldt;

  // Pages and scales of kBatch steps at a time, a run a lane.  A value's scale is 2^(ve + lv), its inverse
  // iv 2^-ve; values of nothing but zeros have ve = kNone and count as with a scale of 1.
  constexpr int32_t kNone = -1000;
  // Exponents of a scale below the row's are taken as this one: weights (up to 2^kLazy) times scales
  // are 0 in fp16 from here on anyway, and their sum stays where the factor taken back from it is finite.
  constexpr int32_t kLeast = -32;
  struct Batch {
    int32_t pages, ve;
    float ks, lv, iv;
    uint64_t there;
  } now = {-1, kNone, 0.0f, 0.0f, 1.0f, 0}, next = now;
  auto fetch = [&](int32_t j) {
    const int32_t tok = start + j * M::kStep + lane * kRun;
    next.pages = tok < to ? table[tok >> a.page_log2] : -1;
    next.pages = (uint32_t)next.pages < (uint32_t)a.pages ? next.pages : -1;
    next.there = __ballot(next.pages >= 0);
    float2v sc = {0.0f, 0.0f};
    if (next.pages >= 0)
      sc = *reinterpret_cast<const float2v *>(a.cache + ((int64_t)next.pages * a.hkv + h) * block +
                                              mixllm::kv8_scale_offset(P, D) + (tok & (P - 1)) / kRun * 8);
    const bool some = sc.y > 0.0f;
    const float mant = some ? __builtin_amdgcn_frexp_mantf(sc.y) : 1.0f;  // [1/2, 1)
    next.ks = sc.x;
    next.ve = some ? __builtin_amdgcn_frexp_expf(sc.y) : kNone;
    next.lv = log2f(mant), next.iv = 1.0f / mant;
  };
  // This wave's units of a step: wave, wave + kWaves, .. of its keys, then of its values; with 64
  // channels one of either.
  auto part_of = [&](int i) { return M::kBlocks > 1 ? i / (M::kBlocks / 2) : wave / (R * U); };
  auto unit_of = [&](int i) { return M::kBlocks > 1 ? wave + i % (M::kBlocks / 2) * M::kWaves : wave % (R * U); };
  uint4v raw[M::kBlocks];
  auto load = [&](int32_t j) __attribute__((always_inline)) {
    if (j % M::kBatch == 0) fetch(j);
#pragma unroll
    for (int i = 0; i < M::kBlocks; ++i) {
      const int part = part_of(i), r = unit_of(i) / U, u = unit_of(i) % U;
      const int32_t pg = __builtin_amdgcn_readlane(next.pages, j % M::kBatch * R + r);
      const int32_t in = (start + j * M::kStep + kRun * r) & (P - 1);
      // an absent run reads any memory of the cache; its scores are masked
      raw[i] = *reinterpret_cast<const uint4v *>(a.cache + ((int64_t)(pg < 0 ? 0 : pg) * a.hkv + h) * block +
                                                 (int64_t)part * P * D + (int64_t)in * D + u * 1024 + lane * 16);
    }
  };
  auto store = [&](int32_t j) __attribute__((always_inline)) {
    uint8_t *keys = all_keys + (j & 1) * M::kStage, *values = all_values + j % 3 * M::kStage;
    const int m = lane & 15, q = lane >> 4;
#pragma unroll
    for (int i = 0; i < M::kBlocks; ++i) {
      const int part = part_of(i), r = unit_of(i) / U, u = unit_of(i) % U;
      const half8 lo = codes8(raw[i].x, raw[i].y), hi = codes8(raw[i].z, raw[i].w);
      if (part == 0) {  // 16 channels of token m
        const int token = kRun * r + m, unit = 8 * u + 2 * q, turn = M::key_turn(token);
        *reinterpret_cast<half8 *>(keys + (token * M::kKeyUnits + (unit ^ turn)) * 16) = lo;
        *reinterpret_cast<half8 *>(keys + (token * M::kKeyUnits + ((unit + 1) ^ turn)) * 16) = hi;
      } else {  // tokens 4q .. 4q+3 of the channels 16 j + m
        const uint4v l4 = __builtin_bit_cast(uint4v, lo), h4 = __builtin_bit_cast(uint4v, hi);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int ch = 64 * u + 16 * jj + m;
          const uint2v w = jj == 0 ? uint2v{l4.x, l4.y} : jj == 1 ? uint2v{l4.z, l4.w} : jj == 2 ? uint2v{h4.x, h4.y} : uint2v{h4.z, h4.w};
          *reinterpret_cast<uint2v *>(values + (ch * M::kValueUnits + ((2 * r + (q & 1)) ^ M::value_turn(ch))) * 16 + (q >> 1) * 8) = w;
        }
      }
    }
  };
  // Group 1 of the waves is half a step behind group 0 (see below) and stores a step further ahead.
  const int late = M::kTurns && wave >= M::kWaves / 2 ? 1 : 0;
  if (steps > 0) load(0);

  // The wave's query rows, as operands: step e has the channels 16 e + 8 c on.
  const int32_t first = wave * 32, live = t.rows - first;  // rows of this wave, if positive
  half8 q[E];
  float row_scale;
  int32_t row_hi, row_lo;
  {
    const int32_t r = t.row0 + (first + n < t.rows ? first + n : t.rows - 1);
    const int32_t i = r / a.group, head = h * a.group + r % a.group;
    const uint16_t *qp = a.q + (int64_t)(t.q0 + i) * a.ldq + (int64_t)head * D + 8 * c;
    uint4v w[E];
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = *reinterpret_cast<const uint4v *>(qp + 16 * e);
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int d = 0; d < 4; ++d)
        top = fmaxf(top, fmaxf(fabsf(up<BF16>(w[e][d] & 0xFFFFu)), fabsf(up<BF16>(w[e][d] >> 16))));
    top = halves_max(top);
    int p = top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : 0;
    p = p < -100 ? -100 : p;
    const float mul = ldexpf(a.scale < 0.0f ? -1.0f : 1.0f, 14 - p);  // a score's factor is not negative
    row_scale = ldexpf(fabsf(a.scale) * kLog2e, p - 14);
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        q[e][2 * d] = (_Float16)(up<BF16>(w[e][d] & 0xFFFFu) * mul);
        q[e][2 * d + 1] = (_Float16)(up<BF16>(w[e][d] >> 16) * mul);
      }
    const int32_t pos = t.pos0 + i;
    row_hi = pos + 1;
    row_lo = a.window ? pos - a.window + 1 : 0;
  }
  // tokens that some row, and that every row of this wave sees
  const int32_t pos_first = t.pos0 + (t.row0 + first) / a.group;
  const int32_t pos_last = t.pos0 + (t.row0 + (live < 32 ? t.rows : first + 32) - 1) / a.group;
  const int32_t any_lo = a.window ? pos_first - a.window + 1 : 0, any_hi = pos_last + 1;
  const int32_t all_lo = a.window ? pos_last - a.window + 1 : 0, all_hi = pos_first + 1;

  float16v o[J];
  float ref = kLow, l = 0.0f, limit = kLow, peak = -1000.0f;
  int32_t shift = -200;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;

  float16v s[R / 2];
  half8 p[kParts][R];
  auto seen = [&](int32_t j) {  // by a row of this wave
    const int32_t t0 = start + j * M::kStep;
    return live > 0 && t0 < any_hi && t0 + M::kStep > any_lo;
  };
  // The order of `reads` operands' reads and `each` products with every one: reads run kAhead ahead.
  auto reads_ahead = [&](auto reads, auto each) __attribute__((always_inline)) {
    constexpr int kReads = decltype(reads)::value, kEach = decltype(each)::value, kAhead = 6;
    __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
      if (i + kAhead < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
  };
  auto multiply = [&](int32_t j) __attribute__((always_inline)) {  // the last step's values, this one's keys
    if (j > 0 && seen(j - 1)) {
      const uint8_t *values = all_values + (j - 1) % 3 * M::kStage;
#pragma unroll
      for (int jj = 0; jj < J; ++jj) {
        const int ch = 32 * jj + n, turn = M::value_turn(ch);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const half8 w = *reinterpret_cast<const half8 *>(values + (ch * M::kValueUnits + ((2 * r + c) ^ turn)) * 16);
#pragma unroll
          for (int k = 0; k < kParts; ++k) o[jj] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w, p[k][r], o[jj], 0, 0, 0);
        }
      }
      reads_ahead(Const<J * R>(), Const<kParts>());
    }
    if (j < steps && seen(j)) {
      const uint8_t *keys = all_keys + (j & 1) * M::kStage;
#pragma unroll
      for (int x = 0; x < R / 2; ++x)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[x][i] = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int x = 0; x < R / 2; ++x) {
          const int token = 32 * x + n, turn = M::key_turn(token);
          const half8 w = *reinterpret_cast<const half8 *>(keys + (token * M::kKeyUnits + ((2 * e + c) ^ turn)) * 16);
          s[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w, q[e], s[x], 0, 0, 0);
        }
      reads_ahead(Const<R / 2 * E>(), Const<1>());
    }
  };
  auto weigh = [&](int32_t j) __attribute__((always_inline)) {
    if (!seen(j)) return;
    const int32_t t0 = start + j * M::kStep;
    const uint32_t here = (uint32_t)(now.there >> (j % M::kBatch * R)) & ((1u << R) - 1);
    auto of_run = [&](float v, int r) {
      return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), j % M::kBatch * R + r));
    };
    float f[R];
    int32_t ve[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f[r] = row_scale * of_run(now.ks, r);
      ve[r] = __builtin_amdgcn_readlane(now.ve, j % M::kBatch * R + r);  // v < 2^ve
    }
    if (!(t0 >= all_lo && t0 >= from && t0 + M::kStep <= all_hi && t0 + M::kStep <= to && here == (1u << R) - 1)) {
      const int32_t lo = row_lo > from ? row_lo : from, hi = row_hi < to ? row_hi : to;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t tok = t0 + kRun * r + i / 4 * 8 + 4 * c + i % 4;
          // the factor is applied here, so that none of 0 meets the infinity
          const float x = s[r / 2][8 * (r % 2) + i] * f[r];
          s[r / 2][8 * (r % 2) + i] = tok >= lo && tok < hi && (here >> r & 1) ? x : -INFINITY;
        }
        f[r] = 1.0f;
      }
    }
    float m[R], top = -INFINITY, big = -INFINITY;  // of s f: the factors are not negative
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = s[r / 2][8 * (r % 2)];
#pragma unroll
      for (int i = 1; i < 8; ++i) m[r] = fmaxf(m[r], s[r / 2][8 * (r % 2) + i]);
      m[r] *= f[r];
      top = fmaxf(top, m[r]);
      big = fmaxf(big, m[r] - ref + (float)ve[r]);
    }
    if (__any(top > limit || big > (float)shift + kTop)) {
      const float high = halves_max(top), up_to = high > limit ? high : ref;
      const float back = ref - up_to;  // kLow stands for no score so far
      big = -INFINITY;
#pragma unroll
      for (int r = 0; r < R; ++r) big = fmaxf(big, m[r] - up_to + (float)ve[r]);
      peak = fmaxf(peak + back, halves_max(big));
      const int32_t to_shift = (int32_t)fminf(fmaxf(ceilf(peak), -180.0f), 180.0f) - (int32_t)(kTop - kRoom);
      const float fl = __builtin_amdgcn_exp2f(back), fo = __builtin_amdgcn_exp2f(back + (float)(shift - to_shift));
      ref = up_to;
      limit = up_to + kLazy;
      shift = to_shift;
      l *= fl;
#pragma unroll
      for (int jj = 0; jj < J; ++jj) o[jj] *= fo;
    }
    // A weight times a value's scale 2^-shift in one exponential; their sum less that factor is the
    // weights'.
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int32_t below = ve[r] - shift, d = ve[r] == kNone ? 0 : below > kLeast ? below : kLeast;
      const float add = (of_run(now.lv, r) + (float)d) - ref;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = __builtin_amdgcn_exp2f(fmaf(s[r / 2][8 * (r % 2) + i], f[r], add));
        sum += w;
        p[0][r][i] = (_Float16)w;
        if (kParts == 2) p[kParts - 1][r][i] = (_Float16)(w - (float)p[0][r][i]);
      }
      l = fmaf(sum, ldexpf(of_run(now.iv, r), -d), l);
    }
  };
  // Until the workgroup's waves are here; what they wrote to LDS before is seen after.
  auto meet = [&]() __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));  // lgkmcnt(0); loads from memory stay in flight
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // A step is two phases: the products, then the weights with the next codes' way to LDS.  Two waves
  // share a SIMD, and left alone both multiply and then both weigh: so one of them (`late`) is a
  // phase behind the other, and one multiplies while the other weighs.  In phase 2 j group 0
  // multiplies step j and group 1 weighs step j - 1, in phase 2 j + 1 the other way about; step j's
  // codes are stored in phases 2 j - 1 (group 0) and 2 j - 2 (group 1), its keys are read in 2 j and
  // 2 j + 1, its values in 2 j + 2 and 2 j + 3, so two and three stages do.
  if (steps > 0) store(0);
  if (steps > 1) load(1);
  meet();
  if (late) {
    if (steps > 1) store(1);
    if (steps > 2) load(2);
    meet();
  }
  for (int32_t j = 0; j < steps; ++j) {
    if (j % M::kBatch == 0) now = next;
    if (j > 0 && j + 1 + late < steps) load(j + 1 + late);
    multiply(j);
    if (M::kTurns) meet();
    weigh(j);
    if (j + 1 + late < steps) store(j + 1 + late);
    meet();
  }
  multiply(steps);
  if (M::kTurns && !late) meet();

  if (n >= live) return;
  const float sum = [&] {
    const uint2v v = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    return __uint_as_float(v.x) + __uint_as_float(v.y);
  }();
  const int32_t rr = first + n;
  if (a.splits > 1) {
    const int64_t place = ((int64_t)(b * a.tiles + rt) * a.hkv + h) * a.splits + split;
    float *dst = a.ws_o + (place * a.tile_rows + rr) * D;
#pragma unroll
    for (int jj = 0; jj < J; ++jj)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float4v v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ldexpf(o[jj][4 * g + i], shift);
        *reinterpret_cast<float4v *>(dst + 32 * jj + 8 * g + 4 * c) = v;
      }
    if (c == 0) *reinterpret_cast<float2v *>(a.ws_ml + (place * a.tile_rows + rr) * 2) = float2v{ref, sum};
    return;
  }
  const int32_t rg = t.row0 + rr, ii = t.q0 + rg / a.group, hh = h * a.group + rg % a.group;
  const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // NaN stays NaN
  uint16_t *dst = a.out + (int64_t)ii * a.ldo + (int64_t)hh * D;
#pragma unroll
  for (int jj = 0; jj < J; ++jj)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = down<BF16>(ldexpf(o[jj][4 * g + i], shift) * inv);
      *reinterpret_cast<uint2v *>(dst + 32 * jj + 8 * g + 4 * c) = uint2v{v[0] | v[1] << 16, v[2] | v[3] << 16};
    }
  if (c == 0 && a.lse) a.lse[(int64_t)ii * a.hq + hh] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * kLn2;
}

// How the work of a call is cut.  Rows: tiles of 16 or 32 (row, head) pairs of one key/value
// head, or of 256 (128 with 256 channels) where there are kMany or more: 8 requests over 4001 tokens, 32/8
// heads of 128, take 34.8 us with 64 pairs each in tiles of 32 and 39.0 in one large, 44.4 with 128
// in one large and 52.8 in four of 32.  Tokens: equal chunks of each tile.  CUs hold 2 or more
// small workgroups, so about kTarget of them run at the longest length (32 requests of 4001
// tokens 50.3 us with 512, 52.2 with 768, 55.0 with 1024); a CU holds one large one, so as many
// chunks as do not need a second round of kCus (2 x 700 rows of 256 channels 141 us in two
// chunks for each of 176 tiles, whose second round and join take what the idle CUs would save, 139.5
// in one).
constexpr int64_t kTarget = 512, kCus = 256, kMany = 128;

Cut cut_of(int32_t B, int32_t hq, int32_t hkv, int32_t dim, int32_t max_rows, int32_t max_len, int32_t window) {
  Cut k;
  const int64_t rows = (int64_t)max_rows * (hq / hkv);
  k.tile_rows = rows >= kMany ? (dim == 256 ? 128 : 256) : rows <= 16 || dim == 256 ? 16 : 32;
  k.tiles = (int32_t)((rows + k.tile_rows - 1) / k.tile_rows);
  int64_t span = max_len;
  // a tile's rows are at most tile_rows positions, its first chunk starts at a whole run
  if (window && (int64_t)window + k.tile_rows + kRun < span) span = (int64_t)window + k.tile_rows + kRun;
  const int64_t groups = (int64_t)B * hkv * k.tiles;
  const int64_t most = (span + kMinChunk - 1) / kMinChunk;
  const int64_t want = rows >= kMany ? kCus / groups : (kTarget + groups - 1) / groups;
  k.splits = (int32_t)(most < 1 || want <= 1 ? 1 : want < most ? want : most);
  return k;
}

// A call whose largest request has kMany pairs or more may hold requests with few rows too (prompts
// and decodes of one step).  Those up to few_pairs are left to a launch of their own with tiles
// and chunks like a call of decodes, where the batch fills the CUs without them (below it they
// find idle ones) and is uneven enough to pay for two more launches.  No tiles: there is none.  In a
// smaller batch a long decode beside a prompt is walked by one workgroup a head: 15 over 32768 tokens
// take 183 us, a prompt of 1000 rows 84, both in one call 1016.
int32_t few_pairs(int32_t group, int32_t dim) { return (dim == 256 ? 16 : 32) / group * group; }

Cut few_of(int32_t T, int32_t B, int32_t hq, int32_t hkv, int32_t dim, int32_t max_rows, int32_t max_len,
           int32_t window) {
  const int32_t group = hq / hkv, few = few_pairs(group, dim);
  if ((int64_t)max_rows * group < kMany || !few || (int64_t)B * hkv < kCus || 2 * (int64_t)T >= (int64_t)B * max_rows)
    return {0, 0, 1};
  return cut_of(B, hq, hkv, dim, few / group, max_len, window);
}

int64_t parts_of(const Cut &k, int32_t B, int32_t hkv) { return (int64_t)B * k.tiles * hkv * k.splits; }
size_t bytes_of(const Cut &k, int32_t B, int32_t hkv, int32_t dim) {
  return k.splits == 1 ? 0 : (size_t)parts_of(k, B, hkv) * k.tile_rows * (dim + 2) * sizeof(float);
}

template <int D, bool BF16>
void launch_cut(Args8 a, const Cut &k, hipStream_t s) {
  a.tiles = k.tiles, a.tile_rows = k.tile_rows, a.splits = k.splits;
  a.ws_ml = a.ws_o ? a.ws_o + parts_of(k, a.B, a.hkv) * k.tile_rows * D : nullptr;
  dim3 grid((unsigned)(a.splits * a.hkv), (unsigned)a.tiles, (unsigned)a.B), threads(kThreads);
  if (a.tile_rows > 32) {
    // Tiles by the rows of the call where that is fewer (20 requests of 1000 rows among 980 of one row over
    // 2000 tokens: 1150 us; with tiles for each request and without `few` 8636; one of 2000 rows among
    // 31: 152 and 572; two prompts of nearly equal rows 185 either way).
    const int64_t units = (int64_t)a.T * a.group / a.tile_rows + a.B;
    if (units < (int64_t)a.B * a.tiles) {
      a.units = (int32_t)units;
      grid.y = units < 32768 ? (unsigned)units : 32768u;
      grid.z = (unsigned)((units + grid.y - 1) / grid.y);
    }
    hipLaunchKernelGGL((kv8_many_kernel<D, BF16>), grid, dim3(Many<D>::kThreads), 0, s, a);
  } else if (a.tile_rows == 16 && a.tiles == 1) {
    hipLaunchKernelGGL((kv8_attention_kernel<D, 1, true, BF16>), grid, threads, 0, s, a);
  } else if constexpr (D == 256) {  // tiles of 16 rows only
    hipLaunchKernelGGL((kv8_attention_kernel<D, 1, false, BF16>), grid, threads, 0, s, a);
  } else if (a.tiles == 1) {
    hipLaunchKernelGGL((kv8_attention_kernel<D, 2, true, BF16>), grid, threads, 0, s, a);
  } else {
    hipLaunchKernelGGL((kv8_attention_kernel<D, 2, false, BF16>), grid, threads, 0, s, a);
  }
  if (a.splits == 1 || hipPeekAtLastError() != hipSuccess) return;
  launch_join<D, BF16>(a, s);
}

template <int D, bool BF16>
void launch(Args8 a, const Cut &k, const Cut &few, hipStream_t s) {
  const int32_t pairs = few.tiles ? few_pairs(a.group, D) : 0;
  a.least = pairs + 1;
  launch_cut<D, BF16>(a, k, s);
  if (!pairs || hipPeekAtLastError() != hipSuccess) return;
  a.least = 1, a.most = pairs, a.max_rows = pairs / a.group + 1;  // a row more tells the larger requests
  launch_cut<D, BF16>(a, few, s);
}

template <int D>
void launch(const Args8 &a, const Cut &k, const Cut &few, int32_t dtype, hipStream_t s) {
  if (dtype == MIXLLM_BF16) launch<D, true>(a, k, few, s);
  else launch<D, false>(a, k, few, s);
}

}  // namespace

extern "C" size_t mixllm_kv8_attention_workspace_bytes(int32_t T, int32_t B, int32_t q_heads, int32_t kv_heads,
                                                       int32_t dim, int32_t max_rows, int32_t max_len,
                                                       int32_t window) {
  if (!shape_ok(T, B, q_heads, kv_heads, dim, max_rows, max_len, window) || T == 0 || B == 0 || max_rows == 0) return 0;
  const Cut k = cut_of(B, q_heads, kv_heads, dim, max_rows, max_len, window);
  // enough for calls of fewer rows too, whose batch may be uneven where this one is not
  const Cut few = few_of(1, B, q_heads, kv_heads, dim, max_rows, max_len, window);
  const size_t large = bytes_of(k, B, kv_heads, dim), small = bytes_of(few, B, kv_heads, dim);  // one after the other
  return large > small ? large : small;
}

extern "C" int mixllm_kv8_attention(const void *q, int64_t ldq, int32_t dtype, int32_t T, int32_t q_heads,
                                    const void *cache, size_t cache_bytes, int32_t pages, int32_t page,
                                    int32_t kv_heads, int32_t dim, const int32_t *table, int64_t ldt, int32_t width,
                                    const int32_t *lens, const int32_t *cu, int32_t B, int32_t max_rows,
                                    int32_t max_len, float scale, int32_t window, void *out, int64_t ldo, float *lse,
                                    void *workspace, size_t workspace_bytes, void *stream) {
  if (!shape_ok(T, B, q_heads, kv_heads, dim, max_rows, max_len, window) ||
      (dtype != MIXLLM_FP16 && dtype != MIXLLM_BF16))
    return MIXLLM_E_SHAPE;
  if (T == 0 || B == 0 || max_rows == 0) return MIXLLM_OK;
  const int st = mixllm::kv8_check_cache(cache, cache_bytes, pages, page, kv_heads, dim);
  if (st != MIXLLM_OK) return st;
  const int bad = check_call(q, ldq, q_heads, dim, table, ldt, width, lens, cu, out, ldo, lse, workspace);
  if (bad != MIXLLM_OK) return bad;
  const Cut k = cut_of(B, q_heads, kv_heads, dim, max_rows, max_len, window);
  const Cut few = few_of(T, B, q_heads, kv_heads, dim, max_rows, max_len, window);
  if (parts_of(k, B, kv_heads) > 0x7FFFFFFF || parts_of(few, B, kv_heads) > 0x7FFFFFFF || B > 65535 ||
      k.tiles > 65535 || (int64_t)B * max_rows * q_heads > 0x7FFFFFFF)
    return MIXLLM_E_SHAPE;
  const size_t large = bytes_of(k, B, kv_heads, dim), small = bytes_of(few, B, kv_heads, dim);
  if (workspace_bytes < large || workspace_bytes < small) return MIXLLM_E_SPACE;
  if ((large || small) && !workspace) return MIXLLM_E_NULL;
  Args8 a;
  static_cast<Args &>(a) = {static_cast<const uint16_t *>(q), static_cast<const uint8_t *>(cache), table, lens, cu,
                            static_cast<uint16_t *>(out), lse, static_cast<float *>(workspace), nullptr,
                            ldq, ldo, ldt, scale, T, q_heads, kv_heads, q_heads / kv_heads, pages,
                            mixllm::log2_of(page), width, B, max_rows, max_len, window, 0, 0, 1};
  a.least = 0, a.most = INT32_MAX, a.units = 0;
  if (dim == 64) launch<64>(a, k, few, dtype, (hipStream_t)stream);
  else if (dim == 128) launch<128>(a, k, few, dtype, (hipStream_t)stream);
  else launch<256>(a, k, few, dtype, (hipStream_t)stream);
  return mixllm::launch_status();
}
