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
// Codes become fp16 without arithmetic: a nibble masked where it sits in a half is a subnormal
// fp16, c 2^-24 times the power of two of its place, which goes into the row's factor.  The
// matrix instruction takes subnormals, but lines its 32 products up by the exponent of the
// normal range that a subnormal does not reach and cuts what lies more than about 24 bits
// below: measured, products with c 2^-24 lose 2^-15 of the code beside the largest weight.
// All are cut downwards, and scores and outputs are small differences of large sums, so codes
// at bit 0 showed (60000 tokens: fp16 outputs 1.7 times the error of their rounding, lse
// 1.5e-5 off).  So keys move to bit 4 (7 operations for 8 codes instead of 5) and values to
// bits 2 and 6 (6 operations): 1.02 times and 1.8e-6, for 1 to 3% of the time.
//
// The query is scaled by a power of two per row so that it fits fp16 (bf16 inputs lose
// nothing but values 2^-38 below the row's largest); the probability times the value's
// scale is rounded to fp16 (relative 2^-11), scaled by a power of two that follows the
// largest value scale seen so that it stays clear of fp16's subnormals, and for fp16 outputs
// and few rows what that rounding leaves is a second operand.  Statistics, sums and outputs
// are fp32.
//
// What bounds it, at 128 channels: the cache's bytes for decodes (128 requests of up to 8192 tokens,
// 946 MB: 189 us, 5.01 TB/s; the copies alone, nothing computed, 170 us); latency, the join and
// the last workgroups where there is less (32 requests, 127 MB: 36 us, 21.7 at the copy's
// rate); for prompts (2 x 1024 rows: 273 us, 400 TFLOP/s) the registers and the 66 KB of LDS that
// the join of the waves takes, which leave 2 waves per SIMD to hide the making of operands and
// the softmax between the matrix instructions.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm_attend.h"
#include "mixllm_kv4.h"
#include "mixllm_lanes.h"

namespace {

__device__ __forceinline__ uint32_t quarters_max(uint32_t v) {
  uint2v a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = a.x > a.y ? a.x : a.y;
  a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return __builtin_amdgcn_readfirstlane(a.x > a.y ? a.x : a.y);
}

// m - k rounded, or the next value above it where that is more than `most` below m: from
// |m| = 2^23 on fp32's steps are 1 or more, and a power k rounded up by them would take a weight
// times a value's scale past fp16.
__device__ __forceinline__ float less(float m, float k, float most) {
  const float x = m - k;
  return m - x > most ? __uint_as_float(__float_as_uint(x) + (x > 0.0f ? 1 : -1)) : x;
}

// 8 codes of a dword as fp16 operands c 2^-20, in the nibble order 0 4 1 5 2 6 3 7.
constexpr int kKeyBits = 20;
__device__ __forceinline__ half8 codes8(uint32_t w) {
  constexpr uint32_t mask = 0x00F000F0u;
  const uint4v r = {w << 4 & mask, w & mask, w >> 4 & mask, w >> 8 & mask};
  return __builtin_bit_cast(half8, r);
}

// Nibble `nib` of both halves: c 2^-22, or c 2^-18 for odd ones.
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w, int nib) {
  return (nib >= 2 ? w >> 6 : w << 2) & (nib & 1 ? 0x03C003C0u : 0x003C003Cu);
}
constexpr float kEvenUnit = 0x1p-22f, kOddUnit = 0x1p-18f;

typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __attribute__((address_space(3))) void *LdsPtr;
constexpr int kRsrcFlags = 0x00020000;  // raw buffer, 32-bit data format

// Waits until at most N vector-memory operations of this wave are outstanding (vmcnt low
// bits [3:0], high bits [15:14]; the other counts do not wait).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }  // lgkmcnt(0)

// A number as a type: stages are named at compile time, or the compiler takes every read of a
// stage for one of the copies in flight and waits for them all.  With both in one array it
// still does so in every second step; an array per stage takes that wait out too and measures
// 1 to 2% slower (128 decodes of up to 8192 tokens 189.5 us for 188.0), so it stays.
template <int N>
struct Const {
  static constexpr int value = N;
};

// How many query rows a tile has and what follows from it.  16 rows fill the operands'
// columns.  Where a request and head has 8 or 4 at most (a decode step has q_heads / kv_heads),
// a tile has 16 / V rows, V = 2 or 4, and column n stands for row n % (16 / V) over the runs x
// of tokens with x % V = n / (16 / V): the V columns of a row keep statistics and sums of their
// own, like workgroups that split the tokens, and are joined at the end.  The operands are
// zero where a column and a run do not belong together, so the products cost what they cost
// for 16 rows, but the scores, exponentials and parameters, most of the vector operations,
// are 4 per lane for V runs and not for each.  With more than 16 rows a tile has 32, CT = 2
// column blocks that share each operand made of codes (prompts of 2 x 1024 rows: 4% less time
// than with 16).
template <int D, int V>
struct Shape {
  static constexpr int kRows = kCols / V;
  static constexpr int kRuns = V == 1 || D == 256 ? 2 : 4;  // runs of a step
  static constexpr int kSets = kRuns / V;         // scores of a lane and step, in fours
  static constexpr int kTokens = kRuns * kRun;
  // The wave's ring in LDS: a stage is one step; of each run the key codes, the value codes
  // and the parameters of keys then values, copied from memory without passing registers
  // (one instruction moves kSize bytes per lane to consecutive places).  One stage is in
  // flight while one is used.
  static constexpr int kSize = D == 64 ? 4 : 16;           // bytes per lane and instruction of codes
  static constexpr int kCodes = 8 * D / (64 * kSize);      // instructions per run: key or value codes
  static constexpr int kPars = D == 256 ? 2 : 1;           // and parameters, 4 bytes per lane
  static constexpr int kBytes = 16 * D + 256 * kPars;      // bytes of a run
  static constexpr int kStage = kRuns * kBytes;
  static constexpr int kLoads = kRuns * (2 * kCodes + kPars);  // instructions of a stage
};

template <int D, int V, int CT, bool BF16>
__global__ __launch_bounds__(kThreads, 2) void kv4_attention_kernel(Args a) {
  static_assert(CT == 1 || V == 1, "more than one column block only where rows fill them");
  using S = Shape<D, V>;
  constexpr int G = D / 64, W = D / 32, J = D / 16;
  constexpr int kStride = D + 4;  // floats of a column of partial outputs in LDS
  constexpr int kAll = CT * kCols;  // columns of a wave
  constexpr int kRing = 2 * S::kStage, kPartial = kAll * kStride * 4;
  // the rings and, after the loop, the waves' partial outputs
  __shared__ __attribute__((aligned(16))) uint8_t smem[kWaves * (kRing > kPartial ? kRing : kPartial)];
  __shared__ float s_m[kWaves][kAll], s_l[kWaves][kAll];

  const int lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4, part = n / S::kRows;
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

  // The query row of this lane, as operands (zero outside the column's part) and as sums per
  // group of channels.
  int32_t i[CT];  // the row's place in its request
  uint4v raw[CT][W];
#pragma unroll
  for (int z = 0; z < CT; ++z) {
    const int32_t row = kCols * z + n % S::kRows, r = t.row0 + (row < t.rows ? row : t.rows - 1);
    i[z] = r / a.group;
    const int32_t head = h * a.group + r % a.group;
    const uint16_t *qp = a.q + (int64_t)(t.q0 + i[z]) * a.ldq + (int64_t)head * D + 8 * c;
#pragma unroll
    for (int s = 0; s < W; ++s) raw[z][s] = *reinterpret_cast<const uint4v *>(qp + 32 * s);
  }

  const int32_t P = 1 << a.page_log2;
  const int32_t block = mixllm::kv4_block_bytes(P, D);
  const int32_t *table = a.table + b * a.ldt;
  // Where this lane's part of a run is in a block, before the run's own offset.
  const int32_t koff = n * (D / 2) + c * (D / 8), voff = P * (D / 2) + (c * 16 + n) * (D / 8);
  const int32_t pword = lane & (32 * G - 1);  // dword of the run's parameters (D = 256: and the one 64 on)
  const int32_t poff = P * D + pword / (16 * G) * (P * (D / 16)) + pword % (16 * G) * 4;
  const int32_t poff2 = P * D + P * (D / 16) + pword % (16 * G) * 4;  // D = 256: the values' half
  uint8_t *ring = smem + wave * kRing;

  // Copies run x of the step at t0 into a stage; pg: its page, negative for none (then any
  // memory of the cache is copied, to keep the number of instructions).
  auto issue = [&](auto stage, int x, int32_t t0, int32_t pg) {
    uint8_t *to_k = ring + decltype(stage)::value * S::kStage + x * S::kBytes, *to_v = to_k + 8 * D, *to_p = to_v + 8 * D;
    pg = pg < 0 ? 0 : pg;
    const Rsrc rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(a.cache) + ((int64_t)pg * a.hkv + h) * block, (short)0, block, kRsrcFlags);
    const int32_t in = (t0 + kRun * x) & (P - 1), at = in * (D / 2);
#pragma unroll
    for (int e = 0; e < S::kCodes; ++e) {
      if constexpr (D == 64) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)(to_k + e * 256), 4, koff + 4 * e, at, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)(to_v + e * 256), 4, voff + 4 * e, at, 0, 0);
      } else {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)(to_k + e * 1024), 16, koff + 16 * e, at, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)(to_v + e * 1024), 16, voff + 16 * e, at, 0, 0);
      }
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)to_p, 4, poff, in * (4 * G), 0, 0);
    if constexpr (S::kPars == 2)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)(to_p + 256), 4, poff2, in * (4 * G), 0, 0);
  };
  // This wave takes every fourth step, in batches whose pages one load fetches: lane
  // kRuns * j + x has the page of run x of the batch's step j, negative for none.  The first
  // batch's loads start before the query is looked at.
  constexpr int32_t kStride4 = kWaves * S::kTokens, kBatch = 64 / S::kRuns;
  int32_t tb = (from & ~(kRun - 1)) + wave * S::kTokens, steps = 0, pages = -1;
  uint64_t there = 0;
  auto start = [&](auto stage, int32_t j) {
#pragma unroll
    for (int x = 0; x < S::kRuns; ++x)
      issue(stage, x, tb + j * kStride4, __builtin_amdgcn_readlane(pages, S::kRuns * j + x));
  };
  auto fetch = [&]() {  // for the batch at tb < to
    const int32_t tok = tb + lane / S::kRuns * kStride4 + lane % S::kRuns * kRun;
    pages = tok < to ? table[tok >> a.page_log2] : -1;
    pages = (uint32_t)pages < (uint32_t)a.pages ? pages : -1;
    there = __ballot(pages >= 0);
    const int32_t left = (to - tb + kStride4 - 1) / kStride4;
    steps = left < kBatch ? left : kBatch;
    start(Const<0>(), 0);
  };
  if (tb < to) fetch();

  half8 q[CT][V][W];
  float row_scale[CT], qsum[CT][G];
  int32_t row_hi[CT], row_lo[CT];  // the row sees tokens [row_lo, row_hi)
#pragma unroll
  for (int z = 0; z < CT; ++z) {
    float top = 0.0f;
#pragma unroll
    for (int s = 0; s < W; ++s)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        top = fmaxf(top, fmaxf(fabsf(up<BF16>(raw[z][s][w] & 0xFFFFu)), fabsf(up<BF16>(raw[z][s][w] >> 16))));
    top = quarters_max(top);
    int e = top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : 0;  // top in [2^(e-1), 2^e)
    e = e < -100 ? -100 : e;
    const float mul = ldexpf(1.0f, 14 - e), factor = a.scale * kLog2e;
    row_scale[z] = ldexpf(factor, e - 14 + kKeyBits);  // in one step: neither part has to fit fp32
#pragma unroll
    for (int g = 0; g < G; ++g) qsum[z][g] = 0.0f;
#pragma unroll
    for (int s = 0; s < W; ++s) {
      float x[8];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        x[2 * w] = up<BF16>(raw[z][s][w] & 0xFFFFu);
        x[2 * w + 1] = up<BF16>(raw[z][s][w] >> 16);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) qsum[z][s / 2] += x[j];
      half8 v;
#pragma unroll
      for (int p = 0; p < 4; ++p) {  // nibbles p and p + 4
        v[2 * p] = (_Float16)(x[p] * mul);
        v[2 * p + 1] = (_Float16)(x[p + 4] * mul);
      }
#pragma unroll
      for (int y = 0; y < V; ++y) q[z][y][s] = V == 1 || part == y ? v : half8{};
    }
#pragma unroll
    for (int g = 0; g < G; ++g) qsum[z][g] = quarters_sum(qsum[z][g]) * factor;
    const int32_t pos = t.pos0 + i[z];
    row_hi[z] = pos + 1;
    row_lo[z] = a.window ? pos - a.window + 1 : 0;
  }
  // [all_lo, all_hi): tokens that every row of the tile sees
  const int32_t all_hi = t.pos0 + t.row0 / a.group + 1;
  const int32_t all_lo = a.window ? t.pos0 + (t.row0 + t.rows - 1) / a.group - a.window + 1 : 0;

  // The column's running sums are of weights w = 2^(score - ref): ref is the largest score
  // seen, up to kLazy, less a power k (the same in the wave) that keeps w times a value's
  // scale below 2^15 and far above fp16's subnormals.
  float4v o[CT][J];
  // A weight times a value's scale is rounded to fp16 for the product, which would show beside
  // the output's own rounding (fp16: 1.5 times its error, bf16: 1.04), so what it leaves goes
  // through the product as a second operand.  Decodes wait for memory: it costs them 0 to 3% (bf16:
  // 131071 tokens 35.1 -> 36.1 us, 128 requests 184.2 -> 184.4).  Tiles of more rows wait for the
  // products (bf16: prompts of 2 x 1024 rows 222.7 -> 273.6, 32 requests of 5 drafted rows over 4001
  // tokens 43.3 -> 49.6), so there bf16, whose own rounding is 8 times larger, goes without.
  constexpr int kParts = BF16 && V == 1 ? 1 : 2;
  float m[CT], ref[CT], limit[CT], l[CT], bias[CT][G], k = 0.0f;
#pragma unroll
  for (int z = 0; z < CT; ++z) {
#pragma unroll
    for (int j = 0; j < J; ++j) o[z][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    m[z] = ref[z] = limit[z] = kLow;
    l[z] = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) bias[z][g] = 0.0f;
  }
  uint32_t vbits = 0;  // value scales up to this fp16 pattern fit k

  // This lane's dwords of key or value codes of a run.
  auto codes = [&](const uint8_t *src, uint32_t (&w)[W]) {
    if constexpr (D == 64) {
#pragma unroll
      for (int e = 0; e < W; ++e) w[e] = *reinterpret_cast<const uint32_t *>(src + e * 256 + lane * 4);
    } else {
#pragma unroll
      for (int e = 0; e < W / 4; ++e) {
        const uint4v v = *reinterpret_cast<const uint4v *>(src + e * 1024 + lane * 16);
        w[4 * e] = v.x, w[4 * e + 1] = v.y, w[4 * e + 2] = v.z, w[4 * e + 3] = v.w;
      }
    }
  };
  auto params = [&](const uint8_t *src, half2v (&p)[4][G]) {  // of the 4 tokens of this quarter
    const uint4v *q4 = reinterpret_cast<const uint4v *>(src + c * (16 * G));
#pragma unroll
    for (int f = 0; f < G; ++f) {
      const uint4v v = q4[f];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t word = v[e];  // a copy: a bit cast of a vector's element takes its first one
        p[(4 * f + e) / G][(4 * f + e) % G] = __builtin_bit_cast(half2v, word);
      }
    }
  };
  auto at = [](const half2v (&p)[G], int e) { return (float)p[e / 2][e % 2]; };

  // here: bit x says that run x is in the cache.
  auto compute = [&](auto stage, int32_t t0, uint32_t here) __attribute__((always_inline)) {
    const uint8_t *src = ring + decltype(stage)::value * S::kStage;
    float s[CT][S::kSets][4];
#pragma unroll
    for (int z = 0; z < S::kSets; ++z) {
      float4v acc[CT][G];
#pragma unroll
      for (int e = 0; e < CT; ++e)
#pragma unroll
        for (int g = 0; g < G; ++g) acc[e][g] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int y = 0; y < V; ++y) {
        uint32_t w[W];
        codes(src + (z * V + y) * S::kBytes, w);
#pragma unroll
        for (int d = 0; d < W; ++d) {
          const half8 v = codes8(w[d]);
#pragma unroll
          for (int e = 0; e < CT; ++e)
            acc[e][d / 2] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, q[e][y][d], acc[e][d / 2], 0, 0, 0);
        }
      }
      half2v kp[4][G];
      params(src + (z * V + part) * S::kBytes + 16 * D, kp);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < CT; ++e) {
          float dot = 0.0f, add = 0.0f;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            dot = fmaf(at(kp[u], g), acc[e][g][u], dot);
            add = fmaf(at(kp[u], G + g), qsum[e][g], add);
          }
          s[e][z][u] = fmaf(row_scale[e], dot, add);
        }
    }
    half2v vp[S::kSets][4][G];
#pragma unroll
    for (int z = 0; z < S::kSets; ++z) params(src + (z * V + part) * S::kBytes + 16 * D + 64 * G, vp[z]);
    uint32_t vc[S::kRuns][W];  // read here, beside the scores, and not when they are needed
#pragma unroll
    for (int x = 0; x < S::kRuns; ++x) codes(src + x * S::kBytes + 8 * D, vc[x]);
    if (!(t0 >= all_lo && t0 >= from && t0 + S::kTokens <= all_hi && t0 + S::kTokens <= to &&
          here == (1u << S::kRuns) - 1)) {
#pragma unroll
      for (int z = 0; z < S::kSets; ++z)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int32_t tok = t0 + kRun * (z * V + part) + 4 * c + u;
          const bool there = tok < to && tok >= from && (here >> (z * V + part) & 1);
#pragma unroll
          for (int e = 0; e < CT; ++e)
            s[e][z][u] = there && tok < row_hi[e] && tok >= row_lo[e] ? s[e][z][u] : -INFINITY;
          // What lies behind the last token, or in its run before the first one that a row sees,
          // may never have been written and be NaN: no part of a sum, not even times zero.
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t w = __builtin_bit_cast(uint32_t, vp[z][u][g]);
            vp[z][u][g] = __builtin_bit_cast(half2v, there ? w : 0u);
          }
        }
    }
    float top[CT];
    bool over = false;
    uint32_t big = 0;
#pragma unroll
    for (int z = 0; z < S::kSets; ++z)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int e = 0; e < CT; ++e) top[e] = z + u == 0 ? s[e][0][0] : fmaxf(top[e], s[e][z][u]);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t pair = __builtin_bit_cast(uint32_t, vp[z][u][g / 2]);
          const uint32_t v = g % 2 ? pair >> 16 : pair & 0xFFFFu;
          big = v > big ? v : big;
        }
      }
#pragma unroll
    for (int e = 0; e < CT; ++e) over = over || top[e] > limit[e];
    if (__any(over || big > vbits)) {
      if (__any(big > vbits)) {
#pragma unroll
        for (int d = S::kRows; d < kCols; d <<= 1) {
          const uint32_t other = __shfl_xor(big, d);
          big = other > big ? other : big;
        }
        big = quarters_max(big);
        const int32_t e = big >> 10 ? big >> 10 : 1;
        vbits = e << 10 | 0x3FF;
        k = (float)(23 - e);  // a scale below 2^(e-14) times 2^k is below 2^9
      }
#pragma unroll
      for (int e = 0; e < CT; ++e) {
        m[e] = fmaxf(m[e], quarters_max(top[e]));
        limit[e] = -less(-m[e], kLazy, kLazy);
        // weights reach 2^((limit - m) + (m - next)) <= 2^(kLazy + k)
        const float next = less(m[e], k, k + (kLazy - (limit[e] - m[e])));
        const float f = __builtin_amdgcn_exp2f(ref[e] - next);
        ref[e] = next;
        l[e] *= f;
#pragma unroll
        for (int g = 0; g < G; ++g) bias[e][g] *= f;
#pragma unroll
        for (int j = 0; j < J; ++j) o[e][j] *= f;
      }
    }
    half2v p[kParts][CT][S::kSets][G][2];
#pragma unroll
    for (int e = 0; e < CT; ++e)
#pragma unroll
      for (int z = 0; z < S::kSets; ++z)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float w = __builtin_amdgcn_exp2f(s[e][z][u] - ref[e]);
          l[e] += w;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            bias[e][g] = fmaf(at(vp[z][u], G + g), w, bias[e][g]);
            // as a fused sum it takes the fp16 factor as it is
            const _Float16 ps = (_Float16)fmaf(at(vp[z][u], g), w, 0.0f);
            p[0][e][z][g][u / 2][u % 2] = ps;
            if (kParts == 2) p[kParts - 1][e][z][g][u / 2][u % 2] = (_Float16)fmaf(at(vp[z][u], g), w, -(float)ps);
          }
        }
#pragma unroll
    for (int y = 0; y < S::kRuns / 2; ++y) {  // two runs fill an operand
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint4v pw[kParts][CT];
#pragma unroll
        for (int r = 0; r < kParts; ++r)
#pragma unroll
          for (int e = 0; e < CT; ++e)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              if (V == 1) {
                pw[r][e][f] = __builtin_bit_cast(uint32_t, p[r][e][0][g][f]);
                pw[r][e][2 + f] = __builtin_bit_cast(uint32_t, p[r][e][S::kSets - 1][g][f]);
              } else {
                const uint32_t w = __builtin_bit_cast(uint32_t, p[r][e][V == 2 ? y : 0][g][f]);
                const int first = V == 2 ? 0 : 2 * y;  // the column part of this pair's first run
                pw[r][e][f] = part == first ? w : 0u;
                pw[r][e][2 + f] = part == first + 1 ? w : 0u;
              }
            }
        uint32_t w[4];  // pairs of tokens, the 4 nibbles of group g's channels in each half
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          if (D == 64) {
            w[z] = vc[2 * y + z / 2][z % 2];
          } else {
            constexpr int per = D < 128 ? 1 : D / 128;  // dwords of one token
            const int d0 = (z % 2) * 2 * per + g / 2;
            w[z] = __builtin_amdgcn_perm(vc[2 * y + z / 2][d0 + per], vc[2 * y + z / 2][d0], g % 2 ? 0x07060302u : 0x05040100u);
          }
        }
#pragma unroll
        for (int nib = 0; nib < 4; ++nib) {
          const uint4v u = {nibble_pair(w[0], nib), nibble_pair(w[1], nib), nibble_pair(w[2], nib), nibble_pair(w[3], nib)};
#pragma unroll
          for (int r = 0; r < kParts; ++r)
#pragma unroll
            for (int e = 0; e < CT; ++e)
              o[e][4 * g + nib] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                  __builtin_bit_cast(half8, u), __builtin_bit_cast(half8, pw[r][e]), o[e][4 * g + nib], 0, 0, 0);
        }
      }
    }
  };

  while (tb < to) {
    auto step = [&](auto stage, int32_t j) __attribute__((always_inline)) {
      if (j + 1 < steps) {
        wait_lds();  // the stage that is filled now was read in the last step
        start(Const<1 - decltype(stage)::value>(), j + 1);
        wait_vm<S::kLoads>();
      } else {
        wait_vm<0>();
      }
      __builtin_amdgcn_sched_barrier(0);
      compute(stage, tb + j * kStride4, (uint32_t)(there >> (S::kRuns * j)) & ((1u << S::kRuns) - 1));
      __builtin_amdgcn_sched_barrier(0);
    };
    for (int32_t j = 0;;) {
      step(Const<0>(), j);
      if (++j == steps) break;
      step(Const<1>(), j);
      if (++j == steps) break;
    }
    wait_lds();
    tb += kBatch * kStride4;
    if (tb < to) fetch();
  }

  // The columns' statistics and outputs; a row's are V columns of each wave.
#pragma unroll
  for (int z = 0; z < CT; ++z) {
    l[z] = quarters_sum(l[z]);
#pragma unroll
    for (int g = 0; g < G; ++g) bias[z][g] = quarters_sum(bias[z][g]);
    if (c == 0) {
      s_m[wave][kCols * z + n] = ref[z];
      s_l[wave][kCols * z + n] = l[z];
    }
  }
  __syncthreads();  // and every wave is done with its ring
  float *s_o = reinterpret_cast<float *>(smem);
#pragma unroll
  for (int z = 0; z < CT; ++z) {
    float best = ref[z];
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
#pragma unroll
      for (int y = 0; y < V; ++y) best = fmaxf(best, s_m[w][kCols * z + n % S::kRows + y * S::kRows]);
    const float f = __builtin_amdgcn_exp2f(ref[z] - best);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float fo = f * (j & 1 ? 1.0f / kOddUnit : 1.0f / kEvenUnit), fb = f * bias[z][j / 4];
      float4v v;
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = fmaf(o[z][j][u], fo, fb);
      *reinterpret_cast<float4v *>(s_o + (wave * kAll + kCols * z + n) * kStride + 16 * j + 4 * c) = v;
    }
  }
  __syncthreads();
  const int64_t place = ((int64_t)(b * a.tiles + rt) * a.hkv + h) * a.splits + split;
  for (int e = threadIdx.x; e < t.rows * (D / 8); e += kThreads) {
    const int rr = e / (D / 8), ch = e % (D / 8) * 8;
    float top = kLow * 2.0f, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
#pragma unroll
      for (int y = 0; y < V; ++y) top = fmaxf(top, s_m[w][rr + y * S::kRows]);
    float4v v0 = {0.0f, 0.0f, 0.0f, 0.0f}, v1 = v0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
#pragma unroll
      for (int y = 0; y < V; ++y) {
        const int col = rr + y * S::kRows;
        sum = fmaf(s_l[w][col], __builtin_amdgcn_exp2f(s_m[w][col] - top), sum);
        const float *src = s_o + (w * kAll + col) * kStride + ch;
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

// How the work of a call is cut.  Rows: tiles of 4, 8, 16 or 32 (row, head) pairs of one
// key/value head, the fewest that hold them or 32.  Tokens: so many equal chunks of each tile
// that about kTarget workgroups run at the longest length; 256 CUs hold 2 of them each.  32
// requests of up to 4001 tokens, 8 heads: 36.3 us with 512, 40.6 with 1024 (more to join),
// 36.0 with 256, whose single workgroup a CU loses where there are fewer requests.
constexpr int64_t kTarget = 512;

Cut cut_of(int32_t B, int32_t hq, int32_t hkv, int32_t dim, int32_t max_rows, int32_t max_len, int32_t window) {
  Cut k;
  const int64_t rows = (int64_t)max_rows * (hq / hkv);
  k.tile_rows = rows <= 4 && dim < 256 ? 4 : rows <= 8 ? 8 : rows <= 16 || dim == 256 ? 16 : 32;
  k.tiles = (int32_t)((rows + k.tile_rows - 1) / k.tile_rows);
  int64_t span = max_len;
  // a tile's rows are at most tile_rows positions, its first chunk starts at a whole run
  if (window && (int64_t)window + k.tile_rows + kRun < span) span = (int64_t)window + k.tile_rows + kRun;
  const int64_t groups = (int64_t)B * hkv * k.tiles;
  const int64_t most = (span + kMinChunk - 1) / kMinChunk, want = (kTarget + groups - 1) / groups;
  k.splits = (int32_t)(most < 1 || want <= 1 ? 1 : want < most ? want : most);
  return k;
}

template <int D, bool BF16>
void launch(const Args &a, hipStream_t s) {
  const dim3 grid((unsigned)(a.splits * a.hkv), (unsigned)a.tiles, (unsigned)a.B), threads(kThreads);
  constexpr bool kWide = D < 256;  // 256 channels: the registers of 4-row and 32-row tiles are not there
  if (kWide && a.tile_rows == 32)
    hipLaunchKernelGGL((kv4_attention_kernel<D, 1, kWide ? 2 : 1, BF16>), grid, threads, 0, s, a);
  else if (kWide && a.tile_rows == 4)
    hipLaunchKernelGGL((kv4_attention_kernel<D, kWide ? 4 : 2, 1, BF16>), grid, threads, 0, s, a);
  else if (a.tile_rows == 8) hipLaunchKernelGGL((kv4_attention_kernel<D, 2, 1, BF16>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((kv4_attention_kernel<D, 1, 1, BF16>), grid, threads, 0, s, a);
  if (a.splits == 1 || hipPeekAtLastError() != hipSuccess) return;
  launch_join<D, BF16>(a, s);
}

template <int D>
void launch(const Args &a, int32_t dtype, hipStream_t s) {
  if (dtype == MIXLLM_BF16) launch<D, true>(a, s);
  else launch<D, false>(a, s);
}

}  // namespace

extern "C" size_t mixllm_kv4_attention_workspace_bytes(int32_t T, int32_t B, int32_t q_heads, int32_t kv_heads,
                                                       int32_t dim, int32_t max_rows, int32_t max_len,
                                                       int32_t window) {
  if (!shape_ok(T, B, q_heads, kv_heads, dim, max_rows, max_len, window) || T == 0 || B == 0 || max_rows == 0) return 0;
  const Cut k = cut_of(B, q_heads, kv_heads, dim, max_rows, max_len, window);
  if (k.splits == 1) return 0;
  return (size_t)B * k.tiles * kv_heads * k.splits * k.tile_rows * (dim + 2) * sizeof(float);
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
  const int bad = check_call(q, ldq, q_heads, dim, table, ldt, width, lens, cu, out, ldo, lse, workspace);
  if (bad != MIXLLM_OK) return bad;
  const Cut k = cut_of(B, q_heads, kv_heads, dim, max_rows, max_len, window);
  const int64_t parts = (int64_t)B * k.tiles * kv_heads * k.splits;
  if (parts > 0x7FFFFFFF || B > 65535 || k.tiles > 65535 || (int64_t)B * max_rows * q_heads > 0x7FFFFFFF)
    return MIXLLM_E_SHAPE;
  float *ws = static_cast<float *>(workspace);
  if (k.splits > 1) {
    if (workspace_bytes < (size_t)parts * k.tile_rows * (dim + 2) * sizeof(float)) return MIXLLM_E_SPACE;
    if (!ws) return MIXLLM_E_NULL;
  }
  const Args a = {static_cast<const uint16_t *>(q), static_cast<const uint8_t *>(cache), table, lens, cu,
                  static_cast<uint16_t *>(out), lse, ws, ws ? ws + parts * k.tile_rows * dim : nullptr,
                  ldq, ldo, ldt, scale, T, q_heads, kv_heads, q_heads / kv_heads, pages,
                  mixllm::log2_of(page), width, B, max_rows,
                  max_len, window, k.tiles, k.tile_rows, k.splits};
  if (dim == 64) launch<64>(a, dtype, (hipStream_t)stream);
  else if (dim == 128) launch<128>(a, dtype, (hipStream_t)stream);
  else launch<256>(a, dtype, (hipStream_t)stream);
  return mixllm::launch_status();
}
