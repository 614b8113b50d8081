// Writing to the paged cache in 8 bits and reading it back (layout: mixllm_kv8.h).
//
// A run, 16 tokens that follow one another in a page, has one scale for the keys of a head
// and one for its values: x ~ s c, c = clamp(rne(x / s), -127, 127).  Tokens come one at a
// time, so a scale grows as they come:
//   s = max(s_held, max |x| / 127) over the call's tokens of the run,
//   held codes c' = rne(c (s_held / s)),
// and a call that writes a run's first token begins it anew (s_held = 0).  All in fp32 steps.
// A code that was rounded again r times is off by at most (1 + r) / 2 of the run's step; of n
// tokens in random order the scale grows 1 + 1/2 + .. + 1/n times, 3.4 of 16.
//
// 8 heads of 128: 64 rows 6.7 us (the chain slots -> run -> store, two barriers between), 6961 rows of four
// prompts 18.8 us for the 43 MB that a copy moves in 8.5.  There half of a workgroup's rows are
// others' pieces, and a wave lives 4.6 us for two loads and a store one after the other; vector
// operations are a third of it.  Heads one after the other in a workgroup with the next head's
// loads ahead measured no better (22.9 - 27.8), nor did 48 or 64 rows (19.6 - 22.9).  Reading back: 8.5 us
// for those rows, a copy's rate.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm_kv8.h"
#include "mixllm_lanes.h"
#include "mixllm_quant_pair.h"

namespace {

using mixllm::down;
using mixllm::kKv8Run;
using mixllm::kKv8Zero;
using mixllm::quarter_max;
using mixllm::up;

struct Kv8Args {
  uint8_t *cache;
  const int32_t *slots;
  uint16_t *k, *v;
  int64_t ldk, ldv;
  int32_t T, heads, pages, page, page_log2;
};

// C 16-bit values from one place to another, both aligned to their size (16 bytes at most).
template <int C>
__device__ __forceinline__ void copy16(uint16_t *to, const uint16_t *from) {
  if (C == 4) *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(from);
  if (C >= 8) *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
  if (C == 16) *reinterpret_cast<uint4 *>(to + 8) = *reinterpret_cast<const uint4 *>(from + 8);
}

// x with NaN as 0 and what is beyond +-65504 as that.
__device__ __forceinline__ float finite(float x) { return x != x ? 0.0f : fminf(fmaxf(x, -65504.0f), 65504.0f); }

__device__ __forceinline__ uint32_t code_byte(float c) { return (uint32_t)((int)c + kKv8Zero); }

// The four codes of a dword rounded again to a scale 1 / r times as large: c r is exact in the
// fused step but for its own rounding, (u - 128) r = u r - 128 r.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float r) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = __builtin_rintf(fmaf((float)((w >> (8 * i)) & 0xFFu), r, -(float)kKv8Zero * r));
    out |= code_byte(fminf(fmaxf(c, -127.0f), 127.0f)) << (8 * i);
  }
  return out;
}

typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));

// The largest size of a lane's C values, as the bits of a 16-bit type: those of infinities and NaN
// are above all others.
template <int C>
__device__ __forceinline__ uint32_t largest(const uint32_t (&raw)[C / 2]) {
  ushort2v top = {0, 0};
#pragma unroll
  for (int j = 0; j < C / 2; ++j)
    top = __builtin_elementwise_max(top, __builtin_bit_cast(ushort2v, raw[j] & 0x7FFF7FFFu));
  return top.x > top.y ? top.x : top.y;
}

template <bool BF16>
constexpr uint32_t kLargest = BF16 ? 0x477Fu : 0x7BFFu;  // bits of the largest value within +-65504

// The codes of a lane's C values as bytes, four to a dword.  By the reciprocal r of s: x r is within
// 6e-5 of the quotient (|x / s| <= 127), and the sum with 1.5 2^23 rounds it to a whole number
// with its byte in the lowest bits; it is the number of rne(x / s) unless x r lies within 2^-12 of a
// half.  A lane with such a value divides, and so do those with a scale so small that r may be no
// number (r = NaN) or with values past +-65504.
template <int C, bool BF16>
__device__ __forceinline__ void codes_of(const uint32_t (&raw)[C / 2], bool within, float s, float r, uint32_t (&w)[C / 4]) {
  constexpr float kWhole = 12582912.0f + kKv8Zero;
  uint32_t c[C];
  float off = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const float t = up<BF16>(raw[j / 2] >> (16 * (j % 2)) & 0xFFFFu) * r, sum = t + kWhole;
    off = fmaxf(off, fabsf(t - (sum - kWhole)));
    c[j] = __float_as_uint(sum);
  }
  if (!(within && r == r && off <= 0.5f - 0x1p-12f)) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const float x = finite(up<BF16>(raw[j / 2] >> (16 * (j % 2)) & 0xFFFFu));
      c[j] = code_byte(s > 0.0f ? fminf(fmaxf(__builtin_rintf(x / s), -127.0f), 127.0f) : 0.0f);
    }
  }
#pragma unroll
  for (int j = 0; j < C / 4; ++j)
    w[j] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[4 * j + 3], c[4 * j + 2], 0x0C0C0400u),
                                 __builtin_amdgcn_perm(c[4 * j + 1], c[4 * j], 0x0C0C0400u), 0x05040100u);
}

// Rows times heads up to which a workgroup takes 4 rows, and not 16 by half as many lanes (us, 8 heads of
// 128): 64 rows of as many requests 6.5 (9.0 with 16), 700 15.5 (23.6); 1500 of one prompt 15.7 (7.7),
// 6961 of four 52 (18.8).
constexpr int64_t kFewRows = 8192;

// A row begins a piece of a run if the row before it is of another run (or of none, or not
// before it in the run).  A workgroup takes the pieces that begin in its ROWS rows and looks at 16
// rows more, where the last ones end.  16 lanes hold a row until its codes are in LDS; then a wave
// each writes the 1024-byte units of the runs: what was held, rounded again where the scale
// grew, with the new codes in their places.  Values go to LDS in the order of channels 16 j + n
// -> 4 n + j, so that a unit's lane has its four channels of a token in one dword.
template <int D, int ROWS, int EACH, bool BF16>
__global__ __launch_bounds__(16 * (ROWS + kKv8Run) / EACH) void kv8_append_kernel(Kv8Args a) {
  constexpr int C = D / 16, U = D / 64;  // channels of a lane; units of a run's keys or values
  constexpr int kWindow = ROWS + kKv8Run, kQuarters = kWindow / EACH, kWaves = kQuarters / 4, kBatch = 4;
  static_assert(kQuarters * EACH == kWindow && kWaves * 4 == kQuarters && kWindow <= 64, "a lane for each row");
  __shared__ __attribute__((aligned(16))) uint8_t codes[2][kWindow][D];
  __shared__ float tops[2][kWindow], scales[2][kWindow][2];            // of a piece's first row: held, new
  __shared__ __attribute__((aligned(16))) int8_t rows[kWindow][kKv8Run];  // and the rows of the run's places
  const int lane = threadIdx.x & 63, i = threadIdx.x & 15, quarter = threadIdx.x >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t group = blockIdx.x / a.heads, head = blockIdx.x - group * a.heads;
  const int32_t row0 = group * ROWS;
  const uint32_t tokens = (uint32_t)a.pages * (uint32_t)a.page;
  auto row_of = [&](int y) { return quarter + y * kQuarters; };  // this quarter's rows of the window

  alignas(16) uint32_t raw[EACH][2][C / 2];
  auto load = [&](int y) __attribute__((always_inline)) {
    const int64_t row = row0 + row_of(y);
    copy16<C>(reinterpret_cast<uint16_t *>(raw[y][0]), a.k + row * a.ldk + (int64_t)head * D + i * C);
    copy16<C>(reinterpret_cast<uint16_t *>(raw[y][1]), a.v + row * a.ldv + (int64_t)head * D + i * C);
  };
#pragma unroll
  for (int y = 0; y < EACH; ++y)
    if (row_of(y) < ROWS && row0 + row_of(y) < a.T) load(y);  // beside the slots, not after them

  // The window's rows, a lane each: bit r of `live`: row r has a slot; of `begins`: it begins a piece.
  const int32_t mine = row0 + lane;
  const int32_t slot = lane < kWindow && mine < a.T ? a.slots[mine] : -1;
  const int32_t prev = lane < kWindow && mine > 0 && mine <= a.T ? a.slots[mine - 1] : -1;
  const bool has = (uint32_t)slot < tokens, had = (uint32_t)prev < tokens;
  const uint64_t live = __ballot(has);
  const uint64_t begins = __ballot(has && !(had && prev / kKv8Run == slot / kKv8Run && prev < slot));
  // the row that begins the piece of row r, or -1: before this window
  auto head_of = [&](int r) {
    const uint64_t before = begins & (~0ull >> (63 - r));
    return before ? 63 - __builtin_clzll(before) : -1;
  };
  auto end_of = [&](int first) {  // the row behind the piece
    const uint64_t after = (begins | ~live) & (~1ull << first);
    return after ? __builtin_ctzll(after) : 64;
  };
  int lead[EACH];
  bool take[EACH];
  int32_t slot0[EACH], own[EACH];
#pragma unroll
  for (int y = 0; y < EACH; ++y) {
    rows[row_of(y)][i] = -1;
    lead[y] = live >> row_of(y) & 1 ? head_of(row_of(y)) : -1;
    take[y] = lead[y] >= 0 && lead[y] < ROWS;
    slot0[y] = __shfl(slot, take[y] ? lead[y] : 0), own[y] = __shfl(slot, row_of(y));  // every lane takes part
  }

  auto block_of = [&](int32_t s) {
    return a.cache + ((int64_t)(s >> a.page_log2) * a.heads + head) * mixllm::kv8_block_bytes(a.page, D);
  };
  auto scales_of = [&](int32_t s) {
    return reinterpret_cast<float *>(block_of(s) + mixllm::kv8_scale_offset(a.page, D)) + (s & (a.page - 1)) / kKv8Run * 2;
  };
  float held[EACH][2];
#pragma unroll
  for (int y = 0; y < EACH; ++y) {
    if (row_of(y) >= ROWS && take[y]) load(y);
    held[y][0] = held[y][1] = 0.0f;
    if (take[y] && slot0[y] % kKv8Run) held[y][0] = scales_of(slot0[y])[0], held[y][1] = scales_of(slot0[y])[1];
  }
  // A wave's jobs: units job = (piece, keys or values, unit), every kWaves-th, kBatch of them at a
  // time.  The first batch's held units are on their way before anything is computed.
  const uint64_t pieces = begins & ((1ull << ROWS) - 1);
  const int jobs = __builtin_popcountll(pieces) * (2 * U);
  auto first_of = [&](int piece) {
    uint64_t left = pieces;
    for (; piece > 0; --piece) left &= left - 1;
    return __builtin_ctzll(left);
  };
  auto unit_of = [&](int first, int part) {  // part: unit of the keys, then of the values
    const int32_t s0 = __builtin_amdgcn_readlane(slot, first);
    return reinterpret_cast<uint4 *>(block_of(s0) + part / U * a.page * D + (s0 & (a.page - 1)) / kKv8Run * (kKv8Run * D) +
                                     part % U * 1024) + lane;
  };
  uint4 old[kBatch];
  auto fetch = [&](int job0) {
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int job = job0 + e * kWaves;
      old[e] = make_uint4(0, 0, 0, 0);
      if (job >= jobs) continue;
      const int first = first_of(job / (2 * U));
      if (__builtin_amdgcn_readlane(slot, first) % kKv8Run) old[e] = *unit_of(first, job % (2 * U));
    }
  };
  fetch(wave);

  bool within[EACH][2];
#pragma unroll
  for (int y = 0; y < EACH; ++y) {
    within[y][0] = within[y][1] = true;
    if (!take[y]) continue;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const uint32_t bits = largest<C>(raw[y][z]);
      within[y][z] = bits <= kLargest<BF16>;
      float top = up<BF16>(bits);
      if (!within[y][z]) {
        top = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j) top = fmaxf(top, fabsf(finite(up<BF16>(raw[y][z][j / 2] >> (16 * (j % 2)) & 0xFFFFu))));
      }
      top = quarter_max(top);
      if (i == 0) tops[z][row_of(y)] = top;
    }
  }
  __syncthreads();
#pragma unroll
  for (int y = 0; y < EACH; ++y) {
    if (!take[y]) continue;
    const int row = row_of(y), end = end_of(lead[y]);
    if (i == 0) rows[lead[y]][own[y] % kKv8Run] = (int8_t)row;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const float top = quarter_max(lead[y] + i < end ? tops[z][lead[y] + i] : 0.0f);  // 16 rows at most, a lane each
      const float was = held[y][z] > 0.0f && held[y][z] < INFINITY ? held[y][z] : 0.0f, s = fmaxf(was, top / 127.0f);
      if (i == 0 && row == lead[y]) scales[z][row][0] = was, scales[z][row][1] = s;
      const float r = s >= 0x1p-100f ? __builtin_amdgcn_rcpf(s) : NAN;
      uint32_t w[C / 4];
      codes_of<C, BF16>(raw[y][z], within[y][z], s, r, w);
#pragma unroll
      for (int j = 0; j < C / 4; ++j) {
        if (z == 0) {
          reinterpret_cast<uint32_t *>(&codes[0][row][i * C])[j] = w[j];
        } else {
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int ch = i * C + 4 * j + b;
            codes[1][row][ch / 64 * 64 + ch % 16 * 4 + ch / 16 % 4] = (uint8_t)(w[j] >> (8 * b));
          }
        }
      }
    }
  }
  __syncthreads();

  const int n = lane & 15, q = lane >> 4;
  for (int job0 = wave; job0 < jobs; job0 += kBatch * kWaves) {
    if (job0 != wave) fetch(job0);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int job = job0 + e * kWaves;
      if (job >= jobs) break;
      const int first = first_of(job / (2 * U)), part = job % (2 * U), z = part / U, u = part % U;
      const float was = scales[z][first][0], s = scales[z][first][1], r = s > 0.0f ? was / s : 0.0f;
      uint32_t w[4] = {old[e].x, old[e].y, old[e].z, old[e].w};
      if (r != 1.0f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = r == 0.0f ? kKv8Zero * 0x01010101u : rescaled(w[j], r);
      }
      if (z == 0) {  // 16 channels of token n
        const int from = rows[first][n];
        if (from >= 0) {
          const uint4 v = *reinterpret_cast<const uint4 *>(&codes[0][from][64 * u + 16 * q]);
          w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        }
      } else {  // tokens 4q .. 4q+3 of the channels 16 j + n
        const uint32_t from = *reinterpret_cast<const uint32_t *>(&rows[first][4 * q]);
        uint32_t v[4], keep = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int at = (int8_t)(from >> (8 * t));
          v[t] = at < 0 ? 0u : *reinterpret_cast<const uint32_t *>(&codes[1][at][64 * u + 4 * n]);
          keep |= at < 0 ? 0xFFu << (8 * t) : 0u;
        }
        // 4 tokens x 4 channels of bytes, turned
        const uint32_t a0 = __builtin_amdgcn_perm(v[1], v[0], 0x05010400u), a1 = __builtin_amdgcn_perm(v[1], v[0], 0x07030602u);
        const uint32_t b0 = __builtin_amdgcn_perm(v[3], v[2], 0x05010400u), b1 = __builtin_amdgcn_perm(v[3], v[2], 0x07030602u);
        const uint32_t t0 = __builtin_amdgcn_perm(b0, a0, 0x05040100u), t1 = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
        const uint32_t t2 = __builtin_amdgcn_perm(b1, a1, 0x05040100u), t3 = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
        w[0] = (w[0] & keep) | (t0 & ~keep), w[1] = (w[1] & keep) | (t1 & ~keep);
        w[2] = (w[2] & keep) | (t2 & ~keep), w[3] = (w[3] & keep) | (t3 & ~keep);
      }
      *unit_of(first, part) = make_uint4(w[0], w[1], w[2], w[3]);
      if (u == 0 && lane == 0) scales_of(__builtin_amdgcn_readlane(slot, first))[z] = s;
    }
  }
}

// Between what the lanes of a quarter write to LDS and what others of them read: a wave's
// LDS operations are done in order, so only the compiler has to be held.
__device__ __forceinline__ void in_quarter() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// s c, rounded to 16 bits: 16 lanes take a token's keys and values of a head.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void kv8_read_kernel(Kv8Args a) {
  constexpr int C = D / 16, U = D / 64;
  __shared__ __attribute__((aligned(16))) uint16_t turn[16][D];
  const int i = threadIdx.x & 15, quarter = threadIdx.x >> 4;
  const int32_t group = blockIdx.x / a.heads, head = blockIdx.x - group * a.heads, row = group * 16 + quarter;
  const int32_t slot = row < a.T ? a.slots[row] : -1;
  if ((uint32_t)slot >= (uint32_t)a.pages * (uint32_t)a.page) return;  // whole quarters leave
  const int32_t in = slot & (a.page - 1), t = in % kKv8Run;
  const uint8_t *blk = a.cache + ((int64_t)(slot >> a.page_log2) * a.heads + head) * mixllm::kv8_block_bytes(a.page, D);
  const float2 s = reinterpret_cast<const float2 *>(blk + mixllm::kv8_scale_offset(a.page, D))[in / kKv8Run];
  const uint8_t *run = blk + in / kKv8Run * (kKv8Run * D);
  auto value = [&](uint32_t w, int j, float sc) { return (uint16_t)down<BF16>(sc * (float)((int)((w >> (8 * j)) & 0xFFu) - kKv8Zero)); };
  {
    const int ch = i * C;
    const uint8_t *src = run + ch / 64 * 1024 + ch / 16 % 4 * 256 + t * 16 + ch % 16;
    uint32_t w[C / 4];
#pragma unroll
    for (int j = 0; j < C / 4; ++j) w[j] = reinterpret_cast<const uint32_t *>(src)[j];
    alignas(16) uint16_t out[C];
#pragma unroll
    for (int j = 0; j < C; ++j) out[j] = value(w[j / 4], j % 4, s.x);
    copy16<C>(a.k + (int64_t)row * a.ldk + (int64_t)head * D + ch, out);
  }
  const uint8_t *src = run + a.page * D + t / 4 * 256 + i * 16;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint4 w = *reinterpret_cast<const uint4 *>(src + u * 1024);
    turn[quarter][64 * u + i] = value(w.x, t % 4, s.y);
    turn[quarter][64 * u + 16 + i] = value(w.y, t % 4, s.y);
    turn[quarter][64 * u + 32 + i] = value(w.z, t % 4, s.y);
    turn[quarter][64 * u + 48 + i] = value(w.w, t % 4, s.y);
  }
  in_quarter();
  copy16<C>(a.v + (int64_t)row * a.ldv + (int64_t)head * D + i * C, &turn[quarter][i * C]);
}

int check_tokens(const void *k, const void *v, int64_t ldk, int64_t ldv, int32_t dtype, const int32_t *slots, int32_t T,
                 const void *cache, size_t cache_bytes, int32_t pages, int32_t page, int32_t heads, int32_t dim) {
  if (T < 0 || (dtype != MIXLLM_FP16 && dtype != MIXLLM_BF16)) return MIXLLM_E_SHAPE;
  if (T == 0) return MIXLLM_OK;
  const int st = mixllm::kv8_check_cache(cache, cache_bytes, pages, page, heads, dim);
  if (st != MIXLLM_OK) return st;
  const int64_t width = (int64_t)heads * dim;
  // a launch has fewer than 2^32 threads, 512 for 16 rows of a head at most
  if (heads > 65535 || ((int64_t)T + 15) / 16 * heads >= 1 << 23) return MIXLLM_E_SHAPE;
  if (ldk < width || ldv < width || ldk % 8 != 0 || ldv % 8 != 0) return MIXLLM_E_SHAPE;
  if (!k || !v || !slots) return MIXLLM_E_NULL;
  if (!mixllm::is_aligned16(k) || !mixllm::is_aligned16(v) || !mixllm::is_aligned4(slots)) return MIXLLM_E_SHAPE;
  return MIXLLM_OK;
}

template <int D, int ROWS, int EACH>
void launch_append(const Kv8Args &a, int32_t dtype, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.T + ROWS - 1) / ROWS * a.heads)), block(16 * (ROWS + kKv8Run) / EACH);  // heads of the same rows together
  if (dtype == MIXLLM_BF16) hipLaunchKernelGGL((kv8_append_kernel<D, ROWS, EACH, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((kv8_append_kernel<D, ROWS, EACH, false>), grid, block, 0, s, a);
}

template <bool APPEND, int D>
void launch_tokens(const Kv8Args &a, int32_t dtype, hipStream_t s) {
  if (APPEND) {
    if ((int64_t)a.T * a.heads <= kFewRows) launch_append<D, 4, 1>(a, dtype, s);
    else launch_append<D, 16, 2>(a, dtype, s);
    return;
  }
  const dim3 grid((unsigned)(((int64_t)a.T + 15) / 16 * a.heads));
  if (dtype == MIXLLM_BF16) hipLaunchKernelGGL((kv8_read_kernel<D, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((kv8_read_kernel<D, false>), grid, dim3(256), 0, s, a);
}

template <bool APPEND>
int run_tokens(const Kv8Args &a, int32_t dim, int32_t dtype, void *stream) {
  if (dim == 64) launch_tokens<APPEND, 64>(a, dtype, (hipStream_t)stream);
  else if (dim == 128) launch_tokens<APPEND, 128>(a, dtype, (hipStream_t)stream);
  else launch_tokens<APPEND, 256>(a, dtype, (hipStream_t)stream);
  return mixllm::launch_status();
}

}  // namespace

extern "C" size_t mixllm_kv8_page_bytes(int32_t page, int32_t heads, int32_t dim) {
  if (!mixllm::kv4_dim_ok(dim) || !mixllm::kv4_page_ok(page) || heads <= 0) return 0;
  return (size_t)heads * mixllm::kv8_block_bytes(page, dim);
}

extern "C" int mixllm_kv8_append(const void *k, int64_t ldk, const void *v, int64_t ldv, int32_t dtype,
                                 const int32_t *slots, int32_t T, void *cache, size_t cache_bytes, int32_t pages,
                                 int32_t page, int32_t heads, int32_t dim, void *stream) {
  const int st = check_tokens(k, v, ldk, ldv, dtype, slots, T, cache, cache_bytes, pages, page, heads, dim);
  if (st != MIXLLM_OK || T == 0) return st;
  const Kv8Args a = {static_cast<uint8_t *>(cache), slots,
                     const_cast<uint16_t *>(static_cast<const uint16_t *>(k)),
                     const_cast<uint16_t *>(static_cast<const uint16_t *>(v)), ldk, ldv, T, heads, pages, page,
                     mixllm::log2_of(page)};
  return run_tokens<true>(a, dim, dtype, stream);
}

extern "C" int mixllm_kv8_read(const void *cache, size_t cache_bytes, int32_t pages, int32_t page, int32_t heads,
                               int32_t dim, const int32_t *slots, int32_t T, void *k, int64_t ldk, void *v,
                               int64_t ldv, int32_t dtype, void *stream) {
  const int st = check_tokens(k, v, ldk, ldv, dtype, slots, T, cache, cache_bytes, pages, page, heads, dim);
  if (st != MIXLLM_OK || T == 0) return st;
  const Kv8Args a = {const_cast<uint8_t *>(static_cast<const uint8_t *>(cache)), slots, static_cast<uint16_t *>(k),
                     static_cast<uint16_t *>(v), ldk, ldv, T, heads, pages, page, mixllm::log2_of(page)};
  return run_tokens<false>(a, dim, dtype, stream);
}
