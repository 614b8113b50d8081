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

constexpr int kRows = 16;              // rows whose runs a workgroup takes
constexpr int kWindow = 2 * kRows;     // rows it looks at: a run that begins in the last goes on
constexpr int kAppendThreads = 16 * kWindow;
constexpr int kAppendWaves = kAppendThreads / 64;

// A row begins a piece of a run if the row before it is of another run (or of none, or not
// before it in the run).  A workgroup takes the pieces that begin in its 16 rows; 16 lanes
// hold a row, then a wave each writes the whole runs: the codes held before, rounded again
// where the scale grew, and the new ones between them.
template <int D, bool BF16>
__global__ __launch_bounds__(kAppendThreads) void kv8_append_kernel(Kv8Args a) {
  constexpr int C = D / 16, U = D / 64;  // channels of a lane; 1024-byte units of a run
  __shared__ __attribute__((aligned(16))) uint8_t codes[2][kWindow][D];
  __shared__ float tops[2][kWindow];
  const int lane = threadIdx.x & 63, i = threadIdx.x & 15, quarter = threadIdx.x >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t group = blockIdx.x / a.heads, head = blockIdx.x - group * a.heads;
  const int32_t row0 = group * kRows, row = row0 + quarter;
  const uint32_t tokens = (uint32_t)a.pages * (uint32_t)a.page;

  // The window's rows, a lane each: bit r of `live`: row r has a slot; of `begins`: it begins a piece.
  const int32_t mine = row0 + (lane & (kWindow - 1));
  const int32_t slot = mine < a.T ? a.slots[mine] : -1, prev = mine > 0 && mine <= a.T ? a.slots[mine - 1] : -1;
  const bool has = (uint32_t)slot < tokens, had = (uint32_t)prev < tokens;
  const uint32_t live = (uint32_t)__ballot(has);
  const uint32_t begins = (uint32_t)__ballot(has && !(had && prev / kKv8Run == slot / kKv8Run && prev < slot));
  // the row that begins the piece of row r, or -1: before this window
  auto head_of = [&](int r) {
    const uint32_t before = begins & (0xFFFFFFFFu >> (kWindow - 1 - r));
    return before ? 31 - __builtin_clz(before) : -1;
  };
  const int lead = live >> quarter & 1 ? head_of(quarter) : -1;
  const bool take = lead >= 0 && lead < kRows;

  alignas(16) uint32_t raw[2][C / 2];
  float x[2][C];
  if (take) {
    copy16<C>(reinterpret_cast<uint16_t *>(raw[0]), a.k + (int64_t)row * a.ldk + (int64_t)head * D + i * C);
    copy16<C>(reinterpret_cast<uint16_t *>(raw[1]), a.v + (int64_t)row * a.ldv + (int64_t)head * D + i * C);
  }
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      x[z][j] = take ? finite(up<BF16>(raw[z][j / 2] >> (16 * (j % 2)) & 0xFFFFu)) : 0.0f;
      top = fmaxf(top, fabsf(x[z][j]));
    }
    top = quarter_max(top);
    if (i == 0) tops[z][quarter] = top;
  }
  __syncthreads();

  // Where a run is, and its scale before and after.  Rows of a piece: from `first` on.
  auto block_of = [&](int32_t s) { return a.cache + ((int64_t)(s >> a.page_log2) * a.heads + head) * mixllm::kv8_block_bytes(a.page, D); };
  auto end_of = [&](int first) {  // the row behind the piece
    const uint32_t after = first < kWindow - 1 ? (begins | ~live) & (0xFFFFFFFEu << first) : 0;
    return after ? __builtin_ctz(after) : kWindow;
  };
  auto held_of = [&](const uint8_t *blk, int32_t s, int z) {
    const float old = s % kKv8Run ? reinterpret_cast<const float *>(blk + mixllm::kv8_scale_offset(a.page, D))[(s & (a.page - 1)) / kKv8Run * 2 + z] : 0.0f;
    return old > 0.0f && old < INFINITY ? old : 0.0f;
  };
  auto top_of = [&](int first, int end, int z) {
    float top = 0.0f;
    for (int r = first; r < end && r < first + kKv8Run; ++r) top = fmaxf(top, tops[z][r]);
    return top;
  };

  const int32_t s0_of_mine = __shfl(slot, take ? lead : 0);  // every lane takes part
  if (take) {
    const int32_t s0 = s0_of_mine;
    const uint8_t *blk = block_of(s0);
    const int end = end_of(lead);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const float s = fmaxf(held_of(blk, s0, z), top_of(lead, end, z) / 127.0f);
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const float c = s > 0.0f ? fminf(fmaxf(__builtin_rintf(x[z][j] / s), -127.0f), 127.0f) : 0.0f;
        codes[z][quarter][i * C + j] = (uint8_t)code_byte(c);
      }
    }
  }
  __syncthreads();

  const int n = lane & 15, c = lane >> 4;
  int piece = 0;
  for (uint32_t left = begins & ((1u << kRows) - 1); left; left &= left - 1, ++piece) {
    if (piece % kAppendWaves != wave) continue;
    const int first = __builtin_ctz(left), end = end_of(first);
    const int32_t s0 = __builtin_amdgcn_readlane(slot, first);
    uint8_t *blk = block_of(s0);
    // the row of each place of the run, or -1: lane t < 16 looks for place t
    int from = -1;
    for (int r = first; r < end && r < first + kKv8Run; ++r)
      if (__builtin_amdgcn_readlane(slot, r) % kKv8Run == n) from = r;
    float *scales = reinterpret_cast<float *>(blk + mixllm::kv8_scale_offset(a.page, D)) + (s0 & (a.page - 1)) / kKv8Run * 2;
    const int32_t at = (s0 & (a.page - 1)) / kKv8Run * (kKv8Run * D);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const float old = held_of(blk, s0, z), s = fmaxf(old, top_of(first, end, z) / 127.0f);
      const float r = s > 0.0f ? old / s : 0.0f;
      uint8_t *run = blk + z * a.page * D + at;
      if (lane == 0) scales[z] = s;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint4 *unit = reinterpret_cast<uint4 *>(run + u * 1024) + lane;
        uint4 held = make_uint4(0, 0, 0, 0);
        if (s0 % kKv8Run) held = *unit;
        uint32_t w[4] = {held.x, held.y, held.z, held.w};
        if (r != 1.0f) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = rescaled(w[j], r);
        }
        if (z == 0) {  // 16 channels of token n
          if (from >= 0) {
            const uint4 v = *reinterpret_cast<const uint4 *>(&codes[0][from][64 * u + 16 * c]);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
          }
        } else {  // tokens 4c .. 4c+3 of the channels 16 j + n
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int src = __shfl(from, 4 * c + t);
            if (src >= 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = (w[j] & ~(0xFFu << (8 * t))) | (uint32_t)codes[1][src][64 * u + 16 * j + n] << (8 * t);
            }
          }
        }
        *unit = make_uint4(w[0], w[1], w[2], w[3]);
      }
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
  // a launch has fewer than 2^32 threads, 512 for 16 rows of a head
  if (heads > 65535 || ((int64_t)T + 15) / 16 * heads >= 1 << 23) return MIXLLM_E_SHAPE;
  if (ldk < width || ldv < width || ldk % 8 != 0 || ldv % 8 != 0) return MIXLLM_E_SHAPE;
  if (!k || !v || !slots) return MIXLLM_E_NULL;
  if (!mixllm::is_aligned16(k) || !mixllm::is_aligned16(v) || !mixllm::is_aligned4(slots)) return MIXLLM_E_SHAPE;
  return MIXLLM_OK;
}

template <bool APPEND, int D>
void launch_tokens(const Kv8Args &a, int32_t dtype, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.T + 15) / 16 * a.heads));  // heads of the same rows together
  if (APPEND) {
    if (dtype == MIXLLM_BF16) hipLaunchKernelGGL((kv8_append_kernel<D, true>), grid, dim3(kAppendThreads), 0, s, a);
    else hipLaunchKernelGGL((kv8_append_kernel<D, false>), grid, dim3(kAppendThreads), 0, s, a);
  } else {
    if (dtype == MIXLLM_BF16) hipLaunchKernelGGL((kv8_read_kernel<D, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((kv8_read_kernel<D, false>), grid, dim3(256), 0, s, a);
  }
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
