// The linear layer in 8 bits with one scale per token and one per output channel:
//   s_a = max |a| / 127, a_q = clamp(rne(a / s_a), -127, 127)     per row of the activations
//   y[m][n] = (sum_k a_q[m][k] w[n][k]) * (s_a[m] * s_w[n])
// The sum is exact in int32 (K <= 131072), so no split of it changes a result.
//
// Without a scale per group there is nothing between the matrix instructions, so where tokens are many
// they and the power they draw are the bound: 8192^3 541 us, 2030 TOPS, the rate of a library's int8
// product here (2070); 2047 x 14336 x 4096 in 127 us, 1890 TOPS, with 448 tiles on 256 CUs.  With few tokens
// it is the weights' bytes: 4 x 28672 x 8192 in 41 us, 5.7 TB/s.  Between, the copies' latency:
// 512 x 4096 x 4096 takes 15 us (1100 TOPS), 4 x 1024 x 8192 8.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm_kv4.h"
#include "mixllm_lanes.h"
#include "mixllm_quant_pair.h"

namespace {

using mixllm::down;
using mixllm::quarter_max;
using mixllm::up;

typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int16v __attribute__((ext_vector_type(16)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------------------- the quantizer

struct RowsArgs {
  const uint16_t *a;
  int8_t *q;
  float *s;
  int64_t lda, ldq;
  int32_t M, K;
};

// The 16 values of a lane, their largest size and their codes.
struct Values {
  uint4 raw[2];
  __device__ __forceinline__ void load(const uint16_t *src) {
    raw[0] = *reinterpret_cast<const uint4 *>(src);
    raw[1] = *reinterpret_cast<const uint4 *>(src + 8);
  }
  template <bool BF16>
  __device__ __forceinline__ float at(int j) const {
    const uint4 &r = raw[j / 8];
    const uint32_t w = j % 8 / 2 == 0 ? r.x : j % 8 / 2 == 1 ? r.y : j % 8 / 2 == 2 ? r.z : r.w;
    return up<BF16>(w >> (16 * (j % 2)) & 0xFFFFu);
  }
  // By the magnitudes' bits, among which those of infinities and NaN are above all others; a
  // maximum of floats would pass over NaN.  Both come out as the infinity.
  template <bool BF16>
  __device__ __forceinline__ float top() const {
    ushort2v t = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint4 &r = raw[j / 4];
      const uint32_t w = j % 4 == 0 ? r.x : j % 4 == 1 ? r.y : j % 4 == 2 ? r.z : r.w;
      t = __builtin_elementwise_max(t, __builtin_bit_cast(ushort2v, w & 0x7FFF7FFFu));
    }
    const uint32_t bits = t.x > t.y ? t.x : t.y;
    return bits < (BF16 ? 0x7F80u : 0x7C00u) ? up<BF16>(bits) : INFINITY;
  }
  // rne(x / s) by the reciprocal r of s: x r is within 6e-5 of the quotient (|x / s| <= 127), so
  // it rounds to the same number unless it lies within 2^-12 of a half; those divide, and so do
  // all where s is so small that r may not be a number (r = NaN).  A scale of NaN gives codes of 0.
  template <bool BF16>
  __device__ __forceinline__ uint4 codes(float s, float r) const {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = at<BF16>(j), t = x * r;
      float q = __builtin_rintf(t);
      if (!(fabsf(t - q) <= 0.5f - 0x1p-12f)) q = s > 0.0f ? __builtin_rintf(x / s) : 0.0f;
      q = fminf(fmaxf(q, -127.0f), 127.0f);
      w[j / 4] |= ((uint32_t)(int)q & 0xFFu) << (8 * (j % 4));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <int THREADS>
__device__ __forceinline__ float row_top(float top, float *tops) {
  typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
  top = quarter_max(top);
  uint2v v = __builtin_amdgcn_permlane16_swap(__float_as_uint(top), __float_as_uint(top), false, false);
  top = fmaxf(__uint_as_float(v.x), __uint_as_float(v.y));
  v = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
  top = fmaxf(__uint_as_float(v.x), __uint_as_float(v.y));
  if (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) top = fmaxf(top, tops[w]);
  }
  return top;
}

// A row that holds no number somewhere has none as its scale, and so in all its outputs.
__device__ __forceinline__ float scale_of(float top) { return top < INFINITY ? top / 127.0f : NAN; }

__device__ __forceinline__ float inverse(float s) { return s >= 0x1p-100f ? __builtin_amdgcn_rcpf(s) : NAN; }

// A workgroup takes a row, 16 values a thread and chunk, held in registers between the maximum
// and the codes; without chunks rows of any length, which it reads twice.
template <int THREADS, int CHUNKS, bool BF16>
__global__ __launch_bounds__(THREADS) void quant_rows_kernel(RowsArgs a) {
  __shared__ float tops[THREADS / 64];
  const int64_t m = blockIdx.x;
  const uint16_t *src = a.a + m * a.lda;
  int8_t *dst = a.q + m * a.ldq;
  const int32_t first = (int32_t)threadIdx.x * 16;
  float top = 0.0f;
  if constexpr (CHUNKS > 0) {
    Values v[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      v[c].raw[0] = v[c].raw[1] = make_uint4(0, 0, 0, 0);
      if (first + c * THREADS * 16 < a.K) v[c].load(src + first + c * THREADS * 16);
    }
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) top = fmaxf(top, v[c].template top<BF16>());
    const float s = scale_of(row_top<THREADS>(top, tops)), r = inverse(s);
    if (threadIdx.x == 0) a.s[m] = s;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
      if (first + c * THREADS * 16 < a.K)
        *reinterpret_cast<uint4 *>(dst + first + c * THREADS * 16) = v[c].template codes<BF16>(s, r);
  } else {
    Values v;
    for (int32_t e = first; e < a.K; e += THREADS * 16) {
      v.load(src + e);
      top = fmaxf(top, v.template top<BF16>());
    }
    const float s = scale_of(row_top<THREADS>(top, tops)), r = inverse(s);
    if (threadIdx.x == 0) a.s[m] = s;
    for (int32_t e = first; e < a.K; e += THREADS * 16) {
      v.load(src + e);
      *reinterpret_cast<uint4 *>(dst + e) = v.template codes<BF16>(s, r);
    }
  }
}

constexpr int32_t kMaxK = 131072;

template <int THREADS, int CHUNKS, bool BF16>
void launch_rows(const RowsArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((quant_rows_kernel<THREADS, CHUNKS, BF16>), dim3((unsigned)a.M), dim3(THREADS), 0, s, a);
}

// Few rows want many threads for each, many rows more loads in flight in each thread: 4 / 512 / 2047 /
// 8191 rows of 4096 take 5.2 / 5.1 / 10.9 / 32.3 us with 256 threads, 5.6 / 5.3 / 9.2 / 21.6 with 128.
template <bool BF16>
void launch_rows(const RowsArgs &a, hipStream_t s) {
  const bool many = a.M > 1024;
  if (a.K <= 1024) launch_rows<64, 1, BF16>(a, s);
  else if (a.K <= 2048) many ? launch_rows<64, 2, BF16>(a, s) : launch_rows<128, 1, BF16>(a, s);
  else if (a.K <= 4096) many ? launch_rows<128, 2, BF16>(a, s) : launch_rows<256, 1, BF16>(a, s);
  else if (a.K <= 8192) many ? launch_rows<256, 2, BF16>(a, s) : launch_rows<512, 1, BF16>(a, s);
  else if (a.K <= 16384) launch_rows<512, 2, BF16>(a, s);
  else if (a.K <= 32768) launch_rows<1024, 2, BF16>(a, s);
  else launch_rows<1024, 0, BF16>(a, s);
}

// --------------------------------------------------------------------------- the product

struct Gemm8Args {
  const int8_t *a, *w;
  const float *sa, *sw;
  uint16_t *y;
  int64_t lda, ldw, ldy;
  int32_t M, N, K;
  int32_t tiles_m, tiles_n;
  int32_t wide;  // four outputs of a row can be written at once
};

// Outputs of the channels n .. n+3 of token m.
template <bool BF16>
__device__ __forceinline__ void store4(const Gemm8Args &a, int32_t m, int32_t n, int4v acc) {
  if (m >= a.M || n >= a.N) return;
  const float sa = a.sa[m];
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = n + i < a.N ? down<BF16>((float)acc[i] * (sa * a.sw[n + i])) : 0u;
  uint16_t *dst = a.y + (int64_t)m * a.ldy + n;
  if (a.wide && n + 3 < a.N) {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.N) dst[i] = (uint16_t)v[i];
  }
}

typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __attribute__((address_space(3))) void *LdsPtr;
constexpr int kRsrcFlags = 0x00020000;  // raw buffer, 32-bit data format

// Waits until at most N vector-memory operations of this wave are outstanding and its LDS
// operations are done, then for the workgroup's other waves.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Many tokens: a workgroup takes BM tokens x BN channels.  Stages of BK inputs of both go from
// memory to LDS, ST - 1 of them in flight; WM x WN waves share the tile, KS such groups the
// inputs of a stage.  A stage has its rows one after the other, their 16-byte chunks turned by
// the row so that the 16 rows that a read takes at once lie in different banks.
template <int BM_, int BN_, int WM_, int WN_, int KS_, int BK_, int ST_>
struct TileShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KS = KS_, BK = BK_, ST = ST_;
  static constexpr int kWaves = WM * WN * KS, kThreads = 64 * kWaves;
  static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;  // 32 x 32 products of a wave
  static constexpr int kSteps = BK / 32 / KS;                 // of 32 inputs, in a stage
  static constexpr int kChunks = BK / 16;
  static constexpr int kStage = (BM + BN) * BK;
  static constexpr int PA = BM * BK / 1024 / kWaves, PW = BN * BK / 1024 / kWaves;  // copies of a wave and stage
  static_assert(PA * kWaves * 1024 == BM * BK && PW * kWaves * 1024 == BN * BK, "whole copies");
  static_assert((BK == 128 || BK == 256) && ST >= 2, "");
  static __device__ __forceinline__ int turn(int row) { return BK == 128 ? (row >> 1) & 7 : row & 15; }
};

template <class T, bool BF16>
__global__ __launch_bounds__(T::kThreads) void tile_kernel(Gemm8Args a) {
  // One array: the compiler then leaves the reads of a stage to the waits below.  With an array per
  // stage it waits for every copy in flight before each stage's reads.
  __shared__ __attribute__((aligned(1024))) uint8_t sm[T::ST * T::kStage];
  const int lane = threadIdx.x & 63, r = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % T::WM, wn = wave / T::WM % T::WN, slice = wave / (T::WM * T::WN);
  // workgroups go to the 8 XCDs in turn: each takes a run of neighbouring tiles
  const int32_t all = a.tiles_m * a.tiles_n, each = all / 8, more = all % 8;
  const int32_t xcd = blockIdx.x % 8, nth = blockIdx.x / 8;
  const int32_t tile = xcd * each + (xcd < more ? xcd : more) + nth;
  const int32_t m0 = tile % a.tiles_m * T::BM, n0 = tile / a.tiles_m * T::BN;

  const Rsrc ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(a.a) + (int64_t)m0 * a.lda, (short)0, -1, kRsrcFlags);
  const Rsrc rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(a.w) + (int64_t)n0 * a.ldw, (short)0, -1, kRsrcFlags);
  constexpr int kRows = 1024 / T::BK;  // rows of a copy
  uint32_t oa[T::PA], ow[T::PW];       // where this lane's rows begin; rows past the last one are read as that
  int32_t ka[T::PA], kw[T::PW];        // and its place in the stage's inputs
#pragma unroll
  for (int p = 0; p < T::PA; ++p) {
    const int row = (wave * T::PA + p) * kRows + lane / T::kChunks;
    oa[p] = (uint32_t)(m0 + row < a.M ? row : a.M - 1 - m0) * (uint32_t)a.lda;
    ka[p] = ((lane % T::kChunks) ^ T::turn(row)) * 16;
  }
#pragma unroll
  for (int p = 0; p < T::PW; ++p) {
    const int row = (wave * T::PW + p) * kRows + lane / T::kChunks;
    ow[p] = (uint32_t)(n0 + row < a.N ? row : a.N - 1 - n0) * (uint32_t)a.ldw;
    kw[p] = ((lane % T::kChunks) ^ T::turn(row)) * 16;
  }
  auto issue = [&](uint8_t *dst, int32_t k0) {
    const int32_t last = a.K - 16;  // inputs past the row are read as its last ones and count as zero below
#pragma unroll
    for (int p = 0; p < T::PA; ++p) {
      const int32_t k = k0 + ka[p] < last ? k0 + ka[p] : last;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LdsPtr)(dst + (wave * T::PA + p) * 1024), 16, (int)(oa[p] + k), 0, 0, 0);
    }
#pragma unroll
    for (int p = 0; p < T::PW; ++p) {
      const int32_t k = k0 + kw[p] < last ? k0 + kw[p] : last;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (LdsPtr)(dst + T::BM * T::BK + (wave * T::PW + p) * 1024), 16,
                                               (int)(ow[p] + k), 0, 0, 0);
    }
  };

  int16v acc[T::TN][T::TM];
#pragma unroll
  for (int t = 0; t < T::TN; ++t)
#pragma unroll
    for (int u = 0; u < T::TM; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[t][u][i] = 0;
  // A step's operands are read while the step before is multiplied: two sets.
  int4v w[2][T::TN], x[2][T::TM];
  auto read = [&](const uint8_t *src, int s) __attribute__((always_inline)) {
    const uint8_t *xa = src + (wm * T::TM * 32 + r) * T::BK, *xw = src + (T::BM + wn * T::TN * 32 + r) * T::BK;
    const int place = ((2 * (slice * T::kSteps + s) + half) ^ T::turn(r)) * 16;
#pragma unroll
    for (int t = 0; t < T::TN; ++t) w[s % 2][t] = *reinterpret_cast<const int4v *>(xw + t * 32 * T::BK + place);
#pragma unroll
    for (int u = 0; u < T::TM; ++u) x[s % 2][u] = *reinterpret_cast<const int4v *>(xa + u * 32 * T::BK + place);
  };
  auto multiply = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < T::TN; ++t)
#pragma unroll
      for (int u = 0; u < T::TM; ++u)
        acc[t][u] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[s % 2][t], x[s % 2][u], acc[t][u], 0, 0, 0);
  };
  // The order of a step: one read after each of the first products.
  auto mixed = [&]() __attribute__((always_inline)) {
    constexpr int kReads = T::TN + T::TM, kProducts = T::TN * T::TM;
#pragma unroll
    for (int i = 0; i < (kProducts > kReads ? kProducts : kReads); ++i) {
      if (i < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (i < kProducts) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
  };

  constexpr int kAhead = T::ST - 1, kLoads = T::PA + T::PW;
  const int32_t stages = (a.K + T::BK - 1) / T::BK;
  for (int i = 0; i < kAhead && i < stages; ++i) issue(sm + i * T::kStage, i * T::BK);
  int32_t now = 0, next = kAhead * T::kStage;  // where stage j is, and where stage j + kAhead goes
  auto ready = [&](int32_t j) __attribute__((always_inline)) {
    // stage j has landed for all, and all have read stage j - 1
    if (j + kAhead - 1 < stages) wait_and_meet<(kAhead - 1) * kLoads>();
    else wait_and_meet<0>();
    if (j + kAhead < stages) issue(sm + next, (j + kAhead) * T::BK);
  };
  const int32_t whole = a.K / T::BK;
  static_assert(T::kSteps % 2 == 0, "the last step of a stage is in the second set");
  ready(0);
  read(sm, 0);
  for (int32_t j = 0; j < whole; ++j) {
#pragma unroll
    for (int s = 0; s + 1 < T::kSteps; ++s) {
      read(sm + now, s + 1);
      multiply(s);
      mixed();
    }
    now = now + T::kStage == T::ST * T::kStage ? 0 : now + T::kStage;
    next = next + T::kStage == T::ST * T::kStage ? 0 : next + T::kStage;
    ready(j + 1);       // while the last step's operands are in registers
    read(sm + now, 0);  // behind the last stage: read and not used
    multiply(T::kSteps - 1);
    mixed();
  }
  if (whole < stages) {
#pragma unroll
    for (int s = 0; s < T::kSteps; ++s) {
      if (s) read(sm + now, s);
#pragma unroll
      for (int t = 0; t < T::TN; ++t)
        if (whole * T::BK + 16 * (2 * (slice * T::kSteps + s) + half) >= a.K) w[s % 2][t] = int4v{0, 0, 0, 0};
      multiply(s);
    }
  }

  if constexpr (T::KS > 1) {  // the other slices' sums go to the first one through LDS
    constexpr int kSums = T::TN * T::TM * 4 * 64, kGroup = T::WM * T::WN;
    static_assert((T::KS - 1) * kGroup * kSums * 16 <= T::ST * T::kStage, "");
    wait_and_meet<0>();
    int4v *sums = reinterpret_cast<int4v *>(sm) + lane;
    if (slice) {
#pragma unroll
      for (int t = 0; t < T::TN; ++t)
#pragma unroll
        for (int u = 0; u < T::TM; ++u)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            sums[(wave - kGroup) * kSums + ((t * T::TM + u) * 4 + g) * 64] =
                int4v{acc[t][u][4 * g], acc[t][u][4 * g + 1], acc[t][u][4 * g + 2], acc[t][u][4 * g + 3]};
    }
    __syncthreads();
    if (slice) return;
#pragma unroll
    for (int q = 0; q + 1 < T::KS; ++q)
#pragma unroll
      for (int t = 0; t < T::TN; ++t)
#pragma unroll
        for (int u = 0; u < T::TM; ++u)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int4v v = sums[(wave + q * kGroup) * kSums + ((t * T::TM + u) * 4 + g) * 64];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][u][4 * g + i] += v[i];
          }
  }
  const int32_t mw = m0 + wm * T::TM * 32 + r, nw = n0 + wn * T::TN * 32 + half * 4;
  if (a.wide && n0 + T::BN <= a.N) {
    float4v sw[T::TN][4];
#pragma unroll
    for (int t = 0; t < T::TN; ++t)
#pragma unroll
      for (int g = 0; g < 4; ++g) __builtin_memcpy(&sw[t][g], a.sw + nw + t * 32 + g * 8, 16);
#pragma unroll
    for (int u = 0; u < T::TM; ++u) {
      const int32_t m = mw + u * 32;
      if (m >= a.M) continue;
      const float sa = a.sa[m];
      uint16_t *dst = a.y + (int64_t)m * a.ldy + nw;
#pragma unroll
      for (int t = 0; t < T::TN; ++t)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = down<BF16>((float)acc[t][u][4 * g + i] * (sa * sw[t][g][i]));
          *reinterpret_cast<uint2 *>(dst + t * 32 + g * 8) = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
        }
    }
    return;
  }
#pragma unroll
  for (int u = 0; u < T::TM; ++u)
#pragma unroll
    for (int t = 0; t < T::TN; ++t)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        store4<BF16>(a, mw + u * 32, nw + t * 32 + g * 8,
                     int4v{acc[t][u][4 * g], acc[t][u][4 * g + 1], acc[t][u][4 * g + 2], acc[t][u][4 * g + 3]});
}

template <class T, bool BF16>
void launch_tiles(Gemm8Args a, hipStream_t s) {
  a.tiles_m = (a.M + T::BM - 1) / T::BM, a.tiles_n = (a.N + T::BN - 1) / T::BN;
  hipLaunchKernelGGL((tile_kernel<T, BF16>), dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(T::kThreads), 0, s, a);
}

using Tile256x256 = TileShape<256, 256, 2, 4, 1, 128, 2>;
using Tile256x128 = TileShape<256, 128, 4, 2, 1, 128, 3>;
using Tile128x128 = TileShape<128, 128, 2, 2, 2, 128, 4>;
using Tile64x128 = TileShape<64, 128, 2, 2, 2, 128, 4>;
using Tile64x64 = TileShape<64, 64, 2, 2, 2, 128, 4>;
using Tile32x64 = TileShape<32, 64, 1, 2, 4, 256, 3>;
using Tile32x32 = TileShape<32, 32, 1, 1, 4, 256, 4>;

// The tile: how long the tiles' rounds of 256 CUs take (measured for 4096 inputs, while the
// device is not full, where a small tile waits for its copies and a large one for the products),
// and not less than the inputs' bytes.  Measured, us, 4096 inputs, from the largest tile down
// (- : not measured):
//    4 x 4096:     -   -  17  11.6   8.6  7.3  7.2      64 x 4096:     -  -  17  12.4  9.1  7.8  7.3
//  128 x 4096:    43   -  18  12.5   9.4  9.2  9.3     256 x 4096:    48 28  18  12.8 10.4   -    -
//  512 x 4096:    48  29  19  15.0  17.5   -    -      1024 x 4096:   49 30  25  26.4 32.5   -    -
// 2047 x 4096:    54  43  52  58    78     -    -      1024 x 14336:  67 77  96 101  124     -    -
// With 1024, 8192 and 14336 inputs too the tile chosen is the fastest of all, or within 7% of it
// (4 to 2047 tokens, 4096 to 28672 channels).  Only the order counts: as times the estimates are off away
// from 4096 inputs, since what a tile costs once grows with the inputs here (4 x 1024 x 8192: 16 by the
// rule, 7.6 measured).  A tile with room for the tokens twice over is left out, so up to 16 tokens
// have one tile only.
template <bool BF16>
void launch_gemm(const Gemm8Args &a, hipStream_t s) {
  constexpr struct {
    int32_t m, n;
    float us;
  } kind[] = {{32, 32, 7.2f}, {32, 64, 7.6f}, {64, 64, 9.1f}, {64, 128, 12.4f}, {128, 128, 17.9f}, {256, 128, 28.1f}, {256, 256, 42.4f}};
  const float bytes_us = ((float)a.M * (float)a.K + (float)a.N * (float)a.K + 2.0f * (float)a.M * (float)a.N) / 5.5e6f;
  int best = 0;
  float least = INFINITY;
  for (int i = 0; i < 7 && (i == 0 || kind[i].m < 2 * (int64_t)a.M); ++i) {
    const int64_t tiles = ((int64_t)a.M + kind[i].m - 1) / kind[i].m * (((int64_t)a.N + kind[i].n - 1) / kind[i].n);
    const float rounds_us = (float)((tiles + 255) / 256) * kind[i].us * (float)a.K / 4096.0f;
    const float us = (rounds_us > bytes_us ? rounds_us : bytes_us) + 0.1f * rounds_us;
    if (us < least) least = us, best = i;
  }
  switch (best) {
    case 0: return launch_tiles<Tile32x32, BF16>(a, s);
    case 1: return launch_tiles<Tile32x64, BF16>(a, s);
    case 2: return launch_tiles<Tile64x64, BF16>(a, s);
    case 3: return launch_tiles<Tile64x128, BF16>(a, s);
    case 4: return launch_tiles<Tile128x128, BF16>(a, s);
    case 5: return launch_tiles<Tile256x128, BF16>(a, s);
    default: return launch_tiles<Tile256x256, BF16>(a, s);
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
  // rows of a tile are reached by 32-bit offsets, and tiles counted in 32 bits
  if (lda >= 1 << 23 || ldw >= 1 << 23 || ((int64_t)M + 31) / 32 * (((int64_t)N + 31) / 32) >= 1 << 23) return MIXLLM_E_SHAPE;
  const Gemm8Args g = {aq, w, sa, sw, static_cast<uint16_t *>(y), lda, ldw, ldy, M, N, K, 0, 0,
                       ldy % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & 7) == 0};
  if (dtype == MIXLLM_BF16) launch_gemm<true>(g, (hipStream_t)stream);
  else launch_gemm<false>(g, (hipStream_t)stream);
  return mixllm::launch_status();
}
