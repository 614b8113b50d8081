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
typedef float float4v __attribute__((ext_vector_type(4)));

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

// Few tokens: the weights are read once, straight into the matrix instruction's operands.  A
// workgroup takes 16 NT channels and 16 MT tokens, its 8 waves blocks of 64 S inputs in turn, and
// adds their sums through LDS.
constexpr int kStreamWaves = 8;

template <int MT, int NT, bool BF16>
__global__ __launch_bounds__(64 * kStreamWaves) void stream_kernel(Gemm8Args a) {
  constexpr int S = MT > 2 ? 2 : 4, kStreamBlock = 64 * S;
  __shared__ int4v red[kStreamWaves][NT * MT][64];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t n0 = blockIdx.x * (16 * NT);
  const int8_t *pw[NT], *pa[MT];
#pragma unroll
  for (int t = 0; t < NT; ++t) pw[t] = a.w + (int64_t)(n0 + 16 * t + r < a.N ? n0 + 16 * t + r : a.N - 1) * a.ldw;
#pragma unroll
  for (int u = 0; u < MT; ++u) pa[u] = a.a + (int64_t)(16 * u + r < a.M ? 16 * u + r : a.M - 1) * a.lda;
  struct Block {
    int4v w[NT][S], x[MT][S];
  };
  auto load = [&](Block &b, int32_t k0) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      int32_t k = k0 + 64 * s + 16 * c;
      k = k < a.K ? k : a.K - 16;  // what is past the row counts as zero below
#pragma unroll
      for (int t = 0; t < NT; ++t) b.w[t][s] = *reinterpret_cast<const int4v *>(pw[t] + k);
#pragma unroll
      for (int u = 0; u < MT; ++u) b.x[u][s] = *reinterpret_cast<const int4v *>(pa[u] + k);
    }
  };
  int4v acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < MT; ++u) acc[t][u] = int4v{0, 0, 0, 0};
  auto add = [&](Block &b, int32_t k0) {
    if (k0 + kStreamBlock > a.K) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (k0 + 64 * s + 16 * c >= a.K) b.w[t][s] = int4v{0, 0, 0, 0};
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < MT; ++u)
          acc[t][u] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b.w[t][s], b.x[u][s], acc[t][u], 0, 0, 0);
  };
  constexpr int32_t kStep = kStreamWaves * kStreamBlock;
  int32_t k = wave * kStreamBlock;
  if (k < a.K) {
    Block b0, b1;
    load(b0, k);
    for (;;) {
      if (k + kStep < a.K) load(b1, k + kStep);
      __builtin_amdgcn_sched_barrier(0);
      add(b0, k);
      if ((k += kStep) >= a.K) break;
      if (k + kStep < a.K) load(b0, k + kStep);
      __builtin_amdgcn_sched_barrier(0);
      add(b1, k);
      if ((k += kStep) >= a.K) break;
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < MT; ++u) red[wave][t * MT + u][lane] = acc[t][u];
  __syncthreads();
  for (int e = threadIdx.x; e < NT * MT * 64; e += 64 * kStreamWaves) {
    const int tile = e >> 6, l = e & 63;
    int4v sum = red[0][tile][l];
#pragma unroll
    for (int w = 1; w < kStreamWaves; ++w) sum += red[w][tile][l];
    store4<BF16>(a, tile % MT * 16 + (l & 15), n0 + tile / MT * 16 + (l >> 4) * 4, sum);
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

template <int N>
struct Const {
  static constexpr int value = N;
};

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
  static_assert((BK == 64 || BK == 128) && ST >= 2 && ST <= 4, "");
  static __device__ __forceinline__ int turn(int row) { return BK == 64 ? (row >> 2) & 3 : (row >> 1) & 7; }
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
  auto compute = [&](const uint8_t *src, auto last, int32_t k0) __attribute__((always_inline)) {
    const uint8_t *xa = src + (wm * T::TM * 32 + r) * T::BK, *xw = src + (T::BM + wn * T::TN * 32 + r) * T::BK;
#pragma unroll
    for (int s = 0; s < T::kSteps; ++s) {
      const int chunk = 2 * (slice * T::kSteps + s) + half, place = (chunk ^ T::turn(r)) * 16;
      int4v w[T::TN], x[T::TM];
#pragma unroll
      for (int t = 0; t < T::TN; ++t) w[t] = *reinterpret_cast<const int4v *>(xw + t * 32 * T::BK + place);
#pragma unroll
      for (int u = 0; u < T::TM; ++u) x[u] = *reinterpret_cast<const int4v *>(xa + u * 32 * T::BK + place);
      if constexpr (decltype(last)::value) {
#pragma unroll
        for (int t = 0; t < T::TN; ++t)
          if (k0 + 16 * chunk >= a.K) w[t] = int4v{0, 0, 0, 0};
      }
#pragma unroll
      for (int t = 0; t < T::TN; ++t)
#pragma unroll
        for (int u = 0; u < T::TM; ++u) acc[t][u] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[t], x[u], acc[t][u], 0, 0, 0);
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
  for (int32_t j = 0; j < whole; ++j) {
    ready(j);
    compute(sm + now, Const<0>(), 0);
    now = now + T::kStage == T::ST * T::kStage ? 0 : now + T::kStage;
    next = next + T::kStage == T::ST * T::kStage ? 0 : next + T::kStage;
  }
  if (whole < stages) {
    ready(whole);
    compute(sm + now, Const<1>(), whole * T::BK);
  }

  if constexpr (T::KS == 2) {  // the second slice's sums go to the first one through LDS
    static_assert(T::TN * T::TM * 1024 * T::WM * T::WN * 4 <= T::ST * T::kStage, "");
    wait_and_meet<0>();
    int4v *mine = reinterpret_cast<int4v *>(sm) + wave % (T::WM * T::WN) * (T::TN * T::TM * 256) + lane;
    if (slice == 1) {
#pragma unroll
      for (int t = 0; t < T::TN; ++t)
#pragma unroll
        for (int u = 0; u < T::TM; ++u)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            mine[((t * T::TM + u) * 4 + g) * 64] =
                int4v{acc[t][u][4 * g], acc[t][u][4 * g + 1], acc[t][u][4 * g + 2], acc[t][u][4 * g + 3]};
    }
    __syncthreads();
    if (slice == 1) return;
#pragma unroll
    for (int t = 0; t < T::TN; ++t)
#pragma unroll
      for (int u = 0; u < T::TM; ++u)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int4v v = mine[((t * T::TM + u) * 4 + g) * 64];
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

template <int MT, int NT, bool BF16>
void launch_stream(const Gemm8Args &a, hipStream_t s) {
  hipLaunchKernelGGL((stream_kernel<MT, NT, BF16>), dim3((unsigned)((a.N + 16 * NT - 1) / (16 * NT))),
                     dim3(64 * kStreamWaves), 0, s, a);
}

using Large = TileShape<256, 256, 2, 4, 1, 64, 4>;
using Middle = TileShape<128, 128, 2, 2, 2, 128, 4>;
using Small = TileShape<64, 128, 2, 2, 2, 128, 3>;

template <bool BF16>
void launch_gemm(const Gemm8Args &a, hipStream_t s) {
  if (a.M <= 16) {
    if (a.N >= 16384) launch_stream<1, 4, BF16>(a, s);
    else if (a.N >= 8192) launch_stream<1, 2, BF16>(a, s);
    else launch_stream<1, 1, BF16>(a, s);
  } else if (a.M <= 32) {
    launch_stream<2, 2, BF16>(a, s);
  } else if (a.M <= 64) {
    launch_stream<4, 2, BF16>(a, s);
  } else {
    auto tiles = [&](int64_t bm, int64_t bn) { return (a.M + bm - 1) / bm * ((a.N + bn - 1) / bn); };
    if (tiles(256, 256) >= 200) launch_tiles<Large, BF16>(a, s);
    else if (tiles(128, 128) >= 200) launch_tiles<Middle, BF16>(a, s);
    else launch_tiles<Small, BF16>(a, s);
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
  if (lda >= 1 << 23 || ldw >= 1 << 23 || ((int64_t)M + 63) / 64 * (((int64_t)N + 15) / 16) >= 1 << 23) return MIXLLM_E_SHAPE;
  const Gemm8Args g = {aq, w, sa, sw, static_cast<uint16_t *>(y), lda, ldw, ldy, M, N, K, 0, 0,
                       ldy % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & 7) == 0};
  if (dtype == MIXLLM_BF16) launch_gemm<true>(g, (hipStream_t)stream);
  else launch_gemm<false>(g, (hipStream_t)stream);
  return mixllm::launch_status();
}
