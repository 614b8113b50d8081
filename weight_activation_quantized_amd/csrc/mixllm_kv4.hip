// The paged key/value cache held in 4 bits: the plan of a step (block tables and slot maps
// from request lengths), the write of new tokens and the read back of tokens.
//
// The pages time linear layers only; they name a quantized cache as orthogonal to the
// layer's quantization (talk notes, KV 量子化との直交性) and describe no kernel for it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm_kv4.h"

namespace {

// ---------------------------------------------------------------------------------------
// The plan.
//
// Everything is a prefix sum over the requests (pages given back, pages needed, tokens
// added) and then a scatter of independent items.  The traffic is a few bytes per request
// and 8 bytes per token, so the time is latency: the sums run in one workgroup, whose
// threads also move the pages (found by bisection in the prefix sums held in LDS, so one
// long request's pages spread over all threads).
// ---------------------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;

struct PlanArgs {
  const int32_t *fresh, *lens, *count;
  int32_t *table, *pool, *lens_out, *count_out, *cu, *slots, *pos;
  int64_t ldt;
  int32_t B, width, F, page_log2, pages, tokens;
};

// Inclusive sum over a wave's lanes.
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t u = __shfl_up(v, d);
    if ((int)(threadIdx.x & 63) >= d) v += u;
  }
  return v;
}

// Exclusive sum over the workgroup; `total` gets the sum of all.  `tmp`: kPlanWaves words.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *tmp, int64_t *total) {
  const int wave = threadIdx.x >> 6;
  const int64_t inc = wave_scan(v);
  __syncthreads();  // tmp may still be read from the last call
  if ((threadIdx.x & 63) == 63) tmp[wave] = inc;
  __syncthreads();
  int64_t base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const int64_t t = tmp[w];
    if (w < wave) base += t;
    sum += t;
  }
  *total = sum;
  return base + inc - v;
}

// Last index i of [0, n) with first[i] <= k (first ascending, first[0] <= k).
__device__ __forceinline__ int find(const int32_t *first, int n, int32_t k) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= k) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t slot_of(const PlanArgs &a, int b, int32_t p) {
  const int32_t pg = a.table[b * a.ldt + (p >> a.page_log2)];
  return (uint32_t)pg < (uint32_t)a.pages ? (pg << a.page_log2) + (p & ((1 << a.page_log2) - 1)) : -1;
}

// Slot and position of the tokens t of [t0, tokens) in steps of `step`, except the first of
// each request, which the sums' kernel wrote: the position of a token is that of its
// request's first one plus its distance from it, and a request without a slot for its first
// token has none for the others.
__device__ __forceinline__ void plan_tokens(const PlanArgs &a, int32_t t0, int32_t step) {
  const int32_t total = a.cu[a.B];
  for (int64_t t = t0; t < a.tokens; t += step) {
    if (t >= total) {
      a.slots[t] = -1;
      a.pos[t] = 0;
      continue;
    }
    const int b = find(a.cu, a.B, (int32_t)t);
    const int32_t first = a.cu[b];
    if (t == first) continue;
    const int32_t p = a.pos[first] + ((int32_t)t - first);
    a.pos[t] = p;
    a.slots[t] = a.slots[first] < 0 ? -1 : slot_of(a, b, p);
  }
}

template <bool TOKENS>
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs a) {
  __shared__ int64_t tmp[kPlanWaves];
  __shared__ int32_t first[kPlanThreads], from[kPlanThreads], many[kPlanThreads];
  const int tid = threadIdx.x;
  const int32_t cap = a.width << a.page_log2, page = 1 << a.page_log2;  // fits: checked on the host
  int32_t count = *a.count;
  count = count < 0 ? 0 : count > a.F ? a.F : count;

  // Pages of requests that ended go on top of the free ones, in the order of the requests.
  int64_t given = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid, n = a.B - b0 < kPlanThreads ? a.B - b0 : kPlanThreads;
    int32_t have = 0;
    if (b < a.B && a.fresh[b] < 0) {
      const int32_t held = a.lens[b] < 0 ? 0 : a.lens[b] < cap ? a.lens[b] : cap;
      have = (int32_t)(((uint32_t)held + page - 1) >> a.page_log2);
    }
    int64_t sum;
    first[tid] = (int32_t)block_scan(have, tmp, &sum);
    __syncthreads();
    for (int32_t k = tid; k < sum; k += kPlanThreads) {
      const int i = find(first, n, k);
      const int64_t at = count + given + k;
      if (at < a.F) a.pool[at] = a.table[(int64_t)(b0 + i) * a.ldt + (k - first[i])];
    }
    given += sum;
    __syncthreads();
  }
  const int32_t top = (int32_t)(count + given < a.F ? count + given : a.F);

  // New pages come from the top, request by request; from the first request on that the
  // pool cannot serve, none that needs a page gets one.
  int64_t needed = 0, rows = 0;
  int32_t taken = 0, refused = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid, n = a.B - b0 < kPlanThreads ? a.B - b0 : kPlanThreads;
    const bool in = b < a.B;
    const int32_t f = in ? a.fresh[b] : 0;
    const int32_t len = in ? a.lens[b] : 0;
    const int32_t held = len < 0 ? 0 : len < cap ? len : cap;
    const int32_t add = f > 0 ? f : 0;
    const bool ended = f < 0, fits = add <= cap - held;
    const int32_t have = (int32_t)(((uint32_t)held + page - 1) >> a.page_log2);
    const int32_t need = ended || !fits ? 0 : (int32_t)(((uint32_t)(held + add) + page - 1) >> a.page_log2) - have;
    int64_t sum, sum_add;
    const int64_t pre = needed + block_scan(need, tmp, &sum);
    const int64_t row = rows + block_scan(add, tmp, &sum_add);
    const bool ok = ended || (fits && (need == 0 || pre + need <= top));
    first[tid] = (int32_t)(pre - needed);
    from[tid] = have;
    many[tid] = ok ? need : 0;
    if (ok && need > 0) taken = (int32_t)(pre + need);
    if (in) {
      refused += !ok;
      a.lens_out[b] = ended ? 0 : ok ? held + add : held;
      a.cu[b] = (int32_t)(row < 0x7FFFFFFF ? row : 0x7FFFFFFF);
    }
    __syncthreads();
    for (int32_t k = tid; k < sum; k += kPlanThreads) {
      const int i = find(first, n, k);
      if (k - first[i] < many[i])
        a.table[(int64_t)(b0 + i) * a.ldt + from[i] + (k - first[i])] = a.pool[top - 1 - needed - k];
    }
    needed += sum;
    rows += sum_add;
    __syncthreads();  // the pages above are in the table before the slots read it
    if (in && add > 0 && row < a.tokens) {
      a.pos[row] = held;
      a.slots[row] = ok ? slot_of(a, b, held) : -1;
    }
  }
  if (tid == 0) a.cu[a.B] = (int32_t)(rows < 0x7FFFFFFF ? rows : 0x7FFFFFFF);
  int64_t out;
  block_scan(refused, tmp, &out);
  // taken is the same prefix sum in every thread that has one: the largest is the last
  __syncthreads();
  if (tid == 0) first[0] = 0;
  __syncthreads();
  atomicMax(&first[0], taken);
  __syncthreads();
  if (tid == 0) {
    a.count_out[0] = top - first[0];
    a.count_out[1] = (int32_t)out;
  }
  if (TOKENS) plan_tokens(a, tid, kPlanThreads);
}

__global__ __launch_bounds__(256) void plan_tokens_kernel(PlanArgs a) {
  plan_tokens(a, (int32_t)(blockIdx.x * 256 + threadIdx.x), (int32_t)(gridDim.x * 256));
}

// Up to this many token rows the sums' workgroup writes them itself.
constexpr int32_t kPlanOneLaunch = 4096;

// ---------------------------------------------------------------------------------------
// The write and the read back.
//
// A quarter wave (16 lanes) owns one head of one token; a wave owns one head of four
// consecutive rows.  Keys: lane i holds channels i * D/16 .. (one wide load), the minimum
// and maximum of a group of 64 go over 64 / (D/16) lanes.  Values: lane n holds channels
// 16 j + n, so its word is complete and the four quarters' words of consecutive tokens are
// neighbours in the cache.
// ---------------------------------------------------------------------------------------

constexpr int kDppXor1 = 0xB1;        // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;        // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;
constexpr int kDppMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Minimum and maximum over LANES (4, 8 or 16) neighbouring lanes of a quarter.
template <int LANES>
__device__ __forceinline__ void lanes_minmax(float &lo, float &hi) {
  lo = fminf(lo, dpp<kDppXor1>(lo));
  hi = fmaxf(hi, dpp<kDppXor1>(hi));
  lo = fminf(lo, dpp<kDppXor2>(lo));
  hi = fmaxf(hi, dpp<kDppXor2>(hi));
  if (LANES >= 8) {
    lo = fminf(lo, dpp<kDppHalfMirror>(lo));
    hi = fmaxf(hi, dpp<kDppHalfMirror>(hi));
  }
  if (LANES >= 16) {
    lo = fminf(lo, dpp<kDppMirror>(lo));
    hi = fmaxf(hi, dpp<kDppMirror>(hi));
  }
}

template <bool BF16>
__device__ __forceinline__ float to_f32(uint32_t bits) {
  if (BF16) return __uint_as_float(bits << 16);
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

template <bool BF16>
__device__ __forceinline__ uint32_t from_f32(float v) {
  if (BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

// NaN becomes 0 and infinities the largest fp16: a cache never holds a parameter that is
// not finite, so a token that a row does not see cannot reach the row's sums.
__device__ __forceinline__ float tame(float x) {
  return x != x ? 0.0f : fminf(fmaxf(x, -65504.0f), 65504.0f);
}

struct Group {
  float s, m;
  uint32_t s16, m16;
};

// Scale and minimum of a group, every step in fp32 with IEEE division, stored as fp16.
__device__ __forceinline__ Group group_of(float lo, float hi) {
  Group g;
  g.m16 = from_f32<false>(lo);
  g.s16 = from_f32<false>((hi - lo) / 15.0f);
  if (g.s16 == 0 && hi > lo) g.s16 = 1;  // 2^-24
  g.m = to_f32<false>(g.m16);
  g.s = to_f32<false>(g.s16);
  return g;
}

__device__ __forceinline__ uint32_t code_of(float x, const Group &g) {
  if (g.s16 == 0) return 0;
  return (uint32_t)fminf(fmaxf(__builtin_rintf((x - g.m) / g.s), 0.0f), 15.0f);
}

struct TokenArgs {
  uint8_t *cache;
  const int32_t *slots;
  uint16_t *k, *v;
  int64_t ldk, ldv;
  int32_t T, heads, pages, page, page_log2;
};

// The cache block of this quarter's (row, head), or nullptr where there is nothing to do;
// `tok` is the token's place in its page.
template <int D>
__device__ __forceinline__ uint8_t *block_of(const TokenArgs &a, int32_t row, int32_t head, int32_t &tok) {
  const int32_t slot = row < a.T ? a.slots[row] : -1;
  if ((uint32_t)slot >= (uint32_t)(a.pages * a.page)) return nullptr;
  const int32_t pg = slot >> a.page_log2;
  tok = slot & (a.page - 1);
  return a.cache + ((int64_t)pg * a.heads + head) * mixllm::kv4_block_bytes(a.page, D);
}

// Byte of lane i's key codes inside a token's D/2 bytes.
template <int D>
__device__ __forceinline__ int key_byte(int i) {
  if (D == 64) return (i & 7) / 2 * (D / 8) + (i >> 3) * 4 + (i & 1) * 2;
  if (D == 128) return (i & 3) * (D / 8) + (i >> 2) * 4;
  return (i & 1) * 2 * (D / 8) + (i >> 1) * 4;  // D = 256: this dword and the one D/8 bytes on
}

template <int D, bool BF16>
__global__ __launch_bounds__(256) void kv4_append_kernel(TokenArgs a) {
  constexpr int C = D / 16, G = D / 64;
  const int i = threadIdx.x & 15;
  const int32_t row = blockIdx.x * 16 + (threadIdx.x >> 4), head = blockIdx.y;
  int32_t tok = 0;
  uint8_t *blk = block_of<D>(a, row, head, tok);
  if (!blk) return;  // whole quarters leave: the lane moves below stay inside a quarter
  float x[C];
  uint32_t c[C];
  {  // keys
    const uint16_t *src = a.k + (int64_t)row * a.ldk + head * D + i * C;
    alignas(16) uint16_t raw[C];
    if (C == 4) *reinterpret_cast<uint2 *>(raw) = *reinterpret_cast<const uint2 *>(src);
    if (C >= 8) *reinterpret_cast<uint4 *>(raw) = *reinterpret_cast<const uint4 *>(src);
    if (C == 16) *reinterpret_cast<uint4 *>(raw + 8) = *reinterpret_cast<const uint4 *>(src + 8);
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      x[j] = tame(to_f32<BF16>(raw[j]));
      lo = fminf(lo, x[j]);
      hi = fmaxf(hi, x[j]);
    }
    lanes_minmax<64 / C>(lo, hi);
    const Group g = group_of(lo, hi);
#pragma unroll
    for (int j = 0; j < C; ++j) c[j] = code_of(x[j], g);
    uint8_t *dst = blk + tok * (D / 2) + key_byte<D>(i);
#pragma unroll
    for (int w = 0; w < (C + 7) / 8; ++w) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < (C < 8 ? C : 8); ++j) word |= c[8 * w + j] << (4 * j);
      if (C == 4) *reinterpret_cast<uint16_t *>(dst) = (uint16_t)word;
      else *reinterpret_cast<uint32_t *>(dst + w * (D / 8)) = word;
    }
    if (i % (64 / C) == 0) {
      uint16_t *par = reinterpret_cast<uint16_t *>(blk + a.page * D + tok * (4 * G));
      par[i / (64 / C)] = (uint16_t)g.s16;
      par[G + i / (64 / C)] = (uint16_t)g.m16;
    }
  }
  {  // values
    const uint16_t *src = a.v + (int64_t)row * a.ldv + head * D + i;
#pragma unroll
    for (int j = 0; j < C; ++j) x[j] = tame(to_f32<BF16>(src[16 * j]));
    uint32_t word[(C + 7) / 8] = {};
    uint16_t *par = reinterpret_cast<uint16_t *>(blk + a.page * D + a.page * (D / 16) + tok * (4 * G));
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float lo = fminf(fminf(x[4 * g], x[4 * g + 1]), fminf(x[4 * g + 2], x[4 * g + 3]));
      float hi = fmaxf(fmaxf(x[4 * g], x[4 * g + 1]), fmaxf(x[4 * g + 2], x[4 * g + 3]));
      lanes_minmax<16>(lo, hi);
      const Group p = group_of(lo, hi);
#pragma unroll
      for (int j = 4 * g; j < 4 * g + 4; ++j) word[j / 8] |= code_of(x[j], p) << (4 * (j % 8));
      if (i == 0) {
        par[g] = (uint16_t)p.s16;
        par[G + g] = (uint16_t)p.m16;
      }
    }
    uint8_t *dst = blk + a.page * (D / 2) + ((tok / 4 * 16 + i) * 4 + tok % 4) * (D / 32);
    if (C == 4) *reinterpret_cast<uint16_t *>(dst) = (uint16_t)word[0];
    if (C == 8) *reinterpret_cast<uint32_t *>(dst) = word[0];
    if (C == 16) *reinterpret_cast<uint2 *>(dst) = make_uint2(word[0], word[(C + 7) / 8 - 1]);
  }
}

// x = m + s c: the product is exact in fp32, so is rounded once there and once to 16 bits.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void kv4_read_kernel(TokenArgs a) {
  constexpr int C = D / 16, G = D / 64;
  const int i = threadIdx.x & 15;
  const int32_t row = blockIdx.x * 16 + (threadIdx.x >> 4), head = blockIdx.y;
  int32_t tok = 0;
  const uint8_t *blk = block_of<D>(a, row, head, tok);
  if (!blk) return;
  {
    const uint16_t *par = reinterpret_cast<const uint16_t *>(blk + a.page * D + tok * (4 * G));
    const float s = to_f32<false>(par[i / (64 / C)]), m = to_f32<false>(par[G + i / (64 / C)]);
    const uint8_t *src = blk + tok * (D / 2) + key_byte<D>(i);
    alignas(16) uint16_t out[C];
#pragma unroll
    for (int w = 0; w < (C + 7) / 8; ++w) {
      const uint32_t word = C == 4 ? *reinterpret_cast<const uint16_t *>(src)
                                   : *reinterpret_cast<const uint32_t *>(src + w * (D / 8));
#pragma unroll
      for (int j = 0; j < (C < 8 ? C : 8); ++j)
        out[8 * w + j] = (uint16_t)from_f32<BF16>(m + s * (float)((word >> (4 * j)) & 15));
    }
    uint16_t *dst = a.k + (int64_t)row * a.ldk + head * D + i * C;
    if (C == 4) *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(out);
    if (C >= 8) *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<uint4 *>(out);
    if (C == 16) *reinterpret_cast<uint4 *>(dst + 8) = *reinterpret_cast<uint4 *>(out + 8);
  }
  {
    const uint16_t *par = reinterpret_cast<const uint16_t *>(blk + a.page * D + a.page * (D / 16) + tok * (4 * G));
    const uint8_t *src = blk + a.page * (D / 2) + ((tok / 4 * 16 + i) * 4 + tok % 4) * (D / 32);
    uint16_t *dst = a.v + (int64_t)row * a.ldv + head * D + i;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t c = (src[j / 2] >> (4 * (j & 1))) & 15;
      dst[16 * j] = (uint16_t)from_f32<BF16>(to_f32<false>(par[G + j / 4]) + to_f32<false>(par[j / 4]) * (float)c);
    }
  }
}

int check_tokens(const void *k, const void *v, int64_t ldk, int64_t ldv, int32_t dtype, const int32_t *slots, int32_t T,
                 const void *cache, size_t cache_bytes, int32_t pages, int32_t page, int32_t heads, int32_t dim) {
  if (T < 0 || (dtype != MIXLLM_FP16 && dtype != MIXLLM_BF16)) return MIXLLM_E_SHAPE;
  if (T == 0) return MIXLLM_OK;
  const int st = mixllm::kv4_check_cache(cache, cache_bytes, pages, page, heads, dim);
  if (st != MIXLLM_OK) return st;
  const int64_t width = (int64_t)heads * dim;
  if (heads > 65535 || ldk < width || ldv < width || ldk % 8 != 0 || ldv % 8 != 0) return MIXLLM_E_SHAPE;
  if (!k || !v || !slots) return MIXLLM_E_NULL;
  if (!mixllm::is_aligned16(k) || !mixllm::is_aligned16(v) || !mixllm::is_aligned4(slots)) return MIXLLM_E_SHAPE;
  return MIXLLM_OK;
}

template <bool APPEND, int D>
void launch_tokens(const TokenArgs &a, int32_t dtype, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)a.T + 15) / 16), (unsigned)a.heads);
  if (APPEND) {
    if (dtype == MIXLLM_BF16) hipLaunchKernelGGL((kv4_append_kernel<D, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((kv4_append_kernel<D, false>), grid, dim3(256), 0, stream, a);
  } else {
    if (dtype == MIXLLM_BF16) hipLaunchKernelGGL((kv4_read_kernel<D, true>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((kv4_read_kernel<D, false>), grid, dim3(256), 0, stream, a);
  }
}

template <bool APPEND>
int run_tokens(const TokenArgs &a, int32_t dim, int32_t dtype, void *stream) {
  if (dim == 64) launch_tokens<APPEND, 64>(a, dtype, (hipStream_t)stream);
  else if (dim == 128) launch_tokens<APPEND, 128>(a, dtype, (hipStream_t)stream);
  else launch_tokens<APPEND, 256>(a, dtype, (hipStream_t)stream);
  return mixllm::launch_status();
}

}  // namespace

extern "C" size_t mixllm_kv4_page_bytes(int32_t page, int32_t heads, int32_t dim) {
  if (!mixllm::kv4_dim_ok(dim) || !mixllm::kv4_page_ok(page) || heads <= 0) return 0;
  return (size_t)heads * mixllm::kv4_block_bytes(page, dim);
}

extern "C" int mixllm_kv_plan(const int32_t *fresh, const int32_t *lens, int32_t B, int32_t *table, int64_t ldt,
                              int32_t width, int32_t *pool, int32_t F, const int32_t *count, int32_t page,
                              int32_t pages, int32_t *lens_out, int32_t *count_out, int32_t *cu, int32_t *slots,
                              int32_t *pos, int32_t tokens, void *stream) {
  if (B < 0 || tokens < 0 || F < 0 || width <= 0 || ldt < width || pages <= 0 || !mixllm::kv4_page_ok(page))
    return MIXLLM_E_SHAPE;
  if ((int64_t)pages * page > 0x7FFFFFFF || (int64_t)width * page > 0x7FFFFFFF ||
      (int64_t)B * width > 0x7FFFFFFF || B > 0x7FFFFFFF - kPlanThreads)
    return MIXLLM_E_SHAPE;
  if (!count || !count_out || !cu || (F && !pool) || (B && (!fresh || !lens || !table || !lens_out)) ||
      (tokens && (!slots || !pos)))
    return MIXLLM_E_NULL;
  const void *all[] = {fresh, lens, table, pool, count, lens_out, count_out, cu, slots, pos};
  for (const void *p : all)
    if (!mixllm::is_aligned4(p)) return MIXLLM_E_SHAPE;
  const PlanArgs a = {fresh, lens, count, table, pool, lens_out, count_out, cu, slots, pos, ldt, B, width, F,
                      mixllm::log2_of(page), pages, tokens};
  if (tokens <= kPlanOneLaunch) {
    hipLaunchKernelGGL((plan_kernel<true>), dim3(1), dim3(kPlanThreads), 0, (hipStream_t)stream, a);
    return mixllm::launch_status();
  }
  hipLaunchKernelGGL((plan_kernel<false>), dim3(1), dim3(kPlanThreads), 0, (hipStream_t)stream, a);
  const int st = mixllm::launch_status();
  if (st != MIXLLM_OK) return st;
  const int32_t blocks = (tokens - 1) / 256 + 1;
  hipLaunchKernelGGL(plan_tokens_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0,
                     (hipStream_t)stream, a);
  return mixllm::launch_status();
}

extern "C" int mixllm_kv4_append(const void *k, int64_t ldk, const void *v, int64_t ldv, int32_t dtype,
                                 const int32_t *slots, int32_t T, void *cache, size_t cache_bytes, int32_t pages,
                                 int32_t page, int32_t heads, int32_t dim, void *stream) {
  const int st = check_tokens(k, v, ldk, ldv, dtype, slots, T, cache, cache_bytes, pages, page, heads, dim);
  if (st != MIXLLM_OK || T == 0) return st;
  const TokenArgs a = {static_cast<uint8_t *>(cache), slots,
                       const_cast<uint16_t *>(static_cast<const uint16_t *>(k)),
                       const_cast<uint16_t *>(static_cast<const uint16_t *>(v)), ldk, ldv, T, heads, pages, page,
                       mixllm::log2_of(page)};
  return run_tokens<true>(a, dim, dtype, stream);
}

extern "C" int mixllm_kv4_read(const void *cache, size_t cache_bytes, int32_t pages, int32_t page, int32_t heads,
                               int32_t dim, const int32_t *slots, int32_t T, void *k, int64_t ldk, void *v,
                               int64_t ldv, int32_t dtype, void *stream) {
  const int st = check_tokens(k, v, ldk, ldv, dtype, slots, T, cache, cache_bytes, pages, page, heads, dim);
  if (st != MIXLLM_OK || T == 0) return st;
  const TokenArgs a = {const_cast<uint8_t *>(static_cast<const uint8_t *>(cache)), slots,
                       static_cast<uint16_t *>(k), static_cast<uint16_t *>(v), ldk, ldv, T, heads, pages, page,
                       mixllm::log2_of(page)};
  return run_tokens<false>(a, dim, dtype, stream);
}
