// The paged key/value cache held in 4 bits: the plan of a step (block tables and slot maps
// from request lengths), the write of new tokens and the read back of tokens.
//
// The pages time linear layers only; they name a quantized cache as orthogonal to the
// layer's quantization (talk notes, KV 量子化との直交性) and describe no kernel for it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixllm_kv4.h"
#include "mixllm_lanes.h"

namespace {

using mixllm::down;
using mixllm::kDppHalfMirror;
using mixllm::kDppMirror;
using mixllm::kDppXor1;
using mixllm::kDppXor2;
using mixllm::moved;
using mixllm::up;

// ---------------------------------------------------------------------------------------
// The plan.
//
// Everything is a prefix sum over the requests (pages given back, pages needed, tokens
// added) and then a scatter of independent items.  The traffic is a few bytes per request
// and 8 bytes per token, so the time is latency: the sums run in one workgroup, all of them
// at once and across lanes without LDS, and its threads also move the pages.  256 requests of
// one token: 5.1 us (0.1 of it the row limit's; the sums one after the other through LDS
// shuffles: 14.0 us; a launch alone takes about 4).
// ---------------------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;

struct PlanArgs {
  const int32_t *fresh, *lens, *count;
  int32_t *table, *pool, *lens_out, *count_out, *cu, *slots, *pos;
  int64_t ldt;
  int32_t B, width, F, page_log2, pages, tokens;
  int64_t room;  // rows that requests may have: one whose rows end behind it is refused
};

// Inclusive sum over the lanes of a wave: within rows of 16 lanes, then the rows' last
// lanes into the rows behind them.
template <int CTRL, int ROWS>
__device__ __forceinline__ int32_t shifted(int32_t v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int32_t row_scan(int32_t v) {
  v += shifted<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
  v += shifted<0x112, 0xF>(v);
  v += shifted<0x114, 0xF>(v);
  v += shifted<0x118, 0xF>(v);
  return v;
}
__device__ __forceinline__ int32_t wave_scan(int32_t v) {
  v = row_scan(v);
  v += shifted<0x142, 0xA>(v);  // row_bcast 15 into rows 1 and 3
  v += shifted<0x143, 0xC>(v);  // row_bcast 31 into rows 2 and 3
  return v;
}

// A request of this step.
struct Request {
  int32_t held, add, have, need;  // tokens, tokens to add, pages, more pages
  bool ended, fits;
};

__device__ __forceinline__ Request request_of(const PlanArgs &a, int32_t b) {
  const int32_t cap = a.width << a.page_log2, page = 1 << a.page_log2;  // fits: checked on the host
  const int32_t f = b < a.B ? a.fresh[b] : 0, len = b < a.B ? a.lens[b] : 0;
  Request r;
  r.held = len < 0 ? 0 : len < cap ? len : cap;
  r.add = f > 0 ? f : 0;
  r.ended = f < 0;
  r.fits = r.add <= cap - r.held;
  r.have = (int32_t)(((uint32_t)r.held + page - 1) >> a.page_log2);
  r.need = r.ended || !r.fits ? 0 : (int32_t)(((uint32_t)(r.held + r.add) + page - 1) >> a.page_log2) - r.have;
  return r;
}

// Sums over the requests before this one and over all of the workgroup's: pages given back,
// pages needed, and the tokens added in two halves (their sum may pass 32 bits).
struct Sums {
  int32_t back, need, low, high;
  __device__ __forceinline__ int64_t add() const { return ((int64_t)high << 16) + low; }
};

// `tmp`: a word per wave and sum, last read before the caller's next barrier.
__device__ __forceinline__ Sums block_scan(const Request &r, Sums *tmp, Sums *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Sums own = {r.ended ? r.have : 0, r.need, r.add & 0xFFFF, r.add >> 16};
  const Sums inc = {wave_scan(own.back), wave_scan(own.need), wave_scan(own.low), wave_scan(own.high)};
  if (lane == 63) tmp[wave] = inc;
  __syncthreads();
  // each row of 16 lanes sums the waves' totals
  Sums w = tmp[lane & 15];
  const Sums mine = w;
  w = {row_scan(w.back), row_scan(w.need), row_scan(w.low), row_scan(w.high)};
  auto at = [](int32_t v, int l) { return __builtin_amdgcn_readlane(v, l); };
  *total = {at(w.back, 15), at(w.need, 15), at(w.low, 15), at(w.high, 15)};
  const int u = __builtin_amdgcn_readfirstlane(wave);
  return {at(w.back - mine.back, u) + inc.back - own.back, at(w.need - mine.need, u) + inc.need - own.need,
          at(w.low - mine.low, u) + inc.low - own.low, at(w.high - mine.high, u) + inc.high - own.high};
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

__device__ __forceinline__ int32_t slot_on(const PlanArgs &a, int32_t pg, int32_t p) {
  return (uint32_t)pg < (uint32_t)a.pages ? (pg << a.page_log2) + (p & ((1 << a.page_log2) - 1)) : -1;
}

// Slot and position of the tokens t of [t0, tokens) in steps of `step`, except the first of
// each request, which the sums' kernel wrote: the position of a token is that of its
// request's first one plus its distance from it, and a request without a slot for its first
// token has none for the others.
__device__ __forceinline__ void plan_tokens(const PlanArgs &a, const int32_t *cu, int32_t t0, int32_t step) {
  const int32_t total = a.cu[a.B];
  for (int64_t t = t0; t < a.tokens; t += step) {
    if (t >= total) {
      a.slots[t] = -1;
      a.pos[t] = 0;
      continue;
    }
    const int b = find(cu, a.B, (int32_t)t);
    const int32_t first = cu[b];
    if (t == first) continue;
    const int32_t p = a.pos[first] + ((int32_t)t - first);
    a.pos[t] = p;
    a.slots[t] = a.slots[first] < 0 ? -1 : slot_on(a, a.table[b * a.ldt + (p >> a.page_log2)], p);
  }
}

template <bool TOKENS>
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs a) {
  __shared__ Sums tmp[2][kPlanWaves];
  __shared__ int32_t first[kPlanThreads], cu[kPlanThreads];
  __shared__ int32_t s_taken, s_refused;
  const int tid = threadIdx.x;
  if (tid == 0) s_taken = s_refused = 0;  // read after the first barrier
  int32_t count = *a.count;
  count = count < 0 ? 0 : count > a.F ? a.F : count;
  Request r = request_of(a, tid);
  // the page that the request's next token goes to, if the request has it
  int32_t tail = -1;
  if (r.add > 0 && r.held < r.have << a.page_log2) tail = a.table[tid * a.ldt + r.have - 1];

  // Pages of requests that ended go on top of the free ones, in the order of the requests.
  Sums sum;
  Sums pre = block_scan(r, tmp[0], &sum);
  const Sums sum0 = sum;
  int64_t given = 0;
  for (int b0 = 0;;) {
    const int n = a.B - b0 < kPlanThreads ? a.B - b0 : kPlanThreads;
    const int32_t back = b0 ? block_scan(request_of(a, b0 + tid), tmp[1], &sum).back : pre.back;
    first[tid] = back;
    __syncthreads();
    for (int32_t k = tid; k < sum.back; k += kPlanThreads) {
      const int i = find(first, n, k);
      const int64_t at = count + given + k;
      if (at < a.F) a.pool[at] = a.table[(int64_t)(b0 + i) * a.ldt + (k - first[i])];
    }
    given += sum.back;
    __syncthreads();  // the pool is complete, and first free
    if ((b0 += kPlanThreads) >= a.B) break;
  }
  const int32_t top = (int32_t)(count + given < a.F ? count + given : a.F);

  // New pages come from the top, request by request; from the first request on that the
  // pool cannot serve, none that needs a page gets one.
  int64_t needed = 0, rows = 0;
  bool more = false;  // a request has more than one token
  sum = sum0;
  for (int b0 = 0;;) {
    const int b = b0 + tid;
    const bool in = b < a.B;
    if (b0) {
      r = request_of(a, b);
      tail = r.add > 0 && r.held < r.have << a.page_log2 ? a.table[b * a.ldt + r.have - 1] : -1;
      pre = block_scan(r, tmp[0], &sum);
    }
    const int64_t before = needed + pre.need, row = rows + pre.add();
    const bool ok = r.ended || (r.fits && (r.need == 0 || before + r.need <= top) && (r.add == 0 || row + r.add <= a.room));
    if (in) {
      const int32_t at = (int32_t)(row < 0x7FFFFFFF ? row : 0x7FFFFFFF);
      if (ok && r.need > 0) atomicMax(&s_taken, (int32_t)(before + r.need));
      if (!ok) atomicAdd(&s_refused, 1);
      a.lens_out[b] = r.ended ? 0 : ok ? r.held + r.add : r.held;
      a.cu[b] = at;
      if (TOKENS && b0 == 0) cu[tid] = at;
      more = more || r.add > 1;
      if (r.add > 0 && row < a.tokens) {
        const bool fresh_page = r.held == r.have << a.page_log2;  // it starts a page
        a.pos[row] = r.held;
        a.slots[row] = !ok ? -1 : slot_on(a, fresh_page ? a.pool[top - 1 - before] : tail, r.held);
      }
    }
    // A wave hands out its 64 requests' pages: one page by the request's own thread, more by
    // all lanes, request after request (a bisection in the prefix sums for every page of the
    // workgroup took 4 us longer at 5100 pages).
    const int32_t gets = ok ? r.need : 0;
    if (gets == 1) a.table[b * a.ldt + r.have] = a.pool[top - 1 - before];
    for (uint64_t left = __ballot(gets > 1); left; left &= left - 1) {
      const int l = __builtin_ctzll(left);
      const int32_t pages = __builtin_amdgcn_readlane(gets, l), have = __builtin_amdgcn_readlane(r.have, l);
      const int32_t from = top - 1 - __builtin_amdgcn_readlane((int32_t)before, l);  // it gets pages: that fits
      int32_t *row = a.table + (int64_t)(b0 + (tid & ~63) + l) * a.ldt + have;
      for (int32_t j0 = tid & 63; j0 < pages; j0 += 256) {
        int32_t pg[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (j0 + 64 * u < pages) pg[u] = a.pool[from - j0 - 64 * u];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (j0 + 64 * u < pages) row[j0 + 64 * u] = pg[u];
      }
    }
    needed += sum.need;
    rows += sum.add();
    __syncthreads();
    if ((b0 += kPlanThreads) >= a.B) break;
  }
  const int32_t total = (int32_t)(rows < 0x7FFFFFFF ? rows : 0x7FFFFFFF);
  if (tid == 0) {
    a.cu[a.B] = total;
    a.count_out[0] = top - s_taken;
    a.count_out[1] = s_refused;
  }
  if (TOKENS) {
    if (__syncthreads_or(more)) {
      plan_tokens(a, a.B <= kPlanThreads ? cu : a.cu, tid, kPlanThreads);
    } else {  // every row is its request's first
      for (int64_t t = total + tid; t < a.tokens; t += kPlanThreads) {
        a.slots[t] = -1;
        a.pos[t] = 0;
      }
    }
  }
}

__global__ __launch_bounds__(256) void plan_tokens_kernel(PlanArgs a) {
  plan_tokens(a, a.cu, (int32_t)(blockIdx.x * 256 + threadIdx.x), (int32_t)(gridDim.x * 256));
}

// Up to this many token rows the sums' workgroup writes them itself.
constexpr int32_t kPlanOneLaunch = 4096;

// ---------------------------------------------------------------------------------------
// The write and the read back.
//
// A quarter wave (16 lanes) owns one head of one token; a wave owns one head of four
// consecutive rows.  Lane i loads channels i * D/16 .. at once, the minimum and maximum of a
// group of 64 go over 64 / (D/16) lanes.  Keys are stored from there; the values' codes change
// places through LDS so that lane n has channels 16 j + n: its word is then complete, and the
// four quarters' words of consecutive tokens are neighbours in the cache.  Long prompts are
// bound inside the unit: 8191 tokens of 8 heads of 128 take 18.5 us with divisions and fp32
// extremes, 15.3 as written, 12 of it without any store.  About half of that is vector operations
// (13 to 16 per value); the rest was not measured apart: the turn through LDS, a byte at a time,
// and two chains of lane moves, one after the other.  Reading them back takes 8.8.
// ---------------------------------------------------------------------------------------

// Minimum and maximum over LANES (4, 8 or 16) neighbouring lanes of a quarter.
template <int LANES>
__device__ __forceinline__ void lanes_minmax(float &lo, float &hi) {
  lo = fminf(lo, moved<kDppXor1>(lo));
  hi = fmaxf(hi, moved<kDppXor1>(hi));
  lo = fminf(lo, moved<kDppXor2>(lo));
  hi = fmaxf(hi, moved<kDppXor2>(hi));
  if (LANES >= 8) {
    lo = fminf(lo, moved<kDppHalfMirror>(lo));
    hi = fmaxf(hi, moved<kDppHalfMirror>(hi));
  }
  if (LANES >= 16) {
    lo = fminf(lo, moved<kDppMirror>(lo));
    hi = fmaxf(hi, moved<kDppMirror>(hi));
  }
}

// NaN becomes 0 and infinities the largest fp16: a cache never holds a parameter that is
// not finite, so a token that a row does not see cannot reach the row's sums.
__device__ __forceinline__ float tame(float x) {
  return x != x ? 0.0f : fminf(fmaxf(x, -65504.0f), 65504.0f);
}

struct Group {
  float s, m, r;  // r: about 1 / s, 0 where s is
  uint32_t s16, m16;
};

// Scale and minimum of a group, every step in fp32 with IEEE division, stored as fp16.  The
// division by 15 in three steps: q = x RN(1 / 15), then q plus the rounded remainder times
// RN(1 / 15), which is the correctly rounded quotient (so for every fp32 mantissa, tried one by
// one; quotients too small for that round to 0 in fp16).
__device__ __forceinline__ Group group_of(float lo, float hi) {
  Group g;
  g.m16 = down<false>(lo + 0.0f);  // -0 becomes 0
  const float x = hi - lo, q = x * (1.0f / 15.0f);
  g.s16 = down<false>(fmaf(fmaf(-15.0f, q, x), 1.0f / 15.0f, q));
  if (g.s16 == 0 && hi > lo) g.s16 = 1;  // 2^-24
  g.m = up<false>(g.m16);
  g.s = up<false>(g.s16);
  g.r = g.s16 ? __builtin_amdgcn_rcpf(g.s) : 0.0f;
  return g;
}

typedef int16_t short2v __attribute__((ext_vector_type(2)));

// A lane's C 16-bit values, of a group that LANES neighbouring lanes hold: the values as fp32
// and the group's parameters.  The extremes are found on the 16-bit patterns, two at a time,
// made to order as integers (the bits below a set sign flipped); across lanes the maximum and
// the complement of the minimum move as one word.  Where the extremes are not finite (or
// beyond fp16) the group's values are tamed first.
template <int C, int LANES, bool BF16>
__device__ __forceinline__ Group measure(const uint32_t (&raw)[C / 2], float (&x)[C]) {
  short2v hi = {-32768, -32768}, lo = {32767, 32767};
#pragma unroll
  for (int j = 0; j < C / 2; ++j) {
    const short2v w = __builtin_bit_cast(short2v, raw[j]);
    const short2v key = w ^ ((w >> 15) & short2v{32767, 32767});
    hi = __builtin_elementwise_max(hi, key);
    lo = __builtin_elementwise_min(lo, key);
    x[2 * j] = up<BF16>(raw[j] & 0xFFFFu);
    x[2 * j + 1] = up<BF16>(raw[j] >> 16);
  }
  const int16_t top = hi.x > hi.y ? hi.x : hi.y, low = lo.x < lo.y ? lo.x : lo.y;
  short2v both = {top, (int16_t)~low};
  auto merge = [&](uint32_t other) { both = __builtin_elementwise_max(both, __builtin_bit_cast(short2v, other)); };
  merge(moved<kDppXor1>(__builtin_bit_cast(uint32_t, both)));
  merge(moved<kDppXor2>(__builtin_bit_cast(uint32_t, both)));
  if (LANES >= 8) merge(moved<kDppHalfMirror>(__builtin_bit_cast(uint32_t, both)));
  if (LANES >= 16) merge(moved<kDppMirror>(__builtin_bit_cast(uint32_t, both)));
  const int16_t last = BF16 ? 0x477F : 0x7BFF;  // the largest pattern up to 65504
  if (both.x > last || both.y > last) {
    float l = INFINITY, h = -INFINITY;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      x[j] = tame(x[j]);
      l = fminf(l, x[j]);
      h = fmaxf(h, x[j]);
    }
    lanes_minmax<LANES>(l, h);
    return group_of(l, h);
  }
  const short2v ends = {both.x, (int16_t)~both.y};
  const uint32_t w = __builtin_bit_cast(uint32_t, ends ^ ((ends >> 15) & short2v{32767, 32767}));
  return group_of(up<BF16>(w >> 16), up<BF16>(w & 0xFFFFu));
}

// rne((x - m) / s) without a division: the quotient is below 32 (15, more where s is a
// subnormal that was rounded down), so the product with v_rcp_f32's value (within 1 ulp) is
// within 32 (2^-23 + 2^-24) of it, and its rounded value within another 32 2^-24: both round to
// the same integer unless the product lies within 2^-16 of a half-integer, where the IEEE
// division decides, for the lane's whole set.
template <int C>
__device__ __forceinline__ void codes_of(const float *x, const Group &g, uint32_t *c) {
  float v[C], off = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const float t = (x[j] - g.m) * g.r;
    v[j] = __builtin_rintf(t);
    off = fmaxf(off, fabsf(t - v[j]));
  }
  if (off > 0.5f - 0x1p-16f) {
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = __builtin_rintf((x[j] - g.m) / g.s);
  }
#pragma unroll
  for (int j = 0; j < C; ++j) c[j] = (uint32_t)__builtin_amdgcn_fmed3f(v[j], 0.0f, 15.0f);
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

// C 16-bit values from one 16-byte (C = 4: 8-byte) aligned place to another.
template <int C>
__device__ __forceinline__ void copy16(uint16_t *to, const uint16_t *from) {
  if (C == 4) *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(from);
  if (C >= 8) *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
  if (C == 16) *reinterpret_cast<uint4 *>(to + 8) = *reinterpret_cast<const uint4 *>(from + 8);
}

// Between what the lanes of a quarter write to LDS and what others of them read: a wave's
// LDS operations are done in order, so only the compiler has to be held.
__device__ __forceinline__ void in_quarter() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int D, bool BF16>
__global__ __launch_bounds__(256) void kv4_append_kernel(TokenArgs a) {
  constexpr int C = D / 16, G = D / 64;
  // a quarter's codes of values on the way from the lanes that hold a group to those that hold
  // a column
  __shared__ __attribute__((aligned(16))) uint8_t turn[16][D];
  const int i = threadIdx.x & 15, quarter = threadIdx.x >> 4;
  const int32_t group = blockIdx.x / a.heads, head = blockIdx.x - group * a.heads, row = group * 16 + quarter;
  if (row >= a.T) return;  // whole quarters leave: the lane moves and LDS below stay inside a quarter
  alignas(16) uint32_t raw[C / 2], raw_v[C / 2];
  // loaded beside the slot, not after it
  copy16<C>(reinterpret_cast<uint16_t *>(raw), a.k + (int64_t)row * a.ldk + head * D + i * C);
  copy16<C>(reinterpret_cast<uint16_t *>(raw_v), a.v + (int64_t)row * a.ldv + head * D + i * C);
  int32_t tok = 0;
  uint8_t *blk = block_of<D>(a, row, head, tok);
  if (!blk) return;
  constexpr int L = 64 / C;  // lanes of a group
  float x[C];
  uint32_t c[C];
  // Lane 0 writes all groups' parameters: group e's are in lanes e L .., row_ror 16 - e L brings
  // them to lane 0.
  auto store = [&](uint8_t *to, uint32_t s16, uint32_t m16) {
    const uint32_t own = s16 | m16 << 16;
    uint32_t all[4] = {own, 0, 0, 0};
    if (G == 2) all[1] = moved<0x128>(own);
    if (G == 4) all[1] = moved<0x12C>(own), all[2] = moved<0x128>(own), all[3] = moved<0x124>(own);
    auto lows = [](uint32_t u, uint32_t v) { return __builtin_amdgcn_perm(v, u, 0x05040100u); };
    auto highs = [](uint32_t u, uint32_t v) { return __builtin_amdgcn_perm(v, u, 0x07060302u); };
    if (i != 0) return;
    if (G == 1) *reinterpret_cast<uint32_t *>(to) = own;
    if (G == 2) *reinterpret_cast<uint2 *>(to) = make_uint2(lows(all[0], all[1]), highs(all[0], all[1]));
    if (G == 4)
      *reinterpret_cast<uint4 *>(to) = make_uint4(lows(all[0], all[1]), lows(all[2], all[3]), highs(all[0], all[1]),
                                                  highs(all[2], all[3]));
  };
  {  // keys
    const Group g = measure<C, L, BF16>(raw, x);
    codes_of<C>(x, g, c);
    uint8_t *dst = blk + tok * (D / 2) + key_byte<D>(i);
#pragma unroll
    for (int w = 0; w < (C + 7) / 8; ++w) {
      uint32_t word = 0;
#pragma unroll
      for (int j = 0; j < (C < 8 ? C : 8); ++j) word |= c[8 * w + j] << (4 * j);
      if (C == 4) *reinterpret_cast<uint16_t *>(dst) = (uint16_t)word;
      else *reinterpret_cast<uint32_t *>(dst + w * (D / 8)) = word;
    }
    store(blk + a.page * D + tok * (4 * G), g.s16, g.m16);
  }
  {  // values: codes by this lane's channels, then to the columns
    const Group g = measure<C, L, BF16>(raw_v, x);
    codes_of<C>(x, g, c);
#pragma unroll
    for (int j = 0; j < C; ++j) turn[quarter][i * C + j] = (uint8_t)c[j];
    store(blk + a.page * D + a.page * (D / 16) + tok * (4 * G), g.s16, g.m16);
    in_quarter();
    uint32_t word[(C + 7) / 8] = {};
#pragma unroll
    for (int j = 0; j < C; ++j) word[j / 8] |= (uint32_t)turn[quarter][16 * j + i] << (4 * (j % 8));
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
  __shared__ __attribute__((aligned(16))) uint16_t turn[16][D];
  const int i = threadIdx.x & 15, quarter = threadIdx.x >> 4;
  const int32_t group = blockIdx.x / a.heads, head = blockIdx.x - group * a.heads, row = group * 16 + quarter;
  int32_t tok = 0;
  const uint8_t *blk = block_of<D>(a, row, head, tok);
  if (!blk) return;
  {
    const uint16_t *par = reinterpret_cast<const uint16_t *>(blk + a.page * D + tok * (4 * G));
    const float s = up<false>(par[i / (64 / C)]), m = up<false>(par[G + i / (64 / C)]);
    const uint8_t *src = blk + tok * (D / 2) + key_byte<D>(i);
    alignas(16) uint16_t out[C];
#pragma unroll
    for (int w = 0; w < (C + 7) / 8; ++w) {
      const uint32_t word = C == 4 ? *reinterpret_cast<const uint16_t *>(src)
                                   : *reinterpret_cast<const uint32_t *>(src + w * (D / 8));
#pragma unroll
      for (int j = 0; j < (C < 8 ? C : 8); ++j)
        out[8 * w + j] = (uint16_t)down<BF16>(m + s * (float)((word >> (4 * j)) & 15));
    }
    copy16<C>(a.k + (int64_t)row * a.ldk + head * D + i * C, out);
  }
  {
    const uint16_t *par = reinterpret_cast<const uint16_t *>(blk + a.page * D + a.page * (D / 16) + tok * (4 * G));
    const uint8_t *src = blk + a.page * (D / 2) + ((tok / 4 * 16 + i) * 4 + tok % 4) * (D / 32);
    uint32_t word[(C + 7) / 8];
    if (C == 4) word[0] = *reinterpret_cast<const uint16_t *>(src);
    if (C == 8) word[0] = *reinterpret_cast<const uint32_t *>(src);
    if (C == 16) {
      const uint2 w = *reinterpret_cast<const uint2 *>(src);
      word[0] = w.x, word[(C + 7) / 8 - 1] = w.y;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t c = (word[j / 8] >> (4 * (j % 8))) & 15;
      turn[quarter][16 * j + i] =
          (uint16_t)down<BF16>(up<false>(par[G + j / 4]) + up<false>(par[j / 4]) * (float)c);
    }
    in_quarter();
    copy16<C>(a.v + (int64_t)row * a.ldv + head * D + i * C, &turn[quarter][i * C]);
  }
}

int check_tokens(const void *k, const void *v, int64_t ldk, int64_t ldv, int32_t dtype, const int32_t *slots, int32_t T,
                 const void *cache, size_t cache_bytes, int32_t pages, int32_t page, int32_t heads, int32_t dim) {
  if (T < 0 || (dtype != MIXLLM_FP16 && dtype != MIXLLM_BF16)) return MIXLLM_E_SHAPE;
  if (T == 0) return MIXLLM_OK;
  const int st = mixllm::kv4_check_cache(cache, cache_bytes, pages, page, heads, dim);
  if (st != MIXLLM_OK) return st;
  const int64_t width = (int64_t)heads * dim;
  // a launch has fewer than 2^32 threads, 256 for 16 rows of a head
  if (heads > 65535 || ((int64_t)T + 15) / 16 * heads >= 1 << 24) return MIXLLM_E_SHAPE;
  if (ldk < width || ldv < width || ldk % 8 != 0 || ldv % 8 != 0) return MIXLLM_E_SHAPE;
  if (!k || !v || !slots) return MIXLLM_E_NULL;
  if (!mixllm::is_aligned16(k) || !mixllm::is_aligned16(v) || !mixllm::is_aligned4(slots)) return MIXLLM_E_SHAPE;
  return MIXLLM_OK;
}

template <bool APPEND, int D>
void launch_tokens(const TokenArgs &a, int32_t dtype, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)a.T + 15) / 16 * a.heads));  // heads of the same rows together
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

namespace {

int run_plan(const int32_t *fresh, const int32_t *lens, int32_t B, int32_t *table, int64_t ldt, int32_t width,
             int32_t *pool, int32_t F, const int32_t *count, int32_t page, int32_t pages, int32_t *lens_out,
             int32_t *count_out, int32_t *cu, int32_t *slots, int32_t *pos, int32_t tokens, int64_t room,
             void *stream) {
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
                      mixllm::log2_of(page), pages, tokens, room};
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

}  // namespace

extern "C" int mixllm_kv_plan(const int32_t *fresh, const int32_t *lens, int32_t B, int32_t *table, int64_t ldt,
                              int32_t width, int32_t *pool, int32_t F, const int32_t *count, int32_t page,
                              int32_t pages, int32_t *lens_out, int32_t *count_out, int32_t *cu, int32_t *slots,
                              int32_t *pos, int32_t tokens, void *stream) {
  return run_plan(fresh, lens, B, table, ldt, width, pool, F, count, page, pages, lens_out, count_out, cu, slots, pos,
                  tokens, INT64_MAX, stream);
}

extern "C" int mixllm_kv_plan_fit(const int32_t *fresh, const int32_t *lens, int32_t B, int32_t *table, int64_t ldt,
                                  int32_t width, int32_t *pool, int32_t F, const int32_t *count, int32_t page,
                                  int32_t pages, int32_t *lens_out, int32_t *count_out, int32_t *cu, int32_t *slots,
                                  int32_t *pos, int32_t tokens, void *stream) {
  return run_plan(fresh, lens, B, table, ldt, width, pool, F, count, page, pages, lens_out, count_out, cu, slots, pos,
                  tokens, tokens, stream);
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
