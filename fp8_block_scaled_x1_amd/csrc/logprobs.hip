// Log probabilities of given tokens with entropy, rank and the most likely
// alternatives, and their gradient.
//
// With m the row's largest logit and d_i = x_i - m, l = sum exp(d_i) and
// w = sum exp(d_i) d_i give everything that depends on the whole row:
//   logprob of x = (x - m) - log l,  entropy = log l - w / l,
// and both sums join over parts of a row (exp(m' - m) moves them to a larger
// maximum m: l exp(m' - m) and (w + l (m' - m)) exp(m' - m)). One pass: a
// workgroup holds a chunk of 8192 logits in registers, takes its maximum, then
// the two sums, the entries that come before the token, and its best entries; a
// second launch joins a row's parts, or the first one writes the row's result
// where the row is one part.
//
// The exponentials are 2^(c x - c m), c = log2 e, one fused multiply-add each:
// what c m loses by its own rounding is a factor of all of them, known exactly
// and taken back from the sums (|m| below 2^20; beyond, 2^(c (x - m))). An entry
// comes before the token if it is larger, or equal and ahead of it, so in a
// chunk that the token is not in one comparison tells, counted by the scalar
// unit.
//
// Best entries: an entry's key is its value in an order of whole numbers, then
// the lowest index, so keys differ. A wave takes the top-th largest of its
// lanes' own largest values as a bound, found bit by bit with ballots: at least
// `top` entries of the wave reach it. Those of all waves go to LDS, where an
// entry's place is the number of larger keys. Which slot of the list an entry
// gets depends on chance, its place does not. Where more than 2 * top + 32 of a
// wave reach it (some 24 of 20 do, unless many are equal or masked), the bound
// is taken by keys: then only `top` lanes, so 32 * top entries, reach it.
//
// Bound: memory. 2048 rows of 129280 BF16 106 us (5.0 TB/s), with the gradient
// 318 (two reads and a write, 5.0 TB/s); forward with one entry of 50 left and the
// others masked, by whatever value, 109 to 111. With alternatives the chain of a
// workgroup: 96 rows of 129280 FP32 with 20 of them 25 us (17 and 6.4 for the
// join, 2.0 TB/s), without 17.

#include "attn_common.h"
#include "serve_internal.h"

namespace fp8bs {

namespace {

constexpr int kThreads = kLogprobsThreads, kPer = 32, kLpChunk = kThreads * kPer;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// Rows begin at any multiple of a number's size.
typedef u32x4 u32x4_by4 __attribute__((aligned(4)));
typedef u32x4 u32x4_by2 __attribute__((aligned(2)));

template <bool BF16>
__device__ __forceinline__ float number(const void* p, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
  else
    return reinterpret_cast<const float*>(p)[i];
}

// Numbers of a 16-byte access, and the chunk's groups of them per thread: group
// k of thread i begins at entry VEC * (i + kThreads * k). A group that the end
// of the row cuts (the chunk has `n` entries) is read from
// VEC before the end: its first entries are the group before's. A chunk of fewer
// than VEC entries is read entry by entry, by every thread.
template <bool BF16>
struct Layout {
  static constexpr int VEC = BF16 ? 8 : 4, GROUPS = kPer / VEC, SIZE = BF16 ? 2 : 4;
  __device__ __forceinline__ static int nominal(int k) { return VEC * ((int)threadIdx.x + kThreads * k); }
  __device__ __forceinline__ static int at(int k, int n) { return n < VEC ? nominal(k) : min(nominal(k), n - VEC); }
};
template <bool BF16>
__device__ __forceinline__ u32x4 load16(const void* p) {
  if constexpr (BF16)
    return *reinterpret_cast<const u32x4_by2*>(p);
  else
    return *reinterpret_cast<const u32x4_by4*>(p);
}

template <bool BF16>
__device__ __forceinline__ void store16(void* p, u32x4 d) {
  if constexpr (BF16)
    *reinterpret_cast<u32x4_by2*>(p) = d;
  else
    *reinterpret_cast<u32x4_by4*>(p) = d;
}

// The thread's groups of a chunk of `n` entries at `base`, as they are in memory
// (entries that a row does not have: anything).
template <bool BF16>
__device__ __forceinline__ void load_raw(const char* base, int n, u32x4 (&d)[Layout<BF16>::GROUPS]) {
  using L = Layout<BF16>;
  if (n >= L::VEC) {
#pragma unroll
    for (int k = 0; k < L::GROUPS; ++k) d[k] = load16<BF16>(base + (int64_t)L::SIZE * L::at(k, n));
  } else {
    d[0] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < L::VEC; ++i) {
      const uint32_t bits = __float_as_uint(number<BF16>(base, min(i, n - 1)));
      if constexpr (BF16)
        d[0][i / 2] |= i & 1 ? bits : bits >> 16;
      else
        d[0][i] = bits;
    }
#pragma unroll
    for (int k = 1; k < L::GROUPS; ++k) d[k] = d[0];
  }
}
template <bool BF16>
__device__ __forceinline__ void numbers_of(const u32x4 (&d)[Layout<BF16>::GROUPS], float (&x)[kPer]) {
  using L = Layout<BF16>;
#pragma unroll
  for (int k = 0; k < L::GROUPS; ++k)
#pragma unroll
    for (int i = 0; i < L::VEC; ++i) {
      if constexpr (BF16)
        x[8 * k + i] = __uint_as_float(i & 1 ? d[k][i / 2] & 0xFFFF0000u : d[k][i / 2] << 16);
      else
        x[4 * k + i] = __uint_as_float(d[k][i]);
    }
}
// As numbers, and -inf for what is not the thread's own.
template <bool BF16>
__device__ __forceinline__ void entries_of(const u32x4 (&d)[Layout<BF16>::GROUPS], int n, float (&x)[kPer]) {
  using L = Layout<BF16>;
  numbers_of<BF16>(d, x);
  if (n == kLpChunk) return;
#pragma unroll
  for (int k = 0; k < L::GROUPS; ++k) {
    const int at = L::at(k, n), from = L::nominal(k) - at, to = n - at;
#pragma unroll
    for (int i = 0; i < L::VEC; ++i) x[L::VEC * k + i] = i >= from && i < to ? x[L::VEC * k + i] : neg_inf();
  }
}

// Ascending with the value, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float((o >> 31) ? o & 0x7FFFFFFFu : ~o); }
__device__ __forceinline__ uint64_t key_of(float x, int index) { return ((uint64_t)order_of(x) << 32) | (uint32_t)~index; }

__device__ __forceinline__ float wave_max_nan(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = max_nan(v, __shfl_xor(v, d, 64));
  return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// The n-th largest of the wave's values (n <= 64), counted with those that `above` more lanes are known to exceed.
__device__ __forceinline__ uint32_t nth_value(uint32_t v, int n, bool counts = true, int above = 0) {
  uint32_t h = 0;
#pragma unroll 1
  for (int b = 31; b >= 0; --b) {
    const uint32_t c = h | (1u << b);
    const int count = above + (int)__popcll(__ballot(counts && v >= c));
    if (count >= n) h = c;
    if (count == n) break;
  }
  return h;
}

struct Sums {      // of a part of a row
  float m, l, w;
};
// A part's sum moved by the factor e. Where e is 0 the sum has no share,
// whatever its size: an empty part's maximum of -inf, or a masked part's of the
// type's lowest value, makes it -inf or a NaN. (A NaN maximum makes e one.)
__device__ __forceinline__ float moved(float e, float sum) { return e == 0.f ? 0.f : e * sum; }
// x, moved to the larger maximum m.
__device__ __forceinline__ void add_part(Sums& s, const Sums& x) {
  const float m = max_nan(s.m, x.m), ref = m == neg_inf() ? 0.f : m;
  const float a = s.m - ref, b = x.m - ref, ea = exp2_fast(a * kLog2e), eb = exp2_fast(b * kLog2e);
  s.w = moved(ea, s.w + s.l * a) + moved(eb, x.w + x.l * b);
  s.l = s.l * ea + x.l * eb;
  s.m = m;
}

// Sums of exp(x_i - m) and of that times (x_i - m). `usual`: the same for the
// wave, and |m| < kUsual if it is set: c m is below 2^21 then, its rounding
// (`lost`) at most 2^-4. It grows with m, and beyond 2^7 (|m| of some 10^10, a
// mask) the exponentials would leave FP32's range.
constexpr float kUsual = 0x1p20f;
__device__ __forceinline__ void sums_against(const float (&x)[kPer], float m, bool usual, float& l, float& w) {
  l = w = 0.f;
  if (usual) {
    const float m2 = m * kLog2e, lost = fmaf(m, kLog2e, -m2);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float d = fmaf(x[i], kLog2e, -m2), e = exp2_fast(d);
      l += e;
      w = fmaf(e, fmaxf(d, -1000.f), w);      // (0 * -inf; a NaN shows in l)
    }
    const float back = exp2_fast(-lost);
    w = fmaf(-lost, l, w) * back * kLn2;
    l *= back;
  } else {      // masks, -inf and NaN among them: differences first
    const float ref = m == neg_inf() ? 0.f : m;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float d = x[i] - ref, e = exp2_fast(d * kLog2e);
      l += e;
      w += e == 0.f ? 0.f : e * d;
    }
  }
}

// Of `n` entries from `first` on, as entries_of gave them: how many of the
// wave's come before the token y with logit xy. They do if they reach a bound:
// xy itself ahead of the token, the next larger value behind it (0 and -0 are equal).
template <bool BF16>
__device__ __forceinline__ int count_before(const float (&x)[kPer], int first, int n, int y, float xy) {
  using L = Layout<BF16>;
  const uint32_t u = __float_as_uint(xy + 0.f);
  const float larger = __uint_as_float(u == 0 ? 1u : (u >> 31) ? u - 1u : u + 1u);
  int before = 0;
  if (y < first || y >= first + kLpChunk) {
    const float least = y < first ? larger : xy;
#pragma unroll
    for (int i = 0; i < kPer; ++i) before += (int)__popcll(__ballot(x[i] >= least));
  } else {
#pragma unroll
    for (int k = 0; k < L::GROUPS; ++k) {
      const int ahead = y - first - L::at(k, n);
#pragma unroll
      for (int i = 0; i < L::VEC; ++i) before += (int)__popcll(__ballot(x[L::VEC * k + i] >= (i < ahead ? xy : larger)));
    }
  }
  if (xy == neg_inf() && n < kLpChunk && n >= L::VEC) {      // what a cut group holds of another's reached it as -inf
    int other = 0;
    for (int k = 0; k < L::GROUPS; ++k) other += max(0, min(min(L::nominal(k) - L::at(k, n), y - first - L::at(k, n)), (int)L::VEC));
    before -= wave_sum(other);
  }
  return before;
}

// What the log probability of a logit x is taken against: (x - m) - n.
struct Norm {
  float m, n;
};
__device__ __forceinline__ float logprob_of(const Norm& o, float x) { return x == neg_inf() ? x : (x - o.m) - o.n; }

// What is written of a row, by one thread.
template <bool BF16>
__device__ __forceinline__ Norm finish_row(const Logprobs& p, int64_t t, const Sums& s, int before) {
  const bool none = s.m == neg_inf();
  const Norm o{s.m, none ? 0.f : __logf(s.l)};
  const int y = p.targets[t];
  const bool token = y >= 0 && y < p.V;
  p.norm[2 * t] = o.m;
  p.norm[2 * t + 1] = o.n;
  p.entropy[t] = none ? 0.f : o.n - s.w / s.l;
  // (a sum that is NaN shows in the log probability of an entry of -inf too)
  p.logprob[t] = !token ? 0.f : o.n != o.n ? o.n : logprob_of(o, number<BF16>(p.logits, t * p.stride + y));
  p.rank[t] = token ? min(before, p.V - 1) : -1;
  return o;
}

// How many of a list's keys are larger.
__device__ __forceinline__ int keys_before(uint64_t key, const uint64_t* list, int count) {
  int n = 0;
#pragma unroll 8
  for (int j = 0; j < count; ++j) n += list[j] > key;
  return n;
}

__device__ __forceinline__ void put_top(const Logprobs& p, int64_t t, const Norm& o, int place, uint64_t key) {
  p.top_ids[t * p.top + place] = (int)~(uint32_t)key;
  p.top_logprobs[t * p.top + place] = logprob_of(o, value_of((uint32_t)(key >> 32)));
}

// With alternatives: a workgroup has one chunk of a row. The code is kept short
// (what is rare reads the chunk again in loops): with 53 KB of it, all unrolled,
// 546 rows of 12943 took 67 us, with 15 KB 27.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void logprobs_chunk_kernel(const Logprobs p, int chunks) {
  using L = Layout<BF16>;
  extern __shared__ __align__(16) uint64_t list[];      // [waves][kPer * top]
  __shared__ float wmax[kThreads / 64];
  __shared__ uint32_t wbound[kThreads / 64];
  __shared__ float4 wsum[kThreads / 64];
  __shared__ int wcount[kThreads / 64], overflow;
  __shared__ Norm norm;
  const int64_t t = blockIdx.x / chunks;
  const int chunk = (int)(blockIdx.x - t * chunks), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int first = chunk * kLpChunk, n = min(p.V - first, kLpChunk);
  const int y = p.targets[t];
  const bool token = y >= 0 && y < p.V;
  const char* base = reinterpret_cast<const char*>(p.logits) + (t * p.stride + first) * L::SIZE;
  u32x4 raw[L::GROUPS];
  load_raw<BF16>(base, n, raw);
  const float xy = token ? number<BF16>(p.logits, t * p.stride + y) : __builtin_inff();
  float x[kPer];
  entries_of<BF16>(raw, n, x);

  float mine = x[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) mine = max_nan(mine, x[i]);
  float m = wave_max_nan(mine);
  uint32_t bound = nth_value(order_of(mine), p.top);
  if (lane == 0) {
    wmax[wave] = m;
    wbound[wave] = bound;
  }
  if (threadIdx.x == 0) overflow = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kThreads / 64; ++k) {
    m = max_nan(m, wmax[k]);
    bound = max(bound, wbound[k]);
  }

  float l, w;
  sums_against(x, m, fabsf(m) < kUsual, l, w);
  l = wave_sum(l);
  w = wave_sum(w);
  int before = count_before<BF16>(x, first, n, y, xy);
  if (lane == 0) wsum[wave] = make_float4(l, w, __int_as_float(before), 0.f);

  // Candidates of the wave, to its part of the list: entry and index, then keys.
  uint64_t* const own_list = list + wave * kPer * p.top;
  const float least = value_of(bound);
  const int few = min(2 * p.top + 32, kPer * p.top);
  int at = 0;
  if (least > neg_inf()) {      // else too many may reach it, or it is a NaN
#pragma unroll
    for (int k = 0; k < L::GROUPS; ++k) {
      const int index = first + L::at(k, n);
#pragma unroll
      for (int i = 0; i < L::VEC; ++i) {
        const bool reaches = !(x[L::VEC * k + i] < least);
        const uint64_t all = __ballot(reaches);
        if (all == 0) continue;
        const int slot = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
        if (reaches && slot < few) own_list[slot] = ((uint64_t)(uint32_t)(index + i) << 32) | __float_as_uint(x[L::VEC * k + i]);
        at += (int)__popcll(all);
      }
    }
    __builtin_amdgcn_wave_barrier();      // (a wave's LDS accesses keep their order)
    for (int i = lane; i < min(at, few); i += 64)
      own_list[i] = key_of(__uint_as_float((uint32_t)own_list[i]), (int)(own_list[i] >> 32));
  }
  if (lane == 0) wcount[wave] = at;
  if (at > few || !(least > neg_inf())) overflow = 1;
  __syncthreads();
  if (overflow) {      // the same for all; the thread's entries now lie kThreads apart
    auto key_at = [&](int i) { return i < n ? key_of(number<BF16>(base, i), first + i) : (uint64_t)0; };
    uint64_t best = 0;
#pragma unroll 8
    for (int j = 0; j < kPer; ++j) {
      const uint64_t key = key_at(threadIdx.x + kThreads * j);
      best = key > best ? key : best;
    }
    const uint32_t hi = (uint32_t)(best >> 32), lo = (uint32_t)best, h = nth_value(hi, p.top);
    const uint64_t bound = max(((uint64_t)h << 32) | nth_value(lo, p.top, hi == h, (int)__popcll(__ballot(hi > h))), (uint64_t)1);
    at = 0;
#pragma unroll 8
    for (int j = 0; j < kPer; ++j) {
      const uint64_t key = key_at(threadIdx.x + kThreads * j), all = __ballot(key >= bound);
      const int slot = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
      if (key >= bound) own_list[slot] = key;      // at most `top` lanes of the wave reach it
      at += (int)__popcll(all);
    }
    if (lane == 0) wcount[wave] = at;
    __syncthreads();
  }
  Sums s{m, 0.f, 0.f};
  int count = 0;
  before = 0;
#pragma unroll
  for (int k = 0; k < kThreads / 64; ++k) {
    count += wcount[k];
    s.l += wsum[k].x;
    s.w += wsum[k].y;
    before += __float_as_int(wsum[k].z);
  }
  const int64_t o = t * chunks + chunk;
  if (threadIdx.x == 0) {
    if (chunks == 1)
      norm = finish_row<BF16>(p, t, s, before);
    else
      p.part[o] = make_float4(s.m, s.l, s.w, __int_as_float(before));
  }
  if (chunks == 1) __syncthreads();
  for (int i = lane; i < wcount[wave]; i += 64) {
    const uint64_t key = own_list[i];
    int place = 0;
    for (int k = 0; k < kThreads / 64; ++k) place += keys_before(key, list + k * kPer * p.top, wcount[k]);
    if (place >= p.top) continue;
    if (chunks == 1)
      put_top(p, t, norm, place, key);
    else
      p.part_top[o * p.top + place] = key;
  }
  if (chunks > 1)
    for (int i = count + threadIdx.x; i < p.top; i += kThreads) p.part_top[o * p.top + i] = 0;
}

// Without alternatives: a workgroup goes over `per` consecutive chunks of a row
// with the next chunk's loads under way, and a thread keeps its own maximum and
// sums, so the waves meet at the end only.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void logprobs_stream_kernel(const Logprobs p, int chunks, int per, int splits) {
  using L = Layout<BF16>;
  __shared__ float4 wsum[kThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x / splits;
  const int split = (int)(blockIdx.x - t * splits), begin = split * per, end = min(chunks, begin + per);
  const char* row = reinterpret_cast<const char*>(p.logits) + t * p.stride * L::SIZE;
  auto load = [&](int chunk, u32x4 (&d)[L::GROUPS]) {
    const int first = chunk * kLpChunk;
    load_raw<BF16>(row + (int64_t)first * L::SIZE, min(p.V - first, kLpChunk), d);
  };
  u32x4 raw[2][L::GROUPS];
  load(begin, raw[0]);
  const int y = p.targets[t];
  const bool token = y >= 0 && y < p.V;
  const float xy = token ? number<BF16>(row, y) : __builtin_inff();
  Sums mine{neg_inf(), 0.f, 0.f};
  int before = 0;      // of the wave: entries that come before the token
  auto work = [&](int chunk, const u32x4 (&now)[L::GROUPS], u32x4 (&next)[L::GROUPS]) {
    load(min(chunk + 1, end - 1), next);
    const int first = chunk * kLpChunk, n = min(p.V - first, kLpChunk);
    float x[kPer];
    entries_of<BF16>(now, n, x);
    Sums c{x[0], 0.f, 0.f};
#pragma unroll
    for (int i = 1; i < kPer; ++i) c.m = max_nan(c.m, x[i]);
    c.m = max_nan(c.m, mine.m);
    sums_against(x, c.m, __all(fabsf(c.m) < kUsual), c.l, c.w);
    add_part(mine, c);
    before += count_before<BF16>(x, first, n, y, xy);
  };
  for (int chunk = begin; chunk < end; chunk += 2) {
    work(chunk, raw[0], raw[1]);
    if (chunk + 1 >= end) break;
    work(chunk + 1, raw[1], raw[0]);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const Sums o{__shfl_xor(mine.m, d, 64), __shfl_xor(mine.l, d, 64), __shfl_xor(mine.w, d, 64)};
    add_part(mine, o);
  }
  if (lane == 0) wsum[wave] = make_float4(mine.m, mine.l, mine.w, __int_as_float(before));
  __syncthreads();
  if (threadIdx.x > 0) return;
  for (int k = 1; k < kThreads / 64; ++k) {
    add_part(mine, Sums{wsum[k].x, wsum[k].y, wsum[k].z});
    before += __float_as_int(wsum[k].w);
  }
  if (splits == 1)
    finish_row<BF16>(p, t, mine, before);
  else
    p.part[t * splits + split] = make_float4(mine.m, mine.l, mine.w, __int_as_float(before));
}

// A workgroup joins a row's chunks.
template <bool BF16, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_join_kernel(const Logprobs p, int chunks) {
  extern __shared__ __align__(16) uint64_t list[];      // chunks * top
  __shared__ Norm norm;
  __shared__ uint64_t bound;
  __shared__ int count;
  const int64_t t = blockIdx.x;
  const uint64_t* from = TOP ? p.part_top + t * chunks * p.top : nullptr;
  const int keys = TOP ? chunks * p.top : 0;
  const uint64_t early = TOP && threadIdx.x < keys ? from[threadIdx.x] : 0;
  if (threadIdx.x < 64) {
    Sums s{neg_inf(), 0.f, 0.f};
    int before = 0;
    for (int c = threadIdx.x; c < chunks; c += 64) {
      const float4 v = p.part[t * chunks + c];
      add_part(s, Sums{v.x, v.y, v.z});
      before += __float_as_int(v.w);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const Sums o{__shfl_xor(s.m, d, 64), __shfl_xor(s.l, d, 64), __shfl_xor(s.w, d, 64)};
      add_part(s, o);
    }
    before = wave_sum(before);
    if (threadIdx.x == 0) norm = finish_row<BF16>(p, t, s, before);
  } else if (TOP && threadIdx.x < 128) {
    // what is worse than some chunk's last is none of the row's best
    uint64_t most = 1;
    for (int c = threadIdx.x - 64; c < chunks; c += 64) {
      const uint64_t last = from[(int64_t)c * p.top + p.top - 1];
      most = last > most ? last : most;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint64_t o = __shfl_xor((unsigned long long)most, d, 64);
      most = o > most ? o : most;
    }
    if (threadIdx.x == 64) {
      bound = most;
      count = 0;
    }
  }
  if constexpr (TOP) {
    __syncthreads();
    const uint64_t least = bound;
    for (int i = threadIdx.x; i < keys; i += kThreads) {
      const uint64_t key = i == threadIdx.x ? early : from[i];
      if (key >= least) list[atomicAdd(&count, 1)] = key;
    }
    __syncthreads();
    const Norm o = norm;
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const uint64_t key = list[i];
      const int place = keys_before(key, list, count);
      if (place < p.top) put_top(p, t, o, place, key);
    }
  }
}

// The gradient, a chunk of a row at a time: one read and one write of every
// entry and an exponential between them. (What two threads both hold of a cut
// group, both write, the same.)
template <bool BF16>
__global__ __launch_bounds__(kThreads) void logprobs_bwd_kernel(const Logprobs p, int chunks) {
  using L = Layout<BF16>;
  const int64_t t = blockIdx.x / chunks;
  const int first = (int)(blockIdx.x - t * chunks) * kLpChunk, n = min(p.V - first, kLpChunk);
  u32x4 raw[L::GROUPS];
  load_raw<BF16>(reinterpret_cast<const char*>(p.logits) + (t * p.stride + first) * L::SIZE, n, raw);
  char* to = reinterpret_cast<char*>(p.d_logits) + (t * p.V + first) * L::SIZE;
  const int y = p.targets[t];
  const bool token = y >= 0 && y < p.V;
  const Norm o{p.norm[2 * t], p.norm[2 * t + 1]};
  const float entropy = p.entropy[t], gl = token ? p.d_logprob[t] : 0.f, gh = p.d_entropy[t];
  const bool none = o.m == neg_inf();
  const float shift = fmaf(entropy, gh, gl);      // of p's factor
  float x[kPer];
  numbers_of<BF16>(raw, x);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float lp = (x[i] - o.m) - o.n, e = exp2_fast(lp * kLog2e);
    // (0 * -inf; a NaN stays one by e)
    x[i] = none ? 0.f : -e * fmaf(gh, fmaxf(lp, -1000.f), shift);
  }
#pragma unroll
  for (int k = 0; k < L::GROUPS; ++k) {
    const int at = L::at(k, n), mine = y - first - at;
    if (token && !none && mine >= 0 && mine < L::VEC) {
#pragma unroll
      for (int i = 0; i < L::VEC; ++i) x[L::VEC * k + i] += i == mine ? gl : 0.f;
    }
    if (L::nominal(k) >= n) continue;
    if (n < L::VEC) {
#pragma unroll
      for (int i = 0; i < L::VEC; ++i)
        if (i < n) {
          if constexpr (BF16)
            reinterpret_cast<__bf16*>(to)[i] = (__bf16)x[i];
          else
            reinterpret_cast<float*>(to)[i] = x[i];
        }
      continue;
    }
    u32x4 d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16)
        d[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x[8 * k + 2 * i], (__bf16)x[8 * k + 2 * i + 1]});
      else
        d[i] = __float_as_uint(x[4 * k + i]);
    }
    store16<BF16>(to + (int64_t)L::SIZE * at, d);
  }
}

template <bool BF16>
void launch_forward(const Logprobs& p, hipStream_t stream) {
  const int chunks = (int)logprobs_chunks(p.V);
  const dim3 rows((unsigned)p.T), block(kThreads);
  if (p.top > 0) {
    const size_t lds = sizeof(uint64_t) * (kThreads / 64) * kPer * p.top;
    hipLaunchKernelGGL(logprobs_chunk_kernel<BF16>, dim3((unsigned)(p.T * chunks)), block, lds, stream, p, chunks);
    if (chunks > 1)
      hipLaunchKernelGGL((logprobs_join_kernel<BF16, true>), rows, block, sizeof(uint64_t) * chunks * p.top, stream, p, chunks);
    return;
  }
  // Few rows: a chunk per workgroup, many: a row, with eight workgroups per
  // compute unit of a full device between them. 2048 rows of 129280 BF16 106 us,
  // with a chunk per workgroup 140; 4096 of 50000 89 and 120; half or twice as
  // many workgroups change no time by more than 5 %.
  const int64_t want = (2048 + p.T - 1) / p.T;
  const int per = (int)((chunks + want - 1) / want), splits = (chunks + per - 1) / per;
  hipLaunchKernelGGL(logprobs_stream_kernel<BF16>, dim3((unsigned)(p.T * splits)), block, 0, stream, p, chunks, per, splits);
  if (splits > 1) hipLaunchKernelGGL((logprobs_join_kernel<BF16, false>), rows, block, 0, stream, p, splits);
}

}  // namespace

int64_t logprobs_chunks(int64_t V) { return (V + kLpChunk - 1) / kLpChunk; }

hipError_t launch_logprobs(const Logprobs& l, bool bf16, hipStream_t stream) {
  if (bf16)
    launch_forward<true>(l, stream);
  else
    launch_forward<false>(l, stream);
  return hipGetLastError();
}

hipError_t launch_logprobs_bwd(const Logprobs& l, bool bf16, hipStream_t stream) {
  const int chunks = (int)logprobs_chunks(l.V);
  const dim3 grid((unsigned)(l.T * chunks)), block(kThreads);
  if (bf16)
    hipLaunchKernelGGL(logprobs_bwd_kernel<true>, grid, block, 0, stream, l, chunks);
  else
    hipLaunchKernelGGL(logprobs_bwd_kernel<false>, grid, block, 0, stream, l, chunks);
  return hipGetLastError();
}

}  // namespace fp8bs
