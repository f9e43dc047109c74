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
// second launch joins a row's chunks, or the first one writes the row's result
// where the row is one chunk.
//
// Best entries: an entry's key is its value in an order of whole numbers, then
// the lowest index, so keys differ. A wave takes the top-th largest of its
// lanes' own largest keys as a bound, found bit by bit with ballots: at least
// `top` entries of the wave reach it, and only lanes that reach it hold any
// that do, so at most 32 * top. Those of all waves go to LDS, where an entry's
// place is the number of larger ones. Which slot of the list an entry gets
// depends on chance, its place does not.

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
// k of thread i begins at entry VEC * (i + kThreads * k).
template <bool BF16>
struct Layout {
  static constexpr int VEC = BF16 ? 8 : 4, GROUPS = kPer / VEC;
  __device__ __forceinline__ static int at(int k) { return VEC * ((int)threadIdx.x + kThreads * k); }
};

// The thread's entries of the chunk of `n` entries at row + first; those past
// its end read as -inf.
template <bool BF16>
__device__ __forceinline__ void load_chunk(const void* row, int64_t first, int n, float (&x)[kPer]) {
  using L = Layout<BF16>;
  const char* base = reinterpret_cast<const char*>(row) + first * (BF16 ? 2 : 4);
  if (n >= kLpChunk) {
    u32x4 d[L::GROUPS];
#pragma unroll
    for (int k = 0; k < L::GROUPS; ++k) {
      if constexpr (BF16)
        d[k] = *reinterpret_cast<const u32x4_by2*>(base + 2 * L::at(k));
      else
        d[k] = *reinterpret_cast<const u32x4_by4*>(base + 4 * L::at(k));
    }
#pragma unroll
    for (int k = 0; k < L::GROUPS; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
          x[8 * k + 2 * i] = __uint_as_float(d[k][i] << 16);
          x[8 * k + 2 * i + 1] = __uint_as_float(d[k][i] & 0xFFFF0000u);
        } else {
          x[4 * k + i] = __uint_as_float(d[k][i]);
        }
      }
    return;
  }
#pragma unroll
  for (int k = 0; k < L::GROUPS; ++k)
#pragma unroll
    for (int i = 0; i < L::VEC; ++i) {
      const int at = L::at(k) + i;
      x[L::VEC * k + i] = at < n ? number<BF16>(base, at) : neg_inf();
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

// The n-th largest of the wave's keys (n <= 64; lanes without one hold 0).
__device__ __forceinline__ uint64_t nth_key(uint64_t key, int n) {
  const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
  uint32_t h = 0;
  int above = 0;      // keys whose upper half is larger than h in the bits so far settled
#pragma unroll 1
  for (int b = 31; b >= 0; --b) {
    const uint32_t c = h | (1u << b);
    const int count = (int)__popcll(__ballot(hi >= c));
    if (count >= n) h = c;
    if (count == n) return (uint64_t)h << 32;
  }
  above = (int)__popcll(__ballot(hi > h));
  uint32_t l = 0;
  const bool tied = hi == h;
#pragma unroll 1
  for (int b = 31; b >= 0; --b) {
    const uint32_t c = l | (1u << b);
    const int count = above + (int)__popcll(__ballot(tied && lo >= c));
    if (count >= n) l = c;
    if (count == n) break;
  }
  return ((uint64_t)h << 32) | l;
}

struct Sums {      // of a part of a row
  float m, l, w;
};
__device__ __forceinline__ float scaled(float a, float b) { return a == 0.f ? 0.f : a * b; }      // 0 of an empty part stays
// x, moved to the larger maximum m.
__device__ __forceinline__ void add_part(Sums& s, const Sums& x) {
  const float m = max_nan(s.m, x.m), ref = m == neg_inf() ? 0.f : m;
  const float a = s.m - ref, b = x.m - ref, ea = exp2_fast(a * kLog2e), eb = exp2_fast(b * kLog2e);
  // an empty part (maximum -inf) has sums of 0, and -inf * 0 must not become a NaN
  s.w = ea * (s.w + scaled(s.l, a)) + eb * (x.w + scaled(x.l, b));
  s.l = s.l * ea + x.l * eb;
  s.m = m;
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

// Places of the `count` keys in `list` (LDS) in descending order: put(place, key) for the first `top`.
template <typename Put>
__device__ __forceinline__ void place_keys(const uint64_t* list, int count, int top, Put&& put) {
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const uint64_t key = list[i];
    int place = 0;
    for (int j = 0; j < count; ++j) place += list[j] > key;
    if (place < top) put(place, key);
  }
}

__device__ __forceinline__ void put_top(const Logprobs& p, int64_t t, const Norm& o, int place, uint64_t key) {
  p.top_ids[t * p.top + place] = (int)~(uint32_t)key;
  p.top_logprobs[t * p.top + place] = logprob_of(o, value_of((uint32_t)(key >> 32)));
}

template <bool BF16, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_chunk_kernel(const Logprobs p, int chunks) {
  extern __shared__ __align__(16) uint64_t list[];      // kThreads / 64 * kPer * top
  __shared__ float wmax[kThreads / 64];
  __shared__ float4 wsum[kThreads / 64];
  __shared__ Norm norm;
  __shared__ int count;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x / chunks;
  const int chunk = (int)(blockIdx.x - t * chunks), first = chunk * kLpChunk, n = min(p.V - first, kLpChunk);
  const int y = p.targets[t];
  const bool token = y >= 0 && y < p.V;
  float x[kPer];
  load_chunk<BF16>(p.logits, t * p.stride + first, n, x);
  const float xy = token ? number<BF16>(p.logits, t * p.stride + y) : __builtin_inff();

  float m = x[0];
#pragma unroll
  for (int i = 1; i < kPer; ++i) m = max_nan(m, x[i]);
  m = wave_max_nan(m);
  if (lane == 0) wmax[wave] = m;
  if (TOP && threadIdx.x == 0) count = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kThreads / 64; ++k) m = max_nan(m, wmax[k]);
  const float ref = m == neg_inf() ? 0.f : m;
  float l = 0.f, w = 0.f;
  int before = 0;
#pragma unroll
  for (int k = 0; k < Layout<BF16>::GROUPS; ++k)
#pragma unroll
    for (int i = 0; i < Layout<BF16>::VEC; ++i) {
      const float v = x[Layout<BF16>::VEC * k + i], d = v - ref, e = exp2_fast(d * kLog2e);
      l += e;
      w += e == 0.f ? 0.f : e * d;
      before += v > xy || (v == xy && first + Layout<BF16>::at(k) + i < y);
    }
  l = wave_sum(l);
  w = wave_sum(w);
  before = wave_sum(before);
  if (lane == 0) wsum[wave] = make_float4(l, w, __int_as_float(before), 0.f);

  if constexpr (TOP) {
    // the lane's largest key
    uint64_t best = 0;
#pragma unroll
    for (int k = 0; k < Layout<BF16>::GROUPS; ++k)
#pragma unroll
      for (int i = 0; i < Layout<BF16>::VEC; ++i) {
        const int at = Layout<BF16>::at(k) + i;
        const uint64_t key = at < n ? key_of(x[Layout<BF16>::VEC * k + i], first + at) : 0;
        best = key > best ? key : best;
      }
    const uint64_t bound = nth_key(best, p.top);
#pragma unroll
    for (int k = 0; k < Layout<BF16>::GROUPS; ++k)
#pragma unroll
      for (int i = 0; i < Layout<BF16>::VEC; ++i) {
        const int at = Layout<BF16>::at(k) + i;
        const uint64_t key = at < n ? key_of(x[Layout<BF16>::VEC * k + i], first + at) : 0;
        if (key != 0 && key >= bound) list[atomicAdd(&count, 1)] = key;
      }
  }
  __syncthreads();
  Sums s{m, 0.f, 0.f};
  before = 0;
#pragma unroll
  for (int k = 0; k < kThreads / 64; ++k) {
    s.l += wsum[k].x;
    s.w += wsum[k].y;
    before += __float_as_int(wsum[k].z);
  }
  if (chunks == 1) {
    if (threadIdx.x == 0) norm = finish_row<BF16>(p, t, s, before);
    if constexpr (TOP) {
      __syncthreads();
      const Norm o = norm;
      place_keys(list, count, p.top, [&](int place, uint64_t key) { put_top(p, t, o, place, key); });
    }
    return;
  }
  const int64_t o = t * chunks + chunk;
  if (threadIdx.x == 0) p.part[o] = make_float4(s.m, s.l, s.w, __int_as_float(before));
  if constexpr (TOP) {
    place_keys(list, count, p.top, [&](int place, uint64_t key) { p.part_top[o * p.top + place] = key; });
    for (int i = count + threadIdx.x; i < p.top; i += kThreads) p.part_top[o * p.top + i] = 0;
  }
}

// A workgroup joins a row's chunks.
template <bool BF16, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_join_kernel(const Logprobs p, int chunks) {
  extern __shared__ __align__(16) uint64_t list[];      // chunks * top
  __shared__ Norm norm;
  __shared__ uint64_t bound;
  __shared__ int count;
  const int64_t t = blockIdx.x;
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
  }
  if constexpr (TOP) {
    // what is worse than some chunk's last is none of the row's best
    if (threadIdx.x == 0) {
      bound = 1;
      count = 0;
    }
    __syncthreads();
    const uint64_t* from = p.part_top + t * chunks * p.top;
    for (int c = threadIdx.x; c < chunks; c += kThreads)
      atomicMax((unsigned long long*)&bound, (unsigned long long)from[(int64_t)c * p.top + p.top - 1]);
    __syncthreads();
    const uint64_t least = bound;
    for (int i = threadIdx.x; i < chunks * p.top; i += kThreads) {
      const uint64_t key = from[i];
      if (key >= least) list[atomicAdd(&count, 1)] = key;
    }
    __syncthreads();
    const Norm o = norm;
    place_keys(list, count, p.top, [&](int place, uint64_t key) { put_top(p, t, o, place, key); });
  }
}

// The gradient, a chunk of a row at a time: one read and one write of every
// entry and an exponential between them.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void logprobs_bwd_kernel(const Logprobs p, int chunks) {
  using L = Layout<BF16>;
  const int64_t t = blockIdx.x / chunks;
  const int chunk = (int)(blockIdx.x - t * chunks), first = chunk * kLpChunk, n = min(p.V - first, kLpChunk);
  float x[kPer];
  load_chunk<BF16>(p.logits, t * p.stride + first, n, x);
  const int y = p.targets[t];
  const bool token = y >= 0 && y < p.V;
  const Norm o{p.norm[2 * t], p.norm[2 * t + 1]};
  const float entropy = p.entropy[t], gl = token ? p.d_logprob[t] : 0.f, gh = p.d_entropy[t];
  const bool none = o.m == neg_inf();
  const float shift = entropy * gh + gl;      // of p's factor
#pragma unroll
  for (int k = 0; k < L::GROUPS; ++k)
#pragma unroll
    for (int i = 0; i < L::VEC; ++i) {
      float& v = x[L::VEC * k + i];
      const float lp = (v - o.m) - o.n, e = exp2_fast(lp * kLog2e);
      const float g = e == 0.f ? 0.f : -e * fmaf(gh, lp, shift);
      v = none ? 0.f : g + (token && first + L::at(k) + i == y ? gl : 0.f);
    }
  char* base = reinterpret_cast<char*>(p.d_logits) + (t * p.V + first) * (BF16 ? 2 : 4);
  if (n >= kLpChunk) {
#pragma unroll
    for (int k = 0; k < L::GROUPS; ++k) {
      u32x4 d;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF16)
          d[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x[8 * k + 2 * i], (__bf16)x[8 * k + 2 * i + 1]});
        else
          d[i] = __float_as_uint(x[4 * k + i]);
      }
      if constexpr (BF16)
        *reinterpret_cast<u32x4_by2*>(base + 2 * L::at(k)) = d;
      else
        *reinterpret_cast<u32x4_by4*>(base + 4 * L::at(k)) = d;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < L::GROUPS; ++k)
#pragma unroll
    for (int i = 0; i < L::VEC; ++i) {
      const int at = L::at(k) + i;
      if (at < n) {
        if constexpr (BF16)
          reinterpret_cast<__bf16*>(base)[at] = (__bf16)x[L::VEC * k + i];
        else
          reinterpret_cast<float*>(base)[at] = x[L::VEC * k + i];
      }
    }
}

template <bool BF16>
void launch_forward(const Logprobs& p, hipStream_t stream) {
  const int chunks = (int)logprobs_chunks(p.V);
  const dim3 grid((unsigned)(p.T * chunks)), rows((unsigned)p.T), block(kThreads);
  if (p.top > 0) {
    const size_t lds = sizeof(uint64_t) * (kThreads / 64) * kPer * p.top;
    hipLaunchKernelGGL((logprobs_chunk_kernel<BF16, true>), grid, block, lds, stream, p, chunks);
    if (chunks > 1)
      hipLaunchKernelGGL((logprobs_join_kernel<BF16, true>), rows, block, sizeof(uint64_t) * chunks * p.top, stream, p, chunks);
  } else {
    hipLaunchKernelGGL((logprobs_chunk_kernel<BF16, false>), grid, block, 0, stream, p, chunks);
    if (chunks > 1) hipLaunchKernelGGL((logprobs_join_kernel<BF16, false>), rows, block, 0, stream, p, chunks);
  }
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
