// Verification of drafted tokens against the target model's probabilities,
// with given random numbers, and the draw of the token that follows them.
//
// Draft j (token x, proposed with probability q_j(x)) is accepted iff
// u_j * q_j(x) < p_j(x); the accepted ones are the drafts before the first
// that is not. After a rejection at position a the next token follows
// max(p_a - q_a, 0), after the last draft p_n, drawn by inverting the
// cumulative sum at u_next. The weights are taken as whole multiples of 2^-38
// (floor(r * 2^38), r in [0, 1]): their 64-bit sums are exact, so the drawn
// token does not depend on how the vocabulary is split or in which order the
// parts are added. A weight below 2^-38 counts as zero; FP32 sums of that many
// probabilities err by far more.
//
// Only one row of p (and of q) per request is read, once for the sums of its
// chunks and, for the one chunk that holds the token, once more (from L2).
// Chunks of 8192 entries give a request 16 workgroups at a vocabulary of 129280.
// One request: 11 us in a graph, the latency of two launches; 96 requests with
// 4 drafts, FP32: 26 us, 87 MB in 19 us (4.6 TB/s), then 8 us for the one chunk
// of each request, again the latency of a launch and of a chunk's loads.

#include "attn_common.h"
#include "attn_internal.h"

namespace fp8bs {

namespace {

constexpr int kChunk = 8192, kVThreads = kVerifyThreads, kPer = kChunk / kVThreads;      // kPer consecutive entries a thread
constexpr float kWeightOne = 274877906944.0f;      // 2^38

template <bool BF16>
__device__ __forceinline__ float prob(const void* p, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
  else
    return reinterpret_cast<const float*>(p)[i];
}

// floor(r * 2^38) for r clamped to [0, 1]; 0 for NaN.
__device__ __forceinline__ uint64_t weight(float r) {
  return r > 0.f ? (uint64_t)(fminf(r, 1.f) * kWeightOne) : 0ull;
}

struct Row {
  int accepted;     // drafts accepted
  bool rejected;    // the next one was turned down
  int token;        // that draft
};

// Every lane of the wave gets the same answer.
template <bool BF16>
__device__ __forceinline__ Row accept(const VerifyDrafts& v, int b) {
  const int lane = threadIdx.x & 63;
  const int n = min(max(v.n_drafts[b], 0), v.K);
  bool ok = false;
  int x = 0;
  if (lane < n) {
    x = v.drafts[(int64_t)b * v.K + lane];
    if (x >= 0 && x < v.V) {
      const float px = prob<BF16>(v.p, ((int64_t)b * (v.K + 1) + lane) * v.V + x);
      const float qx = v.q ? prob<BF16>(v.q, ((int64_t)b * v.K + lane) * v.V + x) : 1.f;
      ok = v.u[(int64_t)b * v.K + lane] * qx < px;
    }
  }
  const uint64_t turned = __ballot(lane < n && !ok);
  Row r;
  r.rejected = turned != 0;
  r.accepted = r.rejected ? __ffsll((unsigned long long)turned) - 1 : n;
  r.token = __shfl(x, r.accepted & 63, 64);
  return r;
}

// Entries first .. first+3 of a row, 0 past its end. VEC: rows begin and end on
// whole groups of four.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load4(const void* row, int64_t at, int first, int V, float (&x)[4]) {
  if constexpr (VEC) {
    x[0] = x[1] = x[2] = x[3] = 0.f;
    if (first >= V) return;
    if constexpr (BF16) {
      const uint2 d = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(row) + at + first);
      x[0] = __uint_as_float(d.x << 16);
      x[1] = __uint_as_float(d.x & 0xFFFF0000u);
      x[2] = __uint_as_float(d.y << 16);
      x[3] = __uint_as_float(d.y & 0xFFFF0000u);
    } else {
      const float4 d = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(row) + at + first);
      x[0] = d.x;
      x[1] = d.y;
      x[2] = d.z;
      x[3] = d.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = first + k < V ? prob<BF16>(row, at + first + k) : 0.f;
  }
}

// The weights of the kPer entries that begin at `first`, `step` apart in groups
// of four: after a rejection, and plain.
template <bool BF16, bool VEC, typename F>
__device__ __forceinline__ void weights(const VerifyDrafts& v, int b, const Row& r, int first, int step, F&& take) {
  const int64_t prow = ((int64_t)b * (v.K + 1) + r.accepted) * v.V, qrow = ((int64_t)b * v.K + r.accepted) * v.V;
  float p[kPer / 4][4], q[kPer / 4][4];
#pragma unroll
  for (int g = 0; g < kPer / 4; ++g) load4<BF16, VEC>(v.p, prow, first + g * step, v.V, p[g]);
  if (r.rejected && v.q) {
#pragma unroll
    for (int g = 0; g < kPer / 4; ++g) load4<BF16, VEC>(v.q, qrow, first + g * step, v.V, q[g]);
  } else {
#pragma unroll
    for (int g = 0; g < kPer / 4; ++g)
#pragma unroll
      for (int k = 0; k < 4; ++k) q[g][k] = r.rejected && first + g * step + k == r.token ? __builtin_inff() : 0.f;
  }
#pragma unroll
  for (int g = 0; g < kPer / 4; ++g)
#pragma unroll
    for (int k = 0; k < 4; ++k) take(4 * g + k, weight(p[g][k] - q[g][k]), weight(p[g][k]));
}

__device__ __forceinline__ uint64_t wave_sum64(uint64_t x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor((unsigned long long)x, d, 64);
  return x;
}
__device__ __forceinline__ uint64_t wave_scan64(uint64_t x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t y = __shfl_up((unsigned long long)x, d, 64);
    if (lane >= d) x += y;
  }
  return x;
}

template <bool BF16, bool VEC>
__global__ __launch_bounds__(kVThreads) void verify_sum_kernel(const VerifyDrafts v, int chunks) {
  __shared__ uint64_t part[kVThreads / 64][2];
  const int b = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const Row r = accept<BF16>(v, b);
  if (chunk == 0 && threadIdx.x == 0) v.rows[b] = make_int4(r.accepted, r.rejected, r.token, 0);
  uint64_t a = 0, c = 0;
  weights<BF16, VEC>(v, b, r, chunk * kChunk + 4 * (int)threadIdx.x, 4 * kVThreads, [&](int, uint64_t x, uint64_t y) {
    a += x;
    c += y;
  });
  a = wave_sum64(a);
  c = wave_sum64(c);
  if ((threadIdx.x & 63) == 0) {
    part[threadIdx.x >> 6][0] = a;
    part[threadIdx.x >> 6][1] = c;
  }
  __syncthreads();
  if (threadIdx.x < 2)
    v.sums[((int64_t)b * chunks + chunk) * 2 + threadIdx.x] =
        part[0][threadIdx.x] + part[1][threadIdx.x] + part[2][threadIdx.x] + part[3][threadIdx.x];
}

template <bool BF16, bool VEC>
__global__ __launch_bounds__(kVThreads) void verify_pick_kernel(const VerifyDrafts v, int chunks) {
  __shared__ uint64_t waves[kVThreads / 64];
  const int b = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int4 known = v.rows[b];
  const Row r{known.x, known.y != 0, known.z};
  // which weights, and their sum
  const uint64_t* sums = v.sums + (int64_t)b * chunks * 2;
  uint64_t ta = 0, tc = 0;
  for (int c = lane; c < chunks; c += 64) {
    ta += sums[2 * c];
    tc += sums[2 * c + 1];
  }
  ta = wave_sum64(ta);
  tc = wave_sum64(tc);
  const bool plain = ta == 0;          // nothing left of p - q: p itself
  const uint64_t total = plain ? tc : ta;
  if (total > 0) {
    // the token is the first whose running sum passes goal = floor(total * u)
    const float u = fminf(fmaxf(v.u_next[b], 0.f), 1.f - 0x1p-24f);
    const uint64_t m = (uint64_t)(u * 16777216.0f);
    uint64_t goal = (total >> 24) * m + (((total & 0xFFFFFFull) * m) >> 24);
    // its chunk
    uint64_t before = 0;
    int chunk = 0;
    for (int c0 = 0; c0 < chunks; c0 += 64) {
      const uint64_t x = c0 + lane < chunks ? sums[2 * (c0 + lane) + plain] : 0ull;
      const uint64_t incl = before + wave_scan64(x);
      const uint64_t hit = __ballot(incl > goal);
      if (hit) {
        const int l = __ffsll((unsigned long long)hit) - 1;
        chunk = c0 + l;
        before = __shfl((unsigned long long)(incl - x), l, 64);
        break;
      }
      before = __shfl((unsigned long long)incl, 63, 64);
    }
    goal -= before;
    // its thread's consecutive entries, then the entry
    const int first = chunk * kChunk + kPer * (int)threadIdx.x;
    uint64_t mine[kPer], own = 0;
    weights<BF16, VEC>(v, b, r, first, 4, [&](int i, uint64_t x, uint64_t y) {
      mine[i] = plain ? y : x;
      own += mine[i];
    });
    uint64_t incl = wave_scan64(own);
    if (lane == 63) waves[w] = incl;
    __syncthreads();
    for (int k = 0; k < w; ++k) incl += waves[k];
    if (incl > goal && incl - own <= goal) {
      uint64_t run = incl - own;
      int at = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        run += mine[i];
        at += run <= goal;
      }
      v.tokens[(int64_t)b * (v.K + 1) + r.accepted] = first + at;
    }
  } else if (threadIdx.x == 0) {
    v.tokens[(int64_t)b * (v.K + 1) + r.accepted] = -1;
  }
  if (w == 0 && lane <= v.K && lane != r.accepted)
    v.tokens[(int64_t)b * (v.K + 1) + lane] = lane < r.accepted ? v.drafts[(int64_t)b * v.K + lane] : -1;
  if (threadIdx.x == 0) v.accepted[b] = r.accepted;
}

template <bool BF16, bool VEC>
void launch(const VerifyDrafts& v, hipStream_t stream) {
  const int chunks = (int)verify_chunks(v.V);
  hipLaunchKernelGGL((verify_sum_kernel<BF16, VEC>), dim3((unsigned)v.B * chunks), dim3(kVThreads), 0, stream, v, chunks);
  hipLaunchKernelGGL((verify_pick_kernel<BF16, VEC>), dim3((unsigned)v.B), dim3(kVThreads), 0, stream, v, chunks);
}

}  // namespace

int64_t verify_chunks(int64_t V) { return (V + kChunk - 1) / kChunk; }

hipError_t launch_verify_drafts(const VerifyDrafts& v, bool bf16, hipStream_t stream) {
  // Rows of whole groups of four entries, all of them aligned: wide loads (96
  // requests, FP32: 28 us; one entry at a time, vocabulary 129281, 42 us).
  const uintptr_t at = reinterpret_cast<uintptr_t>(v.p) | reinterpret_cast<uintptr_t>(v.q);
  const bool vec = v.V % 4 == 0 && at % (bf16 ? 8 : 16) == 0;
  if (bf16)
    vec ? launch<true, true>(v, stream) : launch<true, false>(v, stream);
  else
    vec ? launch<false, true>(v, stream) : launch<false, false>(v, stream);
  return hipGetLastError();
}

}  // namespace fp8bs
