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

#include "attn_common.h"
#include "attn_internal.h"

namespace fp8bs {

namespace {

constexpr int kChunk = 4096, kVThreads = 256, kPer = kChunk / kVThreads;
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

// The weights of vocabulary entry i: after a rejection, and plain.
template <bool BF16>
__device__ __forceinline__ void weights(const VerifyDrafts& v, int64_t prow, int64_t qrow, const Row& r, int i,
                                        uint64_t& residual, uint64_t& plain) {
  const float p = prob<BF16>(v.p, prow + i);
  plain = weight(p);
  residual = plain;
  if (r.rejected) residual = v.q ? weight(p - prob<BF16>(v.q, qrow + i)) : (i == r.token ? 0ull : plain);
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

template <bool BF16>
__global__ __launch_bounds__(kVThreads) void verify_sum_kernel(const VerifyDrafts v, int chunks) {
  __shared__ uint64_t part[kVThreads / 64][2];
  const int b = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const Row r = accept<BF16>(v, b);
  const int64_t prow = ((int64_t)b * (v.K + 1) + r.accepted) * v.V, qrow = ((int64_t)b * v.K + r.accepted) * v.V;
  uint64_t a = 0, c = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = chunk * kChunk + k * kVThreads + (int)threadIdx.x;
    if (i < v.V) {
      uint64_t x, y;
      weights<BF16>(v, prow, qrow, r, i, x, y);
      a += x;
      c += y;
    }
  }
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

template <bool BF16>
__global__ __launch_bounds__(kVThreads) void verify_pick_kernel(const VerifyDrafts v, int chunks) {
  __shared__ uint64_t seg[kChunk / 64];
  const int b = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const Row r = accept<BF16>(v, b);
  const int64_t prow = ((int64_t)b * (v.K + 1) + r.accepted) * v.V, qrow = ((int64_t)b * v.K + r.accepted) * v.V;
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
  int next = -1;
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
    // its 64 entries, then the entry
    uint64_t mine[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = chunk * kChunk + k * kVThreads + (int)threadIdx.x;
      uint64_t x = 0, y = 0;
      if (i < v.V) weights<BF16>(v, prow, qrow, r, i, x, y);
      mine[k] = plain ? y : x;
      const uint64_t s = wave_sum64(mine[k]);
      if (lane == 0) seg[k * (kVThreads / 64) + w] = s;
    }
    __syncthreads();
    const uint64_t x = seg[lane], incl = wave_scan64(x);
    const int s = __ffsll((unsigned long long)__ballot(incl > goal)) - 1;
    goal -= __shfl((unsigned long long)(incl - x), s, 64);
    if ((s & 3) == w) {
      uint64_t y = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (k == s >> 2) y = mine[k];
      const int e = __ffsll((unsigned long long)__ballot(wave_scan64(y) > goal)) - 1;
      next = chunk * kChunk + s * 64 + e;
      if (lane == 0) v.tokens[(int64_t)b * (v.K + 1) + r.accepted] = next;
    }
  } else if (threadIdx.x == 0) {
    v.tokens[(int64_t)b * (v.K + 1) + r.accepted] = -1;
  }
  if (w == 0 && lane <= v.K && lane != r.accepted)
    v.tokens[(int64_t)b * (v.K + 1) + lane] = lane < r.accepted ? v.drafts[(int64_t)b * v.K + lane] : -1;
  if (threadIdx.x == 0) v.accepted[b] = r.accepted;
}

template <bool BF16>
void launch(const VerifyDrafts& v, hipStream_t stream) {
  const int chunks = (int)verify_chunks(v.V);
  hipLaunchKernelGGL(verify_sum_kernel<BF16>, dim3((unsigned)v.B * chunks), dim3(kVThreads), 0, stream, v, chunks);
  hipLaunchKernelGGL(verify_pick_kernel<BF16>, dim3((unsigned)v.B), dim3(kVThreads), 0, stream, v, chunks);
}

}  // namespace

int64_t verify_chunks(int64_t V) { return (V + kChunk - 1) / kChunk; }

hipError_t launch_verify_drafts(const VerifyDrafts& v, bool bf16, hipStream_t stream) {
  if (bf16)
    launch<true>(v, stream);
  else
    launch<false>(v, stream);
  return hipGetLastError();
}

}  // namespace fp8bs
