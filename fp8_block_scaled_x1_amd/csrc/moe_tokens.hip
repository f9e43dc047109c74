// A whole mixture-of-experts layer for a few tokens: two kernels that read each
// chosen expert's weights once.
//
//   up    h = bf16(silu(G_e x) * (U_e x)) for every (expert, token) that meet
//   down  out_t = bf16(sum over t's experts of w * D_e h)
//
// For a few tokens the layer is the reading of its weights, so every wave
// streams 16-row strips of them straight into registers, in the order in which
// the matrix unit wants them (a lane: 32 consecutive bytes of a row's 128, the
// inner index numbered to match), turns the codes into BF16 (exact) and
// multiplies them with the tokens' numbers, which come from L2. A 128-wide
// partial sum is scaled by its block's scale as it is added (FP32).
//
// up: a workgroup is 16 columns of h of one expert (16 rows of G and of U), its
// waves share the inner dimension and add their sums through LDS. down: a
// workgroup is 16 columns of the output for all experts and tokens, so the sum
// over a token's experts needs no second pass and no atomics; its waves share
// the list of (expert, 128-wide chunk). Sums run in a fixed order.
//
// Which experts are chosen is found by every workgroup from the ids (at most
// 4096 of them): a bitmap in LDS, and a lane per token that looks for the
// workgroup's expert among its token's ids. An id outside [0, E) sets no bit.

#include "attn_common.h"
#include "serve_internal.h"

namespace fp8bs {

namespace {

constexpr int kChunkK = 128;      // inner numbers that share a scale
constexpr int kStrip = 16;        // rows of weights
constexpr int kTiles = kMoeMaxTokens / 16;
constexpr int kUpWaves = 4, kDownWaves = 8;

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// The ids of all slots and a bit per chosen expert.
struct Routing {
  int32_t ids[kMoeMaxTokens * kMoeMaxTopk];
  uint32_t bits[kMoeMaxExperts / 32];
};

template <int THREADS>
__device__ __forceinline__ void load_routing(const MoeTokens& m, Routing& r) {
  if (threadIdx.x < kMoeMaxExperts / 32) r.bits[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < m.T * m.topk; i += THREADS) {
    const int e = m.ids[i];
    r.ids[i] = e;
    if (e >= 0 && e < m.E) atomicOr(&r.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// Lane l of the first 32: the chosen experts of word l (`word`), how many come
// before it; returns how many there are. Every lane of the wave takes part.
__device__ __forceinline__ int count_chosen(const Routing& r, uint32_t& word, int& before) {
  const int lane = threadIdx.x & 63;
  word = lane < kMoeMaxExperts / 32 ? r.bits[lane] : 0;
  const int own = __popc(word);
  int v = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(v, d, 64);
    if (lane >= d) v += x;
  }
  before = v - own;
  return __builtin_amdgcn_readlane(v, 63);
}

__device__ __forceinline__ int nth_bit(uint32_t word, int n) {
  for (; n > 0; --n) word &= word - 1;
  return __ffs((int)word) - 1;
}

// Lane t's token: the first slot in which it names expert e (-1: none) and the
// sum of the weights of all of those.
struct Member {
  int slot;
  float weight;
};
template <bool WEIGHTS>
__device__ __forceinline__ Member member_of(const MoeTokens& m, const Routing& r, int e) {
  const int t = threadIdx.x & 63;
  Member x{-1, 0.f};
  if (t < m.T)
    for (int j = m.topk - 1; j >= 0; --j)
      if (r.ids[t * m.topk + j] == e) {
        x.slot = t * m.topk + j;
        if constexpr (WEIGHTS) x.weight += m.weights[t * m.topk + j];
      }
  return x;
}

// 32 codes of a row (the lane's share of a chunk) and their four operands.
struct Codes {
  uint4 a, b;
  __device__ __forceinline__ void load(const uint8_t* p) {
    a = *reinterpret_cast<const uint4*>(p);
    b = *reinterpret_cast<const uint4*>(p + 16);
  }
  __device__ __forceinline__ bf16x8 operand(int s) const {
    return s == 0 ? e4m3_to_bf16(a.x, a.y) : s == 1 ? e4m3_to_bf16(a.z, a.w) : s == 2 ? e4m3_to_bf16(b.x, b.y) : e4m3_to_bf16(b.z, b.w);
  }
};

__global__ __launch_bounds__(64 * kUpWaves) void moe_up_kernel(const MoeTokens m) {
  __shared__ Routing routing;
  __shared__ int tok[kMoeMaxTokens], slot_of[kMoeMaxTokens];
  __shared__ __align__(16) float sums[kUpWaves][kTiles][2][64][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int strips = m.F / kStrip;
  const int rank = blockIdx.x / strips, strip = blockIdx.x - rank * strips;

  load_routing<64 * kUpWaves>(m, routing);
  uint32_t word;
  int before;
  if (rank >= count_chosen(routing, word, before)) return;
  const uint64_t hit = __ballot(rank >= before && rank < before + __popc(word));
  const int hl = __ffsll((unsigned long long)hit) - 1;
  const int e = __builtin_amdgcn_readfirstlane(32 * hl + nth_bit(__shfl(word, hl, 64), rank - __shfl(before, hl, 64)));
  const Member mine = member_of<false>(m, routing, e);
  const uint64_t members = __ballot(mine.slot >= 0);
  const int count = (int)__popcll(members);
  if (wave == 0 && mine.slot >= 0) {
    const int at = (int)__popcll(members & ((1ull << lane) - 1ull));
    tok[at] = lane;
    slot_of[at] = mine.slot;
  }
  __syncthreads();

  const int tiles = (count + 15) / 16, chunks = m.K / kChunkK;
  const int inner = 32 * (lane >> 4);
  const uint16_t* x[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) x[i] = m.x + (int64_t)tok[min(16 * i + (lane & 15), count - 1)] * m.K + inner;
  const int row = strip * kStrip + (lane & 15);
  const uint8_t* gate = m.w_up + ((int64_t)e * 2 * m.F + row) * m.K + inner;
  const uint8_t* up = gate + (int64_t)m.F * m.K;
  const float* sg = m.s_up + ((int64_t)e * 2 * m.F / kChunkK + strip * kStrip / kChunkK) * chunks;
  const float* su = sg + (int64_t)(m.F / kChunkK) * chunks;

  f32x4 ag[kTiles], au[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) ag[i] = au[i] = zero4();
#pragma unroll 2
  for (int c = wave; c < chunks; c += kUpWaves) {
    Codes g, u;
    g.load(gate + c * kChunkK);
    u.load(up + c * kChunkK);
    const float fg = sg[c], fu = su[c];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      if (i < tiles) {
        f32x4 pg = zero4(), pu = zero4();
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const bf16x8 b = *reinterpret_cast<const bf16x8*>(x[i] + c * kChunkK + 8 * s);
          pg = mfma16(g.operand(s), b, pg);
          pu = mfma16(u.operand(s), b, pu);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ag[i][j] = fmaf(fg, pg[j], ag[i][j]);
          au[i][j] = fmaf(fu, pu[j], au[i][j]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
    if (i < tiles) {
      *reinterpret_cast<f32x4*>(sums[wave][i][0][lane]) = ag[i];
      *reinterpret_cast<f32x4*>(sums[wave][i][1][lane]) = au[i];
    }
  __syncthreads();
  // a thread: one of 16 tokens and one of the strip's columns
  const int col = threadIdx.x & 15, of = threadIdx.x >> 4, from = 16 * (col >> 2) + of;
  for (int i = 0; i < tiles; ++i) {
    const int at = 16 * i + of;
    if (at >= count) break;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < kUpWaves; ++w) {
      g += sums[w][i][0][from][col & 3];
      u += sums[w][i][1][from][col & 3];
    }
    const float h = g / (1.f + exp2_fast(-g * kLog2e)) * u;
    reinterpret_cast<__bf16*>(m.h)[(int64_t)slot_of[at] * m.F + strip * kStrip + col] = (__bf16)h;
  }
}

__global__ __launch_bounds__(64 * kDownWaves) void moe_down_kernel(const MoeTokens m) {
  __shared__ Routing routing;
  __shared__ uint16_t chosen[kMoeMaxExperts];
  __shared__ __align__(16) float sums[kDownWaves][kTiles][64][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int strip = blockIdx.x;

  load_routing<64 * kDownWaves>(m, routing);
  uint32_t word;
  int before;
  const int experts = count_chosen(routing, word, before);
  if (wave == 0)
    for (; word; word &= word - 1) chosen[before++] = (uint16_t)(32 * lane + __ffs((int)word) - 1);
  __syncthreads();

  const int tiles = (m.T + 15) / 16, chunks = m.F / kChunkK;
  const int inner = 32 * (lane >> 4), row = strip * kStrip + (lane & 15);
  const int units = experts * chunks;      // at most 1024 * 512
  const int begin = (int)((int64_t)units * wave / kDownWaves), end = (int)((int64_t)units * (wave + 1) / kDownWaves);
  f32x4 acc[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) acc[i] = zero4();
  for (int unit = begin; unit < end;) {
    const int n = unit / chunks, c0 = unit - n * chunks, c1 = min(chunks, c0 + end - unit);
    unit += c1 - c0;
    const int e = __builtin_amdgcn_readfirstlane((int)chosen[n]);
    const Member mine = member_of<true>(m, routing, e);
    const uint64_t members = __ballot(mine.slot >= 0);
    const uint16_t* h[kTiles];
    float w[kTiles];
    bool in[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      // tokens that did not choose the expert read one that did, and add nothing
      const int of = 16 * i + (lane & 15);
      const uint32_t some = (uint32_t)(members >> (16 * i)) & 0xFFFFu;
      in[i] = (members >> of) & 1;
      w[i] = __shfl(mine.weight, of, 64);
      const int other = some ? 16 * i + __ffs((int)some) - 1 : 0;
      h[i] = m.h + (int64_t)__shfl(mine.slot, in[i] ? of : other, 64) * m.F + inner;
    }
    const uint8_t* down = m.w_down + ((int64_t)e * m.K + row) * m.F + inner;
    const float* sd = m.s_down + ((int64_t)e * (m.K / kChunkK) + strip * kStrip / kChunkK) * chunks;
#pragma unroll 2
    for (int c = c0; c < c1; ++c) {
      Codes d;
      d.load(down + c * kChunkK);
      const float f = sd[c];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        if (i < tiles && ((members >> (16 * i)) & 0xFFFF)) {
          f32x4 part = zero4();
#pragma unroll
          for (int s = 0; s < 4; ++s)
            part = mfma16(d.operand(s), *reinterpret_cast<const bf16x8*>(h[i] + c * kChunkK + 8 * s), part);
          const float fw = f * w[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = in[i] ? fmaf(fw, part[j], acc[i][j]) : acc[i][j];
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
    if (i < tiles) *reinterpret_cast<f32x4*>(sums[wave][i][lane]) = acc[i];
  __syncthreads();
  for (int at = threadIdx.x; at < 16 * m.T; at += 64 * kDownWaves) {
    const int t = at >> 4, col = at & 15;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) v += sums[w][t >> 4][16 * (col >> 2) + (t & 15)][col & 3];
    reinterpret_cast<__bf16*>(m.out)[(int64_t)t * m.K + strip * kStrip + col] = (__bf16)v;
  }
}

}  // namespace

hipError_t launch_moe_tokens(const MoeTokens& m, hipStream_t stream) {
  const int most = m.T * m.topk < m.E ? m.T * m.topk : m.E;
  hipLaunchKernelGGL(moe_up_kernel, dim3((unsigned)(most * (m.F / kStrip))), dim3(64 * kUpWaves), 0, stream, m);
  hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)(m.K / kStrip)), dim3(64 * kDownWaves), 0, stream, m);
  return hipGetLastError();
}

}  // namespace fp8bs
