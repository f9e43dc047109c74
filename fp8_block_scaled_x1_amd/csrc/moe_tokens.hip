// A whole mixture-of-experts layer for a few tokens: two kernels that read each
// chosen expert's weights once (twice if more than 32 tokens chose it), and a
// third that joins sums where the output is narrow.
//
//   up    h = bf16(silu(G_e x) * (U_e x)) for every (expert, token) that meet
//   down  out_t = bf16(sum over t's experts of w * D_e h)
//
// For a few tokens the layer is the reading of its weights. A wave streams 32
// rows of them, 128 codes (a scale's reach) at a time and several such pieces
// ahead in registers, every load eight whole 128-byte rows: in the order that
// the matrix unit wants, 16 rows side by side, every lane of a load is a cache
// line of its own and the address unit takes three times as long. The lanes
// trade through 4 KB of LDS that only the wave uses, turn the codes into BF16
// (exact) and multiply them with the tokens' numbers, which come from L2. A
// 128-wide partial sum is scaled by its block's scale as it is added (FP32).
//
// up: a strip is 16 columns of h of one expert (16 rows of G and of U); a
// workgroup's waves share its inner dimension and add their sums through LDS, or
// have a strip each. down: a workgroup is 32 columns of the output and a share of
// the (expert, 128 wide piece) pairs, which its waves share in turn; an expert's sums go to its
// tokens' places in the wave's LDS when the wave is done with it. Both kernels
// work on an expert's own tokens, packed: with a place for each of 64 tokens
// instead, and zeros added to those that did not choose the expert, the
// registers spilled and reading h took longer than reading weights (64 tokens,
// 4 of 32 experts each, 540 us, now 260). A third launch adds the shares' sums,
// in order, where there are several (added by the last workgroup to be done
// instead, the fences at device scope cost 50 us).
//
// Which experts are chosen is found by every workgroup from the ids (at most
// 4096 of them): a bitmap in LDS, and a lane per token that looks for the
// workgroup's expert among its token's ids. An id outside [0, E) sets no bit.
//
// Bound: memory. 8 of 32 experts of 7168 x 2048 for one token 71 us (352 MB, 5.0
// TB/s), 32 tokens on all 32 of them 264 us (1410 MB, 5.3 TB/s). Small layers:
// launches and a workgroup's start, 5 tokens on 13 of 32 experts of 2048 x 1408
// 36 us (113 MB, 3.1 TB/s), 54 tokens on 8 of 768 x 2816 49 us (52 MB).

#include "attn_common.h"
#include "serve_internal.h"

namespace fp8bs {

namespace {

constexpr int kPiece = 128;       // inner numbers that share a scale
constexpr int kUpWaves = 4, kDownWaves = 8, kJoinThreads = 256;
constexpr int kDeep = 4;          // pieces of weights under way
constexpr int kStripBytes = 32 * kPiece;
constexpr int kSumStride = 36;    // of a token's 32 sums

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// Tokens of an expert that are worked on together. One that more than these
// chose is listed a second time (T <= 64), for the rest of them.
constexpr int kGroup = 32;

// Bytes of the routing, a multiple of 16.
__host__ __device__ __forceinline__ int routing_bytes_of(const MoeTokens& m) {
  return ((m.T > kGroup ? kMoeMaxExperts : 0) + kMoeMaxExperts / 16 + m.T * m.topk + 3) / 4 * 16;
}
// Listed pairs of an expert and a group of its tokens, at most.
__host__ __device__ __forceinline__ int most_listed(const MoeTokens& m) {
  const int slots = m.T * m.topk;
  return m.E + (m.T > kGroup ? slots / (kGroup + 1) : 0) < slots ? m.E + (m.T > kGroup ? slots / (kGroup + 1) : 0) : slots;
}
constexpr int kMostListed = kMoeMaxExperts + kMoeMaxTokens * kMoeMaxTopk / (kGroup + 1);

// The ids of all slots, a bit per chosen expert and one per expert in more
// than kGroup slots, in LDS.
struct Routing {
  uint32_t* bits;      // [2][kMoeMaxExperts / 32]
  int32_t* ids;
  __device__ __forceinline__ Routing(const MoeTokens& m, char* lds, int threads)
      : bits(reinterpret_cast<uint32_t*>(lds)), ids(reinterpret_cast<int32_t*>(lds) + kMoeMaxExperts / 16) {
    int32_t* const slots = ids + m.T * m.topk;      // of an expert
    if (threadIdx.x < kMoeMaxExperts / 16) bits[threadIdx.x] = 0;
    if (m.T > kGroup)
      for (int i = threadIdx.x; i < m.E; i += threads) slots[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < m.T * m.topk; i += threads) {
      const int e = m.ids[i];
      ids[i] = e;
      if (e >= 0 && e < m.E) {
        atomicOr(&bits[e >> 5], 1u << (e & 31));
        if (m.T > kGroup && atomicAdd(&slots[e], 1) == kGroup) atomicOr(&bits[kMoeMaxExperts / 32 + (e >> 5)], 1u << (e & 31));
      }
    }
    __syncthreads();
  }
};
// Lane l of the first 32: the experts of word l (`word`) that are chosen, or
// listed a second time, how many come before it; returns how many there are. Every lane of the wave takes part.
__device__ __forceinline__ int count_listed(const Routing& r, int time, uint32_t& word, int& before) {
  const int lane = threadIdx.x & 63;
  word = lane < kMoeMaxExperts / 32 ? r.bits[kMoeMaxExperts / 32 * time + lane] : 0;
  const int own = __popc(word);
  // inclusive sums of each row of 16 lanes, then the first row's total to the second
  int v = own;
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);      // from the lane 1, 2, 4, 8 below
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  const int row0 = __builtin_amdgcn_readlane(v, 15);
  if (lane >= 16) v += row0;
  before = v - own;
  return __builtin_amdgcn_readlane(v, 31);
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

// A piece of 32 rows as it is loaded: load i has rows 8i .. 8i+7, eight lanes a row.
struct Piece {
  u32x4 w[4];
};
// The wave's 4 KB of LDS; the 16-byte chunks of a row are permuted by the row,
// so that 8 rows at one chunk touch every bank once.
struct Trade {
  char* put;      // of this lane: row lane / 8, chunk lane % 8
  const char* get;
  int c0;         // of row lane % 16: chunks 2q and 2q + 1, q = lane / 16
  __device__ __forceinline__ explicit Trade(char* lds) {
    const int lane = threadIdx.x & 63;
    put = lds + (lane >> 3) * kPiece + (((lane & 7) ^ (lane >> 3)) << 4);
    get = lds + (lane & 15) * kPiece;
    c0 = ((2 * (lane >> 4)) ^ (lane & 7)) << 4;
  }
  __device__ __forceinline__ void write(const Piece& p) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4*>(put + 1024 * i) = p.w[i];
  }
  // The lane's 32 codes of row 16 * a + lane % 16: the inner numbers 32q + 8s .. of operand s.
  __device__ __forceinline__ void read(int a, bf16x8 (&o)[4]) const {
    const u32x4 x = *reinterpret_cast<const u32x4*>(get + 2048 * a + c0), y = *reinterpret_cast<const u32x4*>(get + 2048 * a + (c0 ^ 16));
    o[0] = e4m3_to_bf16(x[0], x[1]);
    o[1] = e4m3_to_bf16(x[2], x[3]);
    o[2] = e4m3_to_bf16(y[0], y[1]);
    o[3] = e4m3_to_bf16(y[2], y[3]);
  }
};

// A tile of 16 tokens' numbers of one piece: lane l has token l % 16.
struct Numbers {
  bf16x8 b[4];
  __device__ __forceinline__ void load(const uint16_t* p) {
#pragma unroll
    for (int s = 0; s < 4; ++s) b[s] = *reinterpret_cast<const bf16x8*>(p + 8 * s);
  }
};

template <int TILES, bool ALONE>
__global__ __launch_bounds__(64 * kUpWaves) void moe_up_kernel(const MoeTokens m) {
  constexpr int kShare = ALONE ? 1 : kUpWaves;      // waves of a strip
  extern __shared__ __align__(16) char lds[];      // routing; the waves' strips, then their sums
  __shared__ int tok[kGroup], slot_of[kGroup];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = m.F / 16 * kShare / kUpWaves;      // of a pair
  int rank = blockIdx.x / blocks;
  const int strip = (int)(blockIdx.x - rank * blocks) * (kUpWaves / kShare) + (ALONE ? wave : 0), part = ALONE ? 0 : wave;

  const Routing routing(m, lds, 64 * kUpWaves);
  char* const area = lds + routing_bytes_of(m);
  uint32_t word;
  int before;
  int group = 0, listed = count_listed(routing, 0, word, before);
  if (rank >= listed) {
    rank -= listed;
    group = 1;
    if (m.T <= kGroup || rank >= count_listed(routing, 1, word, before)) return;
  }
  const uint64_t hit = __ballot(rank >= before && rank < before + __popc(word));
  const int hl = __ffsll((unsigned long long)hit) - 1;
  const int e = __builtin_amdgcn_readfirstlane(32 * hl + nth_bit(__shfl(word, hl, 64), rank - __shfl(before, hl, 64)));

  const int pieces = m.K / kPiece;
  const int n = (pieces - part + kShare - 1) / kShare;      // this wave's: part, part + kShare, ..
  const uint8_t* gate = m.w_up + ((int64_t)e * 2 * m.F + strip * 16 + (lane >> 3)) * m.K + 16 * (lane & 7);
  const uint8_t* up = gate + (int64_t)m.F * m.K;
  // (past the wave's last piece that one again: loads under a condition would make the waits for earlier ones wait for these too)
  auto piece_at = [&](int i) { return part + kShare * max(0, min(i, n - 1)); };
  auto load = [&](Piece& p, int i) {
    const int64_t at = min(piece_at(i), pieces - 1) * kPiece;
    p.w[0] = *reinterpret_cast<const u32x4*>(gate + at);
    p.w[1] = *reinterpret_cast<const u32x4*>(gate + at + 8 * (int64_t)m.K);
    p.w[2] = *reinterpret_cast<const u32x4*>(up + at);
    p.w[3] = *reinterpret_cast<const u32x4*>(up + at + 8 * (int64_t)m.K);
  };
  Piece ring[kDeep];
#pragma unroll
  for (int i = 0; i < kDeep; ++i) load(ring[i], i);

  const Member mine = member_of<false>(m, routing, e);
  const uint64_t members = __ballot(mine.slot >= 0);
  const int count = min((int)__popcll(members) - kGroup * group, kGroup);
  if (count <= 0) return;      // (an expert that some token names twice may have fewer tokens than slots)
  const int place = (int)__popcll(members & ((1ull << lane) - 1ull)) - kGroup * group;
  if (wave == 0 && mine.slot >= 0 && place >= 0 && place < kGroup) {
    tok[place] = lane;
    slot_of[place] = mine.slot;
  }
  __syncthreads();

  const int tiles = (count + 15) / 16;
  const uint16_t* x[TILES];
#pragma unroll
  for (int i = 0; i < TILES; ++i) x[i] = m.x + (int64_t)tok[min(16 * i + (lane & 15), count - 1)] * m.K + 32 * (lane >> 4);
  const float* sg = m.s_up + ((int64_t)e * 2 * m.F / kPiece + strip * 16 / kPiece) * pieces;
  const float* su = sg + (int64_t)(m.F / kPiece) * pieces;
  const Trade trade(area + kStripBytes * wave);
  Numbers b[2][TILES];
  auto load_x = [&](Numbers (&to)[TILES], int i) {
    const int at = min(piece_at(i), pieces - 1) * kPiece;
#pragma unroll
    for (int j = 0; j < TILES; ++j)
      if (j == 0 || j < tiles) to[j].load(x[j] + at);
  };
  load_x(b[0], 0);

  f32x4 ag[TILES], au[TILES];
#pragma unroll
  for (int i = 0; i < TILES; ++i) ag[i] = au[i] = zero4();
  auto step = [&](int i, Piece& p, const Numbers (&now)[TILES], Numbers (&next)[TILES]) {
    const int c = min(piece_at(i), pieces - 1);
    const float fg = sg[c], fu = su[c];
    trade.write(p);
    load(p, i + kDeep);
    load_x(next, i + 1);
    bf16x8 g[4], u[4];
    trade.read(0, g);
    trade.read(1, u);
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      if (j == 0 || j < tiles) {
        f32x4 pg = zero4(), pu = zero4();
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          pg = mfma16(g[s], now[j].b[s], pg);
          pu = mfma16(u[s], now[j].b[s], pu);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ag[j][k] = fmaf(fg, pg[k], ag[j][k]);
          au[j][k] = fmaf(fu, pu[k], au[j][k]);
        }
      }
    }
  };
  static_assert(kDeep == 4, "the ring is unrolled");
  for (int i = 0; i < n; i += kDeep) {
    step(i, ring[0], b[0], b[1]);
    if (i + 1 >= n) break;
    step(i + 1, ring[1], b[1], b[0]);
    if (i + 2 >= n) break;
    step(i + 2, ring[2], b[0], b[1]);
    if (i + 3 >= n) break;
    step(i + 3, ring[3], b[1], b[0]);
  }
  auto gated = [](float g, float u) { return (__bf16)(g / (1.f + exp2_fast(-g * kLog2e)) * u); };
  if constexpr (ALONE) {      // a lane has four of the strip's columns, of token lane % 16
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const int at = 16 * i + (lane & 15);
      bf16x4 b;
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = gated(ag[i][j], au[i][j]);
      if (at < count) *reinterpret_cast<bf16x4*>(m.h + (int64_t)slot_of[at] * m.F + strip * 16 + 4 * (lane >> 4)) = b;
    }
    return;
  }
  typedef float Sums[TILES][2][64][4];
  Sums* const sums = reinterpret_cast<Sums*>(area);
  __syncthreads();      // the strips are done with
#pragma unroll
  for (int i = 0; i < TILES; ++i)
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
    reinterpret_cast<__bf16*>(m.h)[(int64_t)slot_of[at] * m.F + strip * 16 + col] = gated(g, u);
  }
}

template <int TILES>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down_kernel(const MoeTokens m) {
  extern __shared__ __align__(16) char lds[];      // routing; the waves' strips, then their sums
  __shared__ uint16_t listed[kMostListed];      // expert, and kMoeMaxExperts added for its second group of tokens
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int strips = m.K / 32, share = blockIdx.x / strips, strip = blockIdx.x - share * strips;

  const Routing routing(m, lds, 64 * kDownWaves);
  char* const area = lds + routing_bytes_of(m);
  uint32_t word;
  int before;
  int pairs = count_listed(routing, 0, word, before);
  if (wave == 0)
    for (; word; word &= word - 1) listed[before++] = (uint16_t)(32 * lane + __ffs((int)word) - 1);
  if (m.T > kGroup) {
    const int again = count_listed(routing, 1, word, before);
    if (wave == 0)
      for (; word; word &= word - 1) listed[pairs + before++] = (uint16_t)(kMoeMaxExperts + 32 * lane + __ffs((int)word) - 1);
    pairs += again;
  }
  // the wave's sums so far: [T][kSumStride], 32 used (the stride spreads tokens over the banks)
  float* const sums = reinterpret_cast<float*>(area + kDownWaves * kStripBytes);
  float* const own_sums = sums + wave * m.T * kSumStride;
  for (int i = lane; i < m.T * kSumStride / 4; i += 64) reinterpret_cast<f32x4*>(own_sums)[i] = zero4();
  __syncthreads();

  const int pieces = m.F / kPiece;
  const int units = pairs * pieces, parts = m.shares * kDownWaves, part = share * kDownWaves + wave;
  const int begin = (int)((int64_t)units * part / parts), end = (int)((int64_t)units * (part + 1) / parts);
  if (begin < end) {
    struct At {      // a unit: piece c of the n-th listed pair
      int n, c;
    };
    auto next = [&](At& a, int unit) {      // the one after `unit`; the last one stays
      if (unit + 1 >= end) return;
      if (++a.c == pieces) {
        a.c = 0;
        ++a.n;
      }
    };
    const uint8_t* down = m.w_down + (int64_t)(strip * 32 + (lane >> 3)) * m.F + 16 * (lane & 7);
    auto load = [&](Piece& p, const At& a) {
      const int e = __builtin_amdgcn_readfirstlane((int)listed[a.n]) % kMoeMaxExperts;
      const uint8_t* at = down + (int64_t)e * m.K * m.F + a.c * kPiece;
#pragma unroll
      for (int i = 0; i < 4; ++i) p.w[i] = *reinterpret_cast<const u32x4*>(at + 8 * i * (int64_t)m.F);
    };
    const Trade trade(area + kStripBytes * wave);
    At ahead{begin / pieces, 0};
    ahead.c = begin - ahead.n * pieces;
    At now = ahead;
    int to_load = begin;
    Piece ring[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      load(ring[i], ahead);
      next(ahead, to_load++);
    }
    int count = 0;               // the pair's tokens; tile i has those from 16 i on, a lane one
    const uint16_t* h[TILES];    // of the lane's token
    float w[TILES];
    int token[TILES];            // -1: none
    const float* sd = nullptr;
    Numbers b[2][TILES];
    auto load_h = [&](Numbers (&to)[TILES], int c) {
#pragma unroll
      for (int i = 0; i < TILES; ++i)
        if (i == 0 || 16 * i < count) to[i].load(h[i] + c * kPiece);
    };
    auto enter = [&](Numbers (&to)[TILES]) {      // the pair of unit `now`
      const int pair = __builtin_amdgcn_readfirstlane((int)listed[now.n]), e = pair % kMoeMaxExperts;
      const Member mine = member_of<true>(m, routing, e);
      const uint64_t members = __ballot(mine.slot >= 0);
      const int skip = pair < kMoeMaxExperts ? 0 : kGroup;
      count = min(max((int)__popcll(members) - skip, 0), kGroup);
      // the group's n-th token goes to lane n: (slot + 1, token), 0 where there is none; the others go to lanes that nobody asks
      const int place = (int)__popcll(members & ((1ull << lane) - 1ull)) - skip;
      const int to_lane = mine.slot >= 0 && place >= 0 && place < kGroup ? place : 63;
      const int what = __builtin_amdgcn_ds_permute(4 * to_lane, (mine.slot + 1) << 6 | lane);
      const int weight = __builtin_amdgcn_ds_permute(4 * to_lane, __float_as_int(mine.weight));
#pragma unroll
      for (int i = 0; i < TILES; ++i) {
        const int of = 16 * i + (lane & 15), x = __shfl(what, of, 64);
        token[i] = of < count ? x & 63 : -1;
        w[i] = __int_as_float(__shfl(weight, of, 64));
        // where there is no token: the row of the first
        h[i] = m.h + (int64_t)max((__shfl(what, of < count ? of : 0, 64) >> 6) - 1, 0) * m.F + 32 * (lane >> 4);
      }
      sd = m.s_down + ((int64_t)e * (m.K / kPiece) + strip * 32 / kPiece) * pieces;
      load_h(to, now.c);
    };
    f32x4 acc[TILES][2];
#pragma unroll
    for (int i = 0; i < TILES; ++i) acc[i][0] = acc[i][1] = zero4();
    auto leave = [&] {      // the pair's products to its tokens
#pragma unroll
      for (int i = 0; i < TILES; ++i) {
        if (token[i] >= 0) {
          float* const at = own_sums + token[i] * kSumStride + 4 * (lane >> 4);
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            f32x4 v = *reinterpret_cast<const f32x4*>(at + 16 * a);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = fmaf(w[i], acc[i][a][j], v[j]);
            *reinterpret_cast<f32x4*>(at + 16 * a) = v;
          }
        }
        acc[i][0] = acc[i][1] = zero4();
      }
    };
    enter(b[0]);
    auto step = [&](int unit, Piece& p, Numbers (&cur)[TILES], Numbers (&nxt)[TILES]) {
      const float f = sd[now.c];
      trade.write(p);
      load(p, ahead);
      next(ahead, to_load++);
      const bool stays = now.c + 1 < pieces;
      if (stays) load_h(nxt, now.c + 1);
      bf16x8 d[2][4];
      trade.read(0, d[0]);
      trade.read(1, d[1]);
#pragma unroll
      for (int i = 0; i < TILES; ++i) {
        if (i == 0 || 16 * i < count) {
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            f32x4 sum = zero4();
#pragma unroll
            for (int s = 0; s < 4; ++s) sum = mfma16(d[a][s], cur[i].b[s], sum);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][a][j] = fmaf(f, sum[j], acc[i][a][j]);
          }
        }
      }
      next(now, unit);
      if (!stays || unit + 1 == end) leave();
      if (!stays && unit + 1 < end) enter(nxt);
    };
    for (int unit = begin; unit < end; unit += kDeep) {
      step(unit, ring[0], b[0], b[1]);
      if (unit + 1 >= end) break;
      step(unit + 1, ring[1], b[1], b[0]);
      if (unit + 2 >= end) break;
      step(unit + 2, ring[2], b[0], b[1]);
      if (unit + 3 >= end) break;
      step(unit + 3, ring[3], b[1], b[0]);
    }
  }
  __syncthreads();
  // a thread: a token and one of the strip's columns
  auto sum_of = [&](int t, int col) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) v += sums[(w * m.T + t) * kSumStride + col];
    return v;
  };
  __bf16* const out = reinterpret_cast<__bf16*>(m.out) + strip * 32;
  if (m.shares == 1) {
    for (int at = threadIdx.x; at < 32 * m.T; at += 64 * kDownWaves) out[(int64_t)(at >> 5) * m.K + (at & 31)] = (__bf16)sum_of(at >> 5, at & 31);
    return;
  }
  float* const mine = m.part + (int64_t)share * m.T * m.K + strip * 32;
  for (int at = threadIdx.x; at < 32 * m.T; at += 64 * kDownWaves) mine[(int64_t)(at >> 5) * m.K + (at & 31)] = sum_of(at >> 5, at & 31);
}

// The shares' sums, in order: a thread has four numbers.
__global__ __launch_bounds__(kJoinThreads) void moe_join_kernel(const MoeTokens m) {
  const int64_t all = (int64_t)m.T * m.K, at = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 4;
  if (at >= all) return;
  f32x4 v = *reinterpret_cast<const f32x4*>(m.part + at);
  for (int i = 1; i < m.shares; ++i) v += *reinterpret_cast<const f32x4*>(m.part + i * all + at);
  bf16x4 b;
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = (__bf16)v[j];
  *reinterpret_cast<bf16x4*>(m.out + at) = b;
}

template <int TILES>
void launch_tiles(const MoeTokens& m, hipStream_t stream) {
  // the waves' strips, later their sums
  constexpr size_t sums = sizeof(float) * TILES * 2 * 64 * 4, area = sums > kStripBytes ? sums : (size_t)kStripBytes;
  // Waves have strips of their own where there are enough for the device, and
  // none has to wait for the others; shared by a workgroup's waves, strips start
  // sooner. The host knows how many there are at most (experts whose ids all lie
  // elsewhere have none). Whole calls, shared and own, us, "in" so many experts:
  // the others elsewhere, strips in brackets. Two tiles:
  //   32 tokens on 8 experts of 1024 x 512 (256) 20.7 and 25.4, 16 of 1024 x 1024
  //   (1024) 33.1 and 29.3, 32 of 2048 x 512 in 256 (1024) 29.0 and 26.0, 32 of 3584
  //   x 2048 (4096) 156 and 144, 16 of 7168 x 1536 (1536) 144 and 155, 32 of 7168 x
  //   2048 (4096) 281 and 266, but in 256 180 and 189; 54 tokens on 8 of 2048 x 512
  //   (672) 35.5 and 40.6, 64 of 4608 x 1536 (7392) 322 and 307. Rows a multiple of
  //   4096 bytes apart: 32 tokens on 32 of 4096 x 2048 (4096) 184 and 190, of 8192 x
  //   2048 311 and 327.
  // One tile:
  //   5 tokens on 8 of 512 x 512 (256) 14.5 and 15.3, 16 of 512 x 1024 (1024) 21.5
  //   and 19.9, 32 of 2048 x 512 in 64 (960) 21.9 and 24.2, 32 of 2048 x 2048 (4096)
  //   89.5 and 84.3, of 2560 x 2048 (3840) 74.1 and 71.8, of 3584 x 2048 in 64 (3840)
  //   72.7 and 74.1, of 7168 x 2048 (4096) 241 and 246; 16 tokens on 32 of 2560 x
  //   1408 (2816) 81.7 and 79.0, but in 96 66.6 and 68.6.
  const int64_t up_strips = (int64_t)most_listed(m) * (m.F / 16), some = 3 * (int64_t)m.K / 2;
  const bool own = TILES == 1 ? m.K <= 2560 && up_strips >= some
                              : m.K % 4096 != 0 && up_strips >= (m.K > 4096 ? 4096 : some < 1024 ? some : 1024);
  if (own)
    hipLaunchKernelGGL((moe_up_kernel<TILES, true>), dim3((unsigned)(up_strips / kUpWaves)), dim3(64 * kUpWaves),
                       routing_bytes_of(m) + kUpWaves * area, stream, m);
  else
    hipLaunchKernelGGL((moe_up_kernel<TILES, false>), dim3((unsigned)up_strips), dim3(64 * kUpWaves),
                       routing_bytes_of(m) + kUpWaves * area, stream, m);
  hipLaunchKernelGGL(moe_down_kernel<TILES>, dim3((unsigned)(m.shares * (m.K / 32))), dim3(64 * kDownWaves),
                     routing_bytes_of(m) + kDownWaves * (kStripBytes + sizeof(float) * m.T * kSumStride), stream, m);
  if (m.shares > 1)
    hipLaunchKernelGGL(moe_join_kernel, dim3((unsigned)(((int64_t)m.T * m.K / 4 + kJoinThreads - 1) / kJoinThreads)), dim3(kJoinThreads), 0, stream, m);
}

}  // namespace

// Shares of the second kernel's work: some 192 workgroups where the output has
// few strips of columns, but no more than 256, a compute unit each. 5 tokens on
// experts of 2048 x 1408 (64 strips, 3 shares) 50.6 us, unshared 65.0, two shares
// 54.0, five 57.6; 64 tokens on 64 of 2048 x 1024 97, unshared 146, five shares
// 111; 2 tokens on 8 of 512 x 512 (16, 12 shares) 13.8, 8 shares 13.0, 16 15.0. 32
// tokens on 16 experts of 4096 x 1024 (128 strips) two shares 57.4, one 63.0, of
// 4352 x 1024 (136) 69.5 and 62.2, of 5888 x 1024 (184) 78.2 and 70.6.
int moe_shares(int64_t K) {
  const int64_t strips = K / 32, some = (192 + strips - 1) / strips, most = 256 / strips;
  return (int)(some < most ? some : most < 1 ? 1 : most);
}

hipError_t launch_moe_tokens(const MoeTokens& m, hipStream_t stream) {
  // Places for one tile of tokens take fewer registers and leave three workgroups
  // on a compute unit for two. One tile and two, strips shared: 5 tokens on 32
  // experts of 1024 x 2048 49.9 and 57.3 us, of 2048 x 2048 74.3 and 80.1, of 7168 x
  // 2048 190 and 191; 16 tokens of 4096 x 2048 160 and 161, of 7168 x 512 on 8 of them
  // 30.7 and 29.7. Strips of their own: 16 tokens on 32 of 1024 x 2048 55.7 and 56.0.
  // Above 16, an expert's second tile shares its weights.
  if (m.T <= 16)
    launch_tiles<1>(m, stream);
  else
    launch_tiles<2>(m, stream);
  return hipGetLastError();
}

}  // namespace fp8bs
