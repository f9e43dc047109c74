// Latent attention in its absorbed form for decoding, over a paged cache, and
// the same for a batch that shares a long prefix.
//
// With the up-projections folded into the queries and the output, every head
// of a token attends to one shared 576-wide key c_j (512 latent numbers and 64
// rotary ones) whose latent part is also the value:
//   S_ij = scale * q_i . c_j,  P = softmax(S),  O_i = sum_j P_ij c_j[0:512].
// A request's heads (times its query tokens) are the rows of one product, so
// the cached tokens are read once for all of them.
//
// Work: the tokens of all requests are cut into tiles of 64, numbered request
// by request, and group g of G takes the contiguous range
// [g*TT/G, (g+1)*TT/G) of the TT tiles: every group has the same work whatever
// the lengths are, the host never needs the lengths, and a request cut between
// groups leaves at most one partial (maximum, sum, unnormalised output) per
// group and end, which a second kernel joins. A workgroup is one block of NR
// rows in one group; the row blocks of a group sit on one XCD, next to each
// other in time, so the L2 serves the tiles to all but the first.
//
// Tile loop (4 waves): wave w forms the scores of its 16 tokens for all NR
// rows, the waves meet over the row maxima and exchange probabilities through
// LDS, then wave w adds the 64 tokens' values into its 128 output columns. So
// a tile is read from LDS once as keys and once as values whatever NR is (a
// split of the rows over the waves would read it four times).
//
// FP8 cache: codes become BF16 exactly; a group's scale multiplies the partial
// score of its 128 columns (FP32) and the probability that meets its 128
// output columns (wave w's columns are group w), so the latent vector itself
// is never rounded.
//
// Roundings below 32 bits: probabilities (times the scale, FP8) to BF16 for
// the matrix unit (relative 2^-8 at most each, on the terms of a mean), and the output.

#include <atomic>

#include "attn_common.h"
#include "attn_internal.h"

namespace fp8bs {

namespace {

constexpr int kTile = 64;            // tokens per tile
constexpr int kLatent = 512, kRope = 64, kKey = kLatent + kRope;
constexpr int kWaitVmcnt0 = 0x0F70;   // s_waitcnt vmcnt(0), the other counters left alone
constexpr int kJoinThreads = 256;
// The weights' reference only follows the running maximum once that is more
// than 2^8 above it: weights up to 2^8 cost no precision in FP32 or BF16, and
// the accumulators are rescaled a few times per request instead of per tile.
constexpr float kSlack = 8.f;

template <bool FP8, int NW>
struct Tile {
  static constexpr int kRowBytes = FP8 ? kLatent : 2 * kLatent;
  static constexpr int kLatentBytes = kTile * kRowBytes;
  static constexpr int kRopeBytes = kTile * 2 * kRope;
  static constexpr int kScaleBytes = FP8 ? kTile * 16 : 0;
  static constexpr int kBytes = kLatentBytes + kRopeBytes + kScaleBytes;
  static constexpr int kRows = kTile / NW;                  // that one wave loads
  static constexpr int kLoads = FP8 ? kRows / 2 + kRows / 8 + 1 : kRows + kRows / 8;
};

// 16-byte chunk swizzles of LDS row r (the loads permute the source chunks, so
// LDS itself is written linearly). The LDS serves a 16-byte read in groups of
// 16 lanes, {0-3, 12-15, 20-27}, {4-11, 16-19, 28-31} and the same from 32, and
// an 8-byte read in halves of the wave. A key read (lane: row lane%16, chunk
// 4*ks + lane/16) thus meets rows 0-3, 12-15 at one chunk and 4-11 at its
// neighbour; a value read rows 0-7 (8-15) at a pair of chunks, or, for bytes,
// rows 0-7 and 16-23 (8-15, 24-31) at one chunk. All of these touch every bank
// once. Rows of 128 bytes (rotary part): key reads do.
__device__ __forceinline__ int swz_bf16(int r) { return (((r & 7) ^ ((r >> 1) & 4)) << 1) | ((r >> 3) & 1); }
__device__ __forceinline__ int swz_fp8(int r) { return swz_bf16(r) ^ ((r >> 4) & 1); }
__device__ __forceinline__ int swz_rope(int r) { return (r >> 1) & 7; }

// The tiles of a request, and the request a tile belongs to.
struct Cursor {
  int b;        // request
  int len;      // its tokens
  int tile;     // tile inside it
  int tiles;    // its tiles
  int left;     // tiles left in the group's range, this one included
};

__device__ __forceinline__ int clamp_len(const MlaDecode& p, int b) { return min(max(p.lens[b * p.len_stride], 0), p.max_len); }

__device__ __forceinline__ void advance(const MlaDecode& p, Cursor& c) {
  --c.left;
  if (++c.tile < c.tiles || c.left <= 0) return;
  do {
    ++c.b;
    c.len = c.b < p.B ? __builtin_amdgcn_readfirstlane(clamp_len(p, c.b)) : 0;
  } while (c.len == 0 && c.b < p.B);
  c.tile = 0;
  c.tiles = (c.len + kTile - 1) / kTile;
}

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// All tiles of the batch.
__device__ __forceinline__ int total_tiles(const MlaDecode& p) {
  int sum = 0;
  for (int b = threadIdx.x & 63; b < p.B; b += 64) sum += (clamp_len(p, b) + kTile - 1) / kTile;
  return __builtin_amdgcn_readfirstlane(wave_sum(sum));
}

// The cursor of tile t (t < all tiles).
__device__ __forceinline__ Cursor locate(const MlaDecode& p, int t, int left) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    const int len = b0 + lane < p.B ? clamp_len(p, b0 + lane) : 0;
    const int n = (len + kTile - 1) / kTile;
    int incl = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
    const uint64_t hit = __ballot(t < base + incl);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      Cursor c;
      c.b = b0 + l;
      c.len = __builtin_amdgcn_readfirstlane(__shfl(len, l, 64));
      c.tiles = __builtin_amdgcn_readfirstlane(__shfl(n, l, 64));
      c.tile = __builtin_amdgcn_readfirstlane(t - base - __shfl(incl - n, l, 64));
      c.left = left;
      return c;
    }
    base += __shfl(incl, 63, 64);
  }
  return Cursor{p.B, 0, 0, 0, 0};
}

__device__ __forceinline__ int range_start(int g, int total, int groups) {
  return (int)((int64_t)g * total / groups);
}

// The flat cache token (page * page size + slot) of token `tok`, given its
// page's entry in the block table.
__device__ __forceinline__ int page_of(const MlaDecode& p, int tok) {
  return (int)(((uint64_t)(uint32_t)tok * p.page_magic) >> p.page_shift);
}

// Token of row 16*rg + lane%16 of a tile. Tokens past the end repeat the last
// one: always cached, and masked by its position.
__device__ __forceinline__ int row_token(const Cursor& c, int rg, int lane) {
  return min(c.tile * kTile + 16 * rg + (lane & 15), c.len - 1);
}

__device__ __forceinline__ void load_entries(const MlaDecode& p, const Cursor& c, int rg, int lane, uint32_t lds) {
  const int tok = row_token(c, rg, lane);
  dma4(p.table + (int64_t)c.b * p.table_stride + page_of(p, tok), lds);
}

// The wave's kRows rows of a tile, whose block-table entries (of the 16-row
// group they are in) lane%16 holds.
template <bool FP8, int NW>
__device__ __forceinline__ void load_tile(const MlaDecode& p, const Cursor& c, int w, int lane, int entry,
                                          uint32_t lds) {
  using T = Tile<FP8, NW>;
  const int rg = w * T::kRows / 16, r0 = w * T::kRows % 16;
  const int tok = row_token(c, rg, lane);
  const int pg = min(max(entry, 0), p.pages - 1);
  const int64_t flat = (int64_t)pg * p.page + (tok - page_of(p, tok) * p.page);
  const int lo = (int)(uint32_t)flat, hi = (int)(flat >> 32);
  if constexpr (!FP8) {
    // rows of 1024 latent bytes, one per load: the row is wave-uniform
    const int chunk = opaque((lane ^ swz_bf16(r0)) << 4);
#pragma unroll
    for (int i = 0; i < T::kRows; ++i) {
      const int64_t f = ((int64_t)__builtin_amdgcn_readlane(hi, r0 + i) << 32) |
                        (uint32_t)__builtin_amdgcn_readlane(lo, r0 + i);
      dma16_s(p.cache + f * (2 * kKey), (uint32_t)(chunk ^ (swz_bf16(i) << 4)),
              lds + (16 * rg + r0 + i) * T::kRowBytes);
    }
  } else {
    // two rows of 512 code bytes per load
#pragma unroll
    for (int i = 0; i < T::kRows; i += 2) {
      const int64_t f0 = ((int64_t)__builtin_amdgcn_readlane(hi, r0 + i) << 32) |
                         (uint32_t)__builtin_amdgcn_readlane(lo, r0 + i);
      const int64_t f1 = ((int64_t)__builtin_amdgcn_readlane(hi, r0 + i + 1) << 32) |
                         (uint32_t)__builtin_amdgcn_readlane(lo, r0 + i + 1);
      const int r = 16 * rg + r0 + i + (lane >> 5);
      dma16(p.cache + (lane < 32 ? f0 : f1) * kLatent + (((lane & 31) ^ swz_fp8(r)) << 4),
            lds + (16 * rg + r0 + i) * T::kRowBytes);
    }
  }
  // rotary part: 8 rows of 128 bytes per load
#pragma unroll
  for (int i = 0; i < T::kRows; i += 8) {
    const int src = r0 + i + (lane >> 3);
    const int64_t f = ((int64_t)__shfl(hi, src, 64) << 32) | (uint32_t)__shfl(lo, src, 64);
    const int chunk = (lane & 7) ^ swz_rope(16 * rg + src);
    const char* row = FP8 ? p.rope + f * (2 * kRope) : p.cache + f * (2 * kKey) + 2 * kLatent;
    dma16(row + (chunk << 4), lds + T::kLatentBytes + (16 * rg + r0 + i) * (2 * kRope));
  }
  if constexpr (FP8) {
    // the scales of the 16-row group (with 8 waves two of them load the same)
    const int src = lane >> 2;
    const int64_t f = ((int64_t)__shfl(hi, src, 64) << 32) | (uint32_t)__shfl(lo, src, 64);
    dma4(p.scales + f * 16 + (lane & 3) * 4, lds + T::kLatentBytes + T::kRopeBytes + 16 * rg * 16);
  }
}

// TEAMS teams of 4 waves, each with its own NR rows, share the tiles in LDS.
template <int NR, int TEAMS, bool FP8, int NBUF>
__global__ __launch_bounds__(256 * TEAMS) void mla_decode_kernel(const MlaDecode p) {
  constexpr int NW = 4 * TEAMS;
  using T = Tile<FP8, NW>;
  constexpr int NB = NR / 16;                       // 16-row blocks of a team
  constexpr int kProbBytes = kTile * NR * (FP8 ? 4 : 2);
  __shared__ __align__(1024) char tiles[NBUF * T::kBytes];
  __shared__ __align__(16) char team_probs[TEAMS * kProbBytes];
  __shared__ __align__(16) float team_stat[TEAMS * 4 * NR];
  __shared__ __align__(16) int entries[NW][64];

  const int lane = threadIdx.x & 63, n16 = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wave & 3, team = wave >> 2, rg = wave * T::kRows / 16;
  char* const probs = team_probs + team * kProbBytes;
  float* const stat = team_stat + team * 4 * NR;

  // workgroup -> (group, row block): workgroups are dealt over the XCDs one by
  // one; renumbered so that an XCD's are consecutive, row blocks of a group first
  const int per = gridDim.x / kAttnXcds, rest = gridDim.x % kAttnXcds;
  const int xcd = blockIdx.x % kAttnXcds;
  const int wg = xcd * per + min(xcd, rest) + blockIdx.x / kAttnXcds;
  const int g = wg / p.row_blocks;
  const int row0 = ((wg - g * p.row_blocks) * TEAMS + team) * NR;      // the team's first row
  const int total = total_tiles(p);
  const int t0 = range_start(g, total, p.groups), t1 = range_start(g + 1, total, p.groups);
  if (t0 >= t1) return;

  const uint32_t lds_tiles = lds_offset(tiles), lds_entries = lds_offset(entries[wave]);
  Cursor cur = locate(p, t0, t1 - t0);
  Cursor nxt = cur;      // the tile that is loaded next
  Cursor ent = cur;      // the tile whose block-table entries are fetched next
#pragma unroll
  for (int i = 0; i < NBUF - 1; ++i) {
    if (nxt.left > 0) {
      load_entries(p, ent, rg, lane, lds_entries);
      advance(p, ent);
      attn_wait<0>();
      load_tile<FP8, NW>(p, nxt, wave, lane, entries[wave][lane & 15], lds_tiles + i * T::kBytes);
      advance(p, nxt);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }
  if (ent.left > 0) {
    load_entries(p, ent, rg, lane, lds_entries);
    advance(p, ent);
  }

  // LDS offsets of this lane: the swizzles only touch bits that the row and
  // tile offsets leave free, so the chunk is picked by an XOR
  const int krow = 16 * w + n16;                                   // key reads: the wave's token n16
  const int key0 = krow * T::kRowBytes + ((g4 ^ (FP8 ? swz_fp8(krow) : swz_bf16(krow))) << 4);
  const int rope0 = T::kLatentBytes + krow * (2 * kRope) + ((g4 ^ swz_rope(krow)) << 4);
  const int vrow = FP8 ? ((n16 >> 1) & 3) + 4 * g4 + 16 * (n16 >> 3) : 4 * g4 + (n16 >> 2);
  const int val0 = vrow * T::kRowBytes + 8 * (n16 & 1) +
                   (FP8 ? 256 * (w >> 1) + ((8 * (w & 1) ^ swz_fp8(vrow)) << 4)
                        : 256 * w + ((((n16 >> 1) & 1) ^ swz_bf16(vrow)) << 4));

  bf16x8 qf[NB][kKey / 32];
  f32x4 acc[8][NB];
  float m[NB], l[NB];
  int limit[NB];
  bool first = true;
  int buf = 0;

  while (cur.left > 0) {      // a request's part of the range
    const bool whole = cur.tile == 0 && cur.left >= cur.tiles;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = min(row0 + nb * 16 + n16, p.rows - 1);
      const uint16_t* qr = p.q + min((int64_t)cur.b * p.rows + row, p.all_rows - 1) * kKey;
#pragma unroll
      for (int ks = 0; ks < kKey / 32; ++ks) {
        // FP8: a lane reads 16 codes at a time, the slots of two k steps
        const int col = FP8 && ks < 16 ? 64 * (ks >> 1) + 16 * g4 + 8 * (ks & 1) : 32 * ks + 8 * g4;
        qf[nb][ks] = *reinterpret_cast<const bf16x8*>(qr + col);
      }
      limit[nb] = cur.len - (p.tokens - 1 - row / p.heads);
      m[nb] = neg_inf();
      l[nb] = 0.f;
#pragma unroll
      for (int d = 0; d < 8; ++d) acc[d][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // said to the compiler, which would otherwise wait for the queries inside
    // the tile loop and with them for the tiles in flight
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);

    for (bool last = false; !last;) {
    if (nxt.left > 0 && NBUF > 2 && cur.left > 1)
      attn_wait<(NBUF - 2) * (T::kLoads + 1)>();
    else
      attn_wait<0>();
    attn_barrier();
    if (nxt.left > 0) {
      const int entry = entries[wave][lane & 15];
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (ent.left > 0) {
        load_entries(p, ent, rg, lane, lds_entries);
        advance(p, ent);
      }
      const int nbuf = buf == 0 ? NBUF - 1 : buf - 1;
      load_tile<FP8, NW>(p, nxt, wave, lane, entry, lds_tiles + nbuf * T::kBytes);
      advance(p, nxt);
    }
    const char* tl = tiles + buf * T::kBytes;

    // scores of this wave's 16 tokens: D[token 4*g4 + i][row n16]
    f32x4 s[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) s[nb] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (!FP8) {
      const int key = opaque(key0);
#pragma unroll
      for (int ks = 0; ks < 16; ++ks) {
        const bf16x8 a = lds_bf16x8(tl + (key ^ ((ks & 3) << 6)) + (ks >> 2) * 256);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) s[nb] = mfma16(a, qf[nb][ks], s[nb]);
      }
    } else {
      const int key = opaque(key0);
      const char* sp = tl + T::kLatentBytes + T::kRopeBytes + (16 * w + 4 * g4) * 16;
      float sc[4][4];     // [token i][group]
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(sp + 16 * i);
#pragma unroll
        for (int q = 0; q < 4; ++q) sc[i][q] = v[q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 part[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) part[nb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int kp2 = 2 * q + h;      // 64 columns
          const uint4 c = *reinterpret_cast<const uint4*>(tl + (key ^ ((kp2 & 3) << 6)) + (kp2 >> 2) * 256);
          const bf16x8 a0 = e4m3_to_bf16(c.x, c.y), a1 = e4m3_to_bf16(c.z, c.w);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) part[nb] = mfma16(a0, qf[nb][2 * kp2], part[nb]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) part[nb] = mfma16(a1, qf[nb][2 * kp2 + 1], part[nb]);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[nb][i] = fmaf(sc[i][q], part[nb][i], s[nb][i]);
      }
    }
    {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const bf16x8 a = lds_bf16x8(tl + (rope0 ^ (ks << 6)));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) s[nb] = mfma16(a, qf[nb][16 + ks], s[nb]);
      }
    }

    // row maxima over the tile
    const int tok0 = cur.tile * kTile + 16 * w + 4 * g4;
    const bool edge = (cur.tile + 1) * kTile > cur.len - (p.tokens - 1);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[nb][i] *= p.scale_log2;
        if (edge && tok0 + i >= limit[nb]) s[nb][i] = neg_inf();
      }
      float v = fmaxf(fmaxf(s[nb][0], s[nb][1]), fmaxf(s[nb][2], s[nb][3]));
      v = fmaxf(v, __shfl_xor(v, 16, 64));
      v = fmaxf(v, __shfl_xor(v, 32, 64));
      if (g4 == 0) stat[w * NR + nb * 16 + n16] = v;
    }
    attn_barrier();

    // probabilities against the new maxima, into LDS as the value product's operand
    float ref[NB];
    bool grown = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int n = nb * 16 + n16;
      ref[nb] = fmaxf(fmaxf(stat[n], stat[NR + n]), fmaxf(stat[2 * NR + n], stat[3 * NR + n]));
      grown |= ref[nb] > m[nb] + kSlack;
    }
    if (__any(grown)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float mn = fmaxf(m[nb], ref[nb]);
        const float alpha = mn == neg_inf() ? 1.f : exp2_fast(m[nb] - mn);
        m[nb] = mn;
        l[nb] *= alpha;
#pragma unroll
        for (int d = 0; d < 8; ++d) acc[d][nb] *= alpha;
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      ref[nb] = m[nb] == neg_inf() ? 0.f : m[nb];      // nothing visible yet: every weight is 0
      f32x4 e;
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = exp2_fast(s[nb][i] - ref[nb]);
      l[nb] += (e[0] + e[1]) + (e[2] + e[3]);
      // [32-token step w/2][row block][lane], half w%2 of the lane's 8 slots
      const int at = (((w >> 1) * NB + nb) * 64 + lane) * 2 + (w & 1);
      if constexpr (FP8) {
        *reinterpret_cast<f32x4*>(probs + 16 * at) = e;
      } else {
        bf16x4 b;
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = (__bf16)e[i];
        *reinterpret_cast<bf16x4*>(probs + 8 * at) = b;
      }
    }
    attn_barrier();

    // output columns 128w .. +127: D[column 4*g4 + i][row n16]
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int val = opaque(val0);
      bf16x8 pb[NB];
      if constexpr (FP8) {
        const float* sp = reinterpret_cast<const float*>(tl + T::kLatentBytes + T::kRopeBytes) + w;
        float sc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sc[j] = sp[4 * (32 * kk + 16 * (j >> 2) + 4 * g4 + (j & 3))];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const f32x4* e = reinterpret_cast<const f32x4*>(probs + ((kk * NB + nb) * 64 + lane) * 32);
          const f32x4 e0 = e[0], e1 = e[1];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            pb[nb][j] = (__bf16)(e0[j] * sc[j]);
            pb[nb][4 + j] = (__bf16)(e1[j] * sc[4 + j]);
          }
        }
      } else {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) pb[nb] = lds_bf16x8(probs + ((kk * NB + nb) * 64 + lane) * 16);
      }
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        bf16x8 a;
        if constexpr (FP8) {
          const i32x2 c = lds_tr8(tl + (val ^ (d << 4)) + 32 * kk * T::kRowBytes);
          a = e4m3_to_bf16((uint32_t)c[0], (uint32_t)c[1]);
        } else {
          const char* vp = tl + (val ^ (d << 5)) + 32 * kk * T::kRowBytes;
          a = join(lds_tr16(vp), lds_tr16(vp + 16 * T::kRowBytes));
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[d][nb] = mfma16(a, pb[nb], acc[d][nb]);
      }
    }

    last = cur.tile + 1 == cur.tiles || cur.left == 1;
    if (last) {
      // sums over the lanes' and waves' tokens
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float v = l[nb];
        v += __shfl_xor(v, 16, 64);
        v += __shfl_xor(v, 32, 64);
        if (g4 == 0) stat[w * NR + nb * 16 + n16] = v;
      }
      attn_barrier();
      const bool final = whole && !p.join;
      const int64_t part = whole ? 2 * p.groups + cur.b : 2 * g + (first ? 0 : 1);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int n = nb * 16 + n16, row = row0 + n;
        const float sum = (stat[n] + stat[NR + n]) + (stat[2 * NR + n] + stat[3 * NR + n]);
        if (row < p.rows && (int64_t)cur.b * p.rows + row < p.all_rows) {
          if (final) {
            const int64_t o = (int64_t)cur.b * p.rows + row;
            const float inv = sum > 0.f ? 1.f / sum : 0.f;
            uint16_t* op = p.out + o * kLatent + 128 * w + 4 * g4;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              bf16x4 b;
#pragma unroll
              for (int i = 0; i < 4; ++i) b[i] = (__bf16)(acc[d][nb][i] * inv);
              *reinterpret_cast<bf16x4*>(op + 16 * d) = b;
            }
            if (w == 0 && g4 == 0) p.lse[o] = sum > 0.f ? (m[nb] + __builtin_log2f(sum)) * kLn2 : neg_inf();
          } else {
            const int64_t o = part * p.rows + row;
            float* op = p.part + o * kLatent + 128 * w + 4 * g4;
#pragma unroll
            for (int d = 0; d < 8; ++d) *reinterpret_cast<f32x4*>(op + 16 * d) = acc[d][nb];
            if (w == 0 && g4 == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * o) = make_float2(m[nb], sum);
          }
        }
      }
      first = false;
    }
    advance(p, cur);
    buf = buf + 1 == NBUF ? 0 : buf + 1;
    }
  }
}

// Joins the partials of the rows whose request was cut between groups (and, in
// the shared form, the prefix's with the request's own). One wave per row,
// lane l columns 8l .. 8l+7.
struct Joiner {
  float m = neg_inf(), l = 0.f;
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(const MlaDecode& p, int64_t part, int row, int lane) {
    const int64_t at = part * p.rows + row;
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
    const f32x4* src = reinterpret_cast<const f32x4*>(p.part + at * kLatent + 8 * lane);
    const f32x4 a = src[0], b = src[1];
    const float mn = fmaxf(m, ml.x), ref = mn == neg_inf() ? 0.f : mn;
    const float x = exp2_fast(m - ref), y = exp2_fast(ml.x - ref);
    l = fmaf(l, x, ml.y * y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = fmaf(o[i], x, a[i] * y);
      o[4 + i] = fmaf(o[4 + i], x, b[i] * y);
    }
    m = mn;
  }
};

// Adds the partials of one row; false if the row's result is written already.
__device__ __forceinline__ bool add_pieces(const MlaDecode& p, int64_t o, int lane, Joiner& j) {
  const int b = (int)(o / p.rows), row = (int)(o - (int64_t)b * p.rows);
  // tiles before the request, its own and all
  int before = 0, all = 0;
  for (int x = lane; x < p.B; x += 64) {
    const int n = (clamp_len(p, x) + kTile - 1) / kTile;
    all += n;
    before += x < b ? n : 0;
  }
  all = wave_sum(all);
  before = wave_sum(before);
  const int own = (clamp_len(p, b) + kTile - 1) / kTile;
  if (own == 0) return true;
  // the group of tile t is the last whose range starts at or before it
  auto group_of = [&](int t) {
    int g = (int)((int64_t)t * p.groups / all);
    while (g + 1 < p.groups && range_start(g + 1, all, p.groups) <= t) ++g;
    while (range_start(g, all, p.groups) > t) --g;
    return g;
  };
  const int g0 = group_of(before), g1 = group_of(before + own - 1);
  if (g0 == g1) {
    if (!p.join) return false;
    j.add(p, 2 * (int64_t)p.groups + b, row, lane);
    return true;
  }
  for (int g = g0; g <= g1; ++g) {
    const int start = range_start(g, all, p.groups);
    if (start == range_start(g + 1, all, p.groups)) continue;     // an empty range
    j.add(p, 2 * (int64_t)g + (start >= before ? 0 : 1), row, lane);
  }
  return true;
}

__global__ __launch_bounds__(kJoinThreads) void mla_join_kernel(const MlaDecode p, const MlaDecode prefix) {
  const int lane = threadIdx.x & 63;
  const int64_t o = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (o >= p.all_rows) return;
  Joiner j;
  if (!add_pieces(p, o, lane, j)) return;
  if (p.join) add_pieces(prefix, o, lane, j);
  const float inv = j.l > 0.f ? 1.f / j.l : 0.f;
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (__bf16)(j.o[i] * inv);
  *reinterpret_cast<bf16x8*>(p.out + o * kLatent + 8 * lane) = v;
  if (lane == 0) p.lse[o] = j.l > 0.f ? (j.m + __builtin_log2f(j.l)) * kLn2 : neg_inf();
}

int compute_units() {
  static std::atomic<int> cached[64] = {};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (cached[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
    cached[dev] = n;
  }
  return cached[dev];
}

template <int NR, int TEAMS>
void launch_rows(const MlaDecode& p, bool fp8, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.groups * p.row_blocks)), block(256 * TEAMS);
  if (fp8)
    hipLaunchKernelGGL((mla_decode_kernel<NR, TEAMS, true, NR * TEAMS == 16 ? 3 : 2>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((mla_decode_kernel<NR, TEAMS, false, 2>), grid, block, 0, stream, p);
}

void launch_tiles(const MlaDecode& p, bool fp8, hipStream_t stream) {
  if (p.block_rows == 16)
    launch_rows<16, 1>(p, fp8, stream);
  else if (p.block_rows == 32)
    launch_rows<32, 1>(p, fp8, stream);
  else
    launch_rows<32, 2>(p, fp8, stream);
}

}  // namespace

int mla_decode_block_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// Groups that share the tiles (max_tiles: the most there can be, from the
// sizes the host knows), so that groups times row blocks fill the device once.
int mla_decode_groups(int64_t row_blocks, int64_t max_tiles) {
  int64_t g = (compute_units() + row_blocks - 1) / row_blocks;
  if (g > max_tiles) g = max_tiles;
  return (int)(g < 1 ? 1 : g);
}

hipError_t launch_mla_decode(const MlaDecode& own, const MlaDecode* prefix, bool fp8, hipStream_t stream) {
  if (prefix) launch_tiles(*prefix, fp8, stream);
  if (own.max_len > 0) launch_tiles(own, fp8, stream);
  hipLaunchKernelGGL(mla_join_kernel, dim3((unsigned)((own.all_rows + 3) / 4)), dim3(kJoinThreads), 0, stream, own,
                     prefix ? *prefix : own);
  return hipGetLastError();
}

}  // namespace fp8bs
