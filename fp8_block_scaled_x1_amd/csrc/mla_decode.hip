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
// Two teams of four waves, 32 rows each, share the tiles in LDS. A
// wave forms the partial scores of 32 tokens over half of the key's columns
// (so it holds 32 x 288 query numbers only), trades one half of them for its
// partner's (the same tokens, the other columns), and has the scores of 16
// tokens and 32 rows. It turns them into weights, writes them to LDS in the
// order in which the value product's operand wants them, and adds the 64
// tokens' values into its 32 x 128 part of the output. No product is formed
// twice, and 72 + 64 + 16 registers of queries, output and scores leave room
// for operands to be fetched ahead, with two waves per SIMD. The
// row maxima need no exchange of their own: the weights are taken against a
// reference that the team shares and that is only raised (a second exchange,
// for all) when some wave finds a score 2^8 above it.
//
// FP8 cache: codes become BF16 exactly; a group's scale multiplies the partial
// score of its 128 columns (FP32) and the probability that meets its 128
// output columns, so the latent vector itself is never rounded.
//
// Bound, BF16 cache, 64 rows: a tile costs a compute unit 2.9 us from L2, of
// which the products need 1.0 us (matrix unit 0.36 busy at 2.15 GHz) and its 74
// KB into LDS 1.4 us; two tiles fill the LDS, so a tile's phases (scores,
// exchange, weights, values) follow each other for all waves, with only the
// next tile's loads beside them. 192 requests of 32 heads behind 16000 common
// tokens: 0.27 ms, 0.8 PFLOP/s. From HBM a tile costs 3.7 us: 128 requests of
// 300 to 4500 tokens on 128 heads, 387 MB: 0.16 ms with the join. FP8 cache, 32
// rows: 256 MB in 64 us, 4.0 TB/s, bound by the codes' conversion and the same
// phases, half of the waves only loading.
//
// Roundings below 32 bits: probabilities (times the scale, FP8) to BF16 for
// the matrix unit (relative 2^-8 at most each, on the terms of a mean), and the output.

#include <atomic>

#include "mla_paged.h"

namespace fp8bs {

namespace {

constexpr int kTile = kMlaDecodeTile;      // tokens per tile
constexpr int kLatent = 512, kRope = 64, kKey = kLatent + kRope;
// The weights' reference only follows the running maximum once that is more
// than 2^8 above it: weights up to 2^8 cost no precision in FP32 or BF16, and
// the accumulators are rescaled a few times per request instead of per tile.
constexpr float kSlack = 8.f;

__device__ __forceinline__ void advance(const MlaDecode& p, Cursor& c) {
  --c.left;
  if (++c.tile < c.tiles || c.left <= 0) return;
  do {
    ++c.b;
    c.len = c.b < p.B ? __builtin_amdgcn_readfirstlane(clamp_len(p, c.b)) : 0;
  } while (c.len == 0 && c.b < p.B);
  c.tile = 0;
  c.tiles = tiles_of<kTile>(c.len);
}

// Token of the tile's row `lane`. Tokens past the end repeat the last one:
// always cached, and masked by its position.
__device__ __forceinline__ int row_token(const Cursor& c, int lane) { return min(c.tile * kTile + lane, c.len - 1); }

inline int compute_units() {
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

template <bool FP8>
struct Tile {
  static constexpr int kRowBytes = FP8 ? kLatent : 2 * kLatent;
  static constexpr int kLatentBytes = kTile * kRowBytes;
  static constexpr int kRopeBytes = kTile * 2 * kRope;
  static constexpr int kScaleBytes = FP8 ? kTile * 16 : 0;        // [group][token]
  static constexpr int kBytes = kLatentBytes + kRopeBytes + kScaleBytes;
};

__device__ __forceinline__ const char* lane_ptr(const char* base, int64_t off, int from) {
  const uint64_t a = (uint64_t)(base + off);
  return (const char*)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(a >> 32), from) << 32) |
                       (uint32_t)__builtin_amdgcn_readlane((int)a, from));
}

// The wave's ROWS rows of a tile, from row r0, load by load (kLoads of them), so
// that they can be issued between the matrix instructions: a wave that issues
// its loads in one go stands still until the address unit has taken them all.
// Lane l holds row l's block-table entry. The 16-byte chunks are permuted by
// swz256 (swz128) of the row in groups of 16 (8), see mla_tiles.h; LDS itself
// is written linearly.
template <bool FP8, int ROWS>
struct Loader {
  using T = Tile<FP8>;
  static constexpr int kMain = FP8 ? ROWS / 2 : ROWS, kRopes = ROWS / 8, kLoads = kMain + kRopes + (FP8 ? 1 : 0);
  const MlaDecode& p;
  const int r0, lane;
  const uint32_t lds;
  const int64_t flat;
  const int chunk;
  __device__ __forceinline__ static int64_t flat_of(const MlaDecode& p, const Cursor& c, int lane, int entry) {
    const int tok = row_token(c, lane);
    return (int64_t)min(max(entry, 0), p.pages - 1) * p.page + (tok - page_of(p, tok) * p.page);
  }
  __device__ __forceinline__ Loader(const MlaDecode& p_, const Cursor& c, int r0_, int lane_, int entry, uint32_t lds_)
      : p(p_), r0(r0_), lane(lane_), lds(lds_), flat(flat_of(p_, c, lane_, entry)),
        chunk(opaque(((FP8 ? lane_ & 31 : lane_) << 4) ^ (swz256(r0_) << 4))) {}
  __device__ __forceinline__ void issue(int n) const {
    if (n < kMain) {
      if constexpr (!FP8) {      // a row of 1024 latent bytes: the row is wave-uniform
        dma16_s(lane_ptr(p.cache, flat * (2 * kKey), r0 + n), (uint32_t)(chunk ^ (swz256(n) << 4)),
                lds + (r0 + n) * T::kRowBytes);
      } else {                   // two rows of 512 code bytes
        const char* a = lane_ptr(p.cache, flat * kLatent, r0 + 2 * n);
        const char* b = lane_ptr(p.cache, flat * kLatent, r0 + 2 * n + 1);
        dma16((lane < 32 ? a : b) + (chunk ^ ((lane < 32 ? swz256(2 * n) : swz256(2 * n + 1)) << 4)),
              lds + (r0 + 2 * n) * T::kRowBytes);
      }
    } else if (n < kMain + kRopes) {      // rotary part: 8 rows of 128 bytes
      const int i = 8 * (n - kMain), row = r0 + i + (lane >> 3);
      const int64_t f = ((int64_t)__shfl((int)(flat >> 32), row, 64) << 32) | (uint32_t)__shfl((int)flat, row, 64);
      const int c = (lane & 7) ^ swz128(row);
      const char* src = FP8 ? p.rope + f * (2 * kRope) : p.cache + f * (2 * kKey) + 2 * kLatent;
      dma16(src + (c << 4), lds + T::kLatentBytes + (r0 + i) * (2 * kRope));
    } else if constexpr (FP8) {           // 64 tokens' scales of one group (with 8 waves two load the same)
      const int q = r0 >> 4;
      dma4(p.scales + flat * 16 + 4 * q, lds + T::kLatentBytes + T::kRopeBytes + q * 4 * kTile);
    }
  }
};

// Operands of the value product, kAhead steps ahead: step i is the 16 tokens
// i/4 and the wave's 32-column block i%4. at: the lane's offset in step 0.
template <bool FP8>
struct ValueFeed {
  static constexpr int kAhead = 4;
  const char* base;
  int at;
  bf16x8 v[FP8 ? 1 : kAhead];
  i32x2 c[FP8 ? kAhead : 1];
  __device__ __forceinline__ ValueFeed(const char* base_, int at_) : base(base_), at(at_) {}
  __device__ __forceinline__ void fetch(int i) {
    const int row = 16 * (i >> 2), d = i & 3;
    if constexpr (FP8) {
      c[i % kAhead] = lds_tr8(base + (at ^ (d << 5)) + row * Tile<FP8>::kRowBytes);
    } else {
      v[i % kAhead] = join(lds_tr16(base + (at ^ (d << 6)) + row * Tile<FP8>::kRowBytes),
                           lds_tr16(base + (at ^ (d << 6) ^ 32) + (row + 8) * Tile<FP8>::kRowBytes));
    }
  }
  __device__ __forceinline__ bf16x8 get(int i) const {
    if constexpr (FP8)
      return e4m3_to_bf16((uint32_t)c[i % kAhead][0], (uint32_t)c[i % kAhead][1]);
    else
      return v[i % kAhead];
  }
};

constexpr int kTeams = kMlaDecodeBlockRows / 32;

// One problem, or two that do not wait for each other (a prefix and the
// requests' own tokens): workgroups from `split` on belong to the second.
struct Problems {
  MlaDecode p[2];
  int split;
};

template <bool FP8, int NBUF, bool TWO>
__global__ __launch_bounds__(256 * kTeams) __attribute__((amdgpu_waves_per_eu(2))) void mla_decode_kernel(
    const Problems problems) {
  const bool second = TWO && (int)blockIdx.x >= problems.split;
  const MlaDecode& p = problems.p[second];
  const int block = blockIdx.x - (second ? problems.split : 0);
  using T = Tile<FP8>;
  constexpr int NW = 4 * kTeams, kRows = kTile / NW;        // waves; rows of a tile that each loads
  using Load = Loader<FP8, kRows>;
  using Values = ValueFeed<FP8>;
  constexpr int kLoads = Load::kLoads;
  // A wave's slot: the partial scores that its partner sends, then its weights
  // (BF16, or FP32 to meet the scales first); behind them its row maxima and
  // its wish to raise the reference. With NBUF = 2 the entries of the next
  // tile wait in a register instead of in LDS.
  constexpr int kProbBytes = 64 * 8 * (FP8 ? 4 : 2), kSlot = FP8 ? 2048 + 256 : 2048;
  static_assert(NBUF == 2 || NBUF == 3, "tiles in flight");
  __shared__ __align__(1024) char lds_mem[NBUF * T::kBytes + NW * kSlot + (NBUF > 2 ? NW * 256 : 0)];
  char* const tiles = lds_mem;
  char* const slots = lds_mem + NBUF * T::kBytes;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rt = wave >> 2, quarter = wave & 3;     // team; 16 tokens (weights) and 128 columns (output) of the wave
  const int th = quarter >> 1, kh = quarter & 1;    // 32 tokens and half of the key's columns (scores)
  char* const slot = slots + wave * kSlot;
  float* const my_stat = reinterpret_cast<float*>(slot + kProbBytes);
  const char* const team = slots + rt * 4 * kSlot;

  // workgroup -> (group, row block): workgroups are dealt over the XCDs one by
  // one; renumbered so that an XCD's are consecutive, row blocks of a group first
  const int blocks = p.groups * p.row_blocks, per = blocks / kAttnXcds, rest = blocks % kAttnXcds;
  const int xcd = block % kAttnXcds;
  const int wg = xcd * per + min(xcd, rest) + block / kAttnXcds;
  const int g = wg / p.row_blocks;
  Cursor cur = first_tile<kTile>(p, g);
  if (cur.left == 0) return;

  const uint32_t lds_tiles = lds_offset(tiles);
  const int* const entries = reinterpret_cast<const int*>(slots + NW * kSlot + wave * 256);
  const uint32_t lds_entries = lds_offset(entries);
  int entry = 0;         // of row `lane` of the tile that is loaded next (NBUF == 2)
  Cursor nxt = cur;      // the tile that is loaded next
  Cursor ent = cur;      // the tile whose block-table entries are fetched next
  auto fetch_entries = [&] {
    const int* src = p.table + (int64_t)ent.b * p.table_stride + page_of(p, row_token(ent, lane));
    if constexpr (NBUF == 2)
      entry = *src;
    else
      dma4(src, lds_entries);
    advance(p, ent);
  };
  auto start_next = [&](int to) {      // the loads of the tile `nxt`, into buffer `to`
    if constexpr (NBUF > 2) {
      entry = entries[lane];
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    const int e = opaque(entry);      // waited for here, before the next fetch is under way
    const Cursor c = nxt;
    advance(p, nxt);
    if (ent.left > 0) fetch_entries();
    return Load(p, c, wave * kRows, lane, e, lds_tiles + to * T::kBytes);
  };
  fetch_entries();
#pragma unroll
  for (int i = 0; i < NBUF - 1; ++i) {
    attn_wait<0>();
    if (nxt.left > 0) {
      const Load ld = start_next(i);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) ld.issue(n);
    }
  }

  // LDS offsets of this lane: the swizzles only touch bits that the row and
  // tile offsets leave free, so the chunk is picked by an XOR
  const TileLane L(lane);
  // key reads: the 16 tokens whose scores the wave keeps come first
  const int krow = 32 * th + (L.row ^ (16 * kh));
  const int key0 = krow * T::kRowBytes + kh * (T::kRowBytes / 2) + ((L.half ^ L.x256) << 4);
  const int rope0 = T::kLatentBytes + krow * (2 * kRope) + ((L.half ^ L.x128 ^ (4 * kh)) << 4);
  int val0;
  if constexpr (FP8) {
    const int i = (lane & 15) >> 1, row = 4 * L.half + (i & 3) + 8 * (i >> 2);
    val0 = row * T::kRowBytes + 256 * (quarter >> 1) + 8 * (lane & 1) +
           (((8 * (quarter & 1) + ((lane >> 4) & 1)) ^ swz256(row)) << 4);
  } else {
    val0 = L.trow * T::kRowBytes + 256 * quarter + L.tbyte + ((L.tchunk ^ L.tx256) << 4);
  }
  const int scale0 = T::kLatentBytes + T::kRopeBytes + 16 * L.half;      // [group][token]

  const int row = ((wg - g * p.row_blocks) * kTeams + rt) * 32 + L.row;  // this lane's row
  const int late = p.tokens - 1 - min(row, p.rows - 1) / p.heads;        // newest tokens hidden from it
  const bool idle = __builtin_amdgcn_readfirstlane(row) >= p.rows;       // a team without rows

  bf16x8 qf[18];
  f32x16 acc[4];
  float m, l;
  bool first = true;
  int buf = 0;

  while (cur.left > 0) {      // a request's part of the range
    const bool whole = cur.tile == 0 && cur.left >= cur.tiles;
    const uint16_t* qr = p.q + min((int64_t)cur.b * p.rows + min(row, p.rows - 1), p.all_rows - 1) * kKey;
#pragma unroll
    for (int ks = 0; ks < 16; ++ks) {
      // FP8: a lane reads 16 codes at a time, the slots of two k steps
      const int col = FP8 ? 32 * (ks >> 1) + 16 * L.half + 8 * (ks & 1) : 16 * ks + 8 * L.half;
      qf[ks] = *reinterpret_cast<const bf16x8*>(qr + 256 * kh + col);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      qf[16 + ks] = *reinterpret_cast<const bf16x8*>(qr + kLatent + 32 * kh + 16 * ks + 8 * L.half);
    m = neg_inf();
    l = 0.f;
#pragma unroll
    for (int d = 0; d < 4; ++d) acc[d] = zero16();
    operands_loaded();

    for (bool last = false; !last;) {
      auto step = [&] {
        last = cur.tile + 1 == cur.tiles || cur.left == 1;
        if (last) return;
        advance(p, cur);
        buf = buf + 1 == NBUF ? 0 : buf + 1;
      };
      // any wave's wish to raise the reference: the answer is the same for all
      auto raised = [&] {
        return __any(*reinterpret_cast<const float*>(slots + (lane % NW) * kSlot + kProbBytes + 128) != 0.f) != 0;
      };
      if (nxt.left > 0 && NBUF > 2)
        attn_wait<kLoads>();
      else
        attn_wait<0>();
      attn_barrier();
      const int at = buf * T::kBytes;      // of the tile in LDS
      const char* tl = tiles + at;

      // partial scores: D[token drow(i) ^ 16 kh][row lane%32] of 32 tokens,
      // operands fetched kAhead steps ahead, the next tile's loads in between
      f32x16 x;
      const int key = opaque(key0 + at), rope = rope0 + at;
      auto partial = [&](auto&& between) {
        if constexpr (!FP8) {
          constexpr int kAhead = 6;
          bf16x8 kf[kAhead];
          auto fetch = [&](int ks) {
            return lds_bf16x8(ks < 16 ? tiles + (key ^ ((ks & 7) << 5)) + (ks >> 3) * 256 : tiles + (rope ^ ((ks & 1) << 5)));
          };
          x = zero16();
#pragma unroll
          for (int ks = 0; ks < kAhead; ++ks) kf[ks] = fetch(ks);
#pragma unroll
          for (int ks = 0; ks < 18; ++ks) {
            __builtin_amdgcn_sched_barrier(0);
            x = mfma32(kf[ks % kAhead], qf[ks], x);
            if (ks + kAhead < 18) kf[ks % kAhead] = fetch(ks + kAhead);
            between(ks);
          }
          __builtin_amdgcn_sched_barrier(0);
        } else {
          constexpr int kAhead = 3;
          uint4 kc[kAhead];
          auto fetch = [&](int h) { return *reinterpret_cast<const uint4*>(tiles + (key ^ (h << 5))); };
          f32x16 z[2] = {zero16(), zero16()};      // 128 columns with one scale a token each
#pragma unroll
          for (int h = 0; h < kAhead; ++h) kc[h] = fetch(h);
          const bf16x8 r0 = lds_bf16x8(tiles + rope), r1 = lds_bf16x8(tiles + (rope ^ 32));
#pragma unroll
          for (int h = 0; h < 8; ++h) {            // 32 columns
            __builtin_amdgcn_sched_barrier(0);
            const uint4 c = kc[h % kAhead];
            const bf16x8 a0 = e4m3_to_bf16(c.x, c.y), a1 = e4m3_to_bf16(c.z, c.w);
            if (h + kAhead < 8) kc[h % kAhead] = fetch(h + kAhead);
            z[h >> 2] = mfma32(a0, qf[2 * h], z[h >> 2]);
            between(2 * h);
            z[h >> 2] = mfma32(a1, qf[2 * h + 1], z[h >> 2]);
            between(2 * h + 1);
          }
          x = mfma32(r0, qf[16], zero16());
          between(16);
          x = mfma32(r1, qf[17], x);
          between(17);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              const f32x4 sc =
                  *reinterpret_cast<const f32x4*>(tl + scale0 + 4 * kTile * (2 * kh + q) + 4 * (32 * th + ((8 * i4) ^ (16 * kh))));
#pragma unroll
              for (int j = 0; j < 4; ++j) x[4 * i4 + j] = fmaf(sc[j], z[q][4 * i4 + j], x[4 * i4 + j]);
            }
        }
      };
      if (idle) {      // its share of the loads, and the barriers of the others
        if (nxt.left > 0) {
          const Load ld = start_next(buf == 0 ? NBUF - 1 : buf - 1);
#pragma unroll
          for (int n = 0; n < kLoads; ++n) ld.issue(n);
        }
        if (lane == 0) my_stat[32] = 0.f;
        attn_barrier();
        attn_barrier();
        if (raised()) attn_barrier();
        step();
        continue;
      }
      if (nxt.left > 0) {
        const Load ld = start_next(buf == 0 ? NBUF - 1 : buf - 1);
        partial([&](int i) {
          if (i * kLoads / 18 != (i + 1) * kLoads / 18) ld.issue(i * kLoads / 18);
        });
      } else {
        partial([](int) {});
      }
      // the partner's half of them to its slot, this wave's kept
      f32x4 s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f32x4 give;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = x[4 * i + j];
          give[j] = x[8 + 4 * i + j];
        }
        *reinterpret_cast<f32x4*>(slots + (wave ^ 1) * kSlot + 1024 * i + 16 * lane) = give;
      }
      attn_barrier();
#pragma unroll
      for (int i = 0; i < 2; ++i) s[i] += *reinterpret_cast<const f32x4*>(slot + 1024 * i + 16 * lane);

      // weights of 16 tokens against the team's reference
      const int tok0 = cur.tile * kTile + 16 * quarter + 4 * L.half, seen = cur.len - late;
      if ((cur.tile + 1) * kTile > cur.len - (p.tokens - 1)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (tok0 + 8 * i + j >= seen) s[i][j] = neg_inf();
      }
      float top = max_nan(max_nan(max_nan(s[0][0], s[0][1]), max_nan(s[0][2], s[0][3])),
                          max_nan(max_nan(s[1][0], s[1][1]), max_nan(s[1][2], s[1][3])));
      top = half_max(top) * p.scale_log2;
      float sum;
      auto weigh = [&] {
        const float ref = m == neg_inf() ? 0.f : m;      // nothing visible yet: every weight is 0
        f32x4 e[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) e[i][j] = exp2_fast(fmaf(s[i][j], p.scale_log2, -ref));
        sum = ((e[0][0] + e[0][1]) + (e[0][2] + e[0][3])) + ((e[1][0] + e[1][1]) + (e[1][2] + e[1][3]));
        if constexpr (FP8) {
          *reinterpret_cast<f32x4*>(slot + 16 * lane) = e[0];
          *reinterpret_cast<f32x4*>(slot + 1024 + 16 * lane) = e[1];
        } else {
          bf16x8 b;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            b[j] = (__bf16)e[0][j];
            b[4 + j] = (__bf16)e[1][j];
          }
          *reinterpret_cast<bf16x8*>(slot + 16 * lane) = b;
        }
      };
      weigh();
      // the first values are on their way before the waves meet
      Values vf(tiles, opaque(val0 + at));
#pragma unroll
      for (int i = 0; i < Values::kAhead; ++i) vf.fetch(i);
      if (L.half == 0) my_stat[L.row] = top;
      const bool grown = __any(top > m + kSlack);
      if (lane == 0) my_stat[32] = grown ? 1.f : 0.f;
      attn_barrier();
      if (raised()) {
        float mn = m;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mn = max_nan(mn, reinterpret_cast<const float*>(team + k * kSlot + kProbBytes)[L.row]);
        const float alpha = mn == neg_inf() ? 1.f : exp2_fast(m - mn);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[d] *= alpha;
        weigh();
        attn_barrier();
      }
      l += sum;

      // output: D[column drow(i)][row lane%32] of each 32-column block
      bf16x8 pb[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        if constexpr (!FP8) {
          pb[a] = lds_bf16x8(team + a * kSlot + 16 * lane);
        } else {
          const f32x4 e0 = *reinterpret_cast<const f32x4*>(team + a * kSlot + 16 * lane);
          const f32x4 e1 = *reinterpret_cast<const f32x4*>(team + a * kSlot + 1024 + 16 * lane);
          const char* sp = tl + scale0 + 4 * kTile * quarter + 4 * 16 * a;
          const f32x4 c0 = *reinterpret_cast<const f32x4*>(sp), c1 = *reinterpret_cast<const f32x4*>(sp + 32);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            pb[a][j] = (__bf16)(e0[j] * c0[j]);
            pb[a][4 + j] = (__bf16)(e1[j] * c1[j]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        acc[i & 3] = mfma32(vf.get(i), pb[i >> 2], acc[i & 3]);
        if (i + Values::kAhead < 16) vf.fetch(i + Values::kAhead);
      }
      __builtin_amdgcn_sched_barrier(0);
      step();
    }

    // sums over the lanes' and the waves' tokens
    l = half_sum(l);
    if (L.half == 0) my_stat[L.row] = l;
    attn_barrier();
    l = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) l += reinterpret_cast<const float*>(team + k * kSlot + kProbBytes)[L.row];
    if (row < p.rows && (int64_t)cur.b * p.rows + row < p.all_rows) {
      if (whole && !p.join) {
        const int64_t o = (int64_t)cur.b * p.rows + row;
        const float inv = inverse_of(l);
        uint16_t* op = p.out + o * kLatent + 128 * quarter + 4 * L.half;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            bf16x4 b;
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = (__bf16)(acc[d][4 * i + j] * inv);
            *reinterpret_cast<bf16x4*>(op + 32 * d + 8 * i) = b;
          }
        if (quarter == 0 && L.half == 0) p.lse[o] = lse_of(m, l);
      } else {
        const int64_t o = (whole ? 2 * (int64_t)p.groups + cur.b : 2 * (int64_t)g + (first ? 0 : 1)) * p.rows + row;
        float* op = p.part + o * kLatent + 128 * quarter + 4 * L.half;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = acc[d][4 * i + j];
            *reinterpret_cast<f32x4*>(op + 32 * d + 8 * i) = v;
          }
        if (quarter == 0 && L.half == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * o) = make_float2(m, l);
      }
    }
    first = false;
    advance(p, cur);
    buf = buf + 1 == NBUF ? 0 : buf + 1;
  }
}

// A BF16 tile has 74 KB, so two fit; of the FP8 tiles (41 KB) three do, which
// leaves a tile's loads the time of two.
template <bool TWO>
void launch_tiles(const Problems& two, bool fp8, hipStream_t stream) {
  const MlaDecode& b = two.p[1];
  const dim3 grid((unsigned)(two.split + (TWO ? (int64_t)b.groups * b.row_blocks : 0)));
  if (fp8)
    hipLaunchKernelGGL((mla_decode_kernel<true, 3, TWO>), grid, dim3(256 * kTeams), 0, stream, two);
  else
    hipLaunchKernelGGL((mla_decode_kernel<false, 2, TWO>), grid, dim3(256 * kTeams), 0, stream, two);
}

}  // namespace

// Groups that share the tiles (max_tiles: the most there can be, from the
// sizes the host knows), so that groups times row blocks fill the device once
// and leave nothing for a second time (rounded up instead, 3 blocks of 64 rows
// are 258 workgroups: 3 query tokens of 32 requests on 128 heads 160 us, so
// 107 us).
int mla_decode_groups(int64_t row_blocks, int64_t max_tiles) {
  int64_t g = compute_units() / row_blocks;
  if (g > max_tiles) g = max_tiles;
  return (int)(g < 1 ? 1 : g);
}

hipError_t launch_mla_decode(const MlaDecode& own, const MlaDecode* prefix, bool fp8, hipStream_t stream) {
  // A prefix and the requests' own tokens in one launch: alone, neither of two
  // small problems fills the device (prefix of 1000, 6 requests of 16 heads:
  // 23 us, in two launches 30 us).
  const MlaDecode& head = prefix ? *prefix : own;
  const Problems two{{head, own}, head.groups * (int)head.row_blocks};
  if (prefix && own.max_len > 0)
    launch_tiles<true>(two, fp8, stream);
  else if (prefix || own.max_len > 0)
    launch_tiles<false>(two, fp8, stream);
  launch_mla_join<kTile>(own, head, prefix != nullptr, stream);
  return hipGetLastError();
}

}  // namespace fp8bs
