// What the kernels of the absorbed latent attention share whatever their cache
// holds: the tiles of all requests cut into equal ranges, and the join of the
// partial results that the cuts leave. TILE: tokens of a tile.
#pragma once

#include "attn_internal.h"
#include "mla_tiles.h"

namespace fp8bs {

namespace {

constexpr int kLatentDim = 512, kJoinThreads = 256;

// The tiles of a request, and the request a tile belongs to.
struct Cursor {
  int b;        // request
  int len;      // its tokens
  int tile;     // tile inside it
  int tiles;    // its tiles
  int left;     // tiles left in the group's range, this one included
};

__device__ __forceinline__ int clamp_len(const MlaDecode& p, int b) { return min(max(p.lens[b * p.len_stride], 0), p.max_len); }

__device__ __forceinline__ int wave_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(v, d, 64);
    if (lane >= d) v += x;
  }
  return v;
}

// The groups' ranges of `total` tiles: consecutive, of equal length but for one
// tile, the longer ones (and, if there are fewer tiles than groups, those that
// have any) first.
struct Ranges {
  int each, longer;
  __device__ __forceinline__ Ranges(int total, int groups)
      : each(total / groups), longer(total - total / groups * groups) {}
  __device__ __forceinline__ int start(int g) const { return g * each + min(g, longer); }
  __device__ __forceinline__ int of(int t) const {      // the group of tile t
    const int head = longer * (each + 1);
    return t < head ? t / (each + 1) : longer + (t - head) / max(each, 1);
  }
};

template <int TILE>
__device__ __forceinline__ int tiles_of(int len) { return (len + TILE - 1) / TILE; }

// The range of group g as a cursor on its first tile (left = 0: it has none).
template <int TILE>
__device__ __forceinline__ Cursor first_tile(const MlaDecode& p, int g) {
  const int lane = threadIdx.x & 63;
  // tiles of all requests; up to 64 requests are read once
  int len = 0, incl = 0, total = 0;
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    len = b0 + lane < p.B ? clamp_len(p, b0 + lane) : 0;
    incl = wave_scan(tiles_of<TILE>(len));
    total += __builtin_amdgcn_readlane(incl, 63);
  }
  const Ranges r(total, p.groups);
  const int t = r.start(g), left = r.start(g + 1) - t;
  if (left <= 0) return Cursor{0, 0, 0, 0, 0};
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    if (p.B > 64) {
      len = b0 + lane < p.B ? clamp_len(p, b0 + lane) : 0;
      incl = wave_scan(tiles_of<TILE>(len));
    }
    const uint64_t hit = __ballot(t < base + incl);
    if (hit) {
      const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
      Cursor c;
      c.b = b0 + l;
      c.len = __builtin_amdgcn_readlane(len, l);
      c.tiles = tiles_of<TILE>(c.len);
      c.tile = t - base - (__builtin_amdgcn_readlane(incl, l) - c.tiles);
      c.left = left;
      return c;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return Cursor{0, 0, 0, 0, 0};
}

// The flat cache token (page * page size + slot) of token `tok`, given its
// page's entry in the block table.
__device__ __forceinline__ int page_of(const MlaDecode& p, int tok) {
  return (int)(((uint64_t)(uint32_t)tok * p.page_magic) >> p.page_shift);
}

// Joins the partials of the rows whose request was cut between groups (and, in
// the shared form, the prefix's with the request's own). W waves per row, lane
// l columns 8l .. 8l+7; all pieces' maxima are read at once, so every load of
// a piece's output is under way before the first is needed.
struct Pieces {      // of one row in one problem: at(i), i < n
  int rows, n, row;
  int64_t first;      // the first piece's slot; the others lie 2 slots apart from `rest`
  int64_t rest;
  bool done;          // the row's result is written already
  __device__ __forceinline__ int64_t at(int i) const { return (i == 0 ? first : rest + 2 * (int64_t)i) * rows + row; }
};

template <int TILE>
__device__ __forceinline__ Pieces pieces_of(const MlaDecode& p, int64_t o) {
  const int lane = threadIdx.x & 63;
  const int b = (int)(o / p.rows);
  Pieces r{p.rows, 0, (int)(o - (int64_t)b * p.rows), 0, 0, false};
  int before = 0, all = 0, own = 0;      // tiles before the request, of all, its own
  for (int b0 = 0; b0 < p.B; b0 += 64) {
    const int n = b0 + lane < p.B ? tiles_of<TILE>(clamp_len(p, b0 + lane)) : 0, incl = wave_scan(n);
    if (b >= b0 && b < b0 + 64) {
      own = __builtin_amdgcn_readlane(n, b - b0);
      before = all + __builtin_amdgcn_readlane(incl, b - b0) - own;
    }
    all += __builtin_amdgcn_readlane(incl, 63);
  }
  if (own == 0) return r;
  const Ranges ranges(all, p.groups);
  const int g0 = ranges.of(before), g1 = ranges.of(before + own - 1);
  if (g0 == g1) {
    r.done = !p.join;
    r.n = 1;
    r.first = 2 * (int64_t)p.groups + b;
  } else {
    r.n = g1 - g0 + 1;
    r.first = 2 * (int64_t)g0 + (ranges.start(g0) < before ? 1 : 0);
    r.rest = 2 * (int64_t)g0;
  }
  return r;
}

template <int W, int TILE>
__global__ __launch_bounds__(kJoinThreads) void mla_join_kernel(const MlaDecode p, const MlaDecode prefix) {
  constexpr int kRowsPerBlock = kJoinThreads / 64 / W, kBatch = 4;
  __shared__ float2 ml[W > 1 ? W : 1];
  __shared__ __align__(16) float sums[W > 1 ? W : 1][512];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave % W;
  const int64_t o = (int64_t)blockIdx.x * kRowsPerBlock + wave / W;
  if (o >= p.all_rows) return;
  const Pieces own = pieces_of<TILE>(p, o);
  if (own.done) return;
  Pieces pre{};
  if (p.join) pre = pieces_of<TILE>(prefix, o);
  const int n = own.n + pre.n;
  // this wave's pieces: every W-th
  float m = neg_inf(), l = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int i0 = w; i0 < n; i0 += 64 * W) {
    const int i = i0 + lane * W;      // lane's piece
    const bool mine = i < own.n;
    float2 x = make_float2(neg_inf(), 0.f);
    if (i < n) x = *reinterpret_cast<const float2*>((mine ? p.part_ml : prefix.part_ml) + 2 * (mine ? own.at(i) : pre.at(i - own.n)));
    float mn = x.x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) mn = max_nan(mn, __shfl_xor(mn, d, 64));
    mn = max_nan(mn, m);
    const float ref = mn == neg_inf() ? 0.f : mn;
    const float old = exp2_fast(m - ref), weight = exp2_fast(x.x - ref);
    float add = x.y * weight;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) add += __shfl_xor(add, d, 64);
    l = fmaf(l, old, add);
    m = mn;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] *= old;
    const int count = min(64, (n - i0 + W - 1) / W);
    for (int k0 = 0; k0 < count; k0 += kBatch) {
      f32x4 v[kBatch][2];
      float wt[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int kc = min(k0 + k, count - 1), j = i0 + kc * W;
        const bool a = j < own.n;
        const float* src = (a ? p.part : prefix.part) + (a ? own.at(j) : pre.at(j - own.n)) * kLatentDim + 8 * lane;
        v[k][0] = *reinterpret_cast<const f32x4*>(src);
        v[k][1] = *reinterpret_cast<const f32x4*>(src + 4);
        const float got = __shfl(weight, kc, 64);
        wt[k] = k0 + k < count ? got : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[j] = fmaf(v[k][0][j], wt[k], acc[j]);
          acc[4 + j] = fmaf(v[k][1][j], wt[k], acc[4 + j]);
        }
    }
  }
  if constexpr (W > 1) {
    if (lane == 0) ml[w] = make_float2(m, l);
    __syncthreads();
    float mn = neg_inf();
#pragma unroll
    for (int k = 0; k < W; ++k) mn = max_nan(mn, ml[k].x);
    const float ref = mn == neg_inf() ? 0.f : mn, x = exp2_fast(m - ref);
    l = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) l = fmaf(ml[k].y, exp2_fast(ml[k].x - ref), l);
    m = mn;
    f32x4 a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = acc[j] * x;
      b[j] = acc[4 + j] * x;
    }
    *reinterpret_cast<f32x4*>(&sums[w][8 * lane]) = a;
    *reinterpret_cast<f32x4*>(&sums[w][8 * lane + 4]) = b;
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc[j] = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) acc[j] += sums[k][8 * lane + j];
    }
  }
  const float inv = inverse_of(l);
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (__bf16)(acc[i] * inv);
  *reinterpret_cast<bf16x8*>(p.out + o * kLatentDim + 8 * lane) = v;
  if (lane == 0) p.lse[o] = lse_of(m, l);
}

template <int TILE>
void launch_mla_join(const MlaDecode& own, const MlaDecode& head, bool behind_prefix, hipStream_t stream) {
  // Few rows have many pieces each: a workgroup per row. Many rows have one or
  // two, and a wave per row has less to set up; behind a prefix they all have
  // the prefix's as well. Whole calls of 3000 to 6000 tokens, workgroup and wave
  // per row: 512 rows of one request 33.5 and 36.4 us, 768 of one 38.0 and 37.4,
  // 1024 of one 43.4 and 38.2, of 8 requests 48.2 and 46.8; 16384 rows 178 and
  // 156. Behind a prefix of 8000, of 32 requests 512 rows 50.7 and 60.0, 1024 of
  // 64 65.9 and 66.7, 2048 of 128 93.1 and 92.2. Over the 4-bit cache: 128 rows of
  // one request 28.2 and 33.7, 768 of 6 39.1 and 38.3, 16384 283 and 264.
  if (own.all_rows <= (behind_prefix ? 2048 : 512))
    hipLaunchKernelGGL((mla_join_kernel<4, TILE>), dim3((unsigned)own.all_rows), dim3(kJoinThreads), 0, stream, own, head);
  else
    hipLaunchKernelGGL((mla_join_kernel<1, TILE>), dim3((unsigned)((own.all_rows + 3) / 4)), dim3(kJoinThreads), 0, stream, own, head);
}

}  // namespace

}  // namespace fp8bs
