// Latent attention in its expanded form (prefill and training), forward and
// backward, for a packed batch of requests of any lengths.
//
// Per head h, with q = (q^n, q^r), keys (k^n_h, k^r) whose 64-wide rotary part
// is shared by all heads, and values v_h:
//   S_ij = scale * (q^n_i . k^n_j + q^r_i . k^r_j),  j <= i + Lk - Lq if causal
//   P = softmax(S),  O = P V,  lse_i = log sum_j exp(S_ij)
// and with D_i = dO_i . O_i:
//   dV = P^T dO,  dS = P * (dO V^T - D),  dq = scale dS K,  dk = scale dS^T q,
//   dk^r = sum over the heads of their dk's rotary part.
//
// Roundings below 32 bits: P and dS to BF16 as operands of the matrix unit
// (relative 2^-8 at most, on each term of a sum), O to BF16 before D is formed from it,
// and the outputs. Scores, softmax statistics, D and every sum are FP32; the
// rotary gradient is summed over the heads in FP32, in head order.
//
// All products are 32x32x16 MFMAs, oriented so that the lane that owns a row
// of the score tile owns it in the next product too.

#include <algorithm>
#include <cmath>

#include "attn_internal.h"
#include "device_common.h"
#include "mla_tiles.h"

namespace fp8bs {

namespace {

// Workgroup -> (unit, head). The heads are dealt over the XCDs and taken there
// four at a time, unit by unit: the units of a head that run together share its
// keys and values in L2 (all of an XCD's heads at once would not fit: 8% slower
// with 16 heads of 8192 tokens), and the last units to run, the short ones of
// four heads, leave little of the device idle (a head after the other: 3-12%
// slower).
__device__ __forceinline__ bool unit_of(int units, int H, int& unit, int& head) {
  constexpr int kTogether = 4;
  if (H % kAttnXcds == 0) {
    const int xcd = blockIdx.x % kAttnXcds, slot = blockIdx.x / kAttnXcds, heads = H / kAttnXcds;
    if (slot >= heads * units) return false;
    const int group = slot / (kTogether * units), in = slot - group * kTogether * units;
    const int n = min(kTogether, heads - group * kTogether);
    head = (group * kTogether + in % n) * kAttnXcds + xcd;
    unit = in / n;
    return true;
  }
  head = blockIdx.x % H;
  unit = blockIdx.x / H;
  return unit < units;
}
unsigned unit_grid(int64_t units, int H) { return (unsigned)(units * H); }

constexpr int kBn = 64;      // keys per tile
constexpr int kNopeTile = kBn * 256, kRopeTile = kBn * 128, kVTile = kBn * 256;
constexpr int kFwdTile = kNopeTile + kRopeTile + kVTile;

// The lane's 32x32x16 operand of 192 query columns (or, offset, 128 of dO).
template <int N>
__device__ __forceinline__ void load_operand(bf16x8 (&f)[N], const uint16_t* row, int half) {
#pragma unroll
  for (int ks = 0; ks < N; ++ks) f[ks] = *reinterpret_cast<const bf16x8*>(row + 16 * ks + 8 * half);
}

// The weights' reference follows the running maximum only once that is more
// than 2^8 above it: weights up to 2^8 cost no precision in FP32 or BF16, and
// the output is rescaled a few times per row instead of per tile.
constexpr float kSlack = 8.f;

// The wave's share of a key tile's loads, one by one: each lane's offsets from
// the tile's first token stay in registers, the tile's base is wave-uniform.
template <int NW>
struct KeyLoader {
  static constexpr int kRows = kBn / NW, kWide = kRows / 4, kLoads = 2 * kWide + kRows / 8;
  static_assert(kRows % 8 == 0, "whole loads per wave");
  uint32_t off[kWide + kRows / 8];
  // last: the tile's last row that exists (rows past it repeat it)
  __device__ __forceinline__ void place(const MlaPrefill& p, int last, int w, int lane) {
#pragma unroll
    for (int n = 0; n < kWide; ++n) {
      const int r = kRows * w + 4 * n + (lane >> 4);
      off[n] = (uint32_t)(min(r, last) * (int)p.kv_stride + (((lane & 15) ^ swz256(r)) << 3)) * 2;
    }
#pragma unroll
    for (int n = 0; n < kRows / 8; ++n) {
      const int r = kRows * w + 8 * n + (lane >> 3);
      off[kWide + n] = (uint32_t)(min(r, last) * (int)p.rope_stride + (((lane & 7) ^ swz128(r)) << 3)) * 2;
    }
  }
  __device__ __forceinline__ void issue(int n, const uint16_t* kv, const uint16_t* kr, int w, uint32_t lds) const {
    if (n < kWide)
      dma16_s(kv, off[n], lds + (kRows * w + 4 * n) * 256);
    else if (n < 2 * kWide)
      dma16_s(kv + kNope, off[n - kWide], lds + kNopeTile + kRopeTile + (kRows * w + 4 * (n - kWide)) * 256);
    else
      dma16_s(kr, off[n - kWide], lds + kNopeTile + (kRows * w + 8 * (n - 2 * kWide)) * 128);
  }
};

// Parts that a block of queries with nt tiles of keys is cut into, `most` at
// the most: no part has fewer than kPartTiles tiles.
constexpr int kPartTiles = 8;
__device__ __forceinline__ int parts_of(int nt, int most) { return max(1, min(most, nt / kPartTiles)); }
constexpr int kJoinSlices = 16;      // workgroups of the join per block of 128 queries: 8 rows each

// Forward: NW waves of 32 queries; key tiles of 64 in three LDS buffers. The
// loop is staggered by one tile: the scores of tile t+1 are formed (matrix
// unit) while the weights of tile t are (vector unit: 32 exponentials a lane,
// about as long as the tile's products), and the values of tile t are added
// while the maxima of tile t+1 are found; so one wave alone keeps both units
// busy, and what it waits for is bridged by the SIMD's second wave. (Formed and
// weighed tile by tile, two chunks of 510 queries with 8000 keys on 32 heads
// took 238 us, so 190.)
//
// 256 queries (NW = 8) halve the tiles' traffic into LDS and give each SIMD
// its second wave; 128 (NW = 4) give twice the workgroups, which can also be
// cut along the keys. Which is taken: see wide_blocks.
//
// Bound by the matrix unit's rate at the clock that the power limit leaves: the
// two long requests run at 1.0 PFLOP/s, 0.53 of the unit's cycles at 1.9 GHz.
// With SPLIT the tiles of a block are shared by several workgroups, which leave
// FP32 partials (output, maximum, sum) for the join below.
template <int NW, bool SPLIT>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2))) void mla_fwd_kernel(const MlaPrefill p,
                                                                                                 int units) {
  constexpr int BM = 32 * NW, NBUF = 3;
  using Load = KeyLoader<NW>;
  __shared__ __align__(1024) char tiles[NBUF * kFwdTile];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int unit, head;
  if (!unit_of(SPLIT ? units * p.parts : units, p.H, unit, head)) return;
  const int part = SPLIT ? unit / units : 0;
  if (SPLIT) unit -= part * units;
  // the last blocks of a causal request see the most keys: they go first
  const ExpertSlot u = locate_expert(p.cu_q, p.B, p.Tq, units - 1 - unit, BM, 1);
  if (u.e < 0) return;
  int k0 = __builtin_amdgcn_readfirstlane(min(max(p.cu_k[u.e], 0), p.Tk));
  const int k1 = __builtin_amdgcn_readfirstlane(min(max(p.cu_k[u.e + 1], k0), p.Tk));
  const int Lq = u.r1 - u.r0;
  int Lk = k1 - k0, off = Lk - Lq;
  const int first = (units - 1 - unit - u.base) * BM;
  const int end = min(first + BM, Lq);                                     // queries of the block
  int kend = p.causal ? min(Lk, max(end + off, 0)) : Lk;                   // keys any of them sees
  int nt = (kend + kBn - 1) / kBn;
  const int parts = SPLIT ? parts_of(nt, p.parts) : 1;
  if (SPLIT) {      // from here on the keys are this part's
    if (part >= parts) return;
    const int t0 = nt * part / parts, skip = t0 * kBn;
    nt = nt * (part + 1) / parts - t0;
    k0 += skip;
    Lk -= skip;
    off -= skip;
    kend = min(kend - skip, nt * kBn);
  }

  const TileLane L(lane);
  const int qi = first + 32 * w + L.row;                                   // this lane's query
  const int qc = min(qi, Lq - 1);
  const int see = p.causal ? min(Lk, qi + off + 1) : Lk;                   // keys it sees
  const int wave_all = p.causal ? min(Lk, first + 32 * w + off + 1) : Lk;  // keys all the wave's queries see
  const int wave_any = p.causal ? min(kend, max(first + 32 * w + 32 + off, 0)) : kend;
  const int wave_nt = first + 32 * w < Lq ? (wave_any + kBn - 1) / kBn : 0;      // its tiles: the first ones

  const uint16_t* kv = p.kv + (int64_t)k0 * p.kv_stride + head * (kNope + kVDim);
  const uint16_t* kr = p.k_rope + (int64_t)k0 * p.rope_stride;
  const uint32_t lds = lds_offset(tiles);
  Load ld;
  ld.place(p, min(Lk, kBn) - 1, w, lane);
  int loaded = 0;      // tiles whose loads are under way
  // the next tile's loads: `kvt`, `krt` its first token
  const uint16_t *kvt = kv, *krt = kr;
  auto loads_begin = [&] {
    if (loaded > 0 && (loaded + 1) * kBn > Lk) ld.place(p, Lk - 1 - loaded * kBn, w, lane);
  };
  auto loads_end = [&] {
    ++loaded;
    kvt += (int64_t)kBn * p.kv_stride;
    krt += (int64_t)kBn * p.rope_stride;
  };

  bf16x8 qf[12];
  load_operand(qf, p.q + (int64_t)(u.r0 + qc) * p.q_stride + head * kQk, L.half);
  const float c = p.scale * kLog2e;
  f32x16 o[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) o[d] = zero16();
  float m = neg_inf(), l = 0.f;      // m: in units of log2
  operands_loaded();
#pragma unroll
  for (int i = 0; i < NBUF - 1; ++i)
    if (i < nt) {
      loads_begin();
#pragma unroll
      for (int n = 0; n < Load::kLoads; ++n) ld.issue(n, kvt, krt, w, lds + i * kFwdTile);
      loads_end();
    }
  const int key0 = at256(L), rope0 = kNopeTile + at128(L), val0 = kNopeTile + kRopeTile + at256t(L);

  // S^T of the tile at LDS offset `at`, operands fetched kAhead steps ahead
  constexpr int kAhead = 4;
  auto products = [&](f32x16 (&s)[2], int at, auto&& between) {
    const int key = opaque(key0 + at), rope = opaque(rope0 + at);
    bf16x8 kf[kAhead];
    auto fetch = [&](int i) {      // step i: k step i/2 of key block i%2
      return i < 16 ? get256(tiles, key, 32 * (i & 1), i >> 1) : get128(tiles, rope, 32 * (i & 1), (i >> 1) - 8);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) kf[i] = fetch(i);
    s[0] = zero16();
    s[1] = zero16();
#pragma unroll
    for (int i = 0; i < 24; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      s[i & 1] = mfma32(kf[i % kAhead], qf[i >> 1], s[i & 1]);
      if (i + kAhead < 24) kf[i % kAhead] = fetch(i + kAhead);
      between(i);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mask = [&](f32x16 (&s)[2], int t) {
    if ((t + 1) * kBn <= wave_all) return;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (t * kBn + 32 * kb + drow(i, L.half) >= see) s[kb][i] = neg_inf();
  };
  // Raises the weights' reference where a tile's maximum asks for it.
  auto raise = [&](float top) {
    top = half_max(top) * c;
    if (__any(top > m + kSlack)) {
      const float mn = max_nan(m, top);
      const float alpha = mn == neg_inf() ? 1.f : exp2_fast(m - mn);
      m = mn;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] *= alpha;
    }
  };
  auto max4 = [](const f32x16& v, int i) { return max_nan(max_nan(v[4 * i], v[4 * i + 1]), max_nan(v[4 * i + 2], v[4 * i + 3])); };

  int buf = 0;
  // Tile t, whose scores are in s; those of tile t+1 go to sn.
  auto step = [&](int t, f32x16 (&s)[2], f32x16 (&sn)[2]) {
    attn_wait<0>();
    attn_barrier();
    const int at = buf * kFwdTile, next = buf + 1 == NBUF ? 0 : buf + 1, prev = buf == 0 ? NBUF - 1 : buf - 1;
    const bool load = loaded < nt;
    if (load) loads_begin();
    auto issue = [&](int n) { ld.issue(n, kvt, krt, w, lds + prev * kFwdTile); };
    if (t < wave_nt) {
      const float ref = m == neg_inf() ? 0.f : m;      // nothing visible yet: every weight is 0
      bf16x8 pb[4];
      float sum[2] = {0.f, 0.f};
      auto weigh = [&](int i) {      // element i of the lane's 32
        const float e = exp2_fast(fmaf(s[i >> 4][i & 15], c, -ref));
        sum[i & 1] += e;
        pb[i >> 3][i & 7] = (__bf16)e;
      };
      auto weigh_at = [&](int i) {      // 32 elements over 24 steps
#pragma unroll
        for (int e = i * 32 / 24; e < (i + 1) * 32 / 24; ++e) weigh(e);
      };
      const bool more = t + 1 < wave_nt;
      if (more && load) {
        products(sn, next * kFwdTile, [&](int i) {
          weigh_at(i);
          if (i * Load::kLoads / 24 != (i + 1) * Load::kLoads / 24) issue(i * Load::kLoads / 24);
        });
      } else {
        if (load) {
#pragma unroll
          for (int n = 0; n < Load::kLoads; ++n) issue(n);
        }
        if (more)
          products(sn, next * kFwdTile, weigh_at);
        else {
#pragma unroll
          for (int i = 0; i < 24; ++i) weigh_at(i);
        }
      }
      l += sum[0] + sum[1];
      if (more) mask(sn, t + 1);
      const int val = opaque(val0 + at);
      bf16x8 vf[kAhead];
      auto fetch = [&](int i) { return get256t(tiles, val, 16 * (i >> 2), i & 3); };      // 16 keys i/4, columns i%4
#pragma unroll
      for (int i = 0; i < kAhead; ++i) vf[i] = fetch(i);
      float top[2] = {neg_inf(), neg_inf()};
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        o[i & 3] = mfma32(vf[i % kAhead], pb[i >> 2], o[i & 3]);
        if (i + kAhead < 16) vf[i % kAhead] = fetch(i + kAhead);
        if (i & 1) top[(i >> 1) & 1] = max_nan(top[(i >> 1) & 1], max4(sn[i >> 3], (i >> 1) & 3));
      }
      __builtin_amdgcn_sched_barrier(0);
      if (more) raise(max_nan(top[0], top[1]));
    } else if (load) {      // nothing here for this wave: only its share of the loads
#pragma unroll
      for (int n = 0; n < Load::kLoads; ++n) issue(n);
    }
    if (load) loads_end();
    buf = next;
  };

  f32x16 sa[2], sb[2];
  if (nt > 0) {
    attn_wait<0>();
    attn_barrier();
    if (wave_nt > 0) {
      products(sa, 0, [](int) {});
      mask(sa, 0);
      float top = neg_inf();
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max_nan(top, max4(sa[i >> 2], i & 3));
      raise(top);
    }
  }
  for (int t = 0; t < nt; t += 2) {
    step(t, sa, sb);
    if (t + 1 < nt) step(t + 1, sb, sa);
  }

  l = half_sum(l);
  if (SPLIT && parts > 1) {
    if (qi < Lq) {
      const int64_t at = ((int64_t)part * p.Tq + u.r0 + qi) * p.H + head;
      float* op = p.part + at * kVDim + 4 * L.half;
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 v;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = o[d][4 * i + j];
          *reinterpret_cast<f32x4*>(op + 32 * d + 8 * i) = v;
        }
      if (L.half == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(m, l);
    }
  } else if (qi < Lq) {
    const float inv = inverse_of(l);
    uint16_t* op = p.out + ((int64_t)(u.r0 + qi) * p.H + head) * kVDim + 4 * L.half;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bf16x4 b;
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = (__bf16)(o[d][4 * i + j] * inv);
        *reinterpret_cast<bf16x4*>(op + 32 * d + 8 * i) = b;
      }
    if (L.half == 0)
      p.lse[(int64_t)head * p.Tq + u.r0 + qi] = lse_of(m, l);
  }
}

// Joins the parts of the blocks that have more than one: 32 lanes a row.
__global__ __launch_bounds__(256) void mla_fwd_join_kernel(const MlaPrefill p, int units) {
  constexpr int BM = 128, kAtOnce = 8;      // parts whose loads are under way together
  const int lane = threadIdx.x & 31, slot = threadIdx.x >> 5;
  const int unit = blockIdx.x / kJoinSlices / p.H, head = blockIdx.x / kJoinSlices % p.H, slice = blockIdx.x % kJoinSlices;
  const ExpertSlot u = locate_expert(p.cu_q, p.B, p.Tq, unit, BM, 1);
  if (u.e < 0) return;
  const int k0 = min(max(p.cu_k[u.e], 0), p.Tk), Lk = min(max(p.cu_k[u.e + 1], k0), p.Tk) - k0;
  const int Lq = u.r1 - u.r0, first = (unit - u.base) * BM, end = min(first + BM, Lq);
  const int kend = p.causal ? min(Lk, max(end + Lk - Lq, 0)) : Lk;
  const int parts = parts_of((kend + kBn - 1) / kBn, p.parts);
  if (parts == 1) return;
  const int64_t step = (int64_t)p.Tq * p.H;      // rows from part to part
  if (const int r = first + 8 * slice + slot; r < end) {
    const int64_t at = (int64_t)(u.r0 + r) * p.H + head;
    float m = neg_inf(), l = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < parts; i0 += kAtOnce) {
      f32x4 v[kAtOnce];
      float2 ml[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int64_t row = at + min(i0 + k, parts - 1) * step;
        v[k] = *reinterpret_cast<const f32x4*>(p.part + row * kVDim + 4 * lane);
        ml[k] = *reinterpret_cast<const float2*>(p.part_ml + 2 * row);
        if (i0 + k >= parts) ml[k] = make_float2(neg_inf(), 0.f);
      }
      float mn = m;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) mn = max_nan(mn, ml[k].x);
      const float ref = mn == neg_inf() ? 0.f : mn, old = exp2_fast(m - ref);
      l *= old;
      o *= old;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float x = exp2_fast(ml[k].x - ref);
        l = fmaf(ml[k].y, x, l);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = i0 + k < parts ? fmaf(v[k][j], x, o[j]) : o[j];
      }
      m = mn;
    }
    const float inv = inverse_of(l);
    bf16x4 b;
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = (__bf16)(o[j] * inv);
    *reinterpret_cast<bf16x4*>(p.out + at * kVDim + 4 * lane) = b;
    if (lane == 0) p.lse[(int64_t)head * p.Tq + u.r0 + r] = lse_of(m, l);
  }
}

// A number as a type, for a function whose code depends on it.
template <int N>
struct Const {
  static constexpr int value = N;
};

constexpr int kBq = 64;
constexpr int kQNope = kBq * 256, kQRope = kBq * 128, kDo = kBq * 256;
constexpr int kBwdTile = kQNope + kQRope + kDo + 2 * kBq * 4;

// Gradients of keys and values: 32 keys are a pair of waves' work, which share
// a SIMD, while 32 queries at a time pass, in tiles of 64 (Q, dO, lse, D). The
// first of the pair forms the scores and the weights, hands the weights (FP32)
// to the second through LDS and adds up dV; the second, a step behind, forms dP
// and dS and adds up dK: 20 products of 32x32x16 each, none formed twice, and
// no more than 48 + 64 (32 + 96) registers of operands and sums, so both fit
// in 256 and one's vector work runs beside the other's products. (One wave for
// both needs 240 for operands and sums alone; alone on its SIMD, with the rest
// in accumulation registers, it took 20-60% longer.) 4096 tokens on 64 heads:
// 0.81 ms, 0.85 PFLOP/s; 20 products of 32 cycles a wave and step leave the
// matrix unit 0.39 busy at 2.2 GHz, the rest is what a step's chain waits for:
// products, exponentials, LDS and the barrier between the two waves.
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) void mla_dkv_kernel(const MlaPrefill p,
                                                                                            int units) {
  constexpr int BK = 128, NBUF = 3, kLoads = 2 + 2 + 1 + 1, kAhead = 6;
  constexpr int kWeights = 32 * 32 * 4;      // a pair's, of one step
  __shared__ __align__(1024) char lds_mem[NBUF * kBwdTile + 2 * 4 * kWeights];
  char* const tiles = lds_mem;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = w & 3;
  int unit, head;
  if (!unit_of(units, p.H, unit, head)) return;
  const ExpertSlot u = locate_expert(p.cu_k, p.B, p.Tk, unit, BK, 1);
  if (u.e < 0) return;
  const int q0 = __builtin_amdgcn_readfirstlane(min(max(p.cu_q[u.e], 0), p.Tq));
  const int q1 = __builtin_amdgcn_readfirstlane(min(max(p.cu_q[u.e + 1], q0), p.Tq));
  const int Lk = u.r1 - u.r0, Lq = q1 - q0, off = Lk - Lq;
  const int kb0 = (unit - u.base) * BK;
  const int key0 = kb0 + 32 * pair;
  const int start = p.causal ? max(0, kb0 - off) : 0;        // first query that sees the block's first key
  const int steps = Lq > start ? (Lq - start + 31) / 32 : 0, nt = (steps + 1) / 2;

  const TileLane L(lane);
  const int key = key0 + L.row, kc = min(key, Lk - 1);
  const uint16_t* qb = p.q + (int64_t)q0 * p.q_stride + head * kQk;
  const uint16_t* db = p.dout + ((int64_t)q0 * p.H + head) * kVDim;
  const float* stat = (w & 1 ? p.delta : p.lse2) + (int64_t)head * p.Tq + q0;      // (four times each, alike)
  const uint32_t lds = lds_offset(tiles);
  // A tile's loads: offsets from its first query in registers, clamped to the
  // last query where the tile has fewer than 64.
  uint32_t off_q[2], off_d[2], off_r, off_s;
  auto place = [&](int last) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int r = 8 * w + 4 * n + (lane >> 4), x = ((lane & 15) ^ swz256(r)) << 3;
      off_q[n] = (uint32_t)(min(r, last) * (int)p.q_stride + x) * 2;
      off_d[n] = (uint32_t)(min(r, last) * p.H * kVDim + x) * 2;
    }
    const int r = 8 * w + (lane >> 3);
    off_r = (uint32_t)(min(r, last) * (int)p.q_stride + (((lane & 7) ^ swz128(r)) << 3)) * 2;
    off_s = (uint32_t)min(lane, last) * 4;
  };
  auto issue = [&](int t, int n, uint32_t at) {
    const int64_t row0 = start + t * kBq;
    const auto uniform = [](uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane(x); };
    if (n < 2)
      dma16_s(qb + row0 * p.q_stride, off_q[n], uniform(at + (8 * w + 4 * n) * 256));
    else if (n < 4)
      dma16_s(db + row0 * (p.H * kVDim), off_d[n - 2], uniform(at + kQNope + kQRope + (8 * w + 4 * (n - 2)) * 256));
    else if (n == 4)
      dma16_s(qb + row0 * p.q_stride + kNope, off_r, uniform(at + kQNope + 8 * w * 128));
    else
      dma4_s(stat + row0, off_s, uniform(at + kQNope + kQRope + kDo + (w & 1) * kBq * 4));
  };
  auto load_tile = [&](int t) {
    const uint32_t to = lds + t % NBUF * kBwdTile;
    if (t == 0 || t == nt - 1) place(min(kBq, Lq - start - t * kBq) - 1);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) issue(t, n, to);
  };
  const float c = p.scale * kLog2e;
  const uint16_t* krow = p.kv + (int64_t)(u.r0 + kc) * p.kv_stride + head * (kNope + kVDim);
  // the pair's weights of steps j and j + 1: [register quad][lane]
  char* const hand = lds_mem + NBUF * kBwdTile + pair * kWeights + 16 * lane;

  // Step j of the loop belongs to the first wave's queries 32 j .. and the
  // second's 32 (j - 1) ..; one barrier each. Even steps begin a tile t = j / 2:
  // it was loaded before, tile t - 2 is free since both are past it.
  auto meet = [&](int j) {
    if (!(j & 1)) attn_wait<0>();
    attn_barrier();
    if (!(j & 1) && (j >> 1) + 1 < nt) load_tile((j >> 1) + 1);
  };

  if (w < 4) {      // scores, weights, dV
    bf16x8 kf[12];
    const uint16_t* rr = p.k_rope + (int64_t)(u.r0 + kc) * p.rope_stride;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) kf[ks] = *reinterpret_cast<const bf16x8*>(krow + 16 * ks + 8 * L.half);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) kf[8 + ks] = *reinterpret_cast<const bf16x8*>(rr + 16 * ks + 8 * L.half);
    f32x16 dv[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) dv[d] = zero16();
    operands_loaded();
    if (nt > 0) load_tile(0);
    const int q_at = at256(L), r_at = kQNope + at128(L), dt_at = kQNope + kQRope + at256t(L);
    const int q_first = p.causal ? key - off : -1, q_all = p.causal ? key0 + 31 - off : -1;
    for (int j = 0; j <= steps; ++j) {
      meet(j);
      if (j == steps) break;      // the second wave's last step
      const int at = (j >> 1) % NBUF * kBwdTile, qr = start + 32 * j;
      const int qa = opaque(q_at + at + (j & 1) * 32 * 256), ra = opaque(r_at + at + (j & 1) * 32 * 128),
                da = opaque(dt_at + at + (j & 1) * 32 * 256);
      bf16x8 f[kAhead];
      f32x16 s = zero16();
      {
        auto fetch = [&](int i) { return i < 8 ? get256(tiles, qa, 0, i) : get128(tiles, ra, 0, i - 8); };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) f[i] = fetch(i);
#pragma unroll
        for (int i = 0; i < 12; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          s = mfma32(f[i % kAhead], kf[i], s);
          if (i + kAhead < 12) f[i % kAhead] = fetch(i + kAhead);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      const float* st = reinterpret_cast<const float*>(tiles + at + kQNope + kQRope + kDo) + 32 * (j & 1) + 4 * L.half;
      f32x4 ls[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ls[i] = *reinterpret_cast<const f32x4*>(st + 8 * i);
      auto fetch = [&](int i) { return get256t(tiles, da, 16 * (i >> 2), i & 3); };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) f[i] = fetch(i);
      if (qr + 32 > Lq || qr < q_all) {      // hide the key from queries that must not see it, and rows past the last
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int qi = qr + drow(i, L.half);
          s[i] = (qi < q_first) | (qi >= Lq) ? neg_inf() : s[i];
        }
      }
      char* const to = hand + (j & 1) * 4 * kWeights;
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        f32x4 e;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          e[k] = exp2_fast(fmaf(s[4 * i4 + k], c, -ls[i4][k]));
          s[4 * i4 + k] = e[k];
        }
        *reinterpret_cast<f32x4*>(to + 1024 * i4) = e;
      }
      const bf16x8 pb[2] = {pack8(s, 0), pack8(s, 1)};
#pragma unroll
      for (int i = 0; i < 8; ++i) {      // D[column drow(i)][key lane%32]
        __builtin_amdgcn_sched_barrier(0);
        dv[i & 3] = mfma32(f[i % kAhead], pb[i >> 2], dv[i & 3]);
        if (i + kAhead < 8) f[i % kAhead] = fetch(i + kAhead);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (key < Lk) {
      uint16_t* out = p.dkv + ((int64_t)(u.r0 + key) * p.H + head) * (kNope + kVDim) + kNope + 4 * L.half;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          bf16x4 b;
#pragma unroll
          for (int k = 0; k < 4; ++k) b[k] = (__bf16)dv[d][4 * i + k];
          *reinterpret_cast<bf16x4*>(out + 32 * d + 8 * i) = b;
        }
    }
  } else {      // dP, dS, dK
    bf16x8 vf[8];
    load_operand(vf, krow + kNope, L.half);
    f32x16 dk[6];
#pragma unroll
    for (int d = 0; d < 6; ++d) dk[d] = zero16();
    operands_loaded();
    if (nt > 0) load_tile(0);
    const int d_at = kQNope + kQRope + at256(L), qt_at = at256t(L), rt_at = kQNope + at128t(L);
    for (int j = 0; j <= steps; ++j) {
      meet(j);
      if (j == 0) continue;      // the first wave's first step
      const int k = j - 1, at = (k >> 1) % NBUF * kBwdTile;
      const int da = opaque(d_at + at + (k & 1) * 32 * 256), qa = opaque(qt_at + at + (k & 1) * 32 * 256),
                ra = opaque(rt_at + at + (k & 1) * 32 * 128);
      bf16x8 f[kAhead];
      f32x16 dp = zero16();
      {
        auto fetch = [&](int i) { return get256(tiles, da, 0, i); };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) f[i] = fetch(i);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          dp = mfma32(f[i % kAhead], vf[i], dp);
          if (i + kAhead < 8) f[i % kAhead] = fetch(i + kAhead);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      const float* st = reinterpret_cast<const float*>(tiles + at + kQNope + kQRope + kDo) + kBq + 32 * (k & 1) + 4 * L.half;
      const char* from = hand + (k & 1) * 4 * kWeights;
      f32x4 e[4], de[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[i] = *reinterpret_cast<const f32x4*>(from + 1024 * i);
        de[i] = *reinterpret_cast<const f32x4*>(st + 8 * i);
      }
      auto fetch = [&](int i) {      // step i: 16 queries i/6, column block i%6
        const int a = 16 * (i / 6), d = i % 6;
        return d < 4 ? get256t(tiles, qa, a, d) : get128t(tiles, ra, a, d - 4);
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) f[i] = fetch(i);
#pragma unroll
      for (int i = 0; i < 16; ++i) dp[i] = e[i >> 2][i & 3] * (dp[i] - de[i >> 2][i & 3]);
      const bf16x8 sb[2] = {pack8(dp, 0), pack8(dp, 1)};
#pragma unroll
      for (int i = 0; i < 12; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        dk[i % 6] = mfma32(f[i % kAhead], sb[i / 6], dk[i % 6]);
        if (i + kAhead < 12) f[i % kAhead] = fetch(i + kAhead);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (key < Lk) {
      uint16_t* out = p.dkv + ((int64_t)(u.r0 + key) * p.H + head) * (kNope + kVDim) + 4 * L.half;
      float* rp = p.rope_part + ((int64_t)head * p.Tk + u.r0 + key) * kRopeDim + 4 * L.half;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          bf16x4 b;
#pragma unroll
          for (int x = 0; x < 4; ++x) b[x] = (__bf16)(dk[d][4 * i + x] * p.scale);
          *reinterpret_cast<bf16x4*>(out + 32 * d + 8 * i) = b;
        }
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          f32x4 v;
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = dk[4 + d][4 * i + x] * p.scale;
          *reinterpret_cast<f32x4*>(rp + 32 * d + 8 * i) = v;
        }
      }
    }
  }
}

// Gradient of the queries: 4 waves of 32 queries over tiles of 64 keys,
// staggered by 32 keys as the keys' gradient is; dS needs no sums between
// workgroups (S and dP are formed a second time instead, 320 of its 512
// multiplications per query and key, so no result depends on any order). 4096
// tokens on 64 heads: 0.63 ms, 0.87 PFLOP/s, bound as the keys' gradient is.
// This kernel also forms what the keys' gradient, launched after it, needs of a
// query: lse in units of log2 (0 if it sees no key: its scores are all masked)
// and D = dO . O, here where dO is in registers already (a kernel
// of its own read 134 MB in 24 us for 4096 tokens on 64 heads).
// D comes from O rounded to BF16. Over many keys that rounding is far below
// those of the weights and of dS; where few keys make O as large as V it is
// their equal (requests of up to 260 tokens: error of dQ and dK 0.0028 of their
// norm instead of 0.0024). A wave whose queries see the first tile alone forms
// D = sum_j P_j dP_j in FP32 instead.
__global__ __launch_bounds__(256, 1) void mla_dq_kernel(const MlaPrefill p, int units) {
  constexpr int NW = 4, BM = 32 * NW, NBUF = 3;
  using Load = KeyLoader<NW>;
  __shared__ __align__(1024) char tiles[NBUF * kFwdTile];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int unit, head;
  if (!unit_of(units, p.H, unit, head)) return;
  const ExpertSlot u = locate_expert(p.cu_q, p.B, p.Tq, units - 1 - unit, BM, 1);
  if (u.e < 0) return;
  const int k0 = __builtin_amdgcn_readfirstlane(min(max(p.cu_k[u.e], 0), p.Tk));
  const int k1 = __builtin_amdgcn_readfirstlane(min(max(p.cu_k[u.e + 1], k0), p.Tk));
  const int Lq = u.r1 - u.r0, Lk = k1 - k0, off = Lk - Lq;
  const int first = (units - 1 - unit - u.base) * BM;
  const int end = min(first + BM, Lq);
  const int kend = p.causal ? min(Lk, max(end + off, 0)) : Lk;
  const int steps = (kend + 31) / 32, nt = (steps + 1) / 2;

  const TileLane L(lane);
  const int qi = first + 32 * w + L.row, qc = min(qi, Lq - 1);
  const int see = p.causal ? min(Lk, qi + off + 1) : Lk;
  const int wave_all = p.causal ? min(Lk, first + 32 * w + off + 1) : Lk;
  const int wave_any = first + 32 * w >= Lq ? 0 : p.causal ? min(kend, max(first + 32 * w + 32 + off, 0)) : Lk;
  const int wave_steps = (wave_any + 31) / 32;

  const uint16_t* kvt = p.kv + (int64_t)k0 * p.kv_stride + head * (kNope + kVDim);      // of the next tile to load
  const uint16_t* krt = p.k_rope + (int64_t)k0 * p.rope_stride;
  const uint32_t lds = lds_offset(tiles);
  Load ld;
  ld.place(p, min(Lk, kBn) - 1, w, lane);
  int loaded = 0;
  auto loads_begin = [&] {
    if (loaded > 0 && (loaded + 1) * kBn > Lk) ld.place(p, Lk - 1 - loaded * kBn, w, lane);
  };
  auto loads_end = [&] {
    ++loaded;
    kvt += (int64_t)kBn * p.kv_stride;
    krt += (int64_t)kBn * p.rope_stride;
  };

  bf16x8 qf[12], df[8];
  load_operand(qf, p.q + (int64_t)(u.r0 + qc) * p.q_stride + head * kQk, L.half);
  load_operand(df, p.dout + ((int64_t)(u.r0 + qc) * p.H + head) * kVDim, L.half);
  bf16x8 of[8];
  load_operand(of, p.out + ((int64_t)(u.r0 + qc) * p.H + head) * kVDim, L.half);
  float lse = p.lse[(int64_t)head * p.Tq + u.r0 + qc];
  const float c = p.scale * kLog2e;
  f32x16 dq[6];
#pragma unroll
  for (int d = 0; d < 6; ++d) dq[d] = zero16();
  operands_loaded();
#pragma unroll
  for (int i = 0; i < NBUF - 1; ++i)
    if (i < nt) {
      loads_begin();
#pragma unroll
      for (int n = 0; n < Load::kLoads; ++n) ld.issue(n, kvt, krt, w, lds + i * kFwdTile);
      loads_end();
    }
  lse = lse == neg_inf() ? 0.f : lse * kLog2e;
  float delta = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) delta = fmaf((float)df[i][k], (float)of[i][k], delta);
  delta = half_sum(delta);
  const int k_at = at256(L), r_at = kNopeTile + at128(L), v_at = kNopeTile + kRopeTile + at256(L);
  const int kt_at = at256t(L), rt_at = kNopeTile + at128t(L);
  constexpr int kAhead = 4;

  // S^T and dP^T of 32 keys (rows: sub * 32 of the tile at LDS offset `at`) by the wave's queries (columns)
  auto products = [&](f32x16& s, f32x16& dp, int at, int sub, auto&& between) {
    const int ka = opaque(k_at + at + sub * 32 * 256), ra = opaque(r_at + at + sub * 32 * 128),
              va = opaque(v_at + at + sub * 32 * 256);
    bf16x8 f[kAhead];
    auto fetch = [&](int i) {
      return i < 8 ? get256(tiles, ka, 0, i) : i < 12 ? get128(tiles, ra, 0, i - 8) : get256(tiles, va, 0, i - 12);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) f[i] = fetch(i);
    s = zero16();
    dp = zero16();
#pragma unroll
    for (int i = 0; i < 20; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      if (i < 12)
        s = mfma32(f[i % kAhead], qf[i], s);
      else
        dp = mfma32(f[i % kAhead], df[i - 12], dp);
      if (i + kAhead < 20) f[i % kAhead] = fetch(i + kAhead);
      between(i);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mask = [&](f32x16& s, int j) {
    if (32 * j + 32 <= wave_all) return;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (32 * j + drow(i, L.half) >= see) s[i] = neg_inf();
  };

  f32x16 s0, dp0, s1, dp1;
  if (nt > 0) {
    if (nt > 1)
      attn_wait<Load::kLoads>();
    else
      attn_wait<0>();
    attn_barrier();
    if (wave_steps > 0) {
      products(s0, dp0, 0, 0, [](int) {});
      mask(s0, 0);
      if (wave_steps <= kBn / 32) {
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) d = fmaf(exp2_fast(fmaf(s0[i], c, -lse)), dp0[i], d);
        if (wave_steps > 1) {
          products(s1, dp1, 0, 1, [](int) {});
          mask(s1, 1);
#pragma unroll
          for (int i = 0; i < 16; ++i) d = fmaf(exp2_fast(fmaf(s1[i], c, -lse)), dp1[i], d);
        }
        delta = half_sum(d);
      }
    }
  }
  if (L.half == 0 && qi < Lq) {
    p.delta[(int64_t)head * p.Tq + u.r0 + qi] = delta;
    p.lse2[(int64_t)head * p.Tq + u.r0 + qi] = lse;
  }
  int buf = 0;      // of the steps' tile
  // Step j, half `sub` of its tile, whose scores and dP are in s and dp; those of step j+1 go to sn and dpn.
  auto step = [&](int j, auto half, f32x16& s, f32x16& dp, f32x16& sn, f32x16& dpn) {
    constexpr int sub = decltype(half)::value;
    const int next = buf + 1 == NBUF ? 0 : buf + 1, prev = buf == 0 ? NBUF - 1 : buf - 1;
    const int at = buf * kFwdTile;
    bool load = false;
    if constexpr (sub == 1) {      // the next step's tile is in LDS for everyone, and the one before this is free
      attn_wait<0>();
      attn_barrier();
      load = loaded < nt;
      if (load) loads_begin();
    }
    auto issue = [&](int n) { ld.issue(n, kvt, krt, w, lds + prev * kFwdTile); };
    if (j < wave_steps) {
      bf16x8 sb[2];
      auto weigh = [&](int i) {      // element i of the lane's 16
        sb[i >> 3][i & 7] = (__bf16)(exp2_fast(fmaf(s[i], c, -lse)) * (dp[i] - delta));
      };
      const int nat = sub ? next * kFwdTile : at;
      const bool more = j + 1 < wave_steps;
      if (more && load)
        products(sn, dpn, nat, sub ^ 1, [&](int i) {
          if (i < 16) weigh(i);
          if (i * Load::kLoads / 20 != (i + 1) * Load::kLoads / 20) issue(i * Load::kLoads / 20);
        });
      else {
        if (load) {
#pragma unroll
          for (int n = 0; n < Load::kLoads; ++n) issue(n);
        }
        if (more)
          products(sn, dpn, nat, sub ^ 1, [&](int i) {
            if (i < 16) weigh(i);
          });
        else {
#pragma unroll
          for (int i = 0; i < 16; ++i) weigh(i);
        }
      }
      if (more) mask(sn, j + 1);
      const int ka = opaque(kt_at + at + sub * 32 * 256), ra = opaque(rt_at + at + sub * 32 * 128);
      bf16x8 f[kAhead];
      auto fetch = [&](int i) {      // step i: 16 keys i/6, column block i%6
        const int a = 16 * (i / 6), k = i % 6;
        return k < 4 ? get256t(tiles, ka, a, k) : get128t(tiles, ra, a, k - 4);
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) f[i] = fetch(i);
#pragma unroll
      for (int i = 0; i < 12; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        dq[i % 6] = mfma32(f[i % kAhead], sb[i / 6], dq[i % 6]);
        if (i + kAhead < 12) f[i % kAhead] = fetch(i + kAhead);
      }
      __builtin_amdgcn_sched_barrier(0);
    } else if (load) {      // nothing here for this wave: only its share of the loads
#pragma unroll
      for (int n = 0; n < Load::kLoads; ++n) issue(n);
    }
    if (load) loads_end();
    if constexpr (sub == 1) buf = next;
  };
  for (int j = 0; j < steps; j += 2) {
    step(j, Const<0>{}, s0, dp0, s1, dp1);
    if (j + 1 < steps) step(j + 1, Const<1>{}, s1, dp1, s0, dp0);
  }
  if (qi < Lq) {
    uint16_t* op = p.dq + ((int64_t)(u.r0 + qi) * p.H + head) * kQk + 4 * L.half;
#pragma unroll
    for (int d = 0; d < 6; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bf16x4 b;
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = (__bf16)(dq[d][4 * i + j] * p.scale);
        *reinterpret_cast<bf16x4*>(op + 32 * d + 8 * i) = b;
      }
  }
}

// dk_rope = sum of the heads' rotary gradients, always in the same order: a
// workgroup's waves take every fourth head each of 256 numbers, so that enough
// loads are under way (one thread for all heads of its numbers: 30 us instead
// of 13 us for 4096 keys on 64 heads, 67 MB).
__global__ __launch_bounds__(256) void mla_rope_sum_kernel(const MlaPrefill p) {
  __shared__ f32x4 sums[3][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t n = (int64_t)p.Tk * kRopeDim, i = ((int64_t)blockIdx.x * 64 + lane) * 4;      // (n: a multiple of 64)
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (i < n) {
#pragma unroll 4
    for (int h = w; h < p.H; h += 4) sum += *reinterpret_cast<const f32x4*>(p.rope_part + h * n + i);
  }
  if (w > 0) sums[w - 1][lane] = sum;
  __syncthreads();
  if (w > 0 || i >= n) return;
  sum = (sum + sums[0][lane]) + (sums[1][lane] + sums[2][lane]);
  bf16x4 b;
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = (__bf16)sum[j];
  *reinterpret_cast<bf16x4*>(p.dk_rope + i) = b;
}

}  // namespace

// Compute units of the MI355X; not asked of the device, so that a workspace's
// size does not depend on it.
static constexpr int kUnits = 256;

// Blocks of `rows` queries on all heads, for requests of average length (the
// host does not know theirs).
static double average_blocks(int64_t Tq, int B, int H, int rows) { return std::ceil((double)Tq / B / rows) * B * H; }

// Few blocks of queries behind many keys leave compute units without work or
// with a second block after the others are done. Cut into s parts, W blocks are
// ceil(W s / CUs) parts after each other on a compute unit (or, causal, the
// longest alone), a part takes 1.3 us per tile and 4 us to begin and end, and
// writing, reading and joining its rows adds 27 ns of the device's time, 8 us
// with the join's launch. The rule takes the s that this makes cheapest, for
// requests of average length.
// Measured, whole against the rule's parts: 512 queries behind 8000 tokens on
// 16 heads 167 and 64 us; 100 behind 100000 on 8 heads 2010 and 158 us; 550 and
// 512 behind 7400 on 32 heads 315 and 272 us. Left whole by the rule, whole
// against two parts: 512 behind 8000 on 128 heads 433 and 456 us, two of 512
// with 1200 keys on 16 heads 35.2 and 37.3 us.
static int narrow_parts(int64_t Tq, int64_t Tk, int B, int H) {
  // (from eight blocks per compute unit on, parts have little left to even out;
  // this bounds the workspace and the launches)
  if (mla_blocks(Tq, B, 128) * H >= 8 * kUnits) return 1;
  constexpr double kTileUs = 1.3, kEndsUs = 4, kJoinUs = 8, kRowsUs = 0.027;
  constexpr int kMost = 16;
  const double q = (double)Tq / B, longest = (double)Tk / B / kBn, mean = std::max(longest - q / (2 * kBn), longest / 2);
  const double W = average_blocks(Tq, B, H, 128);
  int parts = 1;
  double best = 0;
  for (int s = 1; s <= kMost && (s == 1 || s * kPartTiles <= longest); ++s) {
    const double us = std::max(std::ceil(W * s / kUnits) * (mean / s * kTileUs + kEndsUs), longest / s * kTileUs + kEndsUs) +
                      (s > 1 ? kJoinUs + W * s * kRowsUs : 0);
    if (s == 1 || us < best) {
      best = us;
      parts = s;
    }
  }
  return parts;
}

// Blocks of 256 queries where there are more than one and a half of them per
// compute unit. Measured, 256 against 128 queries a block: 4096 tokens on 32
// heads (512 blocks) 172 and 220 us, 3100 behind 30000 on 32 heads (416) 1.99
// and 2.35 ms, two requests of 6000 to 8192 tokens on 128 heads 3.65 and 4.44
// ms. With fewer, 128: 2300 behind 30000 on 32 heads (288) 1.93 and, in parts,
// 1.73 ms, two chunks of 510 behind 7400 on 32 heads (128) 239 and 188 us; in
// between it depends on the lengths (300 blocks: within 10% either way).
// Requests of up to 128 queries have as many blocks of either size, which take
// about as long (100 behind 2000, 16 requests on 32 heads: 132 and 142 us; one
// behind 2000: 108 and 109 us), so only what blocks of 128 in parts are good for
// counts (one behind 30000, 5 requests on 128 heads: 2.10 and 1.86 ms).
static bool wide_blocks(int64_t Tq, int64_t Tk, int B, int H) {
  const double wide = average_blocks(Tq, B, H, 256);
  return wide > 1.5 * kUnits && (wide < average_blocks(Tq, B, H, 128) || narrow_parts(Tq, Tk, B, H) == 1);
}

int mla_prefill_parts(int B, int64_t Tq, int64_t Tk, int H) {
  return B < 1 || wide_blocks(Tq, Tk, B, H) ? 1 : narrow_parts(Tq, Tk, B, H);
}

hipError_t launch_mla_prefill(const MlaPrefill& p, hipStream_t stream) {
  const int64_t wide = mla_blocks(p.Tq, p.B, 256), units = mla_blocks(p.Tq, p.B, 128);
  if (wide_blocks(p.Tq, p.Tk, p.B, p.H)) {
    hipLaunchKernelGGL((mla_fwd_kernel<8, false>), dim3(unit_grid(wide, p.H)), dim3(512), 0, stream, p, (int)wide);
  } else if (p.parts == 1) {
    hipLaunchKernelGGL((mla_fwd_kernel<4, false>), dim3(unit_grid(units, p.H)), dim3(256), 0, stream, p, (int)units);
  } else {
    hipLaunchKernelGGL((mla_fwd_kernel<4, true>), dim3(unit_grid(units * p.parts, p.H)), dim3(256), 0, stream, p,
                       (int)units);
    hipLaunchKernelGGL(mla_fwd_join_kernel, dim3(unit_grid(units * kJoinSlices, p.H)), dim3(256), 0, stream, p, (int)units);
  }
  return hipGetLastError();
}

hipError_t launch_mla_prefill_bwd(const MlaPrefill& p, hipStream_t stream) {
  if (p.Tq > 0) {
    const int64_t units = mla_blocks(p.Tq, p.B, 128);
    hipLaunchKernelGGL(mla_dq_kernel, dim3(unit_grid(units, p.H)), dim3(256), 0, stream, p, (int)units);
  }
  if (p.Tk > 0) {
    const int64_t units = mla_blocks(p.Tk, p.B, 128);
    hipLaunchKernelGGL(mla_dkv_kernel, dim3(unit_grid(units, p.H)), dim3(512), 0, stream, p, (int)units);
    hipLaunchKernelGGL(mla_rope_sum_kernel, dim3((unsigned)(((int64_t)p.Tk * kRopeDim + 255) / 256)), dim3(256), 0,
                       stream, p);
  }
  return hipGetLastError();
}

}  // namespace fp8bs
