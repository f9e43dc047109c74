// Latent attention in its absorbed form over a paged cache held in 4 bits: the
// formulas, the ranges of tiles, the partial results and their join are those
// of the kernel over the BF16 and FP8 caches.
//
// A workgroup has 32 rows; its four waves have one SIMD each and 512 registers.
// Scores: a wave forms those of 16 of a tile's 64 tokens and holds all of the
// rows' queries. A lane is a token and a quarter of its groups: it loads its
// codes from global memory (400 bytes a token, a tile ahead, in
// registers), and the converter turns 8 codes and their group's power of two
// into an exact BF16 operand. An operand is formed once: it goes to the score
// product and, as it is, to the tile's place in LDS, which the value product
// reads transposed (converted a second time for the values, in another layout,
// the registers spilled and 128 rows of 128 requests took 946 us). Values: a
// wave adds all 64 tokens into its 128 columns. Tiles alternate between two
// places, so a tile's values and the next tile's scores are formed together and
// the waves meet once a tile; conversions, matrix instructions and LDS fill
// each other's waits.
//
// Bound: a tile takes 3500 clocks, of which the matrix units need 1088, the
// address unit 1790 and LDS 1460. With one wave on a SIMD the rest is latency:
// without loads, conversions, writes of the numbers to LDS and waits for the
// maxima 2700 would be left, products, weights and the meeting of the waves. 128
// rows of 128 requests of 300 to 4500 tokens 151 us (543 TFLOP/s), 32 rows of 8
// requests of 41000 to 67000 67 us (2.7 TB/s, 465 TFLOP/s), 32 rows of 192
// requests behind a prefix of 16000 317 us (694 TFLOP/s). In graphs over the BF16,
// FP8 and this cache they take 153, 161 and 144 us, 112, 82 and 63, 298, 339 and
// 313 (the kernel over the others has two waves on a SIMD, with half of the key's
// columns each; not built here). Not kept: codes through LDS by direct
// loads (as fast, more code), loads by whole rows, which take a third of the
// address unit's time, with the quarters exchanged between lanes (the prefix's
// call 402 us), loads three tiles ahead (a third copy of the code: 10
// requests of 300 behind a prefix of 12000 50.5 us, now 47; long ones as fast), the waves' wishes looked at beside the next tile's scores (334).
//
// Roundings below 32 bits: the weights to BF16 for the matrix unit (relative 2^-8
// at most each, on the terms of a mean) and the output.

#include <type_traits>
#include <utility>

#include "mla_paged.h"
#include "serve_internal.h"

namespace fp8bs {

namespace {

constexpr int kTile = kFp4Tile, kWaves = 4, kWaveTokens = kTile / kWaves;
static_assert(kTile == 64 && kWaveTokens == 16, "a wave's tokens are the rows of a 16x16x32 product");
constexpr int kLatent = 512, kKey = 576;
constexpr int kRowBytes = 2 * kLatent;
// A tile in LDS: latent numbers, weights (as the value product's operand), row maxima and wishes of the waves.
constexpr int kWeightsAt = kTile * kRowBytes, kStatAt = kWeightsAt + kTile * 32 * 2;
constexpr int kTileBytes = kStatAt + kWaves * 256;
// The weights' reference follows the running maximum once that is more than
// 2^8 above it (weights up to 2^8 cost no precision in FP32 or BF16).
constexpr float kSlack = 8.f;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The next tile of the range; lengths by scalar loads (the kernel writes none
// of them), which leave the tiles' loads in flight alone.
__device__ __forceinline__ void next_tile(const MlaDecode& p, Cursor& c) {
  typedef const __attribute__((address_space(4))) int32_t* scalar_ptr;
  --c.left;
  if (++c.tile < c.tiles || c.left <= 0) return;
  const scalar_ptr lens = (scalar_ptr)(uintptr_t)p.lens;
  do {
    ++c.b;
    c.len = c.b < p.B ? min(max(lens[__builtin_amdgcn_readfirstlane(c.b * p.len_stride)], 0), p.max_len) : 0;
  } while (c.len == 0 && c.b < p.B);
  c.tile = 0;
  c.tiles = tiles_of<kTile>(c.len);
}

struct Problems {
  MlaDecode p[2];
  int split;
};

template <int SEL>
__device__ __forceinline__ uint32_t cvt2(uint32_t codes, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, SEL));
}
// Eight codes of one token and group as an operand.
__device__ __forceinline__ u32x4 cvt8(uint32_t codes, float s) {
  return u32x4{cvt2<0>(codes, s), cvt2<1>(codes, s), cvt2<2>(codes, s), cvt2<3>(codes, s)};
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A lane's part of its token: groups q, 4 + q, 8 + q and 12 + q (q = lane / 16),
// 16 of the rotary numbers, and the token's 16 exponents.
struct Raw {
  u32x4 codes[4];
  bf16x8 rope[2];
  u32x4 exps;
};

// The 16-byte chunks of a token's numbers in LDS are permuted by the token, so
// that 8 tokens at one chunk (written) and 4 at two (read) touch every bank once.
__device__ __forceinline__ int swz(int r) { return ((r & 3) << 1) | ((r >> 2) & 1) | (r & 8); }

// The value of the lane 16 away within a half, combined with this lane's (both get the result).
__device__ __forceinline__ float quarter_max(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max_nan(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float quarter_sum(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <bool TWO>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(1, 1))) void mla_decode_fp4_kernel(
    const Problems problems) {
  const bool second = TWO && (int)blockIdx.x >= problems.split;
  MlaDecode p = problems.p[second];
  // What every tile needs is kept in scalar registers (no instruction): loaded
  // again from the arguments each time, it makes a wave wait for all of its LDS
  // accesses as well (the prefix's call 342 us, then 328).
  auto keep_one = [](auto& x) {
    if constexpr (std::is_pointer_v<std::remove_reference_t<decltype(x)>>) {
      // (a pointer from nowhere would be taken for one into any memory)
      auto* y = (__attribute__((address_space(1))) std::remove_pointer_t<std::remove_reference_t<decltype(x)>>*)x;
      asm("" : "+s"(y));
      x = (std::remove_reference_t<decltype(x)>)y;
    } else {
      asm("" : "+s"(x));
    }
  };
  auto keep = [&](auto&... x) { (keep_one(x), ...); };
  keep(p.cache, p.scales, p.rope, p.table, p.lens, p.table_stride, p.len_stride, p.max_len, p.B, p.pages, p.page, p.page_magic,
       p.page_shift, p.scale_log2, p.tokens);
  const int block = blockIdx.x - (second ? problems.split : 0);
  __shared__ __align__(1024) char tiles[2 * kTileBytes];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tok16 = lane & 15, q4 = lane >> 4;
  const TileLane L(lane);

  // workgroup -> (group, row block), an XCD's consecutive, row blocks of a group first
  const int blocks = p.groups * p.row_blocks, per = blocks / kAttnXcds, rest = blocks % kAttnXcds;
  const int xcd = block % kAttnXcds;
  const int wg = xcd * per + min(xcd, rest) + block / kAttnXcds;
  const int g = wg / p.row_blocks;
  Cursor cur = first_tile<kTile>(p, g);
  if (cur.left == 0) return;

  Cursor nxt = cur;      // the tile that is loaded next
  Cursor ent = cur;      // the tile whose block-table entries are fetched next
  auto token_of = [&](const Cursor& c) { return min(c.tile * kTile + kWaveTokens * wave + tok16, c.len - 1); };
  // Past the range's end its last tile is loaded again: loads under a condition
  // would make the waits for earlier ones wait for these too.
  int entry;
  auto fetch_entry = [&] {
    entry = p.table[(int64_t)ent.b * p.table_stride + page_of(p, token_of(ent))];
    if (ent.left > 1) next_tile(p, ent);
  };
  int64_t slot = 0;      // of the tile that is being loaded
  auto next_slot = [&] {      // of the tile `nxt`, whose entries are here
    const int tok = token_of(nxt);
    slot = min(max(entry, 0), p.pages - 1) * p.page + (tok - page_of(p, tok) * p.page);
    if (nxt.left > 1) next_tile(p, nxt);
    fetch_entry();
  };
  Raw raw;      // of the tile whose scores come next
  auto load_part = [&](int n) {      // 0 .. 3: codes, 4, 5: rotary numbers, 6: exponents
    if (n < 4)
      raw.codes[n] = *reinterpret_cast<const u32x4*>(p.cache + slot * 256 + 16 * q4 + 64 * n);
    else if (n < 6)
      raw.rope[n - 4] = *reinterpret_cast<const bf16x8*>(p.rope + slot * 128 + 16 * q4 + 64 * (n - 4));
    else
      raw.exps = *reinterpret_cast<const u32x4*>(p.scales + slot * 16);
  };
  fetch_entry();
  next_slot();
#pragma unroll
  for (int n = 0; n < 7; ++n) load_part(n);

  // LDS offsets of this lane in a tile: where it writes its token's numbers
  // (16-byte chunk 4 * q4 + s of each 256 bytes, permuted by the token), and
  // where it reads its columns transposed
  const int put0 = (kWaveTokens * wave + tok16) * kRowBytes + (((4 * q4) ^ swz(tok16)) << 4);
  const int val0 = L.trow * kRowBytes + 256 * wave + L.tbyte + ((L.tchunk ^ swz(L.trow)) << 4);
  const int weight0 = kWeightsAt + 1024 * wave + (tok16 + 32 * (q4 & 1)) * 16 + 8 * (q4 >> 1);

  const int row0 = (wg - g * p.row_blocks) * 32;
  const int row = row0 + L.row;      // of the lane's outputs
  int late[2];                       // newest tokens hidden from the rows of its scores
#pragma unroll
  for (int h = 0; h < 2; ++h) late[h] = p.tokens - 1 - min(row0 + 16 * h + tok16, p.rows - 1) / p.heads;

  bf16x8 qf[2][18];
  f32x16 acc[4];
  float m[2], mo, l[2];      // reference of the rows of the lane's scores, of its outputs; sums of its weights
  bool first = true;
  int at = 0;                // offset of the tile whose values come next

  // The rows' queries go through LDS (the place whose values are done with):
  // loaded by each wave as it needs them, a lane a row, they would take the
  // address unit 9400 clocks, 4 us of every request's part; a row's end is
  // padded so that 16 rows at one chunk touch every bank once.
  auto start_piece = [&] {
    constexpr int kChunks = 2 * kKey / 16, kStride = 2 * kKey + 16, kLoads = 8 * kChunks / 64;
    static_assert(32 / kWaves == 8 && 8 * kChunks % 64 == 0 && 32 * kStride <= kWeightsAt, "a wave loads 8 rows");
    char* const stage = tiles + at;
    u32x4 in[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int chunk = 64 * i + lane, r = 8 * wave + chunk / kChunks, c = chunk % kChunks;
      const int64_t from = min((int64_t)cur.b * p.rows + min(row0 + r, p.rows - 1), p.all_rows - 1);
      in[i] = *reinterpret_cast<const u32x4*>(p.q + from * kKey + 8 * c);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int chunk = 64 * i + lane;
      *reinterpret_cast<u32x4*>(stage + (8 * wave + chunk / kChunks) * kStride + 16 * (chunk % kChunks)) = in[i];
    }
    attn_barrier();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const char* qr = stage + opaque((16 * h + tok16) * kStride);
#pragma unroll
      for (int i = 0; i < 16; ++i) qf[h][i] = lds_bf16x8(qr + 256 * (i >> 2) + 64 * q4 + 16 * (i & 3));
#pragma unroll
      for (int i = 0; i < 2; ++i) qf[h][16 + i] = lds_bf16x8(qr + 2 * kLatent + 64 * i + 16 * q4);
      m[h] = neg_inf();
      l[h] = 0.f;
    }
    // (no instruction: the queries stay in the accumulation registers, which the products read as well)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 18; ++i) {
        u32x4 v = __builtin_bit_cast(u32x4, qf[h][i]);
        asm("" : "+a"(v));
        qf[h][i] = __builtin_bit_cast(bf16x8, v);
      }
    mo = neg_inf();
#pragma unroll
    for (int d = 0; d < 4; ++d) acc[d] = zero16();
  };

  // What a tile goes through. Scores: those of the wave's 16 tokens, whose
  // numbers go to the tile's place `to`; as the registers of raw are done with,
  // the next tile's loads follow into them, one at a time (a
  // wave that issues its loads in one go stands still until the address unit
  // has taken them all). Weights against the reference. Values: of the tile at
  // `from`, the one before, 16 products of which half go beside the scores and
  // half beside the weights.
  f32x4 s[2];
  float top[2], sum[2];
  auto weigh = [&](int to) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float ref = m[h] == neg_inf() ? 0.f : m[h];      // nothing visible yet: every weight is 0
      f32x4 e;
      bf16x4 b;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[j] = exp2_fast(fmaf(s[h][j], p.scale_log2, -ref));
        b[j] = (__bf16)e[j];
      }
      sum[h] = (e[0] + e[1]) + (e[2] + e[3]);
      *reinterpret_cast<bf16x4*>(tiles + to + weight0 + 256 * h) = b;
    }
  };
  auto tile_work = [&](auto with_scores, auto with_values, const Cursor& c, int to, int from) {
    constexpr bool S = decltype(with_scores)::value, V = decltype(with_values)::value;
    const int put = opaque(put0 + to), val = opaque(val0 + from);
    bf16x8 pb[4];
    constexpr int kFetch = 4;      // operands of the values under way
    bf16x8 v[kFetch];
    auto fetch = [&](int i) {
      const int t = 16 * (i >> 2), d = i & 3;
      v[i % kFetch] = join(lds_tr16(tiles + (val ^ (d << 6)) + t * kRowBytes),
                           lds_tr16(tiles + (val ^ (d << 6) ^ 128) + (t + 8) * kRowBytes));
    };
    auto value = [&](auto index) {
      constexpr int I = decltype(index)::value;
      acc[I & 3] = mfma32(v[I % kFetch], pb[I >> 2], acc[I & 3]);
      if constexpr (I + kFetch < 16) fetch(I + kFetch);
    };
    if constexpr (V) {
      const char* w = tiles + opaque(from + kWeightsAt + 16 * lane);
#pragma unroll
      for (int a = 0; a < 4; ++a) pb[a] = lds_bf16x8(w + 1024 * a);
#pragma unroll
      for (int i = 0; i < kFetch; ++i) fetch(i);
    }
    float f[4];
    auto score = [&](auto index) {      // 32 of the key's columns
      constexpr int I = decltype(index)::value, P = I >> 2, C = I & 3;
      const u32x4 k = cvt8(raw.codes[P][C], f[P]);
      *reinterpret_cast<u32x4*>(tiles + (put ^ (C << 4)) + 256 * P) = k;
#pragma unroll
      for (int h = 0; h < 2; ++h) s[h] = mfma16(__builtin_bit_cast(bf16x8, k), qf[h][I], s[h]);
    };
    if constexpr (S) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(((raw.exps[i] >> (8 * q4)) & 0xFFu) << 23);
#pragma unroll
      for (int h = 0; h < 2; ++h) s[h] = f32x4{0.f, 0.f, 0.f, 0.f};
      next_slot();
    }
    auto group = [&](auto index) {
      constexpr int I = decltype(index)::value;
      if constexpr (V) value(index);
      if constexpr (S) {
        score(std::integral_constant<int, 2 * I>{});
        score(std::integral_constant<int, 2 * I + 1>{});
        if constexpr (I < 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) s[h] = mfma16(raw.rope[I], qf[h][16 + I], s[h]);
        }
        if constexpr (I == 0) load_part(6);
        if constexpr (I == 2 || I == 4) load_part(4 + (I >> 2));
        if constexpr (I & 1) load_part(I >> 1);
      }
    };
    [&]<int... I>(std::integer_sequence<int, I...>) { (group(std::integral_constant<int, I>{}), ...); }
    (std::make_integer_sequence<int, 8>{});
    if constexpr (S) {
      if ((c.tile + 1) * kTile > c.len - (p.tokens - 1)) {
        const int tok0 = c.tile * kTile + kWaveTokens * wave + 4 * q4;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (tok0 + j >= c.len - late[h]) s[h][j] = neg_inf();
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        top[h] = half_max(quarter_max(max_nan(max_nan(s[h][0], s[h][1]), max_nan(s[h][2], s[h][3])))) * p.scale_log2;
      weigh(to);
      float* const stat = reinterpret_cast<float*>(tiles + to + kStatAt);
      if (q4 < 2) stat[64 * wave + lane] = q4 ? top[1] : top[0];
      if (lane == 0) stat[64 * wave + 32] = 0.f;
      if (top[0] > m[0] + kSlack || top[1] > m[1] + kSlack) stat[64 * wave + 32] = 1.f;
    }
    if constexpr (V) {
      [&]<int... I>(std::integer_sequence<int, I...>) { (value(std::integral_constant<int, I + 8>{}), ...); }
      (std::make_integer_sequence<int, 8>{});
    }
  };

  // The waves meet at a tile's weights. If one wishes the reference raised, all do (the answer is the same for all).
  auto meet = [&](int to) {
    const float* const stat = reinterpret_cast<const float*>(tiles + to + kStatAt);
    attn_barrier();
    if (__any(stat[64 * (lane & 3) + 32] != 0.f)) {
      float n[2] = {m[0], m[1]}, no = mo;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        n[0] = max_nan(n[0], stat[64 * w + tok16]);
        n[1] = max_nan(n[1], stat[64 * w + 16 + tok16]);
        no = max_nan(no, stat[64 * w + L.row]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] *= n[h] == neg_inf() ? 1.f : exp2_fast(m[h] - n[h]);
        m[h] = n[h];
      }
      const float alpha = no == neg_inf() ? 1.f : exp2_fast(mo - no);
      mo = no;
#pragma unroll
      for (int d = 0; d < 4; ++d) acc[d] *= alpha;
      weigh(to);
      attn_barrier();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) l[h] += sum[h];
  };

  auto finish_piece = [&](bool whole) {
    float* const stat = reinterpret_cast<float*>(tiles + at + kStatAt);
    attn_barrier();      // everyone has read the maxima there
#pragma unroll
    for (int h = 0; h < 2; ++h) l[h] = half_sum(quarter_sum(l[h]));
    if (q4 < 2) stat[64 * wave + lane] = q4 ? l[1] : l[0];
    attn_barrier();
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) total += stat[64 * w + L.row];
    if (row < p.rows && (int64_t)cur.b * p.rows + row < p.all_rows) {
      if (whole && !p.join) {
        const int64_t o = (int64_t)cur.b * p.rows + row;
        const float inv = inverse_of(total);
        uint16_t* op = p.out + o * kLatent + 128 * wave + 4 * L.half;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            bf16x4 b;
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = (__bf16)(acc[d][4 * i + j] * inv);
            *reinterpret_cast<bf16x4*>(op + 32 * d + 8 * i) = b;
          }
        if (wave == 0 && L.half == 0) p.lse[o] = lse_of(mo, total);
      } else {
        const int64_t o = (whole ? 2 * (int64_t)p.groups + cur.b : 2 * (int64_t)g + (first ? 0 : 1)) * p.rows + row;
        float* op = p.part + o * kLatent + 128 * wave + 4 * L.half;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = acc[d][4 * i + j];
            *reinterpret_cast<f32x4*>(op + 32 * d + 8 * i) = v;
          }
        if (wave == 0 && L.half == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * o) = make_float2(mo, total);
      }
    }
  };

  // The range, tile by tile: `r` holds the tile whose scores come next. After
  // the last one of a request's part its values are added alone.
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  bool whole = cur.tile == 0 && cur.left >= cur.tiles, fresh = true;
  auto step = [&] {      // returns whether a tile follows
    // (the other place also where nothing is in this one: someone may still read the sums of the last request there)
    if (fresh) {
      start_piece();
      tile_work(yes, no, cur, at ^ kTileBytes, 0);
      fresh = false;
    } else {
      tile_work(yes, yes, cur, at ^ kTileBytes, at);
    }
    at ^= kTileBytes;
    meet(at);
    const bool last = cur.tile + 1 == cur.tiles || cur.left == 1;
    if (last) {
      tile_work(no, yes, cur, 0, at);
      finish_piece(whole);
      first = false;
      fresh = true;
    }
    next_tile(p, cur);
    if (last) whole = cur.left >= cur.tiles;
    return cur.left > 0;
  };
  while (step()) {
  }
}

}  // namespace

hipError_t launch_mla_decode_fp4(const MlaDecode& own, const MlaDecode* prefix, hipStream_t stream) {
  const MlaDecode& head = prefix ? *prefix : own;
  const Problems two{{head, own}, head.groups * (int)head.row_blocks};
  const dim3 block(64 * kWaves);
  if (prefix && own.max_len > 0)
    hipLaunchKernelGGL(mla_decode_fp4_kernel<true>, dim3((unsigned)(two.split + (int64_t)own.groups * own.row_blocks)), block,
                       0, stream, two);
  else if (prefix || own.max_len > 0)
    hipLaunchKernelGGL(mla_decode_fp4_kernel<false>, dim3((unsigned)two.split), block, 0, stream, two);
  launch_mla_join<kTile>(own, head, prefix != nullptr, stream);
  return hipGetLastError();
}

}  // namespace fp8bs
