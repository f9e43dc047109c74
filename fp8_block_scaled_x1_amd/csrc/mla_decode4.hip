// Latent attention in its absorbed form over a paged cache held in 4 bits: the
// formulas, the ranges of tiles, the partial results and their join are those
// of the kernel over the BF16 and FP8 caches.
//
// A tile is 128 tokens, 32 a wave, and the waves of a workgroup do not meet
// before the end of a request's part of the range: a wave holds its 32 rows'
// queries (144 registers) and the whole of its output (256) and has its own
// tiles in LDS. Codes go to LDS as they are (400 bytes a token by direct
// loads, three tiles deep) and are read twice. For the scores a lane is a token
// and reads 32 codes, one group, at a time: the converter makes exact BF16
// operands of codes and the group's power of two. For the output a lane is 16
// columns, half a group, of 8 tokens: the converter gives two columns of one
// token, and a byte permutation pairs tokens. Scores are formed as keys x
// queries, so a lane's weights are the operand of the product with the values.
//
// Roundings below 32 bits: the weights to BF16 for the matrix unit (2^-9
// relative, on the terms of a mean) and the output.

#include <type_traits>

#include "mla_paged.h"
#include "serve_internal.h"

namespace fp8bs {

namespace {

constexpr int kTile = kFp4Tile, kWaves = 4, kWaveTokens = kTile / kWaves;
constexpr int kLatent = 512, kKey = 576;
constexpr int kBufs = 3;
constexpr int kCodeBytes = kWaveTokens * 256, kRopeBytes = kWaveTokens * 128, kScaleBytes = kWaveTokens * 16;
constexpr int kBufBytes = kCodeBytes + kRopeBytes + kScaleBytes;
constexpr int kCodeLoads = 8, kRopeLoads = 4, kLoads = kCodeLoads + kRopeLoads + 1;
// The weights' reference follows the running maximum once that is more than
// 2^8 above it (weights up to 2^8 cost no precision in FP32 or BF16).
constexpr float kSlack = 8.f;
// Output registers that the waves add up at a time, through the buffers of the tile that is done.
constexpr int kJoinRegs = 2;
static_assert(kJoinRegs * 64 * 64 <= kBufBytes, "a register of 16 blocks from 64 lanes");

struct Problems {
  MlaDecode p[2];
  int split;
};

__device__ __forceinline__ float pow2_byte(uint32_t word, int shift) { return __uint_as_float(((word >> shift) & 0xFFu) << 23); }

template <int SEL>
__device__ __forceinline__ uint32_t cvt2(uint32_t codes, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, SEL));
}
// Eight codes of one token and group as an operand.
__device__ __forceinline__ bf16x8 cvt8(uint32_t codes, float s) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(bf16x8, u32x4{cvt2<0>(codes, s), cvt2<1>(codes, s), cvt2<2>(codes, s), cvt2<3>(codes, s)});
}

// A wave's loads of its 32 tokens of a tile: lane l (and l + 32) holds token
// l's slot. The 16-byte chunks of a token's codes lie permuted by its number
// in the tile, those of its rotary numbers by half of it, so that a column of
// chunks touches every LDS bank once.
struct Loader {
  const MlaDecode& p;
  const int lane, slot;
  const uint32_t lds;
  __device__ __forceinline__ void issue(int n) const {
    if (n < kCodeLoads) {
      const int tok = 4 * n + (lane >> 4);
      const int64_t s = __shfl(slot, tok, 64);
      dma16(p.cache + s * 256 + (((lane & 15) ^ (tok & 15)) << 4), lds + 1024 * n);
    } else if (n < kCodeLoads + kRopeLoads) {
      const int i = n - kCodeLoads, tok = 8 * i + (lane >> 3);
      const int64_t s = __shfl(slot, tok, 64);
      dma16(p.rope + s * 128 + (((lane & 7) ^ ((tok >> 1) & 7)) << 4), lds + kCodeBytes + 1024 * i);
    } else if (lane < kWaveTokens) {
      dma16(p.scales + (int64_t)slot * 16, lds + kCodeBytes + kRopeBytes);
    }
  }
};

template <bool TWO>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(1, 1))) void mla_decode_fp4_kernel(
    const Problems problems) {
  const bool second = TWO && (int)blockIdx.x >= problems.split;
  const MlaDecode& p = problems.p[second];
  const int block = blockIdx.x - (second ? problems.split : 0);
  __shared__ __align__(1024) char tiles[kWaves * (kBufs * kBufBytes + 256)];      // then a wave's block-table entries
  __shared__ float2 stats[kWaves][32];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, row32 = lane & 31;

  // workgroup -> (group, row block), an XCD's consecutive, row blocks of a group first
  const int blocks = p.groups * p.row_blocks, per = blocks / kAttnXcds, rest = blocks % kAttnXcds;
  const int xcd = block % kAttnXcds;
  const int wg = xcd * per + min(xcd, rest) + block / kAttnXcds;
  const int g = wg / p.row_blocks;
  Cursor cur = first_tile<kTile>(p, g);
  if (cur.left == 0) return;

  char* const mine = tiles + wave * kBufs * kBufBytes;
  const int* const entries = reinterpret_cast<const int*>(tiles + kWaves * kBufs * kBufBytes + 256 * wave);
  const uint32_t lds_mine = lds_offset(mine), lds_entries = lds_offset(entries);
  Cursor nxt = cur;      // the tile that is loaded next
  Cursor ent = cur;      // the tile whose block-table entries are fetched next
  auto token_of = [&](const Cursor& c) { return min(c.tile * kTile + kWaveTokens * wave + row32, c.len - 1); };
  auto fetch_entries = [&] {
    dma4(p.table + (int64_t)ent.b * p.table_stride + page_of(p, token_of(ent)), lds_entries);
    advance<kTile>(p, ent);
  };
  auto start_next = [&](int to) {      // the loads of the tile `nxt`, into buffer `to`
    const int entry = entries[lane], tok = token_of(nxt);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const Loader ld{p, lane, opaque(min(max(entry, 0), p.pages - 1) * p.page + (tok - page_of(p, tok) * p.page)),
                    lds_mine + to * kBufBytes};
    advance<kTile>(p, nxt);
    if (ent.left > 0) fetch_entries();
    return ld;
  };
  fetch_entries();
#pragma unroll
  for (int i = 0; i < kBufs - 1; ++i) {
    attn_wait<0>();
    if (nxt.left > 0) {
      const Loader ld = start_next(i);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) ld.issue(n);
    }
  }

  // LDS offsets of this lane
  const int key0 = row32 * 256 + ((half ^ (row32 & 15)) << 4);
  const int rope0 = kCodeBytes + row32 * 128 + ((half ^ ((row32 >> 1) & 7)) << 4);
  const int scale0 = kCodeBytes + kRopeBytes + row32 * 16;
  const int val0 = 4 * half * 256 + (((row32 >> 1) ^ (4 * half)) << 4) + 8 * (row32 & 1);
  const int vscale0 = kCodeBytes + kRopeBytes + 4 * half * 16 + (row32 >> 1);

  const int row = (wg - g * p.row_blocks) * 32 + row32;
  const int late = p.tokens - 1 - min(row, p.rows - 1) / p.heads;        // newest tokens hidden from it

  bf16x8 qf[36];
  f32x16 acc[16];
  float m, l;
  bool first = true;
  int buf = 0;

  while (cur.left > 0) {      // a request's part of the range
    const bool whole = cur.tile == 0 && cur.left >= cur.tiles;
    const uint16_t* qr = p.q + min((int64_t)cur.b * p.rows + min(row, p.rows - 1), p.all_rows - 1) * kKey;
#pragma unroll
    for (int i = 0; i < 32; ++i) qf[i] = *reinterpret_cast<const bf16x8*>(qr + 64 * (i >> 2) + 32 * half + 8 * (i & 3));
#pragma unroll
    for (int i = 0; i < 4; ++i) qf[32 + i] = *reinterpret_cast<const bf16x8*>(qr + kLatent + 16 * i + 8 * half);
    m = neg_inf();
    l = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = zero16();
    operands_loaded();

    for (bool last = false; !last;) {
      if (cur.left > 1)      // the next tile's loads may stay in flight
        attn_wait<kLoads>();
      else
        attn_wait<0>();
      const char* tl = mine + buf * kBufBytes;
      const int tok0 = cur.tile * kTile + kWaveTokens * wave;
      if (nxt.left > 0) {
        const Loader ld = start_next(buf == 0 ? kBufs - 1 : buf - 1);
#pragma unroll
        for (int n = 0; n < kLoads; ++n) ld.issue(n);
      }
      if (tok0 < cur.len) {
        const uint4 sw = *reinterpret_cast<const uint4*>(tl + scale0);
        const uint32_t sc[4] = {sw.x >> (8 * half), sw.y >> (8 * half), sw.z >> (8 * half), sw.w >> (8 * half)};
        f32x16 s = zero16();
#pragma unroll
        for (int i = 0; i < 4; ++i) s = mfma32(lds_bf16x8(tl + (rope0 ^ (i << 5))), qf[32 + i], s);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint4 c = *reinterpret_cast<const uint4*>(tl + (key0 ^ (q << 5)));
          const float f = pow2_byte(sc[q >> 1], 16 * (q & 1));
          s = mfma32(cvt8(c.x, f), qf[4 * q], s);
          s = mfma32(cvt8(c.y, f), qf[4 * q + 1], s);
          s = mfma32(cvt8(c.z, f), qf[4 * q + 2], s);
          s = mfma32(cvt8(c.w, f), qf[4 * q + 3], s);
        }
        if (tok0 + kWaveTokens > cur.len - (p.tokens - 1)) {
          const int seen = cur.len - late - tok0;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (drow(i, half) >= seen) s[i] = neg_inf();
        }
        float top = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = max_nan(top, s[i]);
        top = half_max(top) * p.scale_log2;
        if (__any(top > m + kSlack)) {
          const float mn = max_nan(m, top), alpha = mn == neg_inf() ? 1.f : exp2_fast(m - mn);
          m = mn;
          l *= alpha;
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[j] *= alpha;
        }
        const float ref = m == neg_inf() ? 0.f : m;      // nothing visible yet: every weight is 0
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[i] = exp2_fast(fmaf(s[i], p.scale_log2, -ref));
          l += s[i];
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {      // 16 tokens
          const bf16x8 pb = pack8(s, a);
          uint2 c[8];
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = 8 * (e >> 2) + (e & 3);
            c[e] = *reinterpret_cast<const uint2*>(tl + (val0 ^ (r << 4)) + (16 * a + r) * 256);
            f[e] = __uint_as_float((uint32_t)*reinterpret_cast<const uint8_t*>(tl + vscale0 + (16 * a + r) * 16) << 23);
          }
          auto pair_of = [&](auto sel, bool upper) {
            constexpr int SEL = decltype(sel)::value;
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t x = cvt2<SEL>(upper ? c[2 * k].y : c[2 * k].x, f[2 * k]);
              const uint32_t y = cvt2<SEL>(upper ? c[2 * k + 1].y : c[2 * k + 1].x, f[2 * k + 1]);
              lo[k] = __builtin_amdgcn_perm(y, x, 0x05040100u);
              hi[k] = __builtin_amdgcn_perm(y, x, 0x07060302u);
            }
            typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
            const int j = 2 * SEL + (upper ? 8 : 0);
            acc[j] = mfma32(__builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], lo[2], lo[3]}), pb, acc[j]);
            acc[j + 1] = mfma32(__builtin_bit_cast(bf16x8, u32x4{hi[0], hi[1], hi[2], hi[3]}), pb, acc[j + 1]);
          };
          pair_of(std::integral_constant<int, 0>{}, false);
          pair_of(std::integral_constant<int, 1>{}, false);
          pair_of(std::integral_constant<int, 2>{}, false);
          pair_of(std::integral_constant<int, 3>{}, false);
          pair_of(std::integral_constant<int, 0>{}, true);
          pair_of(std::integral_constant<int, 1>{}, true);
          pair_of(std::integral_constant<int, 2>{}, true);
          pair_of(std::integral_constant<int, 3>{}, true);
        }
      }
      last = cur.tile + 1 == cur.tiles || cur.left == 1;
      if (!last) {
        advance<kTile>(p, cur);
        buf = buf + 1 == kBufs ? 0 : buf + 1;
      }
    }

    // the waves' sums, against the largest of their references
    l = half_sum(l);
    if (half == 0) stats[wave][row32] = make_float2(m, l);
    attn_barrier();
    float mm = neg_inf();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mm = max_nan(mm, stats[w][row32].x);
    const float ref = mm == neg_inf() ? 0.f : mm, part = exp2_fast(m - ref);
    // a thread sums 4 columns of a row: lane `from` of every wave has that row
    const int from = threadIdx.x >> 2, c4 = threadIdx.x & 3, orow = (wg - g * p.row_blocks) * 32 + (from & 31);
    float om = neg_inf(), ol = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) om = max_nan(om, stats[w][from & 31].x);
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      ol = fmaf(stats[w][from & 31].y, exp2_fast(stats[w][from & 31].x - (om == neg_inf() ? 0.f : om)), ol);
    const bool stored = orow < p.rows && (int64_t)cur.b * p.rows + orow < p.all_rows;
    const bool final_result = whole && !p.join;
    const int64_t o = final_result ? (int64_t)cur.b * p.rows + orow
                                   : (whole ? 2 * (int64_t)p.groups + cur.b : 2 * (int64_t)g + (first ? 0 : 1)) * p.rows + orow;
    const float inv = inverse_of(ol);
    char* const slab = mine + buf * kBufBytes;
#pragma unroll
    for (int i0 = 0; i0 < 16; i0 += kJoinRegs) {
#pragma unroll
      for (int i = 0; i < kJoinRegs; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          f32x4 v;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = acc[4 * c + j][i0 + i] * part;
          *reinterpret_cast<f32x4*>(slab + 4096 * i + 64 * lane + ((c ^ ((lane >> 2) & 3)) << 4)) = v;
        }
      attn_barrier();
#pragma unroll
      for (int i = 0; i < kJoinRegs; ++i) {
        f32x4 v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
          v += *reinterpret_cast<const f32x4*>(tiles + (w * kBufs + buf) * kBufBytes + 4096 * i + 64 * from +
                                               ((c4 ^ ((from >> 2) & 3)) << 4));
        const int col = 16 * drow(i0 + i, from >> 5) + 4 * c4;
        if (stored) {
          if (final_result) {
            bf16x4 b;
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = (__bf16)(v[j] * inv);
            *reinterpret_cast<bf16x4*>(p.out + o * kLatent + col) = b;
          } else {
            *reinterpret_cast<f32x4*>(p.part + o * kLatent + col) = v;
          }
        }
      }
      attn_barrier();
    }
    if (stored && from < 32 && c4 == 0) {
      if (final_result)
        p.lse[o] = lse_of(om, ol);
      else
        *reinterpret_cast<float2*>(p.part_ml + 2 * o) = make_float2(om, ol);
    }
    first = false;
    advance<kTile>(p, cur);
    buf = buf + 1 == kBufs ? 0 : buf + 1;
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
