// Latent vectors quantized as they are written into a paged cache, and read
// back.
//
// A wave takes a token: 512 latent numbers are 16 bytes a lane, so a group of
// 128 (FP8) is a DPP row and a group of 32 (FP4) four lanes, and every row that
// is read or written is one access of the wave. The token's request is the one
// whose range of the packed rows holds it, found by 64-way search of the
// offsets. The arithmetic of a token is a few dozen instructions; what bounds
// these kernels is the chain offset -> length -> table entry -> slot at the
// small end (96 requests of 1 to 3 tokens: 3.3 us either way) and memory at the
// large one (36900 tokens, FP8: written in 15.5 us, read in 14.6, 4.5 TB/s).

#include "attn_common.h"
#include "device_common.h"
#include "fp8bs_serve.h"
#include "serve_internal.h"

namespace fp8bs {

namespace {

constexpr int kWaves = 4;

// The request b with cu[b] <= t < cu[b+1] and the token's position in it; -1
// if there is none. Wave-uniform. The first level that fits in 64 lanes is read
// at once; 4096 requests take two levels.
struct Place {
  int64_t pos;
  int b;
};

__device__ __forceinline__ Place place_of(const MlaCache& c, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, span = c.B;
  for (;;) {
    const int step = (span + 63) >> 6;
    const int i = min(lo + step * (lane + 1), c.B);
    const bool below = c.cu[i] <= t && lo + step * (lane + 1) <= c.B;
    lo += step * (int)__popcll(__ballot(below));
    if (lo >= c.B) return Place{-1, -1};
    if (step == 1) break;
    span = min(step, c.B - lo);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int first = c.cu[lo], end = c.cu[lo + 1];
  if (t < first || t >= end) return Place{-1, -1};
  return Place{(int64_t)c.lens[lo] - (end - t), lo};
}

// The page that holds position pos of request b, as the table says.
__device__ __forceinline__ int entry_of(const MlaCache& c, const Place& at, int& slot) {
  const int page = (int)(((uint64_t)(uint32_t)at.pos * c.page_magic) >> c.page_shift);
  slot = (int)at.pos - page * c.page;
  return c.table[at.b * c.width + page];
}

__device__ __forceinline__ float pow2_of(int byte) { return __uint_as_float((uint32_t)byte << 23); }

// The exponent (127 added) of a group of 32 from its largest magnitude, a BF16
// number: the smallest e with amax <= 6 * 2^e = 1.5 * 2^(e+2), so the number's
// own exponent less 2, or less 1 if its mantissa is above 1.5; at least -126.
__device__ __forceinline__ int fp4_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return 127;
  return max((int)(u >> 23) - 2 + ((u & 0x7FFFFFu) > 0x400000u ? 1 : 0), 1);
}

template <int KIND>
__global__ __launch_bounds__(64 * kWaves) void cache_write_kernel(const MlaCache c) {
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6));
  if (t >= c.T) return;
  const uint4 d = *reinterpret_cast<const uint4*>(c.latent + t * c.latent_stride + 8 * lane);
  uint4 r = make_uint4(0, 0, 0, 0);
  if (lane < 8) r = *reinterpret_cast<const uint4*>(c.out_rope + t * c.rope_stride + 8 * lane);
  const Place at = place_of(c, t);
  if (at.pos < 0 || at.pos >= c.max_len) return;
  int in_page;
  const int page = entry_of(c, at, in_page);
  if (page < 0 || page >= c.pages) return;
  const int64_t slot = (int64_t)page * c.page + in_page;
  if constexpr (KIND == FP8BS_CACHE_BF16) {
    char* row = c.cache + slot * 1152;
    *reinterpret_cast<uint4*>(row + 16 * lane) = d;
    if (lane < 8) *reinterpret_cast<uint4*>(row + 1024 + 16 * lane) = r;
  } else {
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
    float v[8], amax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    if constexpr (KIND == FP8BS_CACHE_FP8) {
      const GroupDiv g = group_div<true>(row16_max(amax));
      *reinterpret_cast<uint2*>(c.cache + slot * 512 + 8 * lane) =
          make_uint2(e4m3_div_pack4_bf16(v[0], v[1], v[2], v[3], g), e4m3_div_pack4_bf16(v[4], v[5], v[6], v[7], g));
      if ((lane & 15) == 0) *reinterpret_cast<float*>(c.scales + slot * 16 + 4 * (lane >> 4)) = g.s;
    } else {
      amax = fmaxf(amax, __shfl_xor(amax, 1, 64));
      amax = fmaxf(amax, __shfl_xor(amax, 2, 64));
      const int e = fp4_exponent(amax);
      const float s = pow2_of(e);
      uint32_t q = 0;      // nearest, halfway to even; the converter divides by its scale
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
      *reinterpret_cast<uint32_t*>(c.cache + slot * 256 + 4 * lane) = q;
      if ((lane & 3) == 0) c.scales[slot * 16 + (lane >> 2)] = (char)e;
    }
    if (lane < 8) *reinterpret_cast<uint4*>(c.rope + slot * 128 + 16 * lane) = r;
  }
}

template <int KIND>
__global__ __launch_bounds__(64 * kWaves) void cache_read_kernel(const MlaCache c) {
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6));
  if (t >= c.T) return;
  const Place at = place_of(c, t);
  if (at.b < 0) return;
  uint4 d = make_uint4(0, 0, 0, 0), r = d;
  if (at.pos >= 0 && at.pos < c.max_len) {
    int in_page;
    const int page = min(max(entry_of(c, at, in_page), 0), c.pages - 1);
    const int64_t slot = (int64_t)page * c.page + in_page;
    if constexpr (KIND == FP8BS_CACHE_BF16) {
      const char* row = c.cache + slot * 1152;
      d = *reinterpret_cast<const uint4*>(row + 16 * lane);
      if (lane < 8) r = *reinterpret_cast<const uint4*>(row + 1024 + 16 * lane);
    } else {
      if (lane < 8) r = *reinterpret_cast<const uint4*>(c.rope + slot * 128 + 16 * lane);
      bf16x2 o[4];
      if constexpr (KIND == FP8BS_CACHE_FP8) {
        const uint2 q = *reinterpret_cast<const uint2*>(c.cache + slot * 512 + 8 * lane);
        const float s = *reinterpret_cast<const float*>(c.scales + slot * 16 + 4 * (lane >> 4));
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
          o[2 * i] = bf16x2{(__bf16)(a[0] * s), (__bf16)(a[1] * s)};
          o[2 * i + 1] = bf16x2{(__bf16)(b[0] * s), (__bf16)(b[1] * s)};
        }
      } else {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(c.cache + slot * 256 + 4 * lane);
        const float s = pow2_of((uint8_t)c.scales[slot * 16 + (lane >> 2)]);
        o[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0);
        o[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1);
        o[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2);
        o[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3);
      }
      d = make_uint4(__builtin_bit_cast(uint32_t, o[0]), __builtin_bit_cast(uint32_t, o[1]),
                     __builtin_bit_cast(uint32_t, o[2]), __builtin_bit_cast(uint32_t, o[3]));
    }
  }
  *reinterpret_cast<uint4*>(c.latent + t * c.latent_stride + 8 * lane) = d;
  if (lane < 8) *reinterpret_cast<uint4*>(c.out_rope + t * c.rope_stride + 8 * lane) = r;
}

}  // namespace

hipError_t launch_mla_cache_write(const MlaCache& c, hipStream_t stream) {
  const dim3 grid((unsigned)((c.T + kWaves - 1) / kWaves)), block(64 * kWaves);
  if (c.kind == FP8BS_CACHE_BF16)
    hipLaunchKernelGGL(cache_write_kernel<FP8BS_CACHE_BF16>, grid, block, 0, stream, c);
  else if (c.kind == FP8BS_CACHE_FP8)
    hipLaunchKernelGGL(cache_write_kernel<FP8BS_CACHE_FP8>, grid, block, 0, stream, c);
  else
    hipLaunchKernelGGL(cache_write_kernel<FP8BS_CACHE_FP4>, grid, block, 0, stream, c);
  return hipGetLastError();
}

hipError_t launch_mla_cache_read(const MlaCache& c, hipStream_t stream) {
  const dim3 grid((unsigned)((c.T + kWaves - 1) / kWaves)), block(64 * kWaves);
  if (c.kind == FP8BS_CACHE_BF16)
    hipLaunchKernelGGL(cache_read_kernel<FP8BS_CACHE_BF16>, grid, block, 0, stream, c);
  else if (c.kind == FP8BS_CACHE_FP8)
    hipLaunchKernelGGL(cache_read_kernel<FP8BS_CACHE_FP8>, grid, block, 0, stream, c);
  else
    hipLaunchKernelGGL(cache_read_kernel<FP8BS_CACHE_FP4>, grid, block, 0, stream, c);
  return hipGetLastError();
}

}  // namespace fp8bs
