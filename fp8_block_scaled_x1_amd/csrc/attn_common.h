// Device helpers shared by the attention kernels: operand types, the direct
// global-to-LDS loads, transposing LDS reads and small wave reductions.
//
// MFMA register layout used throughout (32x32x16, lane l of 64): A row l%32 /
// B column l%32, k = 8*(l/32) .. +7; D column l%32, rows 8*(i/4) + 4*(l/32) +
// i%4, i < 16.
// The inner index of a product may be numbered freely as long as A and B
// agree. Every kernel here uses that: with scores formed as keys x queries, a
// lane's D rows (4 consecutive keys at a time) are taken directly as its
// inner-index slots of the product with the values, and the values' operand
// is fetched for the same keys by the transposing LDS read, so probabilities
// never move between lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

typedef __attribute__((address_space(3))) void* lds_void;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kAttnXcds = 8;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void)p);
}

// Direct global -> LDS loads: lane i's 16 (or 4) bytes at `src` go to LDS
// bytes lds + 16*i (4*i), lds wave-uniform. Asm rather than the builtin, whose
// stages the compiler cannot tell apart (it would wait for all of them at
// every LDS read); the caller waits (attn_wait, then a barrier) before the
// bytes are read. No VGPR outputs. No memory clobber either, so that LDS reads
// of other buffers may move past these; the waits and barriers have one.
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "m0");
}
__device__ __forceinline__ void dma16_s(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(lds)
               : "m0");
}
__device__ __forceinline__ void dma4(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(lds) : "m0");
}
__device__ __forceinline__ void dma4_s(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "s"(lds) : "m0");
}

// At most N of the wave's vector-memory operations stay pending (they complete
// in issue order).
template <int N>
__device__ __forceinline__ void attn_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Every vector-memory operation done, said to the compiler too: placed after
// the loads of operands that a loop keeps, it leaves no wait for them (and with
// them for the tiles in flight) inside the loop.
__device__ __forceinline__ void operands_loaded() { __builtin_amdgcn_s_waitcnt(0x0F70); }   // vmcnt(0) alone
// All LDS accesses of the wave done, then meet the other waves. Vector-memory
// loads in flight stay in flight.
__device__ __forceinline__ void attn_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Keeps the compiler from computing what follows from v ahead of the loop (one
// XOR next to its use is cheaper than a register held for the whole loop).
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ bf16x8 lds_bf16x8(const char* p) { return *reinterpret_cast<const bf16x8*>(p); }

// Transposing LDS read of 16-bit elements: each group of 16 lanes reads a
// 4-row x 16-column block, lane j giving the address of 4 consecutive columns
// (row j/4, columns 4*(j%4)..), and receives column j's 4 rows.
__device__ __forceinline__ bf16x4 lds_tr16(const char* p) {
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                        (__attribute__((address_space(3))) s16x4*)(lds_void)p));
}
// The same for bytes: an 8-row x 16-column block, lane j giving row j/2,
// columns 8*(j%2).., receiving column j's 8 rows.
__device__ __forceinline__ i32x2 lds_tr8(const char* p) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(lds_void)p);
}
__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Eight E4M3 codes -> BF16, exact (every E4M3 value is a BF16 value).
__device__ __forceinline__ bf16x8 e4m3_to_bf16(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return join(__builtin_shufflevector(a, b, 0, 1, 2, 3), __builtin_shufflevector(c, d, 0, 1, 2, 3));
}

// The larger of two, NaN if one is (a single instruction for two or three
// operands; fmaxf drops a NaN, and first quiets operands that it cannot rule
// one out for: the long prefill 3.71 ms, so 3.65 ms).
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// The value of the lane 32 away, combined with this lane's (both get the result).
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max_nan(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// What a row's output is multiplied by and its lse, from its reference m (in
// units of log2) and sum l of weights. No key seen: 0 and -inf; a NaN stays one.
__device__ __forceinline__ float inverse_of(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? neg_inf() : (m + __builtin_log2f(l)) * kLn2; }

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

}  // namespace fp8bs
