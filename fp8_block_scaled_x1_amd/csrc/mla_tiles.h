// Tiles of the expanded latent attention kernels in LDS: rows of 128 (256
// bytes) or 64 (128 bytes) BF16 numbers, loaded straight from global memory
// with 16-byte chunks permuted inside each row so that both ways of reading a
// tile (16 rows at one chunk; 4 rows at 4 chunks, transposed) touch every LDS
// bank once.
#pragma once

#include "attn_common.h"

namespace fp8bs {

constexpr int kNope = 128, kRopeDim = 64, kVDim = 128, kQk = kNope + kRopeDim;

__device__ __forceinline__ int swz256(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }
__device__ __forceinline__ int swz128(int r) { return (((r >> 1) & 1) << 2) | ((r >> 2) & 3); }

// Lane constants of the two ways to read a tile.
struct TileLane {
  int row;      // row reads: lane%32
  int half;     // lane/32
  int x256, x128;   // swizzles of that row
  int trow;     // transposed reads: first row of the lane (rows trow and trow + 8)
  int tchunk;   // its chunk inside a block of 32 columns
  int tbyte;    // its byte inside the chunk
  int tx256, tx128;
  __device__ __forceinline__ explicit TileLane(int lane) {
    row = lane & 31;
    half = lane >> 5;
    x256 = swz256(row);
    x128 = swz128(row);
    trow = 4 * half + ((lane & 15) >> 2);
    tchunk = 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
    tbyte = 8 * (lane & 1);
    tx256 = swz256(trow);
    tx128 = swz128(trow);
  }
};

// The two operands of 32x32x16 products that a tile gives. get256 and get128:
// 32 rows from row0, the lane's row lane%32, columns 16*ks + 8*(lane/32) .. +7.
// get256t and get128t, transposed: column 32*block + lane%32 of 16 rows from
// row0 (a multiple of 16), the lane's slots j < 4 rows 4*(lane/32) + j, j >= 4
// rows 8 + 4*(lane/32) + j - 4: the rows that the lane holds of a 32x32
// product. `at` is the offset that at256 and so on give for the lane, plus the
// tile's own (a multiple of 256); the swizzle leaves the column to an XOR of
// it, the row to a constant.
__device__ __forceinline__ int at256(const TileLane& L) { return L.row * 256 + ((L.half ^ L.x256) << 4); }
__device__ __forceinline__ int at128(const TileLane& L) { return L.row * 128 + ((L.half ^ L.x128) << 4); }
__device__ __forceinline__ int at256t(const TileLane& L) { return L.trow * 256 + L.tbyte + ((L.tchunk ^ L.tx256) << 4); }
__device__ __forceinline__ int at128t(const TileLane& L) { return L.trow * 128 + L.tbyte + ((L.tchunk ^ L.tx128) << 4); }
__device__ __forceinline__ bf16x8 get256(const char* lds, int at, int row0, int ks) {
  return lds_bf16x8(lds + (at ^ (ks << 5)) + row0 * 256);
}
__device__ __forceinline__ bf16x8 get128(const char* lds, int at, int row0, int ks) {
  return lds_bf16x8(lds + (at ^ (ks << 5)) + row0 * 128);
}
__device__ __forceinline__ bf16x8 get256t(const char* lds, int at, int row0, int block) {
  return join(lds_tr16(lds + (at ^ (block << 6)) + row0 * 256), lds_tr16(lds + (at ^ (block << 6) ^ 32) + (row0 + 8) * 256));
}
__device__ __forceinline__ bf16x8 get128t(const char* lds, int at, int row0, int block) {
  return join(lds_tr16(lds + (at ^ (block << 6)) + row0 * 128), lds_tr16(lds + (at ^ (block << 6) ^ 32) + (row0 + 8) * 128));
}

// Eight FP32 values of a 32x32 product (registers 8a .. 8a+7) as BF16.
__device__ __forceinline__ bf16x8 pack8(const f32x16& v, int a) {
  bf16x8 r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = (__bf16)v[8 * a + j];
  return r;
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// Row of register i of a 32x32 product for this lane half.
__device__ __forceinline__ int drow(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

}  // namespace fp8bs
