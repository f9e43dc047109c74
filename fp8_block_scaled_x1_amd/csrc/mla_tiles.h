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

// One of a wave's direct loads of a tile: 4 rows of 256 bytes, or 8 of 128,
// from tile row r. Rows past `last` repeat it (they are masked, or their
// results dropped).
__device__ __forceinline__ void load_rows256(const uint16_t* base, int64_t stride, int row0, int last, int r, int lane,
                                             uint32_t lds) {
  const int i = r + (lane >> 4);
  dma16(base + (int64_t)min(row0 + i, last) * stride + (((lane & 15) ^ swz256(i)) << 3), lds + r * 256);
}
__device__ __forceinline__ void load_rows128(const uint16_t* base, int64_t stride, int row0, int last, int r, int lane,
                                             uint32_t lds) {
  const int i = r + (lane >> 3);
  dma16(base + (int64_t)min(row0 + i, last) * stride + (((lane & 7) ^ swz128(i)) << 3), lds + r * 128);
}

// ROWS rows of a tile, spread over NW waves.
template <int ROWS, int NW>
__device__ __forceinline__ void load_tile256(const uint16_t* base, int64_t stride, int row0, int last, int w, int lane,
                                             uint32_t lds) {
  static_assert(ROWS % (4 * NW) == 0, "whole loads per wave");
#pragma unroll
  for (int k = 0; k < ROWS / (4 * NW); ++k) load_rows256(base, stride, row0, last, 4 * (k * NW + w), lane, lds);
}
template <int ROWS, int NW>
__device__ __forceinline__ void load_tile128(const uint16_t* base, int64_t stride, int row0, int last, int w, int lane,
                                             uint32_t lds) {
  static_assert(ROWS % (8 * NW) == 0, "whole loads per wave");
#pragma unroll
  for (int k = 0; k < ROWS / (8 * NW); ++k) load_rows128(base, stride, row0, last, 8 * (k * NW + w), lane, lds);
}

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

// Operand of a 32x32x16 product from 32 rows of a tile starting at row0: the
// lane's row lane%32, columns 16*ks + 8*(lane/32) .. +7.
__device__ __forceinline__ bf16x8 rows256(const char* t, const TileLane& L, int row0, int ks) {
  return lds_bf16x8(t + (row0 + L.row) * 256 + (((2 * ks + L.half) ^ L.x256) << 4));
}
__device__ __forceinline__ bf16x8 rows128(const char* t, const TileLane& L, int row0, int ks) {
  return lds_bf16x8(t + (row0 + L.row) * 128 + (((2 * ks + L.half) ^ L.x128) << 4));
}
// Transposed operand: column 32*block + lane%32 of 16 rows starting at row0
// (a multiple of 16), the lane's slots j < 4 rows 4*(lane/32) + j, j >= 4 rows
// 8 + 4*(lane/32) + j - 4: the rows that the lane holds of a 32x32 product.
__device__ __forceinline__ bf16x8 cols256(const char* t, const TileLane& L, int row0, int block) {
  const char* a = t + (row0 + L.trow) * 256 + L.tbyte;
  return join(lds_tr16(a + (((4 * block + L.tchunk) ^ L.tx256) << 4)),
              lds_tr16(a + 8 * 256 + (((4 * block + L.tchunk) ^ L.tx256 ^ 2) << 4)));
}
__device__ __forceinline__ bf16x8 cols128(const char* t, const TileLane& L, int row0, int block) {
  const char* a = t + (row0 + L.trow) * 128 + L.tbyte;
  return join(lds_tr16(a + (((4 * block + L.tchunk) ^ L.tx128) << 4)),
              lds_tr16(a + 8 * 128 + (((4 * block + L.tchunk) ^ L.tx128 ^ 2) << 4)));
}

// The same reads by offset, for loops that fetch ahead: at is the offset that
// at256 and so on give for the lane, plus the tile's own (a multiple of 256);
// the swizzle leaves the column to an XOR of it, the row to a constant.
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
