// Host side of the attention and serving entry points: checks of arguments, and
// the sizes of one absorbed-attention problem.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "attn_internal.h"
#include "fp8bs_attn.h"

namespace {

constexpr int64_t kI32 = (int64_t)1 << 31;

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
int status_of(hipError_t e) { return e == hipSuccess ? FP8BS_OK : FP8BS_ERR_LAUNCH; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
bool bad_scale(float s) { return !(s > 0.f) || !isfinite(s); }

// A launch has fewer than 2^32 threads.
bool launch_too_large(int64_t workgroups, int threads) { return workgroups > (((int64_t)1 << 32) - 1) / threads; }

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// tok / page = (tok * magic) >> shift for 0 <= tok < 2^31: with 2^L the next
// power of two, the multiplier floor(2^(31+L) / page) + 1 errs by at most 2^L
// in 2^(31+L).
struct PageDiv {
  int shift;
  uint32_t magic;
  explicit PageDiv(int page) {
    int L = 0;
    while (((int64_t)1 << L) < page) ++L;
    shift = 31 + L;
    magic = (uint32_t)(((uint64_t)1 << (31 + L)) / (uint64_t)page + 1);
  }
};

// ---- absorbed form ----

// Sizes of one problem (the requests' own tokens, or the prefix) and its
// share of the workspace.
struct DecodeSizes {
  int B;                        // requests
  int64_t rows, all_rows;       // of a request, of all
  int64_t max_len;
  int groups;
  int64_t row_blocks;
  int64_t pieces;               // partials of a request's rows
  int64_t bytes_out() const { return align256(4 * pieces * rows * 512); }
  int64_t bytes() const { return bytes_out() + align256(4 * pieces * rows * 2); }
};

// The kernel's tokens per tile and rows per workgroup.
struct DecodeShape {
  int tile, block_rows;
};

int decode_sizes(DecodeShape shape, int B, int64_t rows, int64_t all_rows, int64_t width, int page, bool joined,
                 DecodeSizes& s) {
  if (width > kI32 / page - shape.tile) return FP8BS_ERR_TOO_LARGE;
  s.B = B;
  s.rows = rows;
  s.all_rows = all_rows;
  s.max_len = width * page;
  const int64_t tiles = (int64_t)B * ((s.max_len + shape.tile - 1) / shape.tile);
  if (tiles >= kI32) return FP8BS_ERR_TOO_LARGE;
  s.row_blocks = (rows + shape.block_rows - 1) / shape.block_rows;
  s.groups = fp8bs::mla_decode_groups(s.row_blocks, tiles);
  s.pieces = 2 * (int64_t)s.groups + (joined ? B : 0);
  return FP8BS_OK;
}

int decode_plan(DecodeShape shape, int B, int T, int H, int64_t width, int page, int64_t prefix_pages,
                DecodeSizes& own, DecodeSizes& prefix) {
  if (B < 0 || T < 1 || H < 1 || width < 0 || page < 1 || prefix_pages < 0) return FP8BS_ERR_SHAPE;
  const int64_t rows = (int64_t)T * H, all = B * rows;
  if (rows >= 1 << 24 || launch_too_large((all + 3) / 4, 256)) return FP8BS_ERR_TOO_LARGE;      // the join: a wave a row
  int st = decode_sizes(shape, B, rows, all, width, page, prefix_pages > 0, own);
  if (st != FP8BS_OK || prefix_pages == 0) return st;
  // the prefix: every block of everyone's rows is a request over the same tokens
  const int block = (int)std::max<int64_t>(1, std::min<int64_t>(all, shape.block_rows));
  return decode_sizes(shape, (int)((all + block - 1) / block), block, all, prefix_pages, page, true, prefix);
}

void fill(fp8bs::MlaDecode& p, const uint16_t* q, const void* cache, const void* scales, const uint16_t* rope,
          int64_t pages, int page, const int32_t* table, int64_t width, const int32_t* lens, const DecodeSizes& s,
          float scale, uint16_t* out, float* lse, bool join, char*& ws) {
  p.q = q;
  p.cache = static_cast<const char*>(cache);
  p.scales = static_cast<const char*>(scales);
  p.rope = reinterpret_cast<const char*>(rope);
  p.table = table;
  p.lens = lens;
  p.table_stride = width;
  p.len_stride = 1;
  p.B = s.B;
  p.rows = (int)s.rows;
  p.all_rows = s.all_rows;
  p.pages = (int)pages;
  p.page = page;
  p.max_len = (int)s.max_len;
  const PageDiv div(page);
  p.page_shift = div.shift;
  p.page_magic = div.magic;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.row_blocks = (int)s.row_blocks;
  p.groups = s.groups;
  p.join = join;
  p.out = out;
  p.lse = lse;
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + s.bytes_out());
  ws += s.bytes();
}

}  // namespace
