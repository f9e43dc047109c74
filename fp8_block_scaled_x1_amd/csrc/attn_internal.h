// Launchers behind the attention and draft-verification entry points
// (arguments are validated by the ABI layer before any of these is called).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {

// Expanded latent attention: token strides in elements, offsets on the device.
struct MlaPrefill {
  const uint16_t* q;
  const uint16_t* kv;
  const uint16_t* k_rope;
  int64_t q_stride, kv_stride, rope_stride;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, H, Tq, Tk;
  float scale;
  int causal;
  uint16_t* out;       // [Tq][H][128]
  float* lse;          // [H][Tq]
  // forward with the keys of a block of queries in parts
  int parts;           // at most
  float* part;         // [parts][Tq][H][128]
  float* part_ml;      // [parts][Tq][H][2]: maximum, sum
  // backward only
  const uint16_t* dout;   // [Tq][H][128]
  float* delta;           // [H][Tq]
  float* lse2;            // [H][Tq]
  float* rope_part;       // [H][Tk][64]
  uint16_t* dq;           // [Tq][H][192]
  uint16_t* dkv;          // [Tk][H][256]
  uint16_t* dk_rope;      // [Tk][64]
};

// Blocks of `rows` tokens of a packed batch, at most: every request ends inside one.
inline int64_t mla_blocks(int64_t tokens, int B, int rows) { return (tokens + rows - 1) / rows + B; }
// Parts that launch_mla_prefill cuts the keys into at these sizes; 1: no workspace.
int mla_prefill_parts(int B, int64_t Tq, int64_t Tk, int H);
hipError_t launch_mla_prefill(const MlaPrefill& p, hipStream_t stream);
hipError_t launch_mla_prefill_bwd(const MlaPrefill& p, hipStream_t stream);

// Absorbed latent attention over a paged cache.
struct MlaDecode {
  const uint16_t* q;      // [B][rows][576]
  const char* cache;      // BF16 [pages][page][576], or the FP8 codes [pages][page][512]
  const char* scales;     // FP8: [pages][page][4] float32
  const char* rope;       // FP8: [pages][page][64] BF16
  const int32_t* table;   // [B][table_stride]
  const int32_t* lens;    // [B]
  int64_t table_stride;
  int len_stride;         // 0: one length (and, table_stride 0, one table) for all
  int B, rows, tokens, heads;   // rows of a request: tokens * heads
  int64_t all_rows;       // rows of all requests (the last may have fewer)
  int pages, page, max_len;
  uint32_t page_magic;    // tok / page = (tok * page_magic) >> page_shift
  int page_shift;
  float scale_log2;
  int row_blocks, groups;
  int join;               // every piece is a partial, joined with the prefix's
  uint16_t* out;          // [B][rows][512]
  float* lse;             // [B][rows]
  float* part;            // [2 groups + B][rows][512]
  float* part_ml;         // [2 groups + B][rows][2]
};

constexpr int kMlaDecodeTile = 64;      // tokens
// Rows per workgroup: 64 halve the tiles' traffic against 32 (128 rows of 128
// requests: 156 us, with 32 each 200 us); where there are no more than 32, the
// waves of the others only load (32 rows of 8 requests, FP8: 77 us, with
// workgroups of four waves 78 us).
constexpr int kMlaDecodeBlockRows = 64;
int mla_decode_groups(int64_t row_blocks, int64_t max_tiles);
hipError_t launch_mla_decode(const MlaDecode& own, const MlaDecode* prefix, bool fp8, hipStream_t stream);

struct VerifyDrafts {
  const void* p;          // [B][K+1][V]
  const void* q;          // [B][K][V], or null: drafts chosen without chance
  const int32_t* drafts;  // [B][K]
  const int32_t* n_drafts;
  const float* u;         // [B][K]
  const float* u_next;    // [B]
  int B, K, V;
  uint64_t* sums;         // [B][chunks][2]
  int4* rows;             // [B]: accepted, whether one was turned down, its token
  int32_t* tokens;        // [B][K+1]
  int32_t* accepted;      // [B]
};

constexpr int kVerifyThreads = 256;      // of a workgroup: one per request and chunk
int64_t verify_chunks(int64_t V);
hipError_t launch_verify_drafts(const VerifyDrafts& v, bool bf16, hipStream_t stream);

}  // namespace fp8bs
