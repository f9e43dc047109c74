// Launchers behind the serving entry points (arguments are validated by the
// ABI layer before any of these is called).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_internal.h"

namespace fp8bs {

// The newest tokens of packed requests and their slots in a paged cache.
struct MlaCache {
  int kind;                 // FP8BS_CACHE_*
  char* cache;              // BF16 [pages][page][576], codes [pages][page][512] (FP8) or [256] (FP4)
  char* scales;             // FP8: [pages][page][4] float32, FP4: [pages][page][16] uint8
  char* rope;               // FP8, FP4: [pages][page][64] BF16
  uint16_t* latent;         // [T][512], read or written
  uint16_t* out_rope;       // [T][64]
  int64_t latent_stride, rope_stride;
  const int32_t* cu;        // [B+1]
  const int32_t* table;     // [B][width]
  const int32_t* lens;      // [B]
  int64_t width;
  int B, T, pages, page;
  int64_t max_len;          // width * page
  uint32_t page_magic;      // as in MlaDecode
  int page_shift;
};
hipError_t launch_mla_cache_write(const MlaCache& c, hipStream_t stream);
hipError_t launch_mla_cache_read(const MlaCache& c, hipStream_t stream);

constexpr int kFp4Tile = 64;            // tokens of a tile
constexpr int kFp4BlockRows = 32;
hipError_t launch_mla_decode_fp4(const MlaDecode& own, const MlaDecode* prefix, hipStream_t stream);

// A mixture-of-experts layer for few tokens.
struct MoeTokens {
  const uint16_t* x;        // [T][K]
  const int32_t* ids;       // [T][topk]
  const float* weights;     // [T][topk]
  const uint8_t* w_up;      // [E][2F][K]
  const float* s_up;        // [E][2F/128][K/128]
  const uint8_t* w_down;    // [E][K][F]
  const float* s_down;      // [E][K/128][F/128]
  uint16_t* h;              // [T*topk][F] BF16, row of the first slot in which a token names an expert
  float* part;              // [shares][T][K] sums of a share of the second kernel's work
  uint16_t* out;            // [T][K]
  int T, topk, E, K, F, shares;
};
constexpr int kMoeMaxTokens = 64, kMoeMaxTopk = 64, kMoeMaxExperts = 1024;
int moe_shares(int64_t K);
hipError_t launch_moe_tokens(const MoeTokens& m, hipStream_t stream);

struct Logprobs {
  const void* logits;       // [T][V], rows stride apart
  int64_t stride;
  const int32_t* targets;   // [T]
  int64_t T;
  int V, top;
  float *logprob, *entropy;
  float* norm;              // [T][2]: maximum, log of the sum of exponentials against it
  int32_t* rank;
  int32_t* top_ids;
  float* top_logprobs;
  float4* part;             // [T][chunks]: maximum, sum, sum of weighted differences, rank
  uint64_t* part_top;       // [T][chunks][top]
  // gradient
  const float *d_logprob, *d_entropy;
  void* d_logits;           // [T][V]
};
constexpr int kLogprobsThreads = 256;
int64_t logprobs_chunks(int64_t V);
hipError_t launch_logprobs(const Logprobs& l, bool bf16, hipStream_t stream);
hipError_t launch_logprobs_bwd(const Logprobs& l, bool bf16, hipStream_t stream);

}  // namespace fp8bs
