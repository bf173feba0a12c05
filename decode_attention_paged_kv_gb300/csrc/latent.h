// latent.h -- arguments of the kernels on latent caches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dkv {

constexpr int kLatentRope = 64;        // channels of the rotated key
constexpr int kMaxLatentBatch = 16384;

// A cache of rows [latent | rotated key], dense or paged.
struct LatentView {
  uint16_t* p;
  int64_t sb, st;     // elements
  const int32_t* bt;  // paged: block table, row stride bts
  int64_t bts;
  int block, nblocks;  // tokens a block (0: dense), blocks of the pool
  int N;
};

struct LatentAppendArgs {
  int B, T, H, rope_len;
  float eps;
  const uint16_t *c, *k, *q, *norm;
  uint16_t* q_out;
  int64_t c_sb, c_st, k_sb, k_st, q_sb, q_st, q_sh, o_sb, o_st, o_sh;
  const float *cos, *sin;
  const int32_t *lens, *news;
  LatentView cache;
  uint32_t* status;  // nullptr: errors are not reported
};

struct LatentAttnArgs {
  int B, T, H;
  float scale_log2;  // softmax scale times log2(e)
  void* out;
  int out_dtype;  // 0: bf16, 1: fp16, 2: fp32
  int64_t o_sb, o_st, o_sh;
  const int32_t *lens, *news;
  LatentView cache;
  uint32_t* status;
  uint64_t wait_limit_ns;
  bool f16;
  int groups;     // groups of 8 heads of a new token: rows are padded to whole groups
  int row_tiles;  // tiles of the rows (new token, head)
  int splits;     // CTAs that share the tokens of a row tile, at most
  int q_box;      // rows of a query copy: a tile's, or 8
  int ctas;
  int weighted;   // row tiles take CTAs by their tiles (at most kMaxWeighted of them)
  int2* pieces;   // [B, row_tiles]: where a sequence's parts lie
  float* part_ml;  // [splits * row_tiles, 2, rows of a tile, 2]
  float* part_o;   // [splits * row_tiles, 2, rows of a tile, dc]; also of sequences summed so far
};

// How the rows and the work are cut; the workspace follows from it.
struct LatentPlan {
  int tile_rows;  // 16, 32 or 64
  int groups, row_tiles, splits, ctas;
  size_t pieces, part_ml, part_o, total;  // workspace offsets
};
constexpr int kLatentTile = 64;  // tokens
constexpr int kLatentRun = 256;  // tiles of a sequence that are summed up at a time
constexpr int kLatentCtas = 152;
constexpr int kMaxWeighted = 8;

struct PromptArgs {
  int B, H;
  float scale_log2;
  int causal;
  void* out;
  int out_dtype;
  int64_t o_st, o_sh;
  const int32_t *cu_q, *cu_k;
  int total_q, total_k;
  uint32_t* status;
  uint64_t wait_limit_ns;
};

cudaError_t launch_latent_append(int dc, bool f16, bool interleaved, const LatentAppendArgs& a,
                                 cudaStream_t s);
// mql / mqr: maps over q_latent and q_rope {channels, H, T, B}, box {64, q_box, 1, 1}; mc: map
// over the cache {64 channels, tokens, chunks, sequences or blocks}, box one chunk
// of 64 tokens or of a block; all with a 128-byte swizzle.
cudaError_t launch_latent_attn(int dc, int tile_rows, const LatentAttnArgs& a,
                               const CUtensorMap& mql, const CUtensorMap& mqr,
                               const CUtensorMap& mc, cudaStream_t s);
// Maps over q_nope, q_rope, k_nope, v {channels, H, rows, 1}, box {64, 1, 128, 1}, and over
// k_rope {channels, rows, 1, 1}, box {64, 128, 1, 1}; 128-byte swizzle.  blocks: CTAs, as many as
// there can be blocks of 256 queries, times the heads.
cudaError_t launch_prompt_attn(int dn, bool f16, const PromptArgs& a, const CUtensorMap& qn,
                               const CUtensorMap& qr, const CUtensorMap& kn, const CUtensorMap& kr,
                               const CUtensorMap& v, int blocks, cudaStream_t s);

}  // namespace dkv
