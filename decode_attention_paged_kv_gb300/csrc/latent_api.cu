// latent_api.cu -- the extern "C" calls on latent caches and on the pages of paged caches:
// argument validation, workspace layout and launches.  Every argument error is returned
// before anything is launched.

#include <math.h>
#include <stdint.h>

#include "../../include/dkv.h"
#include "api_util.h"
#include "dkv_kernels.h"
#include "latent.h"
#include "pages.h"

namespace {

using namespace dkv::api;
using dkv::ceil_div;

constexpr int64_t kInt32Max = INT32_MAX;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

dkv_status check_cache(const dkv_latent_cache* c, int64_t batch) {
  if (c == nullptr) return DKV_ERR_NULL;
  if (c->dtype != DKV_BF16 && c->dtype != DKV_FP16) return DKV_ERR_DTYPE;
  if ((c->latent_dim != 256 && c->latent_dim != 512) || c->rope_dim != dkv::kLatentRope)
    return DKV_ERR_UNSUPPORTED;
  if (c->seq_len < 1 || c->block_size < 0) return DKV_ERR_SHAPE;
  const int64_t row = c->latent_dim + c->rope_dim;
  if (c->stride_b < 0 || c->stride_t < row) return DKV_ERR_SHAPE;
  if (c->stride_b % 8 || c->stride_t % 8 || !aligned16(c->data)) return DKV_ERR_ALIGN;
  // (byte strides of a tensor map are below 2^40)
  if (c->stride_b >= (int64_t{1} << 39) || c->stride_t >= (int64_t{1} << 39)) return DKV_ERR_SHAPE;
  if (c->block_size == 0) {
    if (c->data == nullptr) return DKV_ERR_NULL;
    return DKV_OK;
  }
  if (c->block_size != 16 && c->block_size != 32 && c->block_size != 64)
    return DKV_ERR_UNSUPPORTED;
  if (c->num_blocks < 1) return DKV_ERR_SHAPE;
  if (c->data == nullptr || c->block_table == nullptr) return DKV_ERR_NULL;
  if (!aligned4(c->block_table)) return DKV_ERR_ALIGN;
  if (c->block_table_stride < 0 ||
      (batch > 1 && c->block_table_stride < ceil_div(c->seq_len, c->block_size)))
    return DKV_ERR_SHAPE;
  return DKV_OK;
}

dkv::LatentView view(const dkv_latent_cache* c) {
  dkv::LatentView v{};
  v.p = static_cast<uint16_t*>(c->data);
  v.sb = c->stride_b;
  v.st = c->stride_t;
  v.N = c->seq_len;
  if (c->block_size > 0) {
    v.block = c->block_size;
    v.nblocks = c->num_blocks;
    v.bt = c->block_table;
    v.bts = c->block_table_stride;
  }
  return v;
}

// Strides of rows that are read in vectors of 8 elements.
dkv_status check_strides(std::initializer_list<int64_t> strides) {
  for (const int64_t s : strides) {
    if (s < 0) return DKV_ERR_SHAPE;
    if (s % 8) return DKV_ERR_ALIGN;
  }
  return DKV_OK;
}

// Strides of an output, stored in vectors of 16 bytes.
dkv_status check_out_strides(int32_t dtype, std::initializer_list<int64_t> strides) {
  const int64_t per = dtype == DKV_FP32 ? 4 : 8;
  for (const int64_t s : strides) {
    if (s < 0) return DKV_ERR_SHAPE;
    if (s % per) return DKV_ERR_ALIGN;
  }
  return DKV_OK;
}

// Rows of queries are padded to groups of 8 heads of one new token; a tile of 16, 32 or
// 64 rows is the smallest that holds them all, else 64.  The tokens are shared by as many
// CTAs as keep every multiprocessor busy once, for all row tiles together.
dkv::LatentPlan latent_plan(const dkv_latent_attn* p, const dkv_latent_cache* c) {
  dkv::LatentPlan L{};
  L.groups = static_cast<int>(ceil_div(p->num_heads, 8));
  const int64_t rows = 8ll * L.groups * p->new_tokens;
  L.tile_rows = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
  L.row_tiles = static_cast<int>(ceil_div(rows, L.tile_rows));
  const int64_t tiles = p->batch * ceil_div(c->seq_len, dkv::kLatentTile);
  const int64_t fit = dkv::kLatentCtas / L.row_tiles;
  const int64_t splits = tiles < fit ? tiles : fit;
  L.splits = static_cast<int>(splits < 1 ? 1 : splits);
  L.ctas = L.splits * L.row_tiles;
  // (a bound that only rises with the sizes, so that a workspace serves smaller calls too)
  const int64_t most = tiles * L.row_tiles;
  int64_t ctas = most < dkv::kLatentCtas ? most : dkv::kLatentCtas;
  // (more CTAs than that have whole sequences: they need room where those are long)
  if (ceil_div(c->seq_len, dkv::kLatentTile) > dkv::kLatentRun && ctas < L.row_tiles)
    ctas = L.row_tiles;
  const size_t slots = 2 * static_cast<size_t>(ctas) * L.tile_rows;
  L.pieces = DKV_WORKSPACE_HEADER_BYTES;
  L.part_ml = align_up(L.pieces + 8 * static_cast<size_t>(p->batch) * L.row_tiles);
  L.part_o = align_up(L.part_ml + 8 * slots);
  L.total = align_up(L.part_o + 4 * slots * c->latent_dim);
  return L;
}

CUtensorMapDataType map_type(int32_t dtype) {
  return dtype == DKV_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// A 4-D map of 16-bit elements with a 128-byte swizzle; strides in elements.  (The stride
// of a dimension of size 1 still has to be a valid, 16-byte multiple.)
bool encode_4d(CUtensorMap* map, int32_t dtype, const void* data, const int64_t (&size)[4],
               const int64_t (&stride)[3], const int (&box)[4]) {
  if (!get_encode()) return false;
  cuuint64_t dims[4], st[3];
  cuuint32_t b[4];
  const cuuint32_t one[4] = {1, 1, 1, 1};
  for (int i = 0; i < 4; ++i) {
    dims[i] = static_cast<cuuint64_t>(size[i]);
    b[i] = static_cast<cuuint32_t>(box[i]);
    if (i > 0) st[i - 1] = size[i] == 1 && stride[i - 1] == 0 ? 16 : 2 * stride[i - 1];
  }
  return g_encode(map, map_type(dtype), 4, const_cast<void*>(data), dims, st, b, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool out_dtype_ok(int32_t t) { return t == DKV_FP32 || t == DKV_BF16 || t == DKV_FP16; }

dkv_status check_attn(const dkv_latent_attn* p, const dkv_latent_cache* cache) {
  if (p == nullptr) return DKV_ERR_NULL;
  if (p->batch < 1 || p->num_heads < 1 || p->new_tokens < 1) return DKV_ERR_SHAPE;
  if (p->batch > dkv::kMaxLatentBatch ||
      static_cast<int64_t>(p->new_tokens) * p->num_heads >= (1 << 20))
    return DKV_ERR_UNSUPPORTED;
  if (!(fabsf(p->scale) < INFINITY)) return DKV_ERR_SHAPE;
  const dkv_status st = check_cache(cache, p->batch);
  if (st != DKV_OK) return st;
  // tiles are counted in 32 bits
  if (p->batch * ceil_div(cache->seq_len, dkv::kLatentTile) > kInt32Max)
    return DKV_ERR_UNSUPPORTED;
  return DKV_OK;
}

}  // namespace

extern "C" {

dkv_status dkv_latent_append(const dkv_latent_append_args* p, const dkv_latent_cache* cache,
                             void* workspace, void* stream) {
  if (p == nullptr) return DKV_ERR_NULL;
  if (p->batch < 1 || p->batch > 65535 || p->num_q_heads < 0 || p->new_tokens < 0 ||
      p->rope_len < 0 || p->interleaved < 0 || p->interleaved > 1 || !(p->eps >= 0.f) ||
      !(p->eps < INFINITY))
    return DKV_ERR_SHAPE;
  dkv_status st = check_cache(cache, p->batch);
  if (st != DKV_OK) return st;
  const bool queries = p->num_q_heads > 0;
  if (p->c == nullptr || p->k == nullptr) return DKV_ERR_NULL;
  if (queries && (p->q == nullptr || p->q_out == nullptr)) return DKV_ERR_NULL;
  if (p->rope_len > 0 && (p->cos == nullptr || p->sin == nullptr)) return DKV_ERR_NULL;
  if (!aligned16(p->c) || !aligned16(p->k) || !aligned16(p->norm) || !aligned16(workspace) ||
      (queries && (!aligned16(p->q) || !aligned16(p->q_out))) ||
      (p->rope_len > 0 && (!aligned16(p->cos) || !aligned16(p->sin))) || !aligned4(p->seq_lens) ||
      !aligned4(p->new_lens))
    return DKV_ERR_ALIGN;
  if ((st = check_strides({p->c_stride_b, p->c_stride_t, p->k_stride_b, p->k_stride_t})) != DKV_OK)
    return st;
  if (queries && (st = check_strides({p->q_stride_b, p->q_stride_t, p->q_stride_h, p->o_stride_b,
                                      p->o_stride_t, p->o_stride_h})) != DKV_OK)
    return st;
  // Without lengths on the device the fit is known here.
  if (p->seq_lens == nullptr && p->new_lens == nullptr && p->new_tokens > cache->seq_len)
    return DKV_ERR_SHAPE;
  if (p->rope_len > 0 && p->seq_lens == nullptr && p->rope_len < cache->seq_len)
    return DKV_ERR_SHAPE;
  // What is written has no element twice.
  const int64_t row = cache->latent_dim + cache->rope_dim;
  const bool paged = cache->block_size > 0;
  if (!distinct(row, {{paged ? cache->num_blocks : p->batch, cache->stride_b},
                      {paged ? cache->block_size : cache->seq_len, cache->stride_t}}))
    return DKV_ERR_SHAPE;
  if (queries && !distinct(cache->rope_dim, {{p->batch, p->o_stride_b},
                                             {p->new_tokens, p->o_stride_t},
                                             {p->num_q_heads, p->o_stride_h}}))
    return DKV_ERR_SHAPE;
  if (p->new_tokens == 0) return DKV_OK;
  if (static_cast<int64_t>(p->new_tokens) * (2 + p->num_q_heads) > kInt32Max / 2)
    return DKV_ERR_UNSUPPORTED;
  dkv::LatentAppendArgs a{};
  a.B = p->batch;
  a.T = p->new_tokens;
  a.H = p->num_q_heads;
  a.rope_len = p->rope_len;
  a.eps = p->eps;
  a.c = static_cast<const uint16_t*>(p->c);
  a.k = static_cast<const uint16_t*>(p->k);
  a.q = static_cast<const uint16_t*>(p->q);
  a.norm = static_cast<const uint16_t*>(p->norm);
  a.q_out = static_cast<uint16_t*>(p->q_out);
  a.c_sb = p->c_stride_b, a.c_st = p->c_stride_t;
  a.k_sb = p->k_stride_b, a.k_st = p->k_stride_t;
  a.q_sb = p->q_stride_b, a.q_st = p->q_stride_t, a.q_sh = p->q_stride_h;
  a.o_sb = p->o_stride_b, a.o_st = p->o_stride_t, a.o_sh = p->o_stride_h;
  a.cos = p->cos;
  a.sin = p->sin;
  a.lens = p->seq_lens;
  a.news = p->new_lens;
  a.cache = view(cache);
  a.status = static_cast<uint32_t*>(workspace);
  return cuda_status(dkv::launch_latent_append(cache->latent_dim, cache->dtype == DKV_FP16,
                                               p->interleaved != 0, a,
                                               static_cast<cudaStream_t>(stream)));
}

size_t dkv_latent_workspace_bytes(const dkv_latent_attn* p, const dkv_latent_cache* cache) {
  if (p == nullptr || cache == nullptr) return 0;
  if (p->batch < 1 || p->num_heads < 1 || p->new_tokens < 1 || cache->seq_len < 1 ||
      p->batch > dkv::kMaxLatentBatch ||
      static_cast<int64_t>(p->new_tokens) * p->num_heads >= (1 << 20) ||
      (cache->latent_dim != 256 && cache->latent_dim != 512))
    return 0;
  return latent_plan(p, cache).total;
}

dkv_status dkv_latent_decode_attn(const dkv_latent_attn* p, const dkv_latent_cache* cache,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  dkv_status st = check_attn(p, cache);
  if (st != DKV_OK) return st;
  if (p->q_latent == nullptr || p->q_rope == nullptr || p->out == nullptr) return DKV_ERR_NULL;
  if (!out_dtype_ok(p->out_dtype)) return DKV_ERR_DTYPE;
  if (!aligned16(p->q_latent) || !aligned16(p->q_rope) || !aligned16(p->out) ||
      !aligned16(workspace) || !aligned4(p->seq_lens) || !aligned4(p->new_lens))
    return DKV_ERR_ALIGN;
  if ((st = check_strides({p->ql_stride_b, p->ql_stride_t, p->ql_stride_h, p->qr_stride_b,
                           p->qr_stride_t, p->qr_stride_h})) != DKV_OK)
    return st;
  if ((st = check_out_strides(p->out_dtype, {p->o_stride_b, p->o_stride_t, p->o_stride_h})) !=
      DKV_OK)
    return st;
  if (!distinct(cache->latent_dim, {{p->batch, p->o_stride_b},
                                    {p->new_tokens, p->o_stride_t},
                                    {p->num_heads, p->o_stride_h}}))
    return DKV_ERR_SHAPE;
  if (workspace == nullptr || workspace_bytes < dkv_latent_workspace_bytes(p, cache))
    return DKV_ERR_WORKSPACE;
  dkv::LatentAttnArgs a{};
  a.B = p->batch;
  a.T = p->new_tokens;
  a.H = p->num_heads;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.out = p->out;
  a.out_dtype = out_code(p->out_dtype);
  a.o_sb = p->o_stride_b, a.o_st = p->o_stride_t, a.o_sh = p->o_stride_h;
  a.lens = p->seq_lens;
  a.news = p->new_lens;
  a.cache = view(cache);
  a.status = static_cast<uint32_t*>(workspace);
  a.wait_limit_ns = (p->flags & DKV_FLAG_FORCE_TIMEOUT) ? 0 : kWaitLimitNs;
  a.f16 = cache->dtype == DKV_FP16;
  const dkv::LatentPlan L = latent_plan(p, cache);
  char* ws = static_cast<char*>(workspace);
  a.groups = L.groups;
  a.row_tiles = L.row_tiles;
  a.splits = L.splits;
  a.ctas = L.ctas;
  a.weighted = p->new_tokens > 1 && p->new_lens != nullptr && L.splits > 1 && L.row_tiles > 1 &&
               L.row_tiles <= dkv::kMaxWeighted;
  a.pieces = reinterpret_cast<int2*>(ws + L.pieces);
  a.part_ml = reinterpret_cast<float*>(ws + L.part_ml);
  a.part_o = reinterpret_cast<float*>(ws + L.part_o);
  if (static_cast<int64_t>(p->batch) * L.row_tiles > kInt32Max) return DKV_ERR_UNSUPPORTED;
  // a query copy takes a tile's rows where they are heads of one new token
  a.q_box = p->new_tokens == 1 || 8 * L.groups % L.tile_rows == 0 ? L.tile_rows : 8;
  const int dc = cache->latent_dim;
  CUtensorMap mql, mqr, mc;
  const int64_t H = p->num_heads, T = p->new_tokens, B = p->batch;
  const int chunks = dc / 64 + 1;
  const bool paged = cache->block_size > 0;
  const int tokens = paged && cache->block_size < dkv::kLatentTile ? cache->block_size
                                                                   : dkv::kLatentTile;
  if (!encode_4d(&mql, cache->dtype, p->q_latent, {dc, H, T, B},
                 {p->ql_stride_h, p->ql_stride_t, p->ql_stride_b}, {64, a.q_box, 1, 1}) ||
      !encode_4d(&mqr, cache->dtype, p->q_rope, {dkv::kLatentRope, H, T, B},
                 {p->qr_stride_h, p->qr_stride_t, p->qr_stride_b}, {64, a.q_box, 1, 1}) ||
      !encode_4d(&mc, cache->dtype, cache->data,
                 {64, paged ? cache->block_size : cache->seq_len, chunks,
                  paged ? cache->num_blocks : B},
                 {cache->stride_t, 64, cache->stride_b},
                 {64, tokens, 1, 1}))
    return DKV_ERR_CUDA;
  return cuda_status(dkv::launch_latent_attn(dc, L.tile_rows, a, mql, mqr, mc,
                                             static_cast<cudaStream_t>(stream)));
}

dkv_status dkv_latent_prompt_attn(const dkv_prompt* p, void* workspace, void* stream) {
  if (p == nullptr) return DKV_ERR_NULL;
  if (p->batch < 1 || p->num_heads < 1 || p->total_q < 0 || p->total_k < 0 ||
      p->num_heads > 65535)
    return DKV_ERR_SHAPE;
  if (p->batch > dkv::kMaxLatentBatch) return DKV_ERR_UNSUPPORTED;
  if ((p->nope_dim != 64 && p->nope_dim != 128) || p->rope_dim != dkv::kLatentRope)
    return DKV_ERR_UNSUPPORTED;
  if ((p->dtype != DKV_BF16 && p->dtype != DKV_FP16) || !out_dtype_ok(p->out_dtype))
    return DKV_ERR_DTYPE;
  if (!(fabsf(p->scale) < INFINITY) || p->causal < 0 || p->causal > 1) return DKV_ERR_SHAPE;
  if (p->cu_q == nullptr || p->cu_k == nullptr) return DKV_ERR_NULL;
  if (p->total_q == 0) return DKV_OK;
  if (p->q_nope == nullptr || p->q_rope == nullptr || p->out == nullptr ||
      (p->total_k > 0 && (p->k_nope == nullptr || p->k_rope == nullptr || p->v == nullptr)))
    return DKV_ERR_NULL;
  if (!aligned16(p->q_nope) || !aligned16(p->q_rope) || !aligned16(p->k_nope) ||
      !aligned16(p->k_rope) || !aligned16(p->v) || !aligned16(p->out) || !aligned16(workspace) ||
      !aligned4(p->cu_q) || !aligned4(p->cu_k))
    return DKV_ERR_ALIGN;
  dkv_status st = check_strides({p->qn_stride_t, p->qn_stride_h, p->qr_stride_t, p->qr_stride_h,
                                 p->kn_stride_t, p->kn_stride_h, p->v_stride_t, p->v_stride_h,
                                 p->kr_stride_t});
  if (st != DKV_OK) return st;
  for (const int64_t s : {p->qn_stride_t, p->qn_stride_h, p->qr_stride_t, p->qr_stride_h,
                          p->kn_stride_t, p->kn_stride_h, p->v_stride_t, p->v_stride_h,
                          p->kr_stride_t})
    if (s >= (int64_t{1} << 39)) return DKV_ERR_SHAPE;
  if ((st = check_out_strides(p->out_dtype, {p->o_stride_t, p->o_stride_h})) != DKV_OK) return st;
  if (!distinct(p->nope_dim, {{p->total_q, p->o_stride_t}, {p->num_heads, p->o_stride_h}}))
    return DKV_ERR_SHAPE;
  dkv::PromptArgs a{};
  a.B = p->batch;
  a.H = p->num_heads;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.causal = p->causal;
  a.out = p->out;
  a.out_dtype = out_code(p->out_dtype);
  a.o_st = p->o_stride_t, a.o_sh = p->o_stride_h;
  a.cu_q = p->cu_q;
  a.cu_k = p->cu_k;
  a.total_q = p->total_q;
  a.total_k = p->total_k;
  a.status = static_cast<uint32_t*>(workspace);
  a.wait_limit_ns = (p->flags & DKV_FLAG_FORCE_TIMEOUT) ? 0 : kWaitLimitNs;
  // (a scale of 0 becomes the smallest: masked scores stay at minus infinity)
  if (a.scale_log2 == 0.f) a.scale_log2 = 1.17549435e-38f;
  const int64_t blocks = (ceil_div(p->total_q, 256) + p->batch) * p->num_heads;
  if (blocks > kInt32Max) return DKV_ERR_UNSUPPORTED;
  const int64_t H = p->num_heads, dn = p->nope_dim, dr = p->rope_dim;
  // (without keys no copy is made; a map needs an address all the same)
  const bool keys = p->total_k > 0;
  const int64_t Tk = keys ? p->total_k : 1;
  const void* none = p->q_nope;
  CUtensorMap qn, qr, kn, kr, v;
  if (!encode_4d(&qn, p->dtype, p->q_nope, {dn, H, p->total_q, 1},
                 {p->qn_stride_h, p->qn_stride_t, 0}, {64, 1, 128, 1}) ||
      !encode_4d(&qr, p->dtype, p->q_rope, {dr, H, p->total_q, 1},
                 {p->qr_stride_h, p->qr_stride_t, 0}, {64, 1, 128, 1}) ||
      !encode_4d(&kn, p->dtype, keys ? p->k_nope : none, {dn, H, Tk, 1},
                 {p->kn_stride_h, p->kn_stride_t, 0}, {64, 1, 128, 1}) ||
      !encode_4d(&kr, p->dtype, keys ? p->k_rope : none, {dr, Tk, 1, 1}, {p->kr_stride_t, 0, 0},
                 {64, 128, 1, 1}) ||
      !encode_4d(&v, p->dtype, keys ? p->v : none, {dn, H, Tk, 1},
                 {p->v_stride_h, p->v_stride_t, 0}, {64, 1, 128, 1}))
    return DKV_ERR_CUDA;
  return cuda_status(dkv::launch_prompt_attn(p->nope_dim, p->dtype == DKV_FP16, a, qn, qr, kn, kr, v,
                                             static_cast<int>(blocks),
                                             static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------------ pages
namespace {

struct PagesLayout {
  size_t snap, plan, taken;                        // fork
  size_t totals, counts, src, dst, count, rank;    // compact
  size_t total;
};
PagesLayout pages_layout(int64_t rows, int64_t cols, int64_t nb) {
  PagesLayout L{};
  size_t off = DKV_WORKSPACE_HEADER_BYTES;
  auto take = [&](size_t* at, size_t bytes) {
    *at = off;
    off = align_up(off + bytes);
  };
  take(&L.snap, 4 * static_cast<size_t>(rows * cols));
  take(&L.plan, sizeof(dkv::RowPlan) * static_cast<size_t>(rows));
  take(&L.taken, 4 * static_cast<size_t>(nb));
  L.total = off;
  off = DKV_WORKSPACE_HEADER_BYTES;
  take(&L.totals, 8);
  take(&L.counts, 4 * static_cast<size_t>(ceil_div(nb, dkv::kCompactChunk)));
  take(&L.src, 4 * static_cast<size_t>(nb));
  take(&L.dst, 4 * static_cast<size_t>(nb));
  take(&L.count, 4 * static_cast<size_t>(nb));
  take(&L.rank, 4 * static_cast<size_t>(nb));
  if (off > L.total) L.total = off;
  return L;
}

bool table_ok(int64_t rows, int64_t cols, int64_t nb) {
  return rows >= 1 && cols >= 1 && nb >= 1 && rows <= dkv::kMaxTableRows &&
         rows * cols + rows <= kInt32Max;
}

// Whether two pools have bytes in common.  Blocks of two pools may alternate in memory
// (keys and values of one tensor); then they lie at one stride.
bool pools_meet(const dkv_pool& x, const dkv_pool& y, int64_t blocks) {
  const uint64_t a = reinterpret_cast<uintptr_t>(x.data), b = reinterpret_cast<uintptr_t>(y.data);
  if (a + (blocks - 1) * x.stride + x.block_bytes <= b ||
      b + (blocks - 1) * y.stride + y.block_bytes <= a)
    return false;
  if (blocks == 1 || x.stride != y.stride) return true;
  const int64_t ahead = static_cast<int64_t>(a - b) % x.stride;  // of x's blocks to y's
  const int64_t d = ahead < 0 ? ahead + x.stride : ahead;
  return d < y.block_bytes || d + x.block_bytes > x.stride;
}

dkv_status check_pages(const dkv_pages* p, void* workspace, size_t bytes, dkv::PagesArgs* g) {
  if (p == nullptr) return DKV_ERR_NULL;
  if (p->rows < 1 || p->cols < 1 || p->num_blocks < 1 || p->block_size < 1 || p->num_pools < 0 ||
      p->num_pools > DKV_MAX_POOLS)
    return DKV_ERR_SHAPE;
  if (!table_ok(p->rows, p->cols, p->num_blocks)) return DKV_ERR_UNSUPPORTED;
  if (p->block_table == nullptr || p->refs == nullptr) return DKV_ERR_NULL;
  if (!aligned4(p->block_table) || !aligned16(p->refs) || !aligned16(workspace))
    return DKV_ERR_ALIGN;
  if (p->rows > 1 && p->table_stride < p->cols) return DKV_ERR_SHAPE;
  g->rows = p->rows;
  g->cols = p->cols;
  g->block = p->block_size;
  g->nb = p->num_blocks;
  g->npools = p->num_pools;
  g->table = p->block_table;
  g->ts = p->rows > 1 ? p->table_stride : 0;
  g->refs = p->refs;
  for (int i = 0; i < p->num_pools; ++i) {
    const dkv_pool& x = p->pools[i];
    if (x.data == nullptr) return DKV_ERR_NULL;
    if (x.block_bytes < 1 || (p->num_blocks > 1 && x.stride < x.block_bytes)) return DKV_ERR_SHAPE;
    const uint64_t bits = reinterpret_cast<uintptr_t>(x.data) | static_cast<uint64_t>(x.block_bytes) |
                          static_cast<uint64_t>(x.stride);
    if (bits & 3u) return DKV_ERR_ALIGN;
    if (x.block_bytes > kInt32Max) return DKV_ERR_UNSUPPORTED;
    if (p->num_blocks > 1 && x.stride > INT64_MAX / 2 / p->num_blocks) return DKV_ERR_SHAPE;
    for (int j = 0; j < i; ++j)  // bytes that are copied twice would be moved in no order
      if (pools_meet(x, p->pools[j], p->num_blocks)) return DKV_ERR_SHAPE;
    g->pool[i] = {static_cast<char*>(x.data), x.stride, x.block_bytes, (bits & 15u) == 0};
  }
  if (workspace == nullptr ||
      bytes < pages_layout(p->rows, p->cols, p->num_blocks).total)
    return DKV_ERR_WORKSPACE;
  g->status = static_cast<uint32_t*>(workspace);
  return DKV_OK;
}

}  // namespace

size_t dkv_pages_workspace_bytes(int32_t rows, int32_t cols, int32_t num_blocks) {
  return table_ok(rows, cols, num_blocks) ? pages_layout(rows, cols, num_blocks).total : 0;
}

dkv_status dkv_kv_pages_fork(const dkv_pages* p, const int32_t* seq_lens, const int32_t* parents,
                             const int32_t* new_lens, void* workspace, size_t workspace_bytes,
                             void* stream) {
  dkv::ForkArgs a{};
  const dkv_status st = check_pages(p, workspace, workspace_bytes, &a.g);
  if (st != DKV_OK) return st;
  if (seq_lens == nullptr) return DKV_ERR_NULL;
  if (!aligned4(seq_lens) || !aligned4(parents) || !aligned4(new_lens)) return DKV_ERR_ALIGN;
  const PagesLayout L = pages_layout(p->rows, p->cols, p->num_blocks);
  char* ws = static_cast<char*>(workspace);
  a.lens = seq_lens;
  a.parents = parents;
  a.news = new_lens;
  a.snap = reinterpret_cast<int32_t*>(ws + L.snap);
  a.plan = reinterpret_cast<dkv::RowPlan*>(ws + L.plan);
  a.taken = reinterpret_cast<int32_t*>(ws + L.taken);
  // a row's CTAs: two vectors of its last page a thread, where that many help
  int64_t bytes = 0;
  for (int i = 0; i < p->num_pools; ++i) bytes += p->pools[i].block_bytes;
  const int64_t want = ceil_div(bytes, 8192);
  a.slices = static_cast<int>(want < 1 ? 1 : (want > 64 ? 64 : want));
  return cuda_status(dkv::launch_fork(a, static_cast<cudaStream_t>(stream)));
}

dkv_status dkv_kv_pages_compact(const dkv_pages* p, int32_t* table_out, int64_t table_out_stride,
                                int32_t* refs_out, int32_t* block_map, void* workspace,
                                size_t workspace_bytes, void* stream) {
  dkv::CompactArgs a{};
  const dkv_status st = check_pages(p, workspace, workspace_bytes, &a.g);
  if (st != DKV_OK) return st;
  if (table_out == nullptr || refs_out == nullptr || block_map == nullptr) return DKV_ERR_NULL;
  if (!aligned4(table_out) || !aligned4(refs_out) || !aligned4(block_map)) return DKV_ERR_ALIGN;
  if (p->rows > 1 && (table_out_stride < p->cols ||
                      (table_out == p->block_table && table_out_stride != p->table_stride)))
    return DKV_ERR_SHAPE;
  if (block_map == refs_out || block_map == p->refs) return DKV_ERR_SHAPE;
  int64_t items = 0;
  for (int i = 0; i < p->num_pools; ++i)
    items += ceil_div(p->pools[i].block_bytes, dkv::kCompactPiece);
  if (items > kInt32Max) return DKV_ERR_UNSUPPORTED;
  const PagesLayout L = pages_layout(p->rows, p->cols, p->num_blocks);
  char* ws = static_cast<char*>(workspace);
  a.table_out = table_out;
  a.ts_out = p->rows > 1 ? table_out_stride : 0;
  a.refs_out = refs_out;
  a.map = block_map;
  a.totals = reinterpret_cast<int32_t*>(ws + L.totals);
  a.counts = reinterpret_cast<int32_t*>(ws + L.counts);
  a.src = reinterpret_cast<int32_t*>(ws + L.src);
  a.dst = reinterpret_cast<int32_t*>(ws + L.dst);
  a.count = reinterpret_cast<int32_t*>(ws + L.count);
  a.rank = reinterpret_cast<int32_t*>(ws + L.rank);
  a.items = static_cast<int>(items);
  const int sms = current_sm_count();
  if (sms <= 0) return DKV_ERR_CUDA;
  return cuda_status(dkv::launch_compact(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
