// latent_attn.cu -- attention of new tokens over a latent cache (the absorbed form).
//
// All heads of a sequence read the same rows, [latent | rotated key], as keys, and their
// latent part as values: with R = heads * new tokens rows of queries a cache row of 1152
// bytes (dc = 512) is worth 2176 R flops, so 16 heads are bound by memory and 128 heads
// nearly as much by the tensor cores.  Both products run on tcgen05:
//   S [R, 64 tokens]   = Q K^T            queries as the M of 64 (rows past R: unused)
//   O^T [dc, R]       += V^T P^T          channels as the M of 128, dc / 128 products
// O lies transposed in tensor memory: as many columns as there are rows of queries for
// every 128 channels, so few heads waste nothing, 64 fit beside two tiles of scores, and
// a tile of the cache in shared memory serves as the first product's K-major operand and
// the second's MN-major one without being moved.
//
// A CTA (one a multiprocessor: a tile of 64 tokens is 72 KB, a tile of 64 queries as
// much) is a warp that copies, a warp that issues the products, and four that do the
// softmax -- a thread a row of scores, so its maximum and sum need no exchange -- and own
// the output.  The weights go to the tile's own rotated-key columns, which nothing reads
// after the first product.  The running maximum moves only when a score passes it by 2^8:
// O is scaled seldom, and weights up to 2^8 lose nothing in 16 bits.
//
// Work: the tiles of all sequences in order are cut into equal shares, one a CTA, so
// ragged batches balance; a sequence that shares cut leaves parts (maximum, sum, O in
// fp32) that a second kernel joins.  Row tiles run side by side on the same tokens, which
// the second of them finds in the L2.

#include "dkv_device.cuh"
#include "dkv_kernels.h"
#include "latent.h"
#include "tcgen05.cuh"

namespace dkv {
namespace {

constexpr int kWarpsSoftmax = 8, kFirstSoftmax = 4;  // warps 4 .. 11
constexpr int kThreads = 32 * (kFirstSoftmax + kWarpsSoftmax);
constexpr int kSoftmaxThreads = 32 * kWarpsSoftmax;
constexpr int kCopyWarps = 3;  // warps 0, 2 and 3 (1: products)
constexpr int kTile = kLatentTile;
constexpr int kStages = 2;
constexpr int kChunkBytes = kTile * 128;  // 64 tokens x 64 channels
constexpr uint64_t kDrainNs = 200000000ull;
constexpr float kRise = 8.f;  // how far (log2) a score may pass the reference
// Shortest share of a CTA, in tiles.
constexpr int kMinShare = 2;

template <int MB, int RT>
struct Shape {
  static constexpr int kChunks = 2 * MB + 1;          // of 64 channels, the rotated key last
  static constexpr int kQBytes = kChunks * RT * 128;
  static constexpr int kStageBytes = kChunks * kChunkBytes;
  static constexpr int kColumns = 128 + MB * RT <= 256 ? 256 : 512;
  static constexpr size_t kSmem = 1024 + kQBytes + kStages * kStageBytes;
};

struct Shared {
  uint64_t full[kStages], empty[kStages], s_full[2], p_ready[2], o_done[2], voted[2], o_free, q_full,
      q_free, drain;
  uint32_t tmem;
  volatile int abort;
  volatile int failed[2];  // a softmax warp's wait expired, by turns
  int seq0, off0;          // where the CTA's share begins
  float top[2][2][64];     // a tile's maxima, of its two halves, by turns
  volatile int rose[2];    // the last tile that a score rose far in, by turns
  float factor[64];
  float stat_l[2][64];
  int64_t row_at[64];  // of the output, -1: not written
};

// Sequence b as a row tile sees it: its length, its new tokens, its tiles.
struct Seq {
  int len, n, tiles;
};
__device__ __forceinline__ Seq sequence(const LatentAttnArgs& a, int b, int first_t) {
  const int len = a.lens != nullptr ? min(a.lens[b], a.cache.N) : a.cache.N;
  const int n = a.news != nullptr ? min(max(a.news[b], 0), a.T) : a.T;
  const int tiles = len > 0 && first_t < n ? (len - 1) / kTile + 1 : 0;
  return {len, n, tiles};
}

// The CTA's share: tiles [begin, end) of the row tile's `total`, in sequence `b` from tile
// `off` on.
struct Share {
  int64_t begin, end, total;
  int splits, split;
  int b, off;
};
__device__ __forceinline__ Share share_of(const LatentAttnArgs& a, int split, int first_t,
                                          Shared& sh) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  Share w{};
  int64_t mine = 0;
  for (int b = tid; b < a.B; b += kThreads) mine += sequence(a, b, first_t).tiles;
  // (2^14 sequences of 2^25 tiles: counted in 64 bits)
  __shared__ unsigned long long all;
  __syncthreads();
  if (tid == 0) all = 0;
  __syncthreads();
  if (mine != 0) atomicAdd(&all, static_cast<unsigned long long>(mine));
  __syncthreads();
  w.total = static_cast<int64_t>(all);
  const int64_t most = (w.total + kMinShare - 1) / kMinShare;
  w.splits = static_cast<int>(most < a.splits ? most : a.splits);
  w.split = split;
  if (split >= w.splits) return w;  // (no work: begin == end)
  w.begin = split * w.total / w.splits;
  w.end = (split + 1) * w.total / w.splits;
  // the sequence that holds tile `begin`
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    const int t = b < a.B ? sequence(a, b, first_t).tiles : 0;
    long long x = t;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long up = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += up;
    }
    __shared__ long long warp_sum[kThreads / 32];
    __syncthreads();
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    long long chunk = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) x += warp_sum[i];
      chunk += warp_sum[i];
    }
    x += before;  // tiles up to and with sequence b
    if (t > 0 && w.begin < x && w.begin >= x - t) {
      sh.seq0 = b;
      sh.off0 = static_cast<int>(w.begin - (x - t));
    }
    before += chunk;
    if (before > w.begin) break;
  }
  __syncthreads();
  w.b = sh.seq0;
  w.off = sh.off0;
  return w;
}

// Walks a share segment by segment: a sequence's consecutive tiles.
struct Walk {
  const LatentAttnArgs& a;
  int first_t;
  int64_t at, end;
  int b, off;
  // the current segment
  Seq seq;
  int tile0, tiles, index;
  __device__ __forceinline__ Walk(const LatentAttnArgs& a_, const Share& w, int first_t_)
      : a(a_), first_t(first_t_), at(w.begin), end(w.end), b(w.b - 1), off(w.off), tiles(0),
        index(-1) {}
  __device__ __forceinline__ bool next() {
    at += tiles;
    if (at >= end) return false;
    do {
      if (++b >= a.B) return false;
      seq = sequence(a, b, first_t);
    } while (seq.tiles == 0);
    tile0 = off;
    off = 0;
    const int64_t left = end - at;
    tiles = static_cast<int>(min(left, static_cast<int64_t>(seq.tiles - tile0)));
    ++index;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return tiles == seq.tiles; }
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit,
                                          volatile int* abort) {
  int ok = 0;
  if (threadIdx.x % 32 == 0) ok = mbar_wait_bounded(bar, parity, limit, abort);
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

__device__ __forceinline__ void store_out(void* out, int dtype, int64_t at, float y) {
  if (dtype == 2)
    static_cast<float*>(out)[at] = y;
  else if (dtype == 1)
    static_cast<__half*>(out)[at] = __float2half_rn(y);
  else
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(y);
}

// Row r of a row tile: its new token and head.
struct Row {
  int t, h;
};
template <int RT>
__device__ __forceinline__ Row row_of(const LatentAttnArgs& a, int rt, int r) {
  const int g = rt * (RT / 8) + r / 8;
  return {g / a.groups, (g % a.groups) * 8 + r % 8};
}

// Copies tiles of the cache, `part` of the copying warps; the first one queries too.
template <int MB, int RT>
__device__ __forceinline__ void copy_loop(const LatentAttnArgs& a, const CUtensorMap* mql,
                                          const CUtensorMap* mqr, const CUtensorMap* mc,
                                          const Share& w, int rt, int first_t, int part,
                                          Shared& sh, uint32_t q_smem, uint32_t k_smem) {
  using S = Shape<MB, RT>;
  constexpr int kPer = (S::kChunks + kCopyWarps - 1) / kCopyWarps;  // chunks of a warp
  const LatentView& c = a.cache;
  const bool pieces = c.block > 0 && c.block < kTile;  // a copy a chunk of a block
  const int c0 = part * kPer, c1 = min(c0 + kPer, S::kChunks);
  int i = 0, segs = 0;
  bool ok = true;
  for (Walk k(a, w, first_t); ok && k.next();) {
    const int b = uniform(k.b), len = uniform(k.seq.len), tile0 = uniform(k.tile0);
    const int tiles = uniform(k.tiles);
    for (int t = 0; t < tiles; ++t, ++i) {
      const int s = i % kStages;
      const int j0 = (tile0 + t) * kTile;
      if (i >= kStages &&
          !warp_wait(smem_u32(&sh.empty[s]), ((i / kStages) & 1) ^ 1, a.wait_limit_ns, &sh.abort)) {
        ok = false;
        break;
      }
      const uint32_t bar = smem_u32(&sh.full[s]), dst = k_smem + s * S::kStageBytes;
      if (!pieces) {
        int blk = b, row = j0;
        if (c.block > 0) {
          blk = c.bt[b * c.bts + (tile0 + t)];
          if (blk < 0 || blk >= c.nblocks) {
            set_status(a.status, kStatusCheck);
            blk = min(max(blk, 0), c.nblocks - 1);
          }
          blk = uniform(blk);
          row = 0;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, S::kStageBytes);
          tma_load_4d(dst, mc, bar, 0, row, 0, blk);
        }
      } else {
        // pages that hold tokens of the sequence
        const int pages = min(kTile / c.block, (len - j0 + c.block - 1) / c.block);
        const int32_t* bt = c.bt + b * c.bts + j0 / c.block;
        if (elect_one()) mbar_arrive_expect_tx(bar, pages * c.block * (c1 - c0) * 128);
        __syncwarp();
        for (int p = 0; p < pages; ++p) {
          int blk = bt[p];
          if (blk < 0 || blk >= c.nblocks) {
            set_status(a.status, kStatusCheck);
            blk = min(max(blk, 0), c.nblocks - 1);
          }
          blk = uniform(blk);
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < kPer; ++x)
              if (c0 + x < c1)
                tma_load_4d(dst + (c0 + x) * kChunkBytes + p * c.block * 128, mc, bar, 0, 0, c0 + x,
                            blk);
          }
          __syncwarp();
        }
      }
      __syncwarp();
      if (t == 0 && part == 0) {  // the segment's queries
        if (segs > 0 &&
            !warp_wait(smem_u32(&sh.q_free), (segs - 1) & 1, a.wait_limit_ns, &sh.abort)) {
          ++i;
          ok = false;
          break;
        }
        const uint32_t qbar = smem_u32(&sh.q_full);
        if (elect_one()) mbar_arrive_expect_tx(qbar, S::kQBytes);
        __syncwarp();
        for (int r = 0; r < RT; r += a.q_box) {
          const Row at = row_of<RT>(a, rt, r);
          if (elect_one()) {
            // (rows past the last head or token are filled with zeros)
#pragma unroll
            for (int x = 0; x < 2 * MB; ++x)
              tma_load_4d(q_smem + x * (RT * 128) + r * 128, mql, qbar, x * 64, at.h, at.t, b);
            tma_load_4d(q_smem + 2 * MB * (RT * 128) + r * 128, mqr, qbar, 0, at.h, at.t, b);
          }
          __syncwarp();
        }
        ++segs;
      }
    }
  }
  if (!ok) {
    sh.abort = 1;
    set_status(a.status, kStatusTimeout);
  }
  // nothing is in flight when the CTA ends (a barrier that a part of the warps has filled
  // only does not complete: the copies are waited for by the time they can take)
  if (threadIdx.x % 32 == 0) {
    for (int x = max(0, i - kStages); x < i; ++x)
      mbar_wait_bounded(smem_u32(&sh.full[x % kStages]), (x / kStages) & 1, kDrainNs, nullptr);
    if (segs > 0) mbar_wait_bounded(smem_u32(&sh.q_full), (segs - 1) & 1, kDrainNs, nullptr);
  }
  __syncwarp();
}

template <int MB, int RT>
struct Issuer {
  using S = Shape<MB, RT>;
  const LatentAttnArgs& a;
  Shared& sh;
  uint32_t q_smem, k_smem, tmem;
  // O^T (+)= V^T P^T of tile i.
  __device__ __forceinline__ void values(int i, bool first) {
    tc_fence_after();
    if (elect_one()) {
      const uint32_t k = k_smem + (i % kStages) * S::kStageBytes;
      const uint32_t p = k + 2 * MB * kChunkBytes;
      const uint32_t desc = mma_desc(a.f16, 128, RT, true, false);
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int t = 0; t < kTile / 16; ++t)
          tc_mma(tmem + 128 + m * RT, smem_desc(k + 2 * m * kChunkBytes + t * 2048, kChunkBytes, 1024),
                 smem_desc(p + t * 32, 16, 1024), desc, t > 0 || !first);
      tc_commit(smem_u32(&sh.o_done[i & 1]));
      tc_commit(smem_u32(&sh.empty[i % kStages]));
    }
    __syncwarp();
  }
  // S = Q K^T of tile i.
  __device__ __forceinline__ void scores(int i, bool last) {
    tc_fence_after();
    if (elect_one()) {
      const uint32_t k = k_smem + (i % kStages) * S::kStageBytes;
      const uint32_t desc = mma_desc(a.f16, 64, kTile, false, false);
#pragma unroll
      for (int c = 0; c < S::kChunks; ++c)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          tc_mma(tmem + (i & 1) * 64, smem_desc(q_smem + c * (RT * 128) + x * 32, 16, 1024),
                 smem_desc(k + c * kChunkBytes + x * 32, 16, 1024), desc, c + x > 0);
      tc_commit(smem_u32(&sh.s_full[i & 1]));
      if (last) tc_commit(smem_u32(&sh.q_free));
    }
    __syncwarp();
  }
};

// Issues a tile's scores when it has arrived, its values when its weights are there,
// whichever comes first: waiting for the next tile while weights are ready would keep the
// tile that they belong to from being replaced.
template <int MB, int RT>
__device__ __forceinline__ void product_loop(const LatentAttnArgs& a, const Share& w, int first_t,
                                             Shared& sh, uint32_t q_smem, uint32_t k_smem) {
  using S = Shape<MB, RT>;
  const int lane = threadIdx.x % 32;
  Issuer<MB, RT> run{a, sh, q_smem, k_smem, static_cast<uint32_t>(uniform(sh.tmem))};
  const int n = uniform(static_cast<int>(w.end - w.begin));
  int ns = 0, nv = 0;  // tiles whose scores, whose values have been issued
  // the segment of the next scores, and what values have to know of theirs
  Walk k(a, w, first_t);
  int at = 0, tiles = 0, tile0 = 0, len = 0, seg = -1, value_seg = -1;
  uint32_t begins = 0;  // bit i % 4: tile i begins a segment
  uint64_t since = 0;
  uint32_t idle = 0;
  bool ok = true;
  while (nv < n) {
    bool moved = false;
    if (nv < ns && warp_test(smem_u32(&sh.p_ready[nv & 1]), (nv >> 1) & 1)) {
      const bool first = begins >> (nv & 3) & 1;
      if (!first || value_seg < 0 || warp_test(smem_u32(&sh.o_free), value_seg & 1)) {
        run.values(nv, first);
        value_seg += first;
        ++nv;
        moved = true;
      }
    }
    if (ns < n && ns - nv < 2) {
      if (at == tiles) {  // a new segment
        k.next();
        at = 0;
        tiles = uniform(k.tiles);
        tile0 = uniform(k.tile0);
        len = uniform(k.seq.len);
        ++seg;
      }
      const int s = ns % kStages;
      if (warp_test(smem_u32(&sh.full[s]), (ns / kStages) & 1) &&
          (at > 0 || warp_test(smem_u32(&sh.q_full), seg & 1))) {
        // rows past the sequence may hold anything: as values they must be 0 (a weight of
        // 0 times NaN is NaN); their scores are masked
        const int valid = len - (tile0 + at) * kTile;
        if (valid < kTile) {
          const uint32_t to = k_smem + s * S::kStageBytes;
          const int words = (kTile - valid) * 8;
          for (int x = lane; x < 2 * MB * words; x += 32)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             to + x / words * kChunkBytes + valid * 128 + x % words * 16),
                         "r"(0)
                         : "memory");
          fence_async_smem();
          __syncwarp();
        }
        begins = (begins & ~(1u << (ns & 3))) | static_cast<uint32_t>(at == 0) << (ns & 3);
        ++at;
        run.scores(ns, at == tiles);
        ++ns;
        moved = true;
      }
    }
    if (moved) {
      since = 0;
      idle = 0;
      continue;
    }
    // nothing to do: give up after the limit (the clock is slow to read: now and then)
    if (++idle % 512 != 0 && a.wait_limit_ns != 0) continue;
    const uint64_t now = globaltimer_ns();
    if (since == 0) since = now;
    const bool over = now - since > a.wait_limit_ns || a.wait_limit_ns == 0 || sh.abort != 0;
    if (__any_sync(0xffffffffu, over)) {
      ok = false;
      break;
    }
  }
  if (!ok) {
    sh.abort = 1;
    set_status(a.status, kStatusTimeout);
  }
  // nothing is in flight when the tensor memory is freed
  if (elect_one()) tc_commit(smem_u32(&sh.drain));
  __syncwarp();
  if (lane == 0) mbar_wait_bounded(smem_u32(&sh.drain), 0, kDrainNs, nullptr);
  __syncwarp();
}

template <int MB, int RT>
__device__ __forceinline__ void softmax_loop(const LatentAttnArgs& a, const Share& w, int rt,
                                             int first_t, Shared& sh, uint32_t k_smem) {
  using S = Shape<MB, RT>;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 - kFirstSoftmax;
  const int quarter = warp % 4, half = warp / 4;  // rows, and tokens of a tile
  // A product with M = 64 leaves rows 16 q .. 16 q + 15 in lanes 32 q .. 32 q + 15.  A
  // thread takes 8 tokens of each of two rows, its neighbours the rest of the half tile.
  const int r0 = 16 * quarter + lane / 4;  // and r0 + 8
  const bool quarter_on = 16 * quarter < RT;
  const uint32_t tq = sh.tmem + (static_cast<uint32_t>(32 * quarter) << 16);
  const Row row[2] = {row_of<RT>(a, rt, min(r0, RT - 1)), row_of<RT>(a, rt, min(r0 + 8, RT - 1))};
  const int token = 32 * half + 2 * (lane % 4);  // the thread's first one of a tile
  int i = 0;
  bool bad = false;
  for (Walk k(a, w, first_t); k.next();) {
    bool on[2];
    int seen[2];
    float m[2] = {-INFINITY, -INFINITY}, ref[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      on[e] = quarter_on && row[e].t < k.seq.n && row[e].h < a.H;
      seen[e] = on[e] ? k.seq.len - k.seq.n + row[e].t + 1 : 0;
    }
    for (int t = 0; t < k.tiles; ++t, ++i) {
      bad |= !mbar_wait_bounded(smem_u32(&sh.s_full[i & 1]), (i >> 1) & 1, a.wait_limit_ns,
                                &sh.abort);
      __syncwarp();
      tc_fence_after();
      const int j0 = (k.tile0 + t) * kTile;
      const uint32_t p = k_smem + (i % kStages) * S::kStageBytes + 2 * MB * kChunkBytes;
      float s[16], top[2] = {-INFINITY, -INFINITY}, sum[2];
      // weights under the current references, into the tile's rotated-key columns
      auto weights = [&]() {
        sum[0] = sum[1] = 0.f;
#pragma unroll
        for (int x = 0; x < 16; x += 2) {
          const int e = x >> 1 & 1, c = token + (x >> 2) * 8;  // row, token
          const float p0 = ex2(s[x] - ref[e]), p1 = ex2(s[x + 1] - ref[e]);
          sum[e] += p0 + p1;
          const uint32_t v = a.f16 ? pack2<true>(p0, p1) : pack2<false>(p0, p1);
          const int r = r0 + 8 * e;
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(p + r * 128 + (((c >> 3) ^ (r & 7)) << 4) +
                                                      (c & 7) * 2),
                       "r"(v)
                       : "memory");
        }
      };
      if (quarter_on) {
        tmem_ld_16x32(tq + (i & 1) * 64 + 32 * half, s);
        tmem_wait_ld();
        if (__all_sync(0xffffffffu, min(seen[0], seen[1]) - j0 >= kTile)) {
#pragma unroll
          for (int x = 0; x < 16; ++x) s[x] *= a.scale_log2;
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int c = token + (x >> 2) * 8 + (x & 1);
            s[x] = c < seen[x >> 1 & 1] - j0 ? s[x] * a.scale_log2 : -INFINITY;
          }
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) top[x >> 1 & 1] = fmaxf(top[x >> 1 & 1], s[x]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
          top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
          if (lane % 4 == 0) sh.top[i & 1][half][r0 + 8 * e] = top[e];
        }
      }
      // the first tile sets the references; later ones keep them unless a score rises far
      // past its row's.  (The tile's number, not a flag: nothing has to be cleared.)
      const bool rise = t == 0 || top[0] > m[0] + kRise || top[1] > m[1] + kRise;
      if (__any_sync(0xffffffffu, rise) && lane == 0) sh.rose[i & 1] = i + 1;
      if (bad) sh.failed[i & 1] = 1;
      mbar_arrive(smem_u32(&sh.voted[i & 1]));
      if (quarter_on && t > 0) weights();
      // (the barrier's other threads are at the same work: this wait is short)
      bad |= !mbar_wait_bounded(smem_u32(&sh.voted[i & 1]), (i >> 1) & 1,
                                a.wait_limit_ns + kDrainNs, nullptr);
      __syncwarp();
      if (sh.failed[i & 1]) {  // (every thread of these warps leaves here)
        sh.abort = 1;
        set_status(a.status, kStatusTimeout);
        return;
      }
      if (sh.rose[i & 1] == i + 1) {
        if (quarter_on) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = r0 + 8 * e;
            const float high = fmaxf(sh.top[i & 1][0][r], sh.top[i & 1][1][r]);
            float f = 1.f;
            if (t == 0) {
              m[e] = high;
            } else if (high > m[e] + kRise) {
              f = ex2(m[e] - high);
              l[e] *= f;
              m[e] = high;
            }
            ref[e] = m[e] == -INFINITY ? 0.f : m[e];
            if (half == 0 && lane % 4 == 0) sh.factor[r] = f;
          }
          weights();
        }
        if (t > 0) {
          named_barrier(1, kSoftmaxThreads);  // the factors are there
          bad |= !mbar_wait_bounded(smem_u32(&sh.o_done[(i - 1) & 1]), ((i - 1) >> 1) & 1,
                                    a.wait_limit_ns, &sh.abort);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int c = half * (MB * RT / 2); c < (half + 1) * (MB * RT / 2); c += 16) {
            float o[16];
            tmem_ld16(tq + 128 + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] *= sh.factor[c % RT + x];
            tmem_st16(tq + 128 + c, o);
          }
          tmem_wait_st();
        }
      }
      if (quarter_on) l[0] += sum[0], l[1] += sum[1];
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(smem_u32(&sh.p_ready[i & 1]));
    }
    // the segment's output
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (quarter_on && lane % 4 == 0) {
        const int r = r0 + 8 * e;
        sh.stat_l[half][r] = l[e];
        if (half == 0)
          sh.row_at[r] = on[e] ? k.b * a.o_sb + row[e].t * a.o_st + row[e].h * a.o_sh : -1;
      }
    }
    // (two barriers by turns: the products of the last two tiles may both be under way,
    // and a parity tells neighbouring phases apart only)
    bad |= !mbar_wait_bounded(smem_u32(&sh.o_done[(i - 1) & 1]), ((i - 1) >> 1) & 1,
                              a.wait_limit_ns, &sh.abort);
    named_barrier(1, kSoftmaxThreads);
    tc_fence_after();
    const int channel = 32 * quarter + lane;
    const int64_t slot = 2 * static_cast<int64_t>(w.split * a.row_tiles + rt) + (k.index > 0);
    const bool whole = k.whole();
    if (!whole && quarter_on && half == 0 && lane % 4 == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* ml = a.part_ml + (slot * RT + r0 + 8 * e) * 2;
        ml[0] = m[e];
        ml[1] = l[e] + sh.stat_l[1][r0 + 8 * e];
      }
    }
#pragma unroll 1
    for (int c = half * (MB * RT / 2); c < (half + 1) * (MB * RT / 2); c += 16) {
      float o[16];
      tmem_ld16(tq + 128 + c, o);
      tmem_wait_ld();
      const int ch = c / RT * 128 + channel;
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int row = c % RT + x;
        if (whole) {
          const float sum = sh.stat_l[0][row] + sh.stat_l[1][row];
          if (sh.row_at[row] >= 0)
            store_out(a.out, a.out_dtype, sh.row_at[row] + ch, sum > 0.f ? o[x] / sum : 0.f);
        } else {
          a.part_o[(slot * RT + row) * (128 * MB) + ch] = o[x];
        }
      }
    }
    tc_fence_before();
    mbar_arrive(smem_u32(&sh.o_free));
    if (threadIdx.x == 32 * kFirstSoftmax && k.tile0 + k.tiles == k.seq.tiles) {
      // the sequence ends here: which shares hold its parts
      const int64_t p0 = k.at - k.tile0;  // its first tile
      const int first = static_cast<int>(((p0 + 1) * w.splits + w.total - 1) / w.total) - 1;
      const int late = first * w.total / w.splits != p0;  // that share began before it
      a.pieces[static_cast<int64_t>(k.b) * a.row_tiles + rt] =
          make_int2(2 * first + late, w.split - first + 1);
    }
  }
  if (bad) {
    sh.abort = 1;
    set_status(a.status, kStatusTimeout);
  }
}

template <int MB, int RT>
__global__ void __launch_bounds__(kThreads, 1)
    latent_attn_kernel(const __grid_constant__ LatentAttnArgs a,
                       const __grid_constant__ CUtensorMap mql,
                       const __grid_constant__ CUtensorMap mqr,
                       const __grid_constant__ CUtensorMap mc) {
  using S = Shape<MB, RT>;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t q_smem = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t k_smem = q_smem + S::kQBytes;
  const int warp = threadIdx.x / 32;
  griddep_launch_dependents();
  if (warp == 1) tmem_alloc(smem_u32(&sh.tmem), S::kColumns);
  if (threadIdx.x == 0) {
    prefetch_tensormap(&mql), prefetch_tensormap(&mqr), prefetch_tensormap(&mc);
    const int copy_warps = a.cache.block > 0 && a.cache.block < kTile ? kCopyWarps : 1;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sh.full[i]), copy_warps);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_ready[i]), kSoftmaxThreads);
      mbar_init(smem_u32(&sh.o_done[i]), 1);
      mbar_init(smem_u32(&sh.voted[i]), kSoftmaxThreads);
    }
    mbar_init(smem_u32(&sh.o_free), kSoftmaxThreads);
    mbar_init(smem_u32(&sh.q_full), 1);
    mbar_init(smem_u32(&sh.q_free), 1);
    mbar_init(smem_u32(&sh.drain), 1);
    sh.abort = 0;
    sh.failed[0] = sh.failed[1] = 0;
    sh.rose[0] = sh.rose[1] = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  const int rt = blockIdx.x % a.row_tiles, split = blockIdx.x / a.row_tiles;
  const int first_t = row_of<RT>(a, rt, 0).t;
  const Share w = share_of(a, split, first_t, sh);
  if (w.begin < w.end) {
    if (warp == 1)
      product_loop<MB, RT>(a, w, first_t, sh, q_smem, k_smem);
    else if (warp == 0 || (warp < 4 && a.cache.block > 0 && a.cache.block < kTile))
      copy_loop<MB, RT>(a, &mql, &mqr, &mc, w, rt, first_t, warp == 0 ? 0 : warp - 1, sh, q_smem,
                        k_smem);
    else if (warp >= kFirstSoftmax)
      softmax_loop<MB, RT>(a, w, rt, first_t, sh, k_smem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(sh.tmem, S::kColumns);
}

// Joins the parts of sequences that several shares cut, a CTA a row; writes the zeros of
// sequences without tokens.
template <int MB, int RT>
__global__ void __launch_bounds__(32 * MB) latent_join_kernel(const LatentAttnArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.x / a.row_tiles, rt = blockIdx.x % a.row_tiles, r = blockIdx.y;
  const Row at = row_of<RT>(a, rt, r);
  const Seq seq = sequence(a, b, row_of<RT>(a, rt, 0).t);
  if (at.t >= seq.n || at.h >= a.H) return;
  const int64_t out = b * a.o_sb + at.t * a.o_st + at.h * a.o_sh + 4 * threadIdx.x;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (seq.tiles > 0) {
    const int2 p = a.pieces[static_cast<int64_t>(b) * a.row_tiles + rt];
    const int first = p.x / 2, late = p.x & 1;
    if (p.y <= 1 || p.x < 0 || first + p.y > a.splits) return;  // whole: written already
    auto slot = [&](int i) {
      return (2 * static_cast<int64_t>((first + i) * a.row_tiles + rt) + (i == 0 ? late : 0)) * RT + r;
    };
    float top = -INFINITY, sum = 0.f;
    for (int i = threadIdx.x % 32; i < p.y; i += 32) top = fmaxf(top, a.part_ml[2 * slot(i)]);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (top == -INFINITY) top = 0.f;  // (no token seen: every sum is 0)
#pragma unroll 4
    for (int i = 0; i < p.y; ++i) {
      const int64_t s = slot(i);
      const float f = ex2(a.part_ml[2 * s] - top);
      const float4 x = *reinterpret_cast<const float4*>(a.part_o + s * (128 * MB) + 4 * threadIdx.x);
      sum += f * a.part_ml[2 * s + 1];
      o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
  }
  if (a.out_dtype == 2) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + out) = o;
  } else {
    const uint32_t lo = a.out_dtype == 1 ? pack2<true>(o.x, o.y) : pack2<false>(o.x, o.y);
    const uint32_t hi = a.out_dtype == 1 ? pack2<true>(o.z, o.w) : pack2<false>(o.z, o.w);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out) = make_uint2(lo, hi);
  }
}

template <int MB, int RT>
cudaError_t launch_t(const LatentAttnArgs& a, const CUtensorMap& mql, const CUtensorMap& mqr,
                     const CUtensorMap& mc, cudaStream_t s) {
  // (an attribute of the device that is current: set on every call, it takes no time)
  cudaError_t e = cudaFuncSetAttribute(latent_attn_kernel<MB, RT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(Shape<MB, RT>::kSmem));
  if (e != cudaSuccess) return e;
  e = launch_pdl(latent_attn_kernel<MB, RT>, dim3(a.ctas), dim3(kThreads), Shape<MB, RT>::kSmem, s,
                 a, mql, mqr, mc);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_join_kernel<MB, RT>, dim3(a.B * a.row_tiles, RT), dim3(32 * MB), 0, s, a);
}

}  // namespace

cudaError_t launch_latent_attn(int dc, int tile_rows, const LatentAttnArgs& a,
                               const CUtensorMap& mql, const CUtensorMap& mqr,
                               const CUtensorMap& mc, cudaStream_t s) {
  if (dc == 512) {
    if (tile_rows == 64) return launch_t<4, 64>(a, mql, mqr, mc, s);
    if (tile_rows == 32) return launch_t<4, 32>(a, mql, mqr, mc, s);
    return launch_t<4, 16>(a, mql, mqr, mc, s);
  }
  if (tile_rows == 64) return launch_t<2, 64>(a, mql, mqr, mc, s);
  if (tile_rows == 32) return launch_t<2, 32>(a, mql, mqr, mc, s);
  return launch_t<2, 16>(a, mql, mqr, mc, s);
}

}  // namespace dkv
