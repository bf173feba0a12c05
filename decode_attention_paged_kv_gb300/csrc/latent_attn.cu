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
// much) is two warps that copy, one that issues the scores, one that issues the values, and
// eight that do the softmax -- 8 tokens of each of two rows a thread, loaded so that all
// lanes have work although 16 rows fill half of them -- and own the output.  The weights go
// to the tile's own rotated-key columns, which nothing reads after the first product.  The
// running maximum moves only when a score passes it by 2^8: O is scaled seldom.  A weight
// is rounded once, by half a step of the type, and relative to 2^-7 of that maximum in fp16,
// so that the tail of a long sequence stays in its range; maxima, sums and O are fp32.
//
// Work: the tiles of all sequences in order are cut into equal shares, one a CTA, so
// ragged batches balance; a sequence that shares cut leaves parts (maximum, sum, O in
// fp32) that a second kernel joins.  Row tiles run side by side on the same tokens, which
// the second of them finds in the L2.
//
// Measured on a GB300 (copy rate 6.78 TB/s), bf16, dc = 512: 16 sequences of 20K tokens with
// 16 heads 71 us dense and on blocks of any size (378 MB: 5.3 TB/s), one of 1M tokens 198 us
// (6.1 TB/s), 32 of 8K with 128 heads 115 us (311 MB; 635 TFLOP/s), 8 of 8K with four new
// tokens and 32 heads 46 us (398 TFLOP/s); one of 1K, 16
// heads, dc = 256: 10 us, most of it the two launches' latencies.  What bounds it: a tile
// passes through copies, scores, softmax and values one after the other, 6000 to 7000
// cycles, and shared memory holds 2 tiles beside 64 queries (2.75 beside 16); the products'
// reads and the copies' writes fill two thirds of the shared memory's 128 bytes a cycle
// meanwhile (2490 cycles a tile of 64 rows, 2240 of 16, against 3300 taken).  What carried
// it: 274 us with one warp that waited for tile after tile, 143 with products issued from
// uniform registers and by readiness, 139 with the softmax's 16-lane loads, 152 -> 142 with
// pieces and tables read ahead, 125 with the products' loops rolled up -- the warps'
// different code shares the instruction caches, and 36 products in a row did not fit --
// 114 with shares found without barriers and outputs stored without a quotient each.

#include "dkv_device.cuh"
#include "dkv_kernels.h"
#include "latent.h"
#include "tcgen05.cuh"

namespace dkv {
namespace {

constexpr int kWarpsSoftmax = 8, kFirstSoftmax = 4;  // warps 4 .. 11
constexpr int kThreads = 32 * (kFirstSoftmax + kWarpsSoftmax);
constexpr int kSoftmaxThreads = 32 * kWarpsSoftmax;
constexpr int kCopyWarps = 2;  // warps 0 and 2 (1 and 3: products)
constexpr int kTile = kLatentTile;
constexpr int kChunkBytes = kTile * 128;  // 64 tokens x 64 channels
constexpr int kPairBytes = 2 * kChunkBytes;
constexpr float kRise = 8.f;  // how far (log2) a score may pass the running maximum
// How far (log2) below that maximum fp16 weights have their reference: the largest are 2^15, and
// those down to 2^-21 of it keep the type's 11 bits (down to 2^-14 otherwise, and none below
// 2^-25: 1M tokens 17.4 below one lost 2.8% of the mass that their sum counts).
constexpr float kHalfRoom = 7.f;
// Tiles up to which each has a CTA; past it a share is two at least.  (us: two sequences of
// 1K tokens, 16 heads: one tile a share 12.8, two 14.1; one of 8K: 19.2 and 16.4, of which
// the join of 128 parts is a third.)
constexpr int kSingleTiles = 32;
constexpr int kContiguous = 1 << 30;  // of a sequence's parts: the CTAs of a row tile follow one another

// Shared memory: queries, then two rings that tiles pass through in pieces -- pairs of
// latent chunks (128 channels, what one product of the values takes) and rotated keys --
// each piece with its barriers, so that a piece is replaced as soon as its last product is
// done.
template <int MB, int RT>
struct Shape {
  static constexpr int kChunks = 2 * MB + 1;  // of 64 channels, the rotated key last
  static constexpr int kQBytes = kChunks * RT * 128;
  static constexpr int kColumns = 128 + MB * RT <= 256 ? 256 : 512;
  static constexpr int kRoom = 232448 - 1024 - 4096 - kQBytes;  // (alignment, static)
  static constexpr int kKeys = kRoom >= 3 * (MB * kPairBytes + kChunkBytes) ? 4
                               : kRoom >= (5 * MB / 2) * kPairBytes + 3 * kChunkBytes ? 3 : 2;
  static constexpr int kPairs0 = (kRoom - kKeys * kChunkBytes) / kPairBytes;
  static constexpr int kPairs = kPairs0 < kKeys * MB ? kPairs0 : kKeys * MB;
  static constexpr int kKeyAt = kPairs * kPairBytes;  // of the rings' memory
  static constexpr size_t kSmem = 1024 + kQBytes + kKeyAt + kKeys * kChunkBytes;
  static_assert(kPairs >= 2 * MB && kPairs <= 16 && kKeys <= 4, "");
};
constexpr int kMaxPairs = 16, kMaxKeys = 4;

struct Shared {
  uint64_t full[kMaxPairs], empty[kMaxPairs], key_full[kMaxKeys], key_empty[kMaxKeys];
  uint64_t s_full[2], p_ready[2], o_done[2], voted[2], o_free, q_full, q_free, drain[2];
  uint32_t tmem;
  uint32_t fills[kMaxPairs], key_fills[kMaxKeys], q_fills;  // copies issued, for the drain
  volatile int abort;
  volatile int failed[2];  // a softmax warp's wait expired, by turns
  float top[2][2][64];     // a tile's maxima, of its two halves, by turns
  volatile int rose[2];    // the last tile that a score rose far in, by turns
  float factor[64], before[64];
  float stat_l[2][64];
  int64_t row_at[64];  // of the output, -1: not written
};

// A place in a ring of N: its index and the parity of its present round.
template <int N>
struct Ring {
  int at = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void step() {
    if (++at == N) at = 0, round ^= 1;
  }
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

// The CTA's share: tiles [begin, end) of its row tile's `total`, in sequence `b` from tile
// `off` on.
struct Share {
  int64_t begin, end, total;
  int rt, first_t;    // the row tile, its first new token
  int splits, split;  // CTAs of the row tile, and which this is
  int first_cta, stride;  // their numbers
  int b, off;
};

// Row r of a row tile: its new token and head.
struct Row {
  int t, h;
};
template <int RT>
__device__ __forceinline__ Row row_of(const LatentAttnArgs& a, int rt, int r) {
  const int g = rt * (RT / 8) + r / 8;
  return {g / a.groups, (g % a.groups) * 8 + r % 8};
}

// Row tiles have as many CTAs each, side by side, so that they are at the same tokens at the
// same time; where sequences have different numbers of new tokens, row tiles of the later
// ones have fewer sequences, and fewer CTAs.  Up to 256 sequences each warp counts for
// itself (all of it took 5000 to 6700 cycles with barriers, 64-bit sums and quotients).
// (Tiles of all sequences together are below 2^31.)
template <int RT>
__device__ __forceinline__ Share share_of(const LatentAttnArgs& a, Shared& sh) {
  __shared__ unsigned int tiles_of[kMaxWeighted];
  const int tid = threadIdx.x, lane = tid % 32;
  const bool alone = a.B <= 256;
  Share w{};
  w.rt = blockIdx.x % a.row_tiles, w.split = blockIdx.x / a.row_tiles;
  w.splits = a.splits, w.first_cta = w.rt, w.stride = a.row_tiles;
  const int counted = a.weighted ? a.row_tiles : 1;
  unsigned int mine_of = 0;  // lane r: tiles of row tile r
  if (!alone) {
    if (tid < counted) tiles_of[tid] = 0;
    __syncthreads();
  }
  for (int r = 0; r < counted; ++r) {
    const int first_t = row_of<RT>(a, a.weighted ? r : w.rt, 0).t;
    unsigned int sum = 0;
    for (int b = alone ? lane : tid; b < a.B; b += alone ? 32 : kThreads)
      sum += sequence(a, b, first_t).tiles;
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == r) mine_of = sum;
    if (!alone && lane == 0) atomicAdd(&tiles_of[r], sum);
  }
  if (!alone) {
    __syncthreads();
    if (lane < counted) mine_of = tiles_of[lane];
  }
  unsigned int total = __shfl_sync(0xffffffffu, mine_of, 0);
  if (a.weighted) {
    unsigned long long all = 0;
    for (int r = 0; r < counted; ++r) all += __shfl_sync(0xffffffffu, mine_of, r);
    int start = 0;
    for (int r = 0; r < counted; ++r) {
      total = __shfl_sync(0xffffffffu, mine_of, r);
      // (one each, and the rest by their tiles)
      const int n = 1 + (all > 0 ? static_cast<int>((a.ctas - a.row_tiles) *
                                                    static_cast<unsigned long long>(total) / all)
                                 : 0);
      w.rt = r, w.split = blockIdx.x - start, w.splits = n;
      if (static_cast<int>(blockIdx.x) < start + n || r == counted - 1) break;
      start += n;
    }
    w.first_cta = start, w.stride = 1;
  }
  w.total = total;
  w.first_t = row_of<RT>(a, w.rt, 0).t;
  const unsigned int most = total <= kSingleTiles ? total : (total + 1) / 2;
  if (most < static_cast<unsigned int>(w.splits)) w.splits = static_cast<int>(most);
  if (w.split >= w.splits) return w;  // (no work: begin == end)
  // split * total / splits, without a product past 32 bits
  const unsigned int each = total / w.splits, rest = total % w.splits;
  w.begin = w.split * each + w.split * rest / w.splits;
  w.end = (w.split + 1) * each + (w.split + 1) * rest / w.splits;
  // the sequence that holds tile `begin`
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    const int t = b < a.B ? sequence(a, b, w.first_t).tiles : 0;
    int x = t;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += up;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, w.begin < before + x);
    if (past != 0) {
      const int from = __ffs(past) - 1;
      w.b = b0 + from;
      w.off = static_cast<int>(w.begin - before) - __shfl_sync(0xffffffffu, x - t, from);
      break;
    }
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  return w;
}

// Walks a share segment by segment: consecutive tiles of a sequence, kLatentRun at most.  The
// products' adders cut off what lies some 2^-26 below the sum so far, which adds up: of equal
// weights and values 0.05% over 128K tokens, 0.6% over 1M, of 1M tokens beside a heavy one
// 1.6%.  So a long sequence is summed up in segments of 16K tokens, which stay below 2^-12,
// joined by additions that round.
struct Walk {
  const LatentAttnArgs& a;
  int first_t;
  int64_t at, end;
  int b, off;
  // the current segment
  Seq seq;
  int tile0, tiles;
  int from, index;  // the sequence's first tile in the share, and its number there
  bool fresh, more;  // the sequence's first segment in the share; others follow
  __device__ __forceinline__ Walk(const LatentAttnArgs& a_, const Share& w, int first_t_)
      : a(a_), first_t(first_t_), at(w.begin), end(w.end), b(w.b - 1), off(w.off), tiles(0),
        index(-1), more(false) {}
  __device__ __forceinline__ bool next() {
    at += tiles;
    if (at >= end) return false;
    fresh = !more;
    if (fresh) {
      do {
        if (++b >= a.B) return false;
        seq = sequence(a, b, first_t);
      } while (seq.tiles == 0);
      tile0 = from = off;
      off = 0;
      ++index;
    } else {
      tile0 += tiles;
    }
    const int64_t left = end - at;
    tiles = static_cast<int>(min(left, static_cast<int64_t>(seq.tiles - tile0)));
    more = tiles > kLatentRun;
    if (more) tiles = kLatentRun;
    return true;
  }
  // The share has the sequence from its first tile to its last, which this segment has.
  __device__ __forceinline__ bool whole() const {
    return from == 0 && tile0 + tiles == seq.tiles;
  }
};

// The same, a tile at a time, for warps that issue products and copies: every value is one
// that the compiler knows to be uniform, and so is the loop over `count` tiles around it
// (in a loop that lanes might leave apart, a product took 57 cycles instead of 34).
struct TileWalk {
  Walk walk;
  int count;                 // tiles of the share
  int b, len, tile, segment;  // of the present one: sequence, its length, tile, segment
  int left;                  // of the segment, with this one
  bool first;                // of the segment
  __device__ __forceinline__ TileWalk(const LatentAttnArgs& a, const Share& w, int first_t)
      : walk(a, w, first_t), count(uniform(static_cast<int>(w.end - w.begin))), segment(-1),
        left(0) {}
  __device__ __forceinline__ void step() {
    first = left <= 1;
    if (first) {
      walk.next();
      b = uniform(walk.b), len = uniform(walk.seq.len), tile = uniform(walk.tile0);
      left = uniform(walk.tiles);
      ++segment;
    } else {
      ++tile;
      --left;
    }
  }
};

__device__ __forceinline__ void store_out(void* out, int dtype, int64_t at, float y) {
  if (dtype == 2)
    static_cast<float*>(out)[at] = y;
  else if (dtype == 1)
    static_cast<__half*>(out)[at] = __float2half_rn(y);
  else
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(y);
}

// What a row's output is multiplied by: 0 where it sees no token, NaN where its sum is.
__device__ __forceinline__ float inverse_sum(float sum) {
  return sum > 0.f ? 1.f / sum : (sum == sum ? 0.f : sum);
}

// Copies tiles of the cache, every second piece; the first of the warps queries too.
template <int MB, int RT>
__device__ __forceinline__ void copy_loop(const LatentAttnArgs& a, const CUtensorMap* mql,
                                          const CUtensorMap* mqr, const CUtensorMap* mc,
                                          const Share& w, int rt, int first_t, int part,
                                          Shared& sh, uint32_t q_smem, uint32_t k_smem) {
  using S = Shape<MB, RT>;
  const LatentView& c = a.cache;
  Ring<S::kPairs> pair;
  Ring<S::kKeys> key;
  const int block = c.block == 0 ? kTile : c.block;  // tokens of a copy
  const int lane = threadIdx.x % 32;
  int turn = 0, ahead = 0;
  uint32_t filled = 0;  // bits: the ring's first round is over (pairs, then keys)
  bool ok = true;
  TileWalk k(a, w, first_t);
  for (int i = 0; ok && i < k.count; ++i) {
    k.step();
    const int b = k.b;
    const int j0 = k.tile * kTile;
    // blocks that hold tokens of the sequence; their table entries are read a tile ahead
    // (a read takes as long as a third of a tile's copies)
    const int blocks = min(kTile / block, (k.len - j0 + block - 1) / block);
    int blk[4] = {b, b, b, b};
    if (c.block > 0) {
      const int32_t* bt = c.bt + b * c.bts + j0 / block;
      int entry = ahead;
      if (k.first) entry = lane < blocks ? bt[lane] : 0;
      if (k.left > 1) {
        const int more = min(kTile / block, (k.len - j0 - kTile + block - 1) / block);
        ahead = lane < more ? bt[kTile / block + lane] : 0;
      }
      if (lane < blocks && (entry < 0 || entry >= c.nblocks)) {
        set_status(a.status, kStatusCheck);
        entry = min(max(entry, 0), c.nblocks - 1);
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) blk[p] = uniform(lane == p ? entry : 0);
    }
    const int row = c.block == 0 ? j0 : 0;
#pragma unroll
    for (int g = 0; g <= MB; ++g) {
      const bool is_key = g == MB;
      const int at = is_key ? key.at : pair.at;
      const uint32_t round = is_key ? key.round : pair.round;
      if (turn == part) {
        const uint32_t empty = smem_u32(is_key ? &sh.key_empty[at] : &sh.empty[at]);
        const uint32_t full = smem_u32(is_key ? &sh.key_full[at] : &sh.full[at]);
        if ((filled >> is_key & 1) && !lanes_wait(true, empty, round ^ 1, a.wait_limit_ns, &sh.abort)) {
          ok = false;
          break;
        }
        const uint32_t dst =
            is_key ? k_smem + S::kKeyAt + at * kChunkBytes : k_smem + at * kPairBytes;
        const int chunks = is_key ? 1 : 2;
        if (elect_one()) {
          if (is_key)
            ++sh.key_fills[at];
          else
            ++sh.fills[at];
          mbar_arrive_expect_tx(full, blocks * block * chunks * 128);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            if (p >= blocks) break;
            tma_load_4d(dst + p * block * 128, mc, full, 0, row, 2 * g, blk[p]);
            if (!is_key)
              tma_load_4d(dst + kChunkBytes + p * block * 128, mc, full, 0, row, 2 * g + 1, blk[p]);
          }
        }
        __syncwarp();
      }
      if (++turn == kCopyWarps) turn = 0;
      if (is_key) {
        key.step();
        if (key.at == 0) filled |= 2;
      } else {
        pair.step();
        if (pair.at == 0) filled |= 1;
      }
    }
    if (ok && k.first && part == 0) {  // the segment's queries
      if (k.segment > 0 &&
          !lanes_wait(true, smem_u32(&sh.q_free), (k.segment - 1) & 1, a.wait_limit_ns, &sh.abort)) {
        ok = false;
        break;
      }
      const uint32_t qbar = smem_u32(&sh.q_full);
      if (elect_one()) {
        mbar_arrive_expect_tx(qbar, S::kQBytes);
        ++sh.q_fills;
      }
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
    }
  }
  if (!ok) {
    sh.abort = 1;
    set_status(a.status, kStatusTimeout);
  }
}

// Rows past the sequence may hold anything: as values they must be 0 (a weight of 0 times
// NaN is NaN); their scores are masked.  Clears rows `valid` and on of a piece (one warp).
__device__ __forceinline__ void clear_rows(uint32_t piece, int valid) {
  const int words = (kTile - valid) * 8;
  for (int x = threadIdx.x % 32; x < 2 * words; x += 32)
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                     piece + x / words * kChunkBytes + valid * 128 + x % words * 16),
                 "r"(0)
                 : "memory");
  fence_async_smem();
  __syncwarp();
}

// Waits (one warp) until no copy into shared memory is in flight.
template <int MB, int RT>
__device__ __forceinline__ void drain_copies(Shared& sh) {
  using S = Shape<MB, RT>;
  const int lane = threadIdx.x % 32;
  if (lane < S::kPairs) {
    if (sh.fills[lane] > 0)
      mbar_wait_bounded(smem_u32(&sh.full[lane]), (sh.fills[lane] - 1) & 1, kDrainNs, nullptr);
  } else if (lane < S::kPairs + S::kKeys) {
    const int x = lane - S::kPairs;
    if (sh.key_fills[x] > 0)
      mbar_wait_bounded(smem_u32(&sh.key_full[x]), (sh.key_fills[x] - 1) & 1, kDrainNs, nullptr);
  } else if (lane == 31 && sh.q_fills > 0) {
    mbar_wait_bounded(smem_u32(&sh.q_full), (sh.q_fills - 1) & 1, kDrainNs, nullptr);
  }
  __syncwarp();
}

// The two products have a warp each, which waits for its operands: one warp for both has
// to choose what is ready, and its tests took longer than a product.

// S = Q K^T of each tile, when it has arrived.
template <int MB, int RT>
__device__ __forceinline__ void score_loop(const LatentAttnArgs& a, const Share& w, int first_t,
                                           Shared& sh, uint32_t q_smem, uint32_t k_smem) {
  using S = Shape<MB, RT>;
  const int lane = threadIdx.x % 32;
  const uint32_t tmem = static_cast<uint32_t>(uniform(sh.tmem));
  const uint32_t desc = mma_desc(a.f16, 64, kTile, false, false);
  Ring<S::kPairs> pair;
  Ring<S::kKeys> key;
  bool ok = true;
  TileWalk k(a, w, first_t);
  for (int i = 0; i < k.count; ++i) {
    k.step();
    // the tile's pieces, a lane each; the queries; that the scores two tiles ago are read
    uint32_t bar = smem_u32(&sh.key_full[key.at]), parity = key.round;
    bool wanted = lane <= MB;
    if (lane < MB) {
      const int x = pair.at + lane, wrap = x >= S::kPairs;
      bar = smem_u32(&sh.full[x - wrap * S::kPairs]);
      parity = pair.round ^ wrap;
    } else if (lane == MB + 1) {
      bar = smem_u32(&sh.q_full), parity = k.segment & 1;
      wanted = k.first;
    } else if (lane == MB + 2) {
      bar = smem_u32(&sh.p_ready[i & 1]), parity = ((i >> 1) & 1) ^ 1;
      wanted = i >= 2;
    }
    ok = lanes_wait(wanted, bar, parity, a.wait_limit_ns, &sh.abort);
    if (!ok) break;
    const int places = uniform(pair.at | key.at << 8 | (i & 1) << 16);
    uint32_t from[MB];
#pragma unroll
    for (int x = 0; x < MB; ++x) {
      const int y = (places & 255) + x;
      from[x] = k_smem + (y >= S::kPairs ? y - S::kPairs : y) * kPairBytes;
    }
    const int valid = k.len - k.tile * kTile;
    if (valid < kTile) {
#pragma unroll
      for (int x = 0; x < MB; ++x) clear_rows(from[x], valid);
    }
    tc_fence_after();
    const uint32_t to = tmem + (places >> 16) * 64;
    const uint32_t last = k_smem + S::kKeyAt + (places >> 8 & 255) * kChunkBytes;
    if (elect_one()) {
#pragma unroll 1
      for (int c = 0; c < S::kChunks; ++c) {
        const int at = (places & 255) + c / 2;
        const uint32_t pair_at = k_smem + (at >= S::kPairs ? at - S::kPairs : at) * kPairBytes;
        const uint32_t k0 = c < 2 * MB ? pair_at + (c & 1) * kChunkBytes : last;
        const uint32_t q0 = q_smem + c * (RT * 128);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          tc_mma(to, smem_desc(q0 + y * 32, 16, 1024), smem_desc(k0 + y * 32, 16, 1024), desc,
                 c + y > 0);
      }
      tc_commit(smem_u32(&sh.s_full[i & 1]));
      if (k.left == 1) tc_commit(smem_u32(&sh.q_free));
    }
    __syncwarp();
#pragma unroll
    for (int x = 0; x < MB; ++x) pair.step();
    key.step();
  }
  if (!ok) {
    sh.abort = 1;
    set_status(a.status, kStatusTimeout);
  }
  drain_products(&sh.drain[0]);
}

// O^T (+)= V^T P^T of each tile, when its weights are there.
template <int MB, int RT>
__device__ __forceinline__ void value_loop(const LatentAttnArgs& a, const Share& w, int first_t,
                                           Shared& sh, uint32_t k_smem) {
  using S = Shape<MB, RT>;
  const int lane = threadIdx.x % 32;
  const uint32_t tmem = static_cast<uint32_t>(uniform(sh.tmem));
  const uint32_t desc = mma_desc(a.f16, 128, RT, true, false);
  Ring<S::kPairs> pair;
  Ring<S::kKeys> key;
  bool ok = true;
  TileWalk k(a, w, first_t);
  for (int i = 0; i < k.count; ++i) {
    k.step();
    // the weights; at a segment's first tile that the last one's output is read
    uint32_t bar = smem_u32(&sh.p_ready[i & 1]), parity = (i >> 1) & 1;
    if (lane == 1) bar = smem_u32(&sh.o_free), parity = (k.segment - 1) & 1;
    ok = lanes_wait(lane == 0 || (lane == 1 && k.first && k.segment > 0), bar, parity,
                    a.wait_limit_ns, &sh.abort);
    if (!ok) break;
    tc_fence_after();
    const int places = uniform(pair.at | key.at << 8 | (k.first ? 0 : 1) << 16);
    Ring<S::kPairs> v;
    v.at = places & 255;
    const uint32_t p = k_smem + S::kKeyAt + (places >> 8 & 255) * kChunkBytes;
    const uint32_t keep = places >> 16;
    if (elect_one()) {
#pragma unroll 1
      for (int m = 0; m < MB; ++m) {
        const uint32_t from = k_smem + v.at * kPairBytes;
#pragma unroll
        for (int x = 0; x < kTile / 16; ++x)
          tc_mma(tmem + 128 + m * RT, smem_desc(from + x * 2048, kChunkBytes, 1024),
                 smem_desc(p + x * 32, 16, 1024), desc, x > 0 ? 1 : keep);
        tc_commit(smem_u32(&sh.empty[v.at]));
        v.step();
      }
      tc_commit(smem_u32(&sh.key_empty[places >> 8 & 255]));
      tc_commit(smem_u32(&sh.o_done[i & 1]));
    }
    __syncwarp();
#pragma unroll
    for (int m = 0; m < MB; ++m) pair.step();
    key.step();
  }
  if (!ok) {
    sh.abort = 1;
    set_status(a.status, kStatusTimeout);
  }
  drain_products(&sh.drain[1]);
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
  const float room = a.f16 ? kHalfRoom : 0.f, far = kRise + room;
  int i = 0;
  Ring<S::kKeys> key;
  bool bad = false;
  float run_m[2], run_l[2];  // of a sequence's segments so far
  for (Walk k(a, w, first_t); k.next();) {
    bool on[2];
    int seen[2];
    // (m: what weights are relative to, 2^m; ref: the same, 0 where no token is seen yet)
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
      const uint32_t p = k_smem + S::kKeyAt + key.at * kChunkBytes;
      key.step();
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
      // (Differences: a sum m + 8 would round to m or m + 16 at 2^27.)
      const bool rise = t == 0 || top[0] - m[0] > far || top[1] - m[1] > far;
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
              m[e] = high - room;
            } else if (high - m[e] > far) {
              f = ex2(m[e] - (high - room));
              l[e] *= f;
              m[e] = high - room;
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
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (k.index > 0);
    const bool whole = k.whole();
    if (!whole || !k.fresh) {
      // the sequence's statistics so far; what its outputs so far and these are multiplied by
      if (quarter_on && half == 0 && lane % 4 == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + 8 * e;
          const float sum = l[e] + sh.stat_l[1][r];
          if (k.fresh) {
            run_m[e] = m[e], run_l[e] = sum;
          } else {
            const float high = fmaxf(run_m[e], m[e]), to = high == -INFINITY ? 0.f : high;
            const float f0 = ex2(run_m[e] - to), f1 = ex2(m[e] - to);
            run_m[e] = high, run_l[e] = run_l[e] * f0 + sum * f1;
            const float inv = whole ? inverse_sum(run_l[e]) : 1.f;
            sh.before[r] = f0 * inv, sh.factor[r] = f1 * inv;
          }
          if (!whole && !k.more) {
            float* ml = a.part_ml + (slot * RT + r) * 2;
            ml[0] = run_m[e];
            ml[1] = run_l[e];
          }
        }
      }
    } else {
      // (a quotient a row, not one an element)
      const int mine = threadIdx.x - 32 * kFirstSoftmax;
      if (mine < RT) sh.factor[mine] = inverse_sum(sh.stat_l[0][mine] + sh.stat_l[1][mine]);
    }
    if (whole || !k.fresh) named_barrier(1, kSoftmaxThreads);
#pragma unroll 1
    for (int c = half * (MB * RT / 2); c < (half + 1) * (MB * RT / 2); c += 16) {
      float o[16];
      tmem_ld16(tq + 128 + c, o);
      const int ch = c / RT * 128 + channel, row0 = c % RT;
      float* part = a.part_o + (slot * RT + row0) * (128 * MB) + ch;
      tmem_wait_ld();
      if (whole || !k.fresh) {
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] *= sh.factor[row0 + x];
      }
      if (!k.fresh) {
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] += part[x * (128 * MB)] * sh.before[row0 + x];
      }
      if (whole) {
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (sh.row_at[row0 + x] >= 0)
            store_out(a.out, a.out_dtype, sh.row_at[row0 + x] + ch, o[x]);
      } else {
#pragma unroll
        for (int x = 0; x < 16; ++x) part[x * (128 * MB)] = o[x];
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
          make_int2(2 * (w.first_cta + first * w.stride) + late,
                    (w.split - first + 1) | (a.weighted ? kContiguous : 0));
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
  // (a barrier a thread or two: one thread alone takes 1000 cycles for all)
  const int tid = threadIdx.x;
  if (tid < S::kPairs) {
    mbar_init(smem_u32(&sh.full[tid]), 1);
    mbar_init(smem_u32(&sh.empty[tid]), 1);
    sh.fills[tid] = 0;
  } else if (tid >= 64 && tid < 64 + S::kKeys) {
    mbar_init(smem_u32(&sh.key_full[tid - 64]), 1);
    mbar_init(smem_u32(&sh.key_empty[tid - 64]), 1);
    sh.key_fills[tid - 64] = 0;
  } else if (tid >= 96 && tid < 98) {
    const int i = tid - 96;
    mbar_init(smem_u32(&sh.s_full[i]), 1);
    mbar_init(smem_u32(&sh.p_ready[i]), kSoftmaxThreads);
    mbar_init(smem_u32(&sh.o_done[i]), 1);
    mbar_init(smem_u32(&sh.voted[i]), kSoftmaxThreads);
    mbar_init(smem_u32(&sh.drain[i]), 1);
    sh.failed[i] = 0;
    sh.rose[i] = 0;
  } else if (tid == 128) {
    prefetch_tensormap(&mql), prefetch_tensormap(&mqr), prefetch_tensormap(&mc);
    mbar_init(smem_u32(&sh.o_free), kSoftmaxThreads);
    mbar_init(smem_u32(&sh.q_full), 1);
    mbar_init(smem_u32(&sh.q_free), 1);
    sh.q_fills = 0;
    sh.abort = 0;
  }
  fence_barrier_init();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  const Share w = share_of<RT>(a, sh);
  const int rt = uniform(w.rt), first_t = uniform(w.first_t);
  if (w.begin < w.end) {
    if (warp == 0 || warp == 2)
      copy_loop<MB, RT>(a, &mql, &mqr, &mc, w, rt, first_t, warp / 2, sh, q_smem, k_smem);
    else if (warp == 1)
      score_loop<MB, RT>(a, w, first_t, sh, q_smem, k_smem);
    else if (warp == 3)
      value_loop<MB, RT>(a, w, first_t, sh, k_smem);
    else
      softmax_loop<MB, RT>(a, w, rt, first_t, sh, k_smem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) drain_copies<MB, RT>(sh);
  if (warp == 1) tmem_dealloc(sh.tmem, S::kColumns);
}

// Joins the parts of sequences that several shares cut, a CTA a row: up to four groups of
// threads share a row's parts, each with four under way at once; writes the zeros of
// sequences without tokens.
constexpr int kJoinGroups = 4;
template <int MB, int RT>
__global__ void __launch_bounds__(32 * MB * kJoinGroups) latent_join_kernel(const LatentAttnArgs a) {
  __shared__ float4 part[kJoinGroups - 1][32 * MB];
  __shared__ float stat[kJoinGroups][2];
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.x / a.row_tiles, rt = blockIdx.x % a.row_tiles, r = blockIdx.y;
  const int tid = threadIdx.x % (32 * MB), group = threadIdx.x / (32 * MB);
  const int groups = blockDim.x / (32 * MB);
  const int2 p = a.pieces[static_cast<int64_t>(b) * a.row_tiles + rt];
  const Row at = row_of<RT>(a, rt, r);
  const Seq seq = sequence(a, b, row_of<RT>(a, rt, 0).t);
  if (at.t >= seq.n || at.h >= a.H) return;
  const int64_t out = b * a.o_sb + at.t * a.o_st + at.h * a.o_sh + 4 * tid;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (seq.tiles > 0) {
    const int first = p.x / 2, late = p.x & 1, parts = p.y & ~kContiguous;
    const int stride = p.y & kContiguous ? 1 : a.row_tiles;
    if (parts <= 1 || p.x < 0 || first + static_cast<int64_t>(parts - 1) * stride >= a.ctas)
      return;  // whole: written already
    float top = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int i0 = group; i0 < parts; i0 += 4 * groups) {
      float4 x[4];
      float m[4], l[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int i = i0 + y * groups;
        m[y] = -INFINITY, l[y] = 0.f, x[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i >= parts) continue;
        const int64_t s = (2 * static_cast<int64_t>(first + i * stride) + (i == 0 ? late : 0)) * RT + r;
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * s);
        m[y] = ml.x, l[y] = ml.y;
        x[y] = *reinterpret_cast<const float4*>(a.part_o + s * (128 * MB) + 4 * tid);
      }
      const float high = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), top);
      if (high == -INFINITY) {  // no token seen so far: sums of 0, or NaN where all scores are
        sum += l[0] + l[1] + l[2] + l[3];
        continue;
      }
      const float f0 = ex2(top - high);
      top = high;
      sum *= f0, o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float f = ex2(m[y] - high);
        sum += f * l[y];
        o.x += f * x[y].x, o.y += f * x[y].y, o.z += f * x[y].z, o.w += f * x[y].w;
      }
    }
    if (tid == 0) stat[group][0] = top, stat[group][1] = sum;
    if (group > 0) part[group - 1][tid] = o;
    __syncthreads();
    if (group > 0) return;
    float high = top;
    for (int g = 1; g < groups; ++g) high = fmaxf(high, stat[g][0]);
    if (high == -INFINITY) high = 0.f;  // (every sum is 0 or NaN, and stays so times 0)
    const float f0 = ex2(top - high);
    sum *= f0, o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
    for (int g = 1; g < groups; ++g) {
      const float f = ex2(stat[g][0] - high);
      const float4 x = part[g - 1][tid];
      sum += f * stat[g][1];
      o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
    }
    const float inv = inverse_sum(sum);
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
  } else if (group > 0) {
    return;
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
  // about as many groups as a sequence has fours of parts (the whole call, us: 32 sequences
  // of three parts, 128 heads: one group 152, four 171; one of 8, 16 heads: 12.4, 10.8)
  const int parts = a.splits / a.B + 1;
  const int groups = parts <= 4 ? 1 : (parts <= 8 ? 2 : kJoinGroups);
  return launch_pdl(latent_join_kernel<MB, RT>, dim3(a.B * a.row_tiles, RT),
                    dim3(32 * MB * groups), 0, s, a);
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
