// prompt_attn.cu -- attention of prompts with keys and values expanded a head (the expanded
// form): softmax(scale (q_nope . k_nope + q_rope . k_rope)) v over ragged sequences, the
// rotated keys shared by the heads.
//
// 2 (2 dn + 64) flops a query and key against some bytes a key: bound by the tensor cores.
// A CTA takes 256 queries of a head, as two tiles of 128 rows that take turns: while one
// tile's scores pass through the softmax the tensor cores work on the other's.  Per key
// tile of 128 and query tile
//   S = Q K^T     M = 128, N = 128, dn + 64 channels: both operands from shared memory
//   O += P V      M = 128, N = dn, 128 tokens: P from tensor memory, where it takes the
//                 place of the scores it was made of (dn = 128) or lies beside them (64: the
//                 next scores are made meanwhile); V as it was copied (MN-major)
// A thread has a row of scores to itself (128 threads a query tile), so the softmax needs
// no exchange; a row's output lies in the lane of its thread, so each warp scales its own
// rows when a score passes the running reference by 2^8, which is seldom.
//
// Keys and values come in pieces of 128 tokens x 64 channels (16 KB) through one ring, the
// keys of the next tile before the values of this one are done with: with 96 KB of
// queries (dn = 128) there is room for 8 pieces, a tile and three fifths.
//
// A CTA stays for further blocks of queries: a warp takes over the launch of a CTA that has
// not begun (cluster launch control) and passes its block on, so that copies run into the
// next block while this one's softmax and output are under way, and blocks go to whichever
// multiprocessor is free.
//
// Maxima, sums and outputs are fp32; a weight is rounded once to the inputs' type for its
// product, and is 2^7 at the running maximum in fp16, so that the tail of many keys stays in
// its range.  Measured on a GB300, bf16: the last 2K tokens of 4 prompts of 8K, 16 heads, dn =
// 128: 425 us, 1.42 PFLOP/s of the 1.9 that a large library product reaches; one prompt of
// 8K 230 us (1.50); 2 of 2K with 128 heads 274 us (1.25); one of 16K, 8 heads, dn = 64 336 us
// (1.23); 16 of 512 tokens, 32 heads, dn = 64 51 us (0.50).  What bounds it: with dn = 128 a
// query tile's chain scores - softmax - values, some 3600 cycles for 2560 of products for two
// tiles; with dn = 64 the softmax's instructions (1540 of products); of short prompts the
// chain's beginning and end.  What carried it, the last 2K of up to 8K tokens of 4 prompts, one
// draw of lengths (others take up to 325 us as it is, 1.12 to 1.41 PFLOP/s): 345 us with one
// warp for both tiles' products, 296 with a warp each in turns, 266 with blocks taken over, 258
// without spilt registers, 244 with weights made two at a time, 234 with products in functions
// of their own (fewer instructions for the caches), 216 with long blocks first; 218 since scores
// far from 0 and sums of many keys are right.  No difference
// made a softmax in halves and a second wait between values and scores; outputs read 32
// columns at a time were 2% slower for short prompts.

#include "dkv_device.cuh"
#include "dkv_kernels.h"
#include "latent.h"
#include "tcgen05.cuh"

namespace dkv {
namespace {

constexpr int kThreads = 384;  // warps: copies, products (two), schedule, 2 x 4 of softmax
constexpr int kRows = 128;     // queries of a tile
constexpr int kKeys = 128;     // keys of a tile
constexpr int kPieceBytes = kKeys * 128;
constexpr int kSlots = 8;  // pieces: of a power of two (10, where there is room: 3% slower)
constexpr float kRise = 8.f;  // how far (log2) a score may pass the running maximum
// What (log2) a weight is at the running maximum: in fp16 the largest are 2^15 then, and those
// down to 2^-21 of the maximum keep the type's 11 bits (down to 2^-14 otherwise, and none below
// 2^-25: 1M keys 17.4 below one lost 2.8% of the mass that their sum counts).
template <bool F16>
constexpr float kAtTop = F16 ? 7.f : 0.f;
// Scaled scores (log2) past which their running maximum is taken away before they are scaled:
// below it a scaled maximum is rounded by 2^-14 at most, which is what weights of the two ways
// differ by; at 2^30 it would be off by 32, and weights with it.
constexpr float kFar = 1024.f;
// Key tiles whose values are summed up at a time, 16K keys: the products' adders cut off what lies
// some 2^-26 below the sum so far, which adds up (of equal weights and values 0.05% over 128K
// keys, 0.6% over 1M; of 1M keys beside a heavy one 1.6%; 16K keys stay below 2^-12).  Tensor
// memory has no room for a second sum, but the row's place in the output has: its mean so far,
// rounded to the output's type, goes there, and what that leaves of the sum stays.  (2K queries
// of 128K keys, 8 heads of 128 channels: 1944 us without, 2022 so, 2101 every 8K keys.)
constexpr int kRun = 128;

// A block of queries of a head.
struct Work {
  int b, h;      // sequence (-1: no more work), head
  int q0, nq;    // its query rows
  int k0, nk;    // its key rows
  int row;       // the first query of the block, within the sequence
  int tiles[2];  // key tiles of the two query tiles
};

struct Shared {
  uint64_t full[kSlots], empty[kSlots];
  uint64_t q_full[2], q_free[2], s_full[2], p_ready[2], o_done[2], o_free[2], turn[2], drain[2];
  uint64_t s_free[2], v_done[2];
  uint64_t work_full[2], work_free[2], taken, wanted;
  alignas(16) uint4 handle;  // of the CTA taken over
  uint32_t tmem;
  // copies issued and CTAs asked for: for the drain; the first slot's also show progress to warps
  // that wait for the end of a block, which 16M keys take 200 ms to reach
  volatile uint32_t fills[kSlots];
  uint32_t q_fills[2], takes;
  volatile int abort;
  Work work[2];  // by turns
};
// Warps that read a block's description: copies, two of products, eight of softmax.
constexpr int kReaders = 11;

struct Bounds {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ Bounds bounds(const PromptArgs& a, int b) {
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k) {
    set_status(a.status, kStatusCheck);
    return {0, 0, 0, 0};
  }
  return {q0, q1 - q0, k0, k1 - k0};
}

// Keys that the query `row` of a sequence sees.
__device__ __forceinline__ int seen_by(const PromptArgs& a, const Work& w, int row) {
  return a.causal ? min(w.nk, max(0, w.nk - w.nq + row + 1)) : w.nk;
}

// Which block a CTA number stands for: sequences in order of their keys (of 32 at a time, the
// most first), within from the last queries to the first (the last see the most keys), heads
// within, so that long blocks begin early and short ones fill the end; as many heads at a time
// as leave their keys in half of the L2 (2 prompts of 2K, 128 heads: 273 us, not 281).  One warp.
struct Finder {
  const PromptArgs& a;
  int b0 = 0;
  long long before = 0;  // blocks of the sequences before b0
  int b;             // the lane's sequence
  Bounds mine;
  long long blocks;  // of it, all heads
  int room, all_heads;  // keys of a head that half of the L2 holds, with their values; of all
  __device__ __forceinline__ Finder(const PromptArgs& a_, int key_bytes)
      : a(a_), room((64 << 20) / key_bytes), all_heads(room / a.H) {
    load();
  }
  __device__ __forceinline__ void load() {
    const int lane = threadIdx.x % 32;
    b = b0 + lane;
    mine = b < a.B ? bounds(a, b) : Bounds{0, 0, 0, 0};
    if (a.B > 1) {
      int before_mine = 0, from = 0;
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        const int nk = __shfl_sync(0xffffffffu, mine.nk, x);
        before_mine += nk > mine.nk || (nk == mine.nk && x < lane);
      }
#pragma unroll
      for (int x = 0; x < 32; ++x)
        if (__shfl_sync(0xffffffffu, before_mine, x) == lane) from = x;
      b = b0 + from;
      mine = {__shfl_sync(0xffffffffu, mine.q0, from), __shfl_sync(0xffffffffu, mine.nq, from),
              __shfl_sync(0xffffffffu, mine.k0, from), __shfl_sync(0xffffffffu, mine.nk, from)};
    }
    blocks = (mine.nq + 2ll * kRows - 1) / (2 * kRows) * a.H;
  }
  __device__ __forceinline__ Work find(long long item) {
    if (item < before) b0 = 0, before = 0, load();
    const int lane = threadIdx.x % 32;
    Work w{};
    w.b = -1;
    while (true) {
      long long x = blocks;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const long long up = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += up;
      }
      const long long end = before + x;
      const uint32_t past = __ballot_sync(0xffffffffu, item < end);
      if (past != 0) {
        const int from = __ffs(past) - 1;
        const int i = static_cast<int>(item - __shfl_sync(0xffffffffu, end - blocks, from));
        w.b = __shfl_sync(0xffffffffu, b, from);
        w.q0 = __shfl_sync(0xffffffffu, mine.q0, from);
        w.nq = __shfl_sync(0xffffffffu, mine.nq, from);
        w.k0 = __shfl_sync(0xffffffffu, mine.k0, from);
        w.nk = __shfl_sync(0xffffffffu, mine.nk, from);
        const int per = (w.nq - 1) / (2 * kRows) + 1;
        int first = 0, heads = a.H, rest = i;
        if (w.nk > all_heads) {  // as many heads at a time as have room
          const int group = max(room / w.nk, 1);
          first = i / (per * group) * group;
          heads = min(group, a.H - first);
          rest = i - first * per;
        }
        w.h = first + rest % heads;
        w.row = (per - 1 - rest / heads) * (2 * kRows);
#pragma unroll
        for (int x2 = 0; x2 < 2; ++x2) {
          const int row = w.row + x2 * kRows;  // of the tile's first query
          const int seen = seen_by(a, w, min(row + kRows, w.nq) - 1);
          w.tiles[x2] = row >= w.nq || seen == 0 ? 0 : (seen - 1) / kKeys + 1;
        }
        return w;
      }
      if (b0 + 32 >= a.B) return w;
      before = __shfl_sync(0xffffffffu, end, 31);
      b0 += 32;
      load();
    }
  }
};

// Takes over the launch of a CTA that has not begun, if there is one: asks ...
__device__ __forceinline__ void take_cta(Shared& sh) {
  ++sh.takes;
  mbar_arrive_expect_tx(smem_u32(&sh.taken), 16);
  fence_async_smem();
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(smem_u32(&sh.handle)),
      "r"(smem_u32(&sh.taken))
      : "memory");
}
// ... and, once the answer is there, which one it was.
__device__ __forceinline__ bool taken_cta(const Shared& sh, uint32_t* cta) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t"
      ".reg .pred p;\n\t"
      ".reg .b128 h;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t"
      "}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(&sh.handle))
      : "memory");
  *cta = x;
  return ok != 0;
}

// Publishes the CTA's blocks, its own first, then those it takes over.
__device__ __forceinline__ void schedule_loop(const PromptArgs& a, int key_bytes, Shared& sh) {
  const int lane = threadIdx.x % 32;
  Finder find(a, key_bytes);
  uint32_t cta = blockIdx.x;
  bool ok = true, more = true;  // more: `cta` is a CTA to stand in for
  for (int j = 0; ok; ++j) {
    Work w{};
    w.b = -1;
    if (more) w = find.find(cta);
    if (j >= 2)
      ok = lanes_wait(true, smem_u32(&sh.work_free[j & 1]), ((j >> 1) - 1) & 1, a.wait_limit_ns,
                      &sh.abort);
    if (ok && lane == 0) {
      sh.work[j & 1] = w;
      mbar_arrive(smem_u32(&sh.work_full[j & 1]));
    }
    __syncwarp();
    if (!more || !ok) break;
    // not before this block's copies are all under way: a block that waits here for its
    // turn is one that another multiprocessor could have begun
    if (w.b >= 0) {
      ok = lanes_wait(true, smem_u32(&sh.wanted), j & 1, a.wait_limit_ns, &sh.abort, &sh.fills[0]);
      if (!ok) break;
    }
    if (lane == 0) take_cta(sh);
    __syncwarp();
    uint32_t turn = j;
    while (true) {
      ok = lanes_wait(true, smem_u32(&sh.taken), turn & 1, a.wait_limit_ns, &sh.abort);
      more = ok && taken_cta(sh, &cta);
      if (w.b >= 0 || !more) break;
      // the grid is for the most blocks that there can be: the rest of it has none, and is
      // taken out of the way sooner than launched
      __syncwarp();
      if (lane == 0) take_cta(sh);
      __syncwarp();
      ++turn;
    }
    if (w.b < 0) break;
  }
  if (!ok) {
    sh.abort = 1;
    set_status(a.status, kStatusTimeout);
  }
}

// The j-th block of the CTA, as the reading warps see it; false: there is none (or no word
// of it: *ok).
__device__ __forceinline__ bool next_work(const PromptArgs& a, Shared& sh, int j, Work* w, bool* ok) {
  *ok = lanes_wait(true, smem_u32(&sh.work_full[j & 1]), (j >> 1) & 1, a.wait_limit_ns, &sh.abort);
  if (!*ok) return false;
  *w = sh.work[j & 1];
  __syncwarp();
  if (w->b >= 0 && threadIdx.x % 32 == 0) mbar_arrive(smem_u32(&sh.work_free[j & 1]));
  return w->b >= 0;
}

template <int DN>
struct Shape {
  static constexpr int kQChunks = DN / 64 + 1, kVChunks = DN / 64;
  static constexpr int kPieces = kQChunks + kVChunks;  // of a key tile
  static constexpr int kQBytes = kQChunks * kPieceBytes;  // of a query tile
  // Tensor memory of a query tile: scores, weights, output.  With 64 channels there is room for
  // weights beside the scores, so the next scores are made while the softmax has these.
  static constexpr bool kApart = DN == 64;
  static constexpr uint32_t kScores = kApart ? 256 : 128;  // from one query tile to the other
  static constexpr uint32_t kWeights = kApart ? 128 : 0;
  static constexpr uint32_t kOutput = kApart ? 192 : 256, kOutputs = kApart ? 256 : 128;
  static constexpr size_t kSmem = 1024 + 2 * kQBytes + kSlots * kPieceBytes;
};

struct Maps {
  CUtensorMap qn, qr, kn, kr, v;
};

template <int DN>
__device__ __forceinline__ void copy_loop(const PromptArgs& a, const Maps& m, Shared& sh,
                                          uint32_t q_smem, uint32_t ring) {
  using S = Shape<DN>;
  bool ok = true;
  int at = 0;
  uint32_t round = 0;
  bool again = false;  // the ring's first round is over
  Work w;
  for (int j = 0; next_work(a, sh, j, &w, &ok); ++j) {
    const int h = uniform(w.h), q = uniform(w.q0 + w.row), k0 = uniform(w.k0);
    const int used = uniform((w.tiles[0] > 0 ? 1 : 0) | (w.tiles[1] > 0 ? 2 : 0));
    const int n = uniform(max(w.tiles[0], w.tiles[1]));
    for (int i = 0; ok && i < max(n, 1); ++i) {
      const int row = k0 + i * kKeys;
#pragma unroll
      for (int c = 0; c < S::kPieces; ++c) {
        if (i == 0 && c == S::kQChunks) {  // the queries, after the first keys
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            ok = j == 0 ||
                 lanes_wait(true, smem_u32(&sh.q_free[x]), (j - 1) & 1, a.wait_limit_ns, &sh.abort);
            if (!ok) break;
            const uint32_t bar = smem_u32(&sh.q_full[x]), to = q_smem + x * S::kQBytes;
            if (elect_one()) {
              ++sh.q_fills[x];
              if (used >> x & 1) {
                mbar_arrive_expect_tx(bar, S::kQBytes);
#pragma unroll
                for (int d = 0; d < S::kQChunks - 1; ++d)
                  tma_load_4d(to + d * kPieceBytes, &m.qn, bar, 64 * d, h, q + x * kRows, 0);
                tma_load_4d(to + (S::kQChunks - 1) * kPieceBytes, &m.qr, bar, 0, h, q + x * kRows, 0);
              } else {
                mbar_arrive(bar);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        if (i >= n) continue;
        if (again &&
            !lanes_wait(true, smem_u32(&sh.empty[at]), round ^ 1, a.wait_limit_ns, &sh.abort)) {
          ok = false;
          break;
        }
        const int slot = uniform(at);
        const uint32_t bar = smem_u32(&sh.full[slot]), to = ring + slot * kPieceBytes;
        if (elect_one()) {
          sh.fills[slot] = sh.fills[slot] + 1;
          mbar_arrive_expect_tx(bar, kPieceBytes);
          if (c < S::kQChunks - 1)
            tma_load_4d(to, &m.kn, bar, 64 * c, h, row, 0);
          else if (c == S::kQChunks - 1)
            tma_load_4d(to, &m.kr, bar, 0, row, 0, 0);
          else
            tma_load_4d(to, &m.v, bar, 64 * (c - S::kQChunks), h, row, 0);
        }
        __syncwarp();
        if (++at == kSlots) at = 0, round ^= 1, again = true;
      }
    }
    if (!ok) break;
    if (elect_one()) mbar_arrive(smem_u32(&sh.wanted));
    __syncwarp();
  }
  if (!ok) {
    sh.abort = 1;
    set_status(a.status, kStatusTimeout);
  }
}

// O (+)= P V of a key tile, by one thread; `base`: its first piece.
template <int DN>
__device__ __forceinline__ void issue_values(Shared& sh, uint32_t ring, uint32_t output_at,
                                             uint32_t weights_at, uint32_t desc, int base, int keep) {
  using S = Shape<DN>;
  // (a product for each piece: two are not neighbours where the ring wraps)
#pragma unroll 1
  for (int c = 0; c < S::kVChunks; ++c) {
    const uint32_t v = ring + (base + c) % kSlots * kPieceBytes;
#pragma unroll
    for (int y = 0; y < kKeys / 16; ++y)
      tc_mma_ts(output_at + c * 64, weights_at + y * 8, smem_desc(v + y * 2048, 16, 1024), desc,
                y > 0 ? 1 : keep);
    tc_commit(smem_u32(&sh.empty[(base + c) % kSlots]));
  }
}
// S = Q K^T of a key tile, likewise.
template <int DN>
__device__ __forceinline__ void issue_scores(Shared& sh, uint32_t ring, uint32_t scores_at,
                                             uint32_t q, uint32_t desc, int base, int x) {
  using S = Shape<DN>;
#pragma unroll 1
  for (int c = 0; c < S::kQChunks; ++c) {
    const uint32_t k = ring + (base + c) % kSlots * kPieceBytes;
#pragma unroll
    for (int y = 0; y < 4; ++y)
      tc_mma(scores_at, smem_desc(q + c * kPieceBytes + y * 32, 16, 1024),
             smem_desc(k + y * 32, 16, 1024), desc, c + y > 0);
  }
  tc_commit(smem_u32(&sh.s_full[x]));
#pragma unroll
  for (int c = 0; c < S::kQChunks; ++c) tc_commit(smem_u32(&sh.empty[(base + c) % kSlots]));
}
// Pieces that this query tile has no use for.
template <int DN>
__device__ __forceinline__ void pass_pieces(Shared& sh, int base, int count) {
  for (int c = 0; c < count; ++c)
    mbar_arrive(smem_u32(&sh.empty[(base + c) % kSlots]));
}
// Rows past the sequence may hold anything; a weight of 0 times NaN is NaN (both query tiles'
// warps clear them: with the same zeros).
template <int DN>
__device__ __forceinline__ void clear_values(uint32_t ring, int base, int valid) {
  using S = Shape<DN>;
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int c = 0; c < S::kVChunks; ++c) {
    const uint32_t v = ring + (base + c) % kSlots * kPieceBytes;
    for (int y = lane; y < (kKeys - valid) * 8; y += 32)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + valid * 128 + y * 16),
                   "r"(0)
                   : "memory");
  }
  fence_async_smem();
  __syncwarp();
}

// Issues query tile x's products, a warp for each query tile: between its products a warp
// spends some 600 cycles on barriers and descriptors, which the other's fill.
// Weights in place of the scores (128 channels): the values, then the next scores, which take
// the place of the weights just used (products of one thread run in order), with one wait for
// all that they need: a second one left the tensor cores idle for 350 cycles.  The query tiles
// take turns: left alone they fall into step, both in the softmax at one time and both at the
// tensor cores at another.
// Weights apart (64 channels): the next scores as soon as the softmax has read these, then
// these values; a query tile's own products run beside its softmax, and no turns are needed.
template <int DN>
__device__ __forceinline__ void product_loop(const PromptArgs& a, bool f16, int x, Shared& sh,
                                             uint32_t q_smem, uint32_t ring) {
  using S = Shape<DN>;
  const int lane = threadIdx.x % 32;
  const uint32_t tmem = static_cast<uint32_t>(uniform(sh.tmem));
  const uint32_t scores_at = tmem + x * S::kScores, weights_at = scores_at + S::kWeights;
  const uint32_t output_at = tmem + S::kOutput + x * S::kOutputs;
  const uint32_t q = q_smem + x * S::kQBytes;
  // (a scale below 0: products of negated queries, so that the softmax takes its size alone)
  const uint32_t score_desc =
      mma_desc(f16, kRows, kKeys, false, false) | (a.scale_log2 < 0.f ? kNegateA : 0u);
  const uint32_t value_desc = mma_desc(f16, kRows, 64, false, true);
  bool ok = true;
  // of the blocks so far: pieces (modulo two rounds of the ring), steps, key tiles of x
  int pieces = 0, steps = 0, done = 0;
  Work w;
  for (int j = 0; next_work(a, sh, j, &w, &ok); ++j) {
    const int n = uniform(max(w.tiles[0], w.tiles[1]));
    const int tiles = uniform(w.tiles[x]), nk = uniform(w.nk);
    // Step i: the values of key tile i - 1 and the scores of key tile i, whose pieces follow
    // one another.  Queries and output are waited for in every block, whatever it uses of them:
    // a warp that went on without would complete a barrier twice before it is looked at.
    for (int i = 0; i <= n; ++i) {
      const bool values = i > 0, scores = i < n;  // what the step has
      const bool use_values = values && i <= tiles, use_scores = i < tiles;  // for x
      const int piece = pieces + i * S::kPieces - S::kVChunks;  // the first: of the values
      const int p = max(piece + lane, 0);
      uint32_t bar = smem_u32(&sh.full[p % kSlots]), parity = (p / kSlots) & 1;
      const bool a_value = lane < S::kVChunks && values;
      const bool a_score = lane >= S::kVChunks && lane < S::kPieces && scores;
      bool value_wait = a_value, score_wait = a_score;
      if (lane == S::kPieces) {
        bar = smem_u32(&sh.p_ready[x]), parity = (done + i - 1) & 1, value_wait = use_values;
      } else if (lane == S::kPieces + 1) {
        bar = smem_u32(&sh.q_full[x]), parity = j & 1, score_wait = i == 0;
      } else if (lane == S::kPieces + 2) {
        if (S::kApart)  // that the softmax has read the scores before
          bar = smem_u32(&sh.s_free[x]), parity = (done + i - 1) & 1,
          score_wait = use_scores && done + i > 0;
        else
          bar = smem_u32(&sh.turn[x]), parity = (steps + i - 1 + x) & 1,
          score_wait = steps + i + x > 0;
      } else if (lane == S::kPieces + 3) {  // that the last block's output has been read
        bar = smem_u32(&sh.o_free[x]), parity = (j - 1) & 1, value_wait = j > 0 && i == min(n, 1);
      }
      const int base = uniform(piece + 8 * kSlots), keep = uniform(i > 1);
      const bool do_values = uniform(use_values), do_scores = uniform(use_scores);
      const int valid = nk - (i - 1) * kKeys;
      if constexpr (S::kApart) {
        ok = lanes_wait(score_wait, bar, parity, a.wait_limit_ns, &sh.abort);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (do_scores)
            issue_scores<DN>(sh, ring, scores_at, q, score_desc, base + S::kVChunks, x);
          else if (scores)
            pass_pieces<DN>(sh, base + S::kVChunks, S::kQChunks);
          // the block's queries are free
          if (i == max(n - 1, 0)) tc_commit(smem_u32(&sh.q_free[x]));
        }
        __syncwarp();
        ok = lanes_wait(value_wait, bar, parity, a.wait_limit_ns, &sh.abort);
        if (!ok) break;
        if (use_values && valid < kKeys) clear_values<DN>(ring, base, valid);
        tc_fence_after();
        if (elect_one()) {
          if (do_values) {
            issue_values<DN>(sh, ring, output_at, weights_at, value_desc, base, keep);
            tc_commit(smem_u32(&sh.v_done[x]));
          } else if (values) {
            pass_pieces<DN>(sh, base, S::kVChunks);
          }
          if (i == n) tc_commit(smem_u32(&sh.o_done[x]));
        }
        __syncwarp();
      } else {
        ok = lanes_wait(value_wait || score_wait, bar, parity, a.wait_limit_ns, &sh.abort);
        if (!ok) break;
        if (use_values && valid < kKeys) clear_values<DN>(ring, base, valid);
        tc_fence_after();
        if (elect_one()) {
          if (do_values)
            issue_values<DN>(sh, ring, output_at, weights_at, value_desc, base, keep);
          else if (values)
            pass_pieces<DN>(sh, base, S::kVChunks);
          // (the other warp takes as long to begin as the scores to issue)
          mbar_arrive(smem_u32(&sh.turn[1 - x]));
          if (do_scores)
            issue_scores<DN>(sh, ring, scores_at, q, score_desc, base + S::kVChunks, x);
          else if (scores)
            pass_pieces<DN>(sh, base + S::kVChunks, S::kQChunks);
          // the block's queries are free; its output is complete
          if (i == max(n - 1, 0)) tc_commit(smem_u32(&sh.q_free[x]));
          if (i == n) tc_commit(smem_u32(&sh.o_done[x]));
        }
        __syncwarp();
      }
    }
    if (!ok) break;
    pieces = (pieces + n * S::kPieces) % (2 * kSlots);
    steps += n + 1;
    done += tiles;
  }
  if (!ok) {
    sh.abort = 1;
    set_status(a.status, kStatusTimeout);
  }
  drain_products(&sh.drain[x]);
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(lo), "f"(hi));
  return x;
}
__device__ __forceinline__ float2 halves_of(uint64_t x) {
  float2 y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(x));
  return y;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 8 channels of the output, as they lie there.
__device__ __forceinline__ void load8(const void* out, int dtype, int64_t at, float (&x)[8]) {
  if (dtype == 2) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(out) + at);
    const float4 u = p[0], w = p[1];
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
    return;
  }
  const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(out) + at);
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = dtype == 1 ? lo16<true>(v[i]) : lo16<false>(v[i]);
    x[2 * i + 1] = dtype == 1 ? hi16<true>(v[i]) : hi16<false>(v[i]);
  }
}
// Stores 8 channels and leaves in x what was stored: rounded, 0 where that is not finite.
__device__ __forceinline__ void store8(void* out, int dtype, int64_t at, float (&x)[8]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    if (dtype != 2) {
      const uint32_t y = dtype == 1 ? pack2<true>(x[i], x[i + 1]) : pack2<false>(x[i], x[i + 1]);
      x[i] = dtype == 1 ? lo16<true>(y) : lo16<false>(y);
      x[i + 1] = dtype == 1 ? hi16<true>(y) : hi16<false>(y);
    }
    x[i] = fabsf(x[i]) < INFINITY ? x[i] : 0.f;
    x[i + 1] = fabsf(x[i + 1]) < INFINITY ? x[i + 1] : 0.f;
    v[i / 2] = dtype == 1 ? pack2<true>(x[i], x[i + 1]) : pack2<false>(x[i], x[i + 1]);
  }
  if (dtype == 2) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]), p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}
__device__ __forceinline__ float inverse_sum(float l) {  // 0 where a row sees no key
  return l > 0.f ? 1.f / l : (l == l ? 0.f : l);
}

// A row's sum in tensor memory: what lies aside of it (a mean of weight `aside`) taken back and,
// if `put`, its mean over the weights' sum l laid aside in its place.  A warp's lanes together.
// (Not inlined: it is seldom called, and the code around it is fetched for every tile; inlined,
// 16 prompts of up to 777 tokens take 66.8 us, not 66.0.)
template <int DN>
__device__ __noinline__ void sum_aside(uint32_t to, void* out, int dtype, int64_t at, bool on,
                                       float aside, float l, bool put) {
  const float inv = inverse_sum(l);
#pragma unroll 1
  for (int c = 0; c < DN; c += 8) {
    float o[8], mean[8];
    tmem_ld8(to + c, o);
    tmem_wait_ld();
    if (on && aside > 0.f) {
      load8(out, dtype, at + c, mean);
#pragma unroll
      for (int y = 0; y < 8; ++y) o[y] = fmaf(mean[y], aside, o[y]);
    }
    if (on && put) {
#pragma unroll
      for (int y = 0; y < 8; ++y) mean[y] = o[y] * inv;
      store8(out, dtype, at + c, mean);
#pragma unroll
      for (int y = 0; y < 8; ++y) o[y] = fmaf(-mean[y], l, o[y]);
    }
    __syncwarp();
    tmem_st8(to + c, o);
  }
  tmem_wait_st();
}

template <int DN, bool F16>
__device__ __forceinline__ void softmax_loop(const PromptArgs& a, int x, Shared& sh) {
  using S = Shape<DN>;
  const int lane = threadIdx.x % 32, quarter = threadIdx.x / 32 % 4;
  const uint32_t tq = sh.tmem + (static_cast<uint32_t>(32 * quarter) << 16);
  const uint32_t ts = tq + x * S::kScores, tp = ts + S::kWeights;
  const uint32_t to = tq + S::kOutput + x * S::kOutputs;
  const float scale = fabsf(a.scale_log2);
  bool ok = true;
  int done = 0;  // key tiles of the blocks so far
  Work w;
  for (int j = 0; next_work(a, sh, j, &w, &ok); ++j) {
    const int row = w.row + x * kRows + 32 * quarter + lane;  // within the sequence
    const bool on = row < w.nq;
    const int seen = on ? seen_by(a, w, row) : 0;
    // m: the running maximum before it is scaled; from and ref are taken from scores before and
    // after that
    float m = -INFINITY, from = 0.f, ref = 0.f, l = 0.f;
    bool far = false;
    auto refer = [&](float high) {  // (the warp's lanes together)
      m = high;
      const bool none = m == -INFINITY;
      from = none ? 0.f : m;
      ref = from * scale - kAtTop<F16>;
      far = __any_sync(0xffffffffu, fabsf(ref) >= kFar);
      if (far) ref = -kAtTop<F16>;
    };
    const int64_t at = static_cast<int64_t>(w.q0 + row) * a.o_st + w.h * a.o_sh;
    float aside = 0.f;  // the sum of the weights whose values' mean lies in the output
    const int n = w.tiles[x];
    for (int i = 0; i < n; ++i, ++done) {
      ok = lanes_wait(true, smem_u32(&sh.s_full[x]), done & 1, a.wait_limit_ns, &sh.abort);
      if (!ok) break;
      tc_fence_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, reinterpret_cast<float(&)[32]>(s[32 * c]));
      tmem_wait_ld();
      if constexpr (S::kApart) {
        tc_fence_before();
        mbar_arrive(smem_u32(&sh.s_free[x]));
      }
      const int limit = seen - i * kKeys;
      if (__any_sync(0xffffffffu, limit < kKeys)) {
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = c < limit ? s[c] : -INFINITY;
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 128; c += 2) top[c / 2 % 4] = max3(top[c / 2 % 4], s[c], s[c + 1]);
      const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      if (i == 0) {
        refer(high);
      } else {
        const bool rise = (high - m) * scale > kRise, put = i % kRun == 0;
        if (__any_sync(0xffffffffu, rise || put)) {
          // (the products of the tile before were done when these scores were: or, apart,
          // are waited for)
          if constexpr (S::kApart) {
            ok = lanes_wait(true, smem_u32(&sh.v_done[x]), (done - 1) & 1, a.wait_limit_ns,
                            &sh.abort);
            if (!ok) break;
            tc_fence_after();
          }
          const float f = rise ? ex2((m - high) * scale) : 1.f;
          refer(rise ? high : m);
          if (put) {
            sum_aside<DN>(to, a.out, a.out_dtype, at, on, aside, l, true);
            aside = l;
          }
          l *= f, aside *= f;
#pragma unroll 1
          for (int c = 0; c < DN; c += 16) {
            float o[16];
            tmem_ld16(to + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] *= f;
            tmem_st16(to + c, o);
          }
        }
      }
      // (by pairs: half the code, which all tiles fetch past)
      if (far) {
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          const float2 y = halves_of(add2(pair_of(s[c], s[c + 1]), pair_of(-from, -from)));
          s[c] = y.x, s[c + 1] = y.y;
        }
      }
      const uint64_t scale2 = pair_of(scale, scale), ref2 = pair_of(-ref, -ref);
      uint64_t sum[4] = {};
      if constexpr (S::kApart) {
        // the weights before these have been used
        if (i > 0) {
          ok = lanes_wait(true, smem_u32(&sh.v_done[x]), (done - 1) & 1, a.wait_limit_ns, &sh.abort);
          if (!ok) break;
          tc_fence_after();
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t p[32];
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          const float2 e =
              halves_of(fma2(pair_of(s[64 * c + 2 * y], s[64 * c + 2 * y + 1]), scale2, ref2));
          const float p0 = ex2(e.x), p1 = ex2(e.y);
          sum[y % 4] = add2(sum[y % 4], pair_of(p0, p1));
          p[y] = pack2<F16>(p0, p1);
        }
        tmem_st32(tp + 32 * c, p);
      }
      const float2 both = halves_of(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
      l += both.x + both.y;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&sh.p_ready[x]));
    }
    // (also where the other query tile alone has keys: until it has been through them)
    if (ok)
      ok = lanes_wait(true, smem_u32(&sh.o_done[x]), j & 1, a.wait_limit_ns, &sh.abort, &sh.fills[0]);
    if (!ok) break;
    tc_fence_after();
    if (__any_sync(0xffffffffu, aside > 0.f))
      sum_aside<DN>(to, a.out, a.out_dtype, at, on, aside, l, false);
    const float inv = inverse_sum(l);
#pragma unroll 1
    for (int c = 0; c < DN; c += 16) {
      float o[16];
      __syncwarp();
      if (n > 0) {
        tmem_ld16(to + c, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int y = 0; y < 16; ++y) o[y] = l > 0.f || l != l ? o[y] * inv : 0.f;
      if (!on) continue;
      if (a.out_dtype == 2) {
        float4* out = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + c);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          out[y] = make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
      } else {
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at + c);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = a.out_dtype == 1 ? pack2<true>(o[8 * y + 2 * e], o[8 * y + 2 * e + 1])
                                    : pack2<false>(o[8 * y + 2 * e], o[8 * y + 2 * e + 1]);
          out[y] = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
    }
    tc_fence_before();
    mbar_arrive(smem_u32(&sh.o_free[x]));
  }
  if (!ok) {
    sh.abort = 1;
    set_status(a.status, kStatusTimeout);
  }
}

template <int DN, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ Maps m) {
  using S = Shape<DN>;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t q_smem = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t ring = q_smem + 2 * S::kQBytes;
  const int warp = threadIdx.x / 32;
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 2);
      sh.fills[i] = 0;
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&sh.q_full[x]), 1);
      mbar_init(smem_u32(&sh.q_free[x]), 1);
      mbar_init(smem_u32(&sh.s_full[x]), 1);
      mbar_init(smem_u32(&sh.p_ready[x]), kRows);
      mbar_init(smem_u32(&sh.o_done[x]), 1);
      mbar_init(smem_u32(&sh.o_free[x]), kRows);
      mbar_init(smem_u32(&sh.turn[x]), 1);
      mbar_init(smem_u32(&sh.s_free[x]), kRows);
      mbar_init(smem_u32(&sh.v_done[x]), 1);
      mbar_init(smem_u32(&sh.drain[x]), 1);
      mbar_init(smem_u32(&sh.work_full[x]), 1);
      mbar_init(smem_u32(&sh.work_free[x]), kReaders);
    }
    mbar_init(smem_u32(&sh.taken), 1);
    mbar_init(smem_u32(&sh.wanted), 1);
    sh.abort = 0;
    sh.q_fills[0] = sh.q_fills[1] = sh.takes = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(&sh.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  // A row of scores and what is made of it need more registers than 168 a thread (65536 among
  // 384), copies and products fewer: the softmax's warps take over 32 each from the others
  // (104 + 2 x 200 = 3 x 168).  Without spilt registers 32 prompts of 256 tokens, 16 heads take
  // 38 us, not 48, the last 2K tokens of 4 x 8K 476, not 484.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0)
      copy_loop<DN>(a, m, sh, q_smem, ring);
    else if (warp <= 2)
      product_loop<DN>(a, F16, warp - 1, sh, q_smem, ring);
    else
      schedule_loop(a, 4 * DN, sh);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    softmax_loop<DN, F16>(a, warp >= 8, sh);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {  // nothing that writes shared memory is in flight when the CTA ends
    const int lane = threadIdx.x;
    if (lane < kSlots && sh.fills[lane] > 0)
      mbar_wait_bounded(smem_u32(&sh.full[lane]), (sh.fills[lane] - 1) & 1, kDrainNs, nullptr);
    if (lane >= 30 && sh.q_fills[lane - 30] > 0)
      mbar_wait_bounded(smem_u32(&sh.q_full[lane - 30]), (sh.q_fills[lane - 30] - 1) & 1, kDrainNs,
                        nullptr);
    if (lane == 29 && sh.takes > 0)
      mbar_wait_bounded(smem_u32(&sh.taken), (sh.takes - 1) & 1, kDrainNs, nullptr);
    __syncwarp();
  }
  if (warp == 1) tmem_dealloc(sh.tmem, 512);
}

template <int DN, bool F16>
cudaError_t launch_t(const PromptArgs& a, const Maps& m, int blocks, cudaStream_t s) {
  // (an attribute of the device that is current: set on every call, it takes no time)
  const cudaError_t e =
      cudaFuncSetAttribute(prompt_attn_kernel<DN, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(Shape<DN>::kSmem));
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_attn_kernel<DN, F16>, dim3(blocks), dim3(kThreads), Shape<DN>::kSmem, s, a,
                    m);
}

}  // namespace

cudaError_t launch_prompt_attn(int dn, bool f16, const PromptArgs& a, const CUtensorMap& qn,
                               const CUtensorMap& qr, const CUtensorMap& kn, const CUtensorMap& kr,
                               const CUtensorMap& v, int blocks, cudaStream_t s) {
  const Maps m{qn, qr, kn, kr, v};
  if (dn == 128) return f16 ? launch_t<128, true>(a, m, blocks, s) : launch_t<128, false>(a, m, blocks, s);
  return f16 ? launch_t<64, true>(a, m, blocks, s) : launch_t<64, false>(a, m, blocks, s);
}

}  // namespace dkv
