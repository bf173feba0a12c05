// attn_fp8.cu -- decode attention over an 8-bit KV cache (exact and
// page-sparse): e4m3 codes with one fp32 scale per 16-token block and kv head.
//
// What it computes (per query head h of batch b, kv head h / G):
//   out = sum_t softmax_t(scale * q . k_t) v_t,
//   k_t = ks(page of t) * code_k(t),   v_t = vs(page of t) * code_v(t)
// over all tokens of the sequence, or over those of the pages selected for h.
//
// The scales never touch the codes.  ks multiplies the page's scores.  vs =
// 2^e * f (1 <= |f| < 2, or f = 0) goes into the softmax weights: beside the
// usual sum l of 2^(s - m) (s: the scores in log2 units), the output accumulates
// w = f * 2^((s - m) + (e - r)) with an integer r, so the weights that meet the
// codes are near 1 at the largest contribution whatever the scales are: a page
// of large values with little weight costs the others no bits.  s - m is exact
// near the maximum and e - r always, so r adds no rounding.  At the end of an
// item o = 2^r * sum w code, the usual partial.
//
// m and r are references, not the exact maxima: they move only when a score
// passes m, or a weight passes 1, by more than 2^kSlack (fp16 holds w < 2^9
// without loss), which after a warp's first pages is rare.  So a step needs no
// reduction across lanes, only a vote, and rarely rescales.
//
// Structure as in the 16-bit kernel: a persistent grid pulls work items
// (batch, kv head, chunk of pages) from a counter; one producer warp streams
// pages by TMA tensor copies (one 16 x d byte box a tensor and page, d-byte
// swizzle) into per-warp sub-rings of two-page shared-memory stages; four
// consumer warps compute.  Codes become fp16 in registers (exact: e4m3 is a
// subset of fp16) and are always the MMA's A operand, so that all of its 16 rows
// work; the query heads are the columns:
//   * S^T = K Q^T, tokens x heads.  One ldmatrix word of lane (g, t4) is four
//     consecutive channels 16 c + 4 t4 .. + 3 of token g, which two conversions
//     turn into the A fragments of k-step c; the query's B fragments take the
//     same channel order.
//   * O^T = V^T P^T, channels x heads.  One transposed ldmatrix word is the
//     channel pair (2 g, 2 g + 1) of tokens 2 t4 and 2 t4 + 1; a byte permute
//     and two conversions make the A fragments whose rows g and g + 8 are the
//     channels 16 c + 2 g and 16 c + 2 g + 1.
// The weights are split into fp16 hi + lo (22 significant bits).  Columns, by
// the query heads GL that a kv head may have in an instantiation:
//   GL = 8  columns are heads; hi and lo are two products into one sum.
//   GL = 4  columns 0-3 hold the hi halves and 4-7 the lo halves of 4 heads: one
//           product.  The query fills both column halves, so lanes t4 < 2 find
//           the first page's scores of all heads and t4 >= 2 the second's: 4 of
//           the stage's 128 scores a lane.
//   GL = 1  even columns hi, odd columns lo; the query fills every column and
//           each lane keeps one of the stage's 32 scores.
// Weights reach the B fragments by 8 x 8 transposes (movmatrix), or shuffles for
// one head.  A bf16 query is scaled by a power of two per head so that its
// largest component lies in [2^14, 2^15): exact in fp16 for every component
// within 2^28 of it; the scores are scaled back.
//
// Bound by HBM: a token's K and V are 2 d bytes, once.  Measured on a GB300 (copy
// rate 6.79 TB/s), 32 query / 8 kv heads, d = 128, with the merge: 16 sequences
// of 32K tokens 158 us dense (6.8 TB/s), 165 us paged (6.5), ragged 116 us
// (6.1); one of 1M tokens 303 us (7.1).  At d = 64 a page is the same work for
// half the bytes, and its chain of dependent steps shows: 16 x 32K 86 us dense
// (6.3), 95 us paged (5.6); 8 x 32 heads of 8K, one query head each, 47 us (5.7).
// What the layout is worth, at 16 x 32K, d = 128: with the heads on the MMA's M
// side (8 of 16 rows, four to eight scores a lane, exact running maxima) and two
// CTAs an SM, 183 us dense and 190 us paged.  Two pages a box in a dense cache
// read in order save the 8K shape 5 us.  A small call costs about 7 us, two
// kernels' chains of dependent loads.
//
// Every mbarrier wait is bounded; on expiry the kernel records a timeout in
// the status word, stops issuing, drains the copies it issued and exits.

#include <math.h>

#include "dkv_device.cuh"
#include "dkv_kernels.h"
#include "per_device.h"

namespace dkv {
namespace {

constexpr uint64_t kDrainLimitNs = 200000000ull;  // 200 ms for the whole drain
constexpr int kListPages = 64;                    // pages of an item listed at a time
constexpr int kMaxRagged = 128;    // sequences whose items are counted by their lengths
constexpr float kSlack = 8.f;      // how far, in log2 units, a reference may be passed
constexpr float kUnset = -3.402823466e38f;  // a reference before the first token: the
                                            // lowest value, so every finite score passes it

struct ItemDesc {
  int item;     // work item, -1: no more work
  int n_pages;  // pages in the item
};

// GL: query heads a kv head may have (1, 4 or 8).
template <int D, int GL>
struct Fp8Cfg {
  static constexpr int kPagesPerStage = 2;
  static constexpr int kTileBytes = kPage * D;      // one tensor's page of codes
  // K codes of both pages | V codes of both
  static constexpr int kVOffset = kPagesPerStage * kTileBytes;
  static constexpr int kStageBytes = 2 * kVOffset;
  // Three CTAs an SM, each with 64 KiB of pages in flight.  64 channels take
  // fewer registers, and a page's work, the same for half the bytes, has more
  // latency to hide: four with 48 KiB (16 x 32K paged, 4 query heads a kv head,
  // 101 -> 99 us, the select at 8 x 8K 36.8 -> 34.8).
  static constexpr int kCtas = D == 64 ? 4 : 3;
  static constexpr int kStages = (kCtas == 3 ? 64 : 48) * 1024 / kStageBytes;
  // The warps' states of 8 heads are merged in two turns of 4.
  static constexpr int kTurns = GL == 8 ? 2 : 1;
  static constexpr int kMergeRows = GL / kTurns;
  static constexpr int kSub = kStages / kConsumerWarps;    // stages per consumer warp
  static constexpr int kIssueLanes = kStages < 16 ? kStages : 16;
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kMetaOffset = kBarOffset + (2 * kStages + 4) * 8;
  static constexpr int kDescOffset = kMetaOffset + kStages * kPagesPerStage * 16;
  static constexpr int kMergeOffset = kDescOffset + 2 * 8;
  static constexpr int kMergeRow = D + 3;  // o[D], max m, sum l, exponent r
  static constexpr int kListOffset =
      (kMergeOffset + (kConsumerWarps - 1) * kMergeRows * kMergeRow * 4 + 15) / 16 * 16;
  static constexpr int kBlockOffset = kListOffset + 16 * kListPages;
  static constexpr int kFirstOffset = kBlockOffset + 4 * kListPages;
  static constexpr int kMiscOffset = kFirstOffset + 4 * kMaxRagged;
  static constexpr int kSmemBytes = 1024 + kMiscOffset + 16;
  static_assert(kTileBytes % 1024 == 0, "tiles keep the swizzle's alignment");
  static_assert(kStages % kConsumerWarps == 0, "one sub-ring per consumer warp");
  static_assert(kIssueLanes % kConsumerWarps == 0, "an issuing lane feeds one warp");
  static_assert(kMetaOffset % 16 == 0 && kListOffset % 16 == 0, "16-byte rows");
  static_assert((kSmemBytes + 1024) * kCtas <= 228 * 1024, "the CTAs fit an SM");
};

// Shared address of 16-byte chunk c of token t in a tile of 16 rows of D bytes
// written with D-byte swizzle: rows of 128 bytes, the chunk XORed with t % 8,
// or rows of 64 bytes, the chunk XORed with (t / 2) % 4.
template <int D>
__device__ __forceinline__ uint32_t code_addr(uint32_t base, int t, int c) {
  return base + static_cast<uint32_t>(t * D + ((D == 128 ? c ^ (t & 7) : c ^ ((t >> 1) & 3)) << 4));
}

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"r"(kConsumerWarps * 32) : "memory");
}

// Barrier over the consumer warps that also ORs `flag` across them, so every
// consumer takes the same branch afterwards.
__device__ __forceinline__ bool consumers_any(bool flag) {
  uint32_t res;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(res)
      : "r"(static_cast<uint32_t>(flag)), "r"(kConsumerWarps * 32)
      : "memory");
  return res != 0;
}

// Two e4m3 codes (the low / high half of w) as a packed fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3_lo2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

// 2^x, 0 for x = -inf (results below 2^-126 are 0: a weight that small is lost
// beside the largest, which is above 1/2: r is rounded up).
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The transpose of an 8 x 8 matrix of 16-bit values, two of a row a lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ void store_out(void* out, int out_dtype, int64_t off, float v) {
  if (out_dtype == 2) {
    static_cast<float*>(out)[off] = v;
  } else if (out_dtype == 1) {
    static_cast<__half*>(out)[off] = __float2half_rn(v);
  } else {
    static_cast<__nv_bfloat16*>(out)[off] = __float2bfloat16_rn(v);
  }
}

template <int D, bool F16, bool SPARSE, int GL>
__global__ void __launch_bounds__(kAttnThreads, Fp8Cfg<D, GL>::kCtas) attn_fp8_kernel(
    const AttnArgs a, const __grid_constant__ CUtensorMap mk,
    const __grid_constant__ CUtensorMap mv) {
  using C = Fp8Cfg<D, GL>;
  constexpr int kQ = C::kPagesPerStage;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t full0 = sbase + C::kBarOffset;
  const uint32_t empty0 = full0 + 8 * C::kStages;
  const uint32_t dfull0 = empty0 + 8 * C::kStages;
  const uint32_t dempty0 = dfull0 + 16;
  // per page of a stage: page, head mask, K scale, V scale
  int4* stage_meta = reinterpret_cast<int4*>(smem + C::kMetaOffset);
  volatile ItemDesc* desc = reinterpret_cast<volatile ItemDesc*>(smem + C::kDescOffset);
  float* mrg = reinterpret_cast<float*>(smem + C::kMergeOffset);
  int4* list = reinterpret_cast<int4*>(smem + C::kListOffset);  // the same, of listed pages
  int* blocks = reinterpret_cast<int*>(smem + C::kBlockOffset);  // paged: their pool blocks
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOffset);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(dfull0 + 8 * s, 1);
      mbar_init(dempty0 + 8 * s, 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kConsumerWarps && lane == 0) {
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
  }
  griddep_launch_dependents();
  // With per-unit ready flags the sparse path waits for each unit's selection
  // as it takes the unit's items (the selection kernel lets this grid start
  // only once every earlier kernel has finished).
  const bool unit_flags = SPARSE && a.unit_ready != nullptr;
  if (!unit_flags) griddep_wait();
  __syncthreads();
  // One chunk a unit: the item is its rows' whole result, written to out here.
  const bool whole = a.n_chunks == 1;

  if (warp == kConsumerWarps) {
    // ------------------------------------------------------------ producer
    // Lane 0 fetches items and publishes their descriptors.  Stage q of an
    // item (pages 2 q, 2 q + 1) goes to consumer warp q % 4; lanes
    // 0 .. kIssueLanes - 1 issue one stage each per round.
    //
    // An item's pages are listed in parts of kListPages: page, mask, block and
    // scales.  That takes four or five dependent loads (work counter -> length
    // or union -> block table -> scales), about 3 us, in which the ring would
    // run dry; so the next part is listed step by step between the rounds of
    // the current one, each step using what the one before loaded.
    const uint64_t pol = l2_evict_first_policy();
    // (the maps' boxes are two pages high for a dense cache read in order)
    const bool pair_boxes = !SPARSE && a.bt == nullptr;
    const int my_w = lane & 3;  // consumer warp this lane feeds
    const bool issuer = lane < C::kIssueLanes;
    int wc = 0;           // stages issued so far to warp my_w
    bool failed = false;  // a lane gave up waiting for a free slot
    // Exact attention over sequences of their own lengths: tickets count the
    // chunks that hold pages, sequence by sequence (heads inside), so no ticket
    // is spent on an empty one.  seq_end[b]: the chunks of sequences 0 .. b.
    int* seq_end = reinterpret_cast<int*>(smem + C::kFirstOffset);
    const bool by_length = !SPARSE && a.lens != nullptr && a.B <= kMaxRagged && !whole;
    int n_tickets = a.n_items;
    if (by_length) {
      int sum = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int bb = b0 + lane;
        int c = 0;
        if (bb < a.B)
          c = static_cast<int>(ceil_div(ceil_div(max(0, min(a.lens[bb], a.N)), kPage),
                                        a.pages_per_chunk));
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int up = __shfl_up_sync(0xffffffffu, c, o);
          if (lane >= o) c += up;
        }
        if (bb < a.B) seq_end[bb] = sum + c;
        sum += __shfl_sync(0xffffffffu, c, 31);
      }
      __syncwarp();
      n_tickets = sum * a.Hkv;  // (at most n_items)
    }
    constexpr int kPer = kListPages / 32;
    // The part being listed, and where its listing has got to.
    int item = 0, n = 0, b = 0, kvh = 0, unit = 0, first = 0, l0 = 0;
    int step = 0;
    // Taking an item before the current one is done costs balance at the end:
    // only where a CTA gets several, and not while selections are still coming.
    const bool ahead = !unit_flags && a.n_items >= 4 * static_cast<int>(gridDim.x);
    int ticket = 0, count = 0, len = 0;
    int page[kPer], mask[kPer], blk[kPer];
    float ks[kPer], vs[kPer];
    constexpr int kListed = 6;
    bool fresh = true;  // no ticket taken yet
    const bool counted = n_tickets > static_cast<int>(gridDim.x);  // CTAs take several
    // One step; with `block`, a step that has to wait does.
    auto advance = [&](bool block) {
      switch (step) {
        case 0:  // a new item: the CTA's own number first, then from the counter
          if (fresh)
            ticket = blockIdx.x;
          else if (!counted)
            ticket = n_tickets;
          else if (lane == 0)
            ticket = static_cast<int>(gridDim.x + atomicAdd(a.work_counter, 1u));
          fresh = false;
          step = 1;
          break;
        case 1: {
          item = __shfl_sync(0xffffffffu, ticket, 0);
          l0 = 0;
          if (item >= n_tickets) {
            item = -1;
            n = 0;
            step = kListed;
            break;
          }
          if (by_length) {
            // the first sequence that ends past the ticket's chunk
            const int at = item / a.Hkv;
            kvh = item % a.Hkv;
            b = 0;
            for (int b0 = 0; b0 < a.B; b0 += 32) {
              const int bb = b0 + lane;
              b += __popc(__ballot_sync(0xffffffffu, bb < a.B && seq_end[bb] <= at));
            }
            const int c = at - (b > 0 ? seq_end[b - 1] : 0);
            unit = b * a.Hkv + kvh;
            item = unit * a.n_chunks + c;
            first = c * a.pages_per_chunk;
          } else {
            unit = item / a.n_chunks;
            first = item % a.n_chunks * a.pages_per_chunk;  // (sparse: once the union is known)
            kvh = unit % a.Hkv;
            b = unit / a.Hkv;
          }
          len = a.lens != nullptr ? a.lens[b] : a.N;
          step = SPARSE ? 2 : 3;
          if constexpr (!SPARSE) break;
          [[fallthrough]];
        }
        case 2:  // sparse: the union's size, once the unit's selection is there
          if constexpr (SPARSE) {
            if (unit_flags) {
              int rdy = 1;
              if (lane == 0)
                rdy = block ? flag_wait_bounded(a.unit_ready + unit, a.wait_limit_ns, abort_flag)
                            : ld_acquire_gpu(a.unit_ready + unit) != 0u;
              if (!__shfl_sync(0xffffffffu, rdy, 0)) {
                if (!block) break;  // asked again
                if (lane == 0 && *abort_flag == 0) {
                  set_status(a.status, kStatusTimeout);
                  *abort_flag = 1;
                }
                item = -1;  // stop: publish the end of work
                n = 0;
                step = kListed;
                break;
              }
            }
            count = __ldcg(a.union_count + unit);
          }
          step = 3;
          break;
        case 3:  // the part's pages
          if (l0 == 0) {
            int part = a.pages_per_chunk;
            if constexpr (SPARSE) {
              part = fp8_part_pages(count, a.n_chunks);
              first = item % a.n_chunks * part;
            } else {
              count = static_cast<int>(ceil_div(min(len, a.N), kPage));
            }
            n = len <= 0 ? 0 : max(0, min(count - first, part));
            if (n == 0 && !whole) {  // no partial is read for it
              step = 0;
              break;
            }
          }
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int j = l0 + lane + 32 * i;
            page[i] = first + j;
            mask[i] = 0xff;
            if constexpr (SPARSE) {
              if (j < n) {
                const int2 e = __ldcg(a.union_list +
                                      static_cast<int64_t>(unit) * a.union_stride + first + j);
                page[i] = e.x;
                mask[i] = e.y;
              }
            }
          }
          step = 4;
          if constexpr (SPARSE) break;
          [[fallthrough]];
        case 4:
          if (a.bt != nullptr) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              if (l0 + lane + 32 * i < n) blk[i] = a.bt[b * a.bts + page[i]];
          }
          step = 5;
          break;
        case 5: {
          const float* kscale = a.k8.scale + kvh * a.k8.sh;
          const float* vscale = a.v8.scale + kvh * a.v8.sh;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            if (l0 + lane + 32 * i >= n) continue;
            if (a.bt != nullptr) {
              // An entry outside [0, num_blocks) is clamped into it, so no copy
              // leaves the pool, and reported as a failed check.
              if (blk[i] < 0 || blk[i] >= a.nblocks) set_status(a.status, kStatusCheck);
              blk[i] = min(max(blk[i], 0), a.nblocks - 1);
              ks[i] = kscale[blk[i] * a.k8.sb];
              vs[i] = vscale[blk[i] * a.v8.sb];
            } else {
              ks[i] = kscale[b * a.k8.sb + page[i]];
              vs[i] = vscale[b * a.v8.sb + page[i]];
            }
          }
          step = kListed;
          break;
        }
        default: break;
      }
    };
    while (step != kListed) advance(true);
    for (int k = -1;;) {
      // The listed part becomes the current one: its registers go to the list.
      const int c_item = item, c_n = n, c_b = b, c_kvh = kvh, c_l0 = l0;
      const int ln = min(kListPages, n - l0);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int j = lane + 32 * i;
        if (j < ln) {
          list[j] = make_int4(page[i], mask[i], __float_as_int(ks[i]), __float_as_int(vs[i]));
          blocks[j] = blk[i];
        }
      }
      __syncwarp();
      if (c_l0 == 0) {  // a new item: publish it
        const int slot = ++k & 1;
        int ok = 1;
        if (lane == 0 && k >= 2) {
          ok = mbar_wait_bounded(dempty0 + 8 * slot, ((k >> 1) - 1) & 1, a.wait_limit_ns,
                                 abort_flag);
          if (!ok && *abort_flag == 0) {
            set_status(a.status, kStatusTimeout);
            *abort_flag = 1;
          }
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        if (lane == 0) {
          desc[slot].item = c_item;
          desc[slot].n_pages = c_n;
          mbar_arrive(dfull0 + 8 * slot);  // release: consumers see the descriptor
        }
        if (c_item < 0) break;
      }
      // What is listed next: the item's next part, or a new item.
      l0 += kListPages;
      step = l0 < n ? 3 : 0;
      bool lok = true;
      for (int j0 = 0; j0 < ln; j0 += C::kIssueLanes * kQ) {
        const int j = j0 + lane * kQ;  // first page of this lane's stage
        if (issuer && j < ln) {
          const int c = wc + (j / kQ >> 2);
          const int s = my_w * C::kSub + c % C::kSub;  // warp my_w's sub-ring, in order
          if (c >= C::kSub &&
              !mbar_wait_bounded(empty0 + 8 * s, ((c / C::kSub) - 1) & 1, a.wait_limit_ns,
                                 abort_flag)) {
            lok = false;
          } else {
            const int cnt = min(kQ, ln - j);
#pragma unroll
            for (int t = 0; t < kQ; ++t)
              if (t < cnt) stage_meta[s * kQ + t] = list[j + t];
            const uint32_t dst = sbase + s * C::kStageBytes;
            const uint32_t bar = full0 + 8 * s;
            // {channel, token, -, kv head, batch} of the cache, or
            // {channel, token in block, -, kv head, block} of a pool
            if (pair_boxes) {  // a box of both pages (past the end: zeros)
              mbar_arrive_expect_tx(bar, C::kStageBytes);
              const int y = list[j].x * kPage;
              tma_load_5d_hint(dst, &mk, bar, 0, y, 0, c_kvh, c_b, pol);
              tma_load_5d_hint(dst + C::kVOffset, &mv, bar, 0, y, 0, c_kvh, c_b, pol);
            } else {
              mbar_arrive_expect_tx(bar, cnt * 2 * C::kTileBytes);
#pragma unroll
              for (int t = 0; t < kQ; ++t) {
                if (t < cnt) {
                  const int y = a.bt != nullptr ? 0 : list[j + t].x * kPage;
                  const int z = a.bt != nullptr ? blocks[j + t] : c_b;
                  const uint32_t d = dst + t * C::kTileBytes;
                  tma_load_5d_hint(d, &mk, bar, 0, y, 0, c_kvh, z, pol);
                  tma_load_5d_hint(d + C::kVOffset, &mv, bar, 0, y, 0, c_kvh, z, pol);
                }
              }
            }
          }
        }
        lok = __all_sync(0xffffffffu, lok);
        if (!lok) break;
        if (step != kListed && (ahead || step > 0)) advance(false);
      }
      const int nq = static_cast<int>(ceil_div(ln, kQ));  // stages of this part
      wc += nq > my_w ? (nq - my_w + 3) >> 2 : 0;
      if (!lok) {
        failed = true;
        break;
      }
      while (step != kListed) advance(true);
    }
    if (lane == 0 && failed && *abort_flag == 0) {
      set_status(a.status, kStatusTimeout);
      *abort_flag = 1;
    }
    __syncwarp();
    // (a limit of 0, the test hook: the consumers may give up after this check)
    if (lane < kConsumerWarps && (*abort_flag || a.wait_limit_ns == 0)) {
      // Let every copy this CTA issued land before it exits: lane w waits for
      // the last kSub slots of warp w's sub-ring (slots never issued just run
      // into the deadline).
      const uint64_t deadline = globaltimer_ns() + kDrainLimitNs;
      for (int c = max(0, wc - C::kSub); c < wc; ++c) {
        const uint64_t now = globaltimer_ns();
        if (now >= deadline) break;
        mbar_wait_bounded(full0 + 8 * (my_w * C::kSub + c % C::kSub), (c / C::kSub) & 1,
                          deadline - now, nullptr);
      }
    }
    __syncwarp();
    if (lane == 0 && counted) {
      // The last CTA to stop fetching work resets the counters for the next
      // call (every earlier fetch is ordered before its ticket by the fence).
      __threadfence();
      if (atomicAdd(a.exit_counter, 1u) == gridDim.x - 1) {
        atomicExch(a.work_counter, 0u);
        atomicExch(a.exit_counter, 0u);
      }
    }
    // The grid ends only after the selection grid has (so the kernels after
    // this one, which wait for this grid alone, see every selection output).
    if (unit_flags) griddep_wait();
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, t4 = lane & 3;
  const int mtx = lane >> 3, mrow = lane & 7;
  // This lane's score columns 2 t4 + e are heads h0 + e, on page `pt` of a stage
  // (GL = 8: on both).
  const int h0 = GL == 8 ? 2 * t4 : (GL == 4 ? 2 * (t4 & 1) : 0);
  const int pt = t4 >> 1;
  int mycnt = 0;  // stages this warp has taken from its sub-ring
  // Exits are taken by all four consumer warps together (consumers_any), so no
  // warp is ever left waiting at a consumer barrier.
  for (int k = 0;; ++k) {
    const int slot = k & 1;
    const bool dok = mbar_wait_bounded(dfull0 + 8 * slot, (k >> 1) & 1, a.wait_limit_ns,
                                       abort_flag);
    if (consumers_any(!dok)) {
      if (threadIdx.x == 0) {
        set_status(a.status, kStatusTimeout);
        *abort_flag = 1;
      }
      return;
    }
    const int item = desc[slot].item, n_pages = desc[slot].n_pages;
    if (item < 0) return;  // the same descriptor for every consumer warp
    const int chunk = item % a.n_chunks;
    const int unit = item / a.n_chunks;
    const int kvh = unit % a.Hkv, b = unit / a.Hkv;
    const int Nb = seq_len_of(a.lens, b, a.N);  // tokens this sequence attends

    // The query's B fragments: k-step c of lane (g, t4) is channels
    // 16 c + 4 t4 .. + 3 of the head of column g, in fp16.
    uint32_t qa[D / 16][2];
    float qs[2];  // the lane's heads' factor from products to log2 units
    {
      const int head = GL == 1 ? 0 : g & (GL - 1);
      const bool head_ok = head < a.G;
      const uint16_t* qrow = static_cast<const uint16_t*>(a.q) + b * a.q_sb +
                             static_cast<int64_t>(kvh * a.G + (head_ok ? head : 0)) * a.q_sh +
                             4 * t4;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint2 w = head_ok ? *reinterpret_cast<const uint2*>(qrow + 16 * c) : make_uint2(0u, 0u);
        qa[c][0] = w.x;
        qa[c][1] = w.y;
      }
      qs[0] = qs[1] = a.scale_log2;
      if constexpr (!F16) {
        // 2^up brings the head's largest component into [2^14, 2^15)
        uint32_t top = 0;  // its bits: bf16 magnitudes order as integers
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            top = max(top, max(qa[c][i] & 0x7fffu, (qa[c][i] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int up = min(126, 14 + 127 - static_cast<int>(top >> 7));
        const float f = __int_as_float((127 + up) << 23);
        const float down = a.scale_log2 * __int_as_float((127 - up) << 23);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qs[e] = __shfl_sync(0xffffffffu, down, 4 * (GL == 1 ? 0 : h0 + e));
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qa[c][i] = pack2<true>(lo16<false>(qa[c][i]) * f, hi16<false>(qa[c][i]) * f);
      }
    }
    // Per head of the lane: the references m and r, the largest (s - m) + e that r
    // was set for, and the lane's part of the sum l.
    constexpr int kE = GL == 1 ? 1 : 2;             // heads of a lane
    constexpr int kT = GL == 8 ? kQ : 1;            // pages of a lane
    constexpr int kN = GL == 1 ? 1 : 2;             // tokens of a lane, page and head
    float m_ref[kE], v_ref[kE], r_ref[kE], l_run[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) m_ref[e] = v_ref[e] = kUnset, r_ref[e] = l_run[e] = 0.f;
    float acc[D / 16][4];  // tile c: channels 16 c + 2 g (0, 1) and + 1 (2, 3), columns 2 t4 + e
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;

    bool aborted = false;
    for (int sq = warp; sq * kQ < n_pages; sq += kConsumerWarps) {
      const int s = warp * C::kSub + mycnt % C::kSub;
      const bool ok = mbar_wait_bounded(full0 + 8 * s, (mycnt / C::kSub) & 1, a.wait_limit_ns,
                                        abort_flag);
      ++mycnt;
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) {
          set_status(a.status, kStatusTimeout);
          *abort_flag = 1;
        }
        aborted = true;
        break;
      }
      const int cnt = min(kQ, n_pages - sq * kQ);
      const uint32_t st = sbase + s * C::kStageBytes;

      // S^T = K Q^T: sc[t][0 .. 3] = tokens g and g + 8 (2, 3) of page t in
      // columns 2 t4 and 2 t4 + 1 (1, 3).
      float sc[kQ][4];
#pragma unroll
      for (int t = 0; t < kQ; ++t) {
        sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
        if (t < cnt) {
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t r[4];  // [chunk c, c + 1][tokens 0-7, 8-15]
            ldsm_x4(code_addr<D>(st + t * C::kTileBytes, 8 * (mtx & 1) + mrow, c + (mtx >> 1)),
                    r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              mma16816<true>(sc[t], e4m3_lo2(r[2 * i]), e4m3_lo2(r[2 * i + 1]),
                             e4m3_hi2(r[2 * i]), e4m3_hi2(r[2 * i + 1]), qa[c + i][0],
                             qa[c + i][1]);
          }
        }
      }

      // The lane's scores in log2 units: sv[t][e][n] of page t (GL = 8; else page
      // pt), head h0 + e, token g + 8 n (GL = 1: token g + 8 (t4 & 1)).
      float sv[kT][kE][kN], ve[kT], vf[kT];
      bool ragged = false;
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        const int page_t = GL == 8 ? t : pt;
        const bool have = page_t < cnt;
        const int4 meta = stage_meta[s * kQ + page_t];
        const float ks = __int_as_float(meta.z);
        // vs = 2^ve * vf (a scale below 2^-126 counts as 0)
        const uint32_t vb = static_cast<uint32_t>(meta.w);
        const int ex = (vb >> 23) & 0xff;
        ve[t] = static_cast<float>(ex - 127);
        vf[t] = ex == 0 ? 0.f : __uint_as_float((vb & 0x807fffffu) | 0x3f800000u);
#pragma unroll
        for (int e = 0; e < kE; ++e)
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            const int i = GL == 1 ? 0 : 2 * n + e;
            float raw = GL == 8 ? sc[t][i] : (pt ? sc[1][i] : sc[0][i]);
            if constexpr (GL == 1) raw = (t4 & 1) ? (pt ? sc[1][2] : sc[0][2]) : raw;
            sv[t][e][n] = raw * (qs[e] * ks);
          }
        const bool past = have && Nb - meta.x * kPage < kPage;  // (no sum passes 2^31)
        ragged |= past;
        if (SPARSE || !have || past) {
          // Token i of a page counts for head h if it lies in the sequence and
          // bit (h << sub_log2) + (i >> (4 - sub_log2)) of the mask is set.
          const int sl = SPARSE ? a.sub_log2 : 0;
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            const int i = g + 8 * (GL == 1 ? t4 & 1 : n);
            const bool in = have && meta.x * kPage + i < Nb;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
              const bool on =
                  !SPARSE || ((meta.y >> (((h0 + e) << sl) + (sl ? i >> (4 - sl) : 0))) & 1);
              if (!in || !on) sv[t][e][n] = -INFINITY;
            }
          }
        }
      }
      ragged = __any_sync(0xffffffffu, ragged);

      // x = s - m, y = x + (e - r): 2^x into l, f 2^y into the weights.
      float x[kT][kE][kN], y[kT][kE][kN], top = -INFINITY;
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int e = 0; e < kE; ++e)
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            x[t][e][n] = sv[t][e][n] - m_ref[e];
            y[t][e][n] = x[t][e][n] + (ve[t] - r_ref[e]);
            top = fmaxf(top, fmaxf(x[t][e][n], y[t][e][n]));
          }
      if (__any_sync(0xffffffffu, top > kSlack)) {
        // New references: the running maxima with this stage's.  (s - m) + e, not s
        // + e: beside a large s the exponent would have no digits left.
        constexpr int kFirst = GL == 8 ? 4 : (GL == 4 ? 2 : 1);  // lanes of other heads
        float m_new[kE], pv[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          float pm = -INFINITY;
#pragma unroll
          for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int n = 0; n < kN; ++n) pm = fmaxf(pm, sv[t][e][n]);
#pragma unroll
          for (int o = kFirst; o < 32; o *= 2)
            pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, o));
          m_new[e] = fmaxf(m_ref[e], pm);
          pv[e] = -INFINITY;  // (stays so where no token of the stage counts)
#pragma unroll
          for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int n = 0; n < kN; ++n)
              pv[e] = fmaxf(pv[e], (sv[t][e][n] - m_new[e]) + ve[t]);
#pragma unroll
          for (int o = kFirst; o < 32; o *= 2)
            pv[e] = fmaxf(pv[e], __shfl_xor_sync(0xffffffffu, pv[e], o));
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          if (pv[e] != -INFINITY) {
            const float down = m_ref[e] - m_new[e];  // (unset: 2^down is 0)
            v_ref[e] = fmaxf(v_ref[e] + down, pv[e]);
            const float r_new = ceilf(v_ref[e]);
            l_run[e] *= exp2_fast(down);
            const float alpha = exp2_fast(down + (r_ref[e] - r_new));
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              acc[c][e] *= alpha;
              acc[c][2 + e] *= alpha;
              if constexpr (GL == 1) acc[c][1] *= alpha, acc[c][3] *= alpha;
            }
            m_ref[e] = m_new[e];
            r_ref[e] = r_new;
          }
#pragma unroll
          for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              x[t][e][n] = sv[t][e][n] - m_ref[e];
              y[t][e][n] = x[t][e][n] + (ve[t] - r_ref[e]);
            }
        }
      }
      if (ragged) {
        // Slots past the sequence's end hold anything: zero those V codes
        // (their weights are 0, but 0 * NaN is not).
        for (int t = 0; t < cnt; ++t) {
          const int nt = min(kPage, Nb - stage_meta[s * kQ + t].x * kPage);
          uint8_t* vt = smem + s * C::kStageBytes + C::kVOffset + t * C::kTileBytes;
          for (int i = lane; i < (kPage - nt) * (D / 16); i += 32)
            *reinterpret_cast<uint4*>(vt + nt * D + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        // (before the slot goes back to the copy engine)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      float w[kT][kE][kN];
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int e = 0; e < kE; ++e)
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            l_run[e] += exp2_fast(x[t][e][n]);
            w[t][e][n] = exp2_fast(y[t][e][n]) * vf[t];
          }

      // B fragments of P^T: pb[t][n] = tokens 2 t4 + 8 n, + 1 of page t in column
      // g; GL = 8: pl the lo halves.
      uint32_t pb[kQ][2], pl[kQ][2];
      if constexpr (GL == 1) {
        const __half wh = __float2half_rn(w[0][0][0]);
        const __half2 w2 = __halves2half2(wh, __float2half_rn(w[0][0][0] - __half2float(wh)));
        const uint32_t wp = *reinterpret_cast<const uint32_t*>(&w2);
        const uint32_t pick = (g & 1) ? 0x7632u : 0x5410u;
#pragma unroll
        for (int t = 0; t < kQ; ++t)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            pb[t][n] = __byte_perm(__shfl_sync(0xffffffffu, wp, 8 * t4 + 2 * t + n),
                                   __shfl_sync(0xffffffffu, wp, 8 * t4 + 4 + 2 * t + n), pick);
      } else if constexpr (GL == 4) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint32_t hi, lo;
          split_pair<true>(w[0][0][n], w[0][1][n], hi, lo);
          // page 0's lo halves for lanes t4 >= 2, page 1's hi halves for t4 < 2
          const uint32_t other = __shfl_xor_sync(0xffffffffu, pt ? hi : lo, 2);
          pb[0][n] = movmatrix_trans(pt ? other : hi);
          pb[1][n] = movmatrix_trans(pt ? lo : other);
        }
      } else {
#pragma unroll
        for (int t = 0; t < kQ; ++t)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            uint32_t hi, lo;
            split_pair<true>(w[t][0][n], w[t][1][n], hi, lo);
            pb[t][n] = movmatrix_trans(hi);
            pl[t][n] = movmatrix_trans(lo);
          }
      }

      // O^T += V^T P^T
#pragma unroll
      for (int t = 0; t < kQ; ++t) {
        if (t < cnt) {
          const uint32_t vt = st + C::kVOffset + t * C::kTileBytes;
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t r[4];  // [chunk c, c + 1][tokens 0-7, 8-15]
            ldsm_x4_trans(code_addr<D>(vt, 8 * (mtx & 1) + mrow, c + (mtx >> 1)), r[0], r[1], r[2],
                          r[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // bytes (token 2 t4: even, odd; token 2 t4 + 1: even, odd channel)
              // to (even, even; odd, odd)
              const uint32_t y0 = __byte_perm(r[2 * i], 0u, 0x3120);
              const uint32_t y8 = __byte_perm(r[2 * i + 1], 0u, 0x3120);
              const uint32_t a0 = e4m3_lo2(y0), a1 = e4m3_hi2(y0);
              const uint32_t a2 = e4m3_lo2(y8), a3 = e4m3_hi2(y8);
              mma16816<true>(acc[c + i], a0, a1, a2, a3, pb[t][0], pb[t][1]);
              if constexpr (GL == 8)
                mma16816<true>(acc[c + i], a0, a1, a2, a3, pl[t][0], pl[t][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * s);
    }

    // Sum up over the lanes: l over the tokens; o over the hi and lo columns,
    // which leaves head h0 + e's channels 16 c + 2 g + i in acc[c][2 i + e] of
    // the lanes t4 < kOwners.
#pragma unroll
    for (int e = 0; e < kE; ++e)
#pragma unroll
      for (int o = GL == 8 ? 4 : (GL == 4 ? 2 : 1); o < 32; o *= 2)
        l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], o);
    if constexpr (GL == 4) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[c][i] += __shfl_xor_sync(0xffffffffu, acc[c][i], 2);
    } else if constexpr (GL == 1) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) acc[c][0] += acc[c][1], acc[c][2] += acc[c][3];
    }
    constexpr int kOwners = GL == 8 ? 4 : (GL == 4 ? 2 : 1);

    // Warps 1-3 hand their states to warp 0, which merges them with its own
    // (ascending warp order) and writes the item's partial.
    // The barrier also tells that warp 0 is done with the merge area, and that all
    // have read the item's descriptor.
    if (consumers_any(aborted)) return;
    if (threadIdx.x == 0) mbar_arrive(dempty0 + 8 * slot);
#pragma unroll
    for (int turn = 0; turn < C::kTurns; ++turn) {
      // this turn's heads of the lane, and their row in a warp's part of the area
      const int e0 = C::kTurns == 2 ? turn : 0, e1 = C::kTurns == 2 ? turn + 1 : kE;
      const int row0 = C::kTurns == 2 ? t4 - turn : h0;  // (+ e)
      if (turn > 0) consumers_sync();  // warp 0 has read the turn before
      if (warp > 0 && t4 < kOwners) {
#pragma unroll
        for (int e = e0; e < e1; ++e) {
          float* r = mrg + ((warp - 1) * C::kMergeRows + row0 + e) * C::kMergeRow;
          if (g == 0) {
            r[D] = m_ref[e];
            r[D + 1] = l_run[e];
            r[D + 2] = r_ref[e];
          }
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            r[16 * c + 2 * g] = acc[c][e];
            r[16 * c + 2 * g + 1] = acc[c][2 + e];
          }
        }
      }
      consumers_sync();
      if (warp > 0 || t4 >= kOwners) continue;
#pragma unroll
      for (int e = e0; e < e1; ++e) {
        if (h0 + e >= a.G) continue;
        const float* rows = mrg + (row0 + e) * C::kMergeRow;  // of warp 1
        constexpr int kNext = C::kMergeRows * C::kMergeRow;   // to the next warp's
        float M = m_ref[e];
#pragma unroll
        for (int v = 1; v < kConsumerWarps; ++v) M = fmaxf(M, rows[(v - 1) * kNext + D]);
        // f: 2^(m - M + r), the weight of a warp's o (unset: 0, or o is 0)
        float f[kConsumerWarps];
        f[0] = exp2f((m_ref[e] - M) + r_ref[e]);
        float L = exp2f(m_ref[e] - M) * l_run[e];
#pragma unroll
        for (int v = 1; v < kConsumerWarps; ++v) {
          const float* r = rows + (v - 1) * kNext;
          f[v] = exp2f((r[D] - M) + r[D + 2]);
          L += exp2f(r[D] - M) * r[D + 1];
        }
        const int64_t row = static_cast<int64_t>(b) * a.Hq + kvh * a.G + h0 + e;
        const int64_t pi = row * a.n_chunks + chunk;
        float* po = a.part_o + pi * D;
        const int64_t oo = b * a.o_sb + (kvh * a.G + h0 + e) * a.o_sh;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          float2 O = make_float2(f[0] * acc[c][e], f[0] * acc[c][2 + e]);
          const int ch = 16 * c + 2 * g;
#pragma unroll
          for (int v = 1; v < kConsumerWarps; ++v) {
            const float* r = rows + (v - 1) * kNext + ch;
            O.x += f[v] * r[0];
            O.y += f[v] * r[1];
          }
          if (whole) {  // (an empty sequence: 0; NaN scores have their way)
            store_out(a.out, a.out_dtype, oo + ch, n_pages > 0 ? O.x / L : 0.f);
            store_out(a.out, a.out_dtype, oo + ch + 1, n_pages > 0 ? O.y / L : 0.f);
          } else {
            *reinterpret_cast<float2*>(po + ch) = O;
          }
        }
        if (g == 0 && !whole) {
          a.part_ml[2 * pi] = M > kUnset ? M : -INFINITY;
          a.part_ml[2 * pi + 1] = L;
        }
      }
    }
  }
}

// Resident CTAs per SM of one instantiation, at most Fp8Cfg::kCtas; computed once
// a device (the shared-memory limit is set per device too).
template <int D, bool F16, bool SPARSE, int GL>
cudaError_t ctas_per_sm_t(int* out) {
  using C = Fp8Cfg<D, GL>;
  static PerDevice known;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return per_device(known, dev, cudaSuccess, out, [](int* n) {
    auto kern = attn_fp8_kernel<D, F16, SPARSE, GL>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, kAttnThreads, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (*n < 1) return cudaErrorInvalidConfiguration;
    if (*n > C::kCtas) *n = C::kCtas;
    return cudaSuccess;
  });
}

template <int D, bool F16, bool SPARSE, int GL>
cudaError_t launch_t(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int num_sms,
                     cudaStream_t s) {
  int per_sm = 0;
  const cudaError_t e = ctas_per_sm_t<D, F16, SPARSE, GL>(&per_sm);
  if (e != cudaSuccess) return e;
  const int64_t want = static_cast<int64_t>(num_sms) * per_sm;
  const int grid = static_cast<int>(a.n_items < want ? a.n_items : want);
  return launch_pdl(attn_fp8_kernel<D, F16, SPARSE, GL>, dim3(grid), dim3(kAttnThreads),
                    Fp8Cfg<D, GL>::kSmemBytes, s, a, mk, mv);
}

// f.run<D, F16, SPARSE, GL>() for the run-time values, G query heads a kv head.
template <bool SPARSE, int GL, typename F>
cudaError_t dispatch_type(int d, bool f16, const F& f) {
  if (d == 128)
    return f16 ? f.template run<128, true, SPARSE, GL>() : f.template run<128, false, SPARSE, GL>();
  return f16 ? f.template run<64, true, SPARSE, GL>() : f.template run<64, false, SPARSE, GL>();
}
template <bool SPARSE, typename F>
cudaError_t dispatch_group(int G, int d, bool f16, const F& f) {
  if (G == 1) return dispatch_type<SPARSE, 1>(d, f16, f);
  return G <= 4 ? dispatch_type<SPARSE, 4>(d, f16, f) : dispatch_type<SPARSE, 8>(d, f16, f);
}
template <typename F>
cudaError_t dispatch(bool sparse, int G, int d, bool f16, const F& f) {
  return sparse ? dispatch_group<true>(G, d, f16, f) : dispatch_group<false>(G, d, f16, f);
}

struct Launch {
  const AttnArgs& a;
  const CUtensorMap &mk, &mv;
  int num_sms;
  cudaStream_t s;
  template <int D, bool F16, bool SPARSE, int GL>
  cudaError_t run() const {
    return launch_t<D, F16, SPARSE, GL>(a, mk, mv, num_sms, s);
  }
};
struct Ctas {
  int* out;
  template <int D, bool F16, bool SPARSE, int GL>
  cudaError_t run() const {
    return ctas_per_sm_t<D, F16, SPARSE, GL>(out);
  }
};

}  // namespace

cudaError_t launch_attn_fp8(int d, bool f16, bool sparse, const AttnArgs& a, const CUtensorMap& mk,
                            const CUtensorMap& mv, int num_sms, cudaStream_t s) {
  return dispatch(sparse, a.G, d, f16, Launch{a, mk, mv, num_sms, s});
}

cudaError_t attn_fp8_ctas_per_sm(int d, bool f16, bool sparse, int* out) {
  return dispatch(sparse, 8, d, f16, Ctas{out});  // the most shared memory
}

}  // namespace dkv
