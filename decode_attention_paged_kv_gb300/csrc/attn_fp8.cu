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
// usual running max m of the scores s (log2 units) and sum l of 2^(s - m), the
// output accumulates w = f * 2^((s - m) + (e - r)) with an integer r kept at
// ceil(max(s + e) - m), so the weights that meet the codes stay below 2 and
// the largest is near 1 whatever the scales are: a page of large values with
// little weight costs the others no bits.  s - m is exact near the maximum and
// e - r always, so a second maximum adds no rounding.  At the end of an item
// o = 2^r * sum w code, the usual partial.
//
// Structure as in the 16-bit kernel: a persistent grid pulls work items
// (batch, kv head, chunk of pages) from a counter; one producer warp streams
// pages by TMA tensor copies (one 16 x d byte box a tensor and page, d-byte
// swizzle) into per-warp sub-rings of shared-memory stages; four consumer warps
// compute.  Codes become fp16 in registers (exact: e4m3 is a subset of fp16):
//   * S = Q K^T: one ldmatrix word of lane (g, t4) is four consecutive channels
//     16 c + 4 t4 .. + 3 of token g, which two conversions turn into the B
//     fragment of k-step c; the query's A fragments take the same channel order.
//   * O += P V: one transposed ldmatrix word is the channel pair (2 g, 2 g + 1)
//     of tokens 2 t4 and 2 t4 + 1; a byte permute and two conversions make the B
//     fragments of two output tiles, the even and the odd channels of 16 c ..
//     16 c + 15 (output tile 2 c + e, column n is channel 16 c + 2 n + e).
// A bf16 query is scaled by a power of two per head so that its largest
// component lies in [2^14, 2^15): exact in fp16 for every component within 2^28
// of it; the scores are scaled back.  The weights are split into fp16 hi + lo
// (A rows 0-7 / 8-15), 22 significant bits.
//
// Every mbarrier wait is bounded; on expiry the kernel records a timeout in
// the status word, stops issuing, drains the copies it issued and exits.

#include <math.h>

#include "dkv_device.cuh"
#include "dkv_kernels.h"

namespace dkv {
namespace {

constexpr uint64_t kDrainLimitNs = 200000000ull;  // 200 ms for the whole drain
constexpr int kListPages = 128;                   // pages of an item listed at a time

struct ItemDesc {
  int item;     // work item, -1: no more work
  int n_pages;  // pages in the item
};

template <int D, bool MHA>
struct Fp8Cfg {
  // Three CTAs fit an SM where a thread needs at most 128 registers.
  static constexpr int kCtas = MHA || D == 64 ? 3 : 2;
  static constexpr int kPagesPerStage = 2;
  static constexpr int kTileBytes = kPage * D;      // one tensor's page of codes
  static constexpr int kSlotBytes = 2 * kTileBytes;  // K codes | V codes
  static constexpr int kStageBytes = kPagesPerStage * kSlotBytes;
  static constexpr int kRing = MHA ? 64 * 1024 : (D == 64 ? 48 * 1024 : 96 * 1024);
  static constexpr int kStages = kRing / kStageBytes;
  static constexpr int kSub = kStages / kConsumerWarps;    // stages per consumer warp
  static constexpr int kIssueLanes = kStages < 16 ? kStages : 16;
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kMetaOffset = kBarOffset + (2 * kStages + 4) * 8;
  static constexpr int kDescOffset = kMetaOffset + kStages * kPagesPerStage * 16;
  static constexpr int kMergeOffset = kDescOffset + 2 * 8;
  static constexpr int kMergeRow = D + 3;  // o[D], max m, sum l, exponent r
  static constexpr int kListOffset =
      (kMergeOffset + (kConsumerWarps - 1) * (MHA ? 1 : 8) * kMergeRow * 4 + 15) / 16 * 16;
  static constexpr int kBlockOffset = kListOffset + 16 * kListPages;
  static constexpr int kMiscOffset = kBlockOffset + 4 * kListPages;
  static constexpr int kSmemBytes = 1024 + kMiscOffset + 16;
  static_assert(kSlotBytes % 1024 == 0, "tiles keep the swizzle's alignment");
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
// beside the largest, which is at least 1).
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The largest of a warp's values (no NaN), in every lane: one integer reduction
// over order-preserving keys (a float's bits, the magnitude bits flipped when
// negative; the map is its own inverse).
__device__ __forceinline__ float warp_max(float x) {
  const int b = __float_as_int(x);
  const int k = __reduce_max_sync(0xffffffffu, b >= 0 ? b : b ^ 0x7fffffff);
  return __int_as_float(k >= 0 ? k : k ^ 0x7fffffff);
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

template <int D, bool F16, bool SPARSE, bool MHA>
__global__ void __launch_bounds__(kAttnThreads, MHA || D == 64 ? Fp8Cfg<D, MHA>::kCtas : 0)
    attn_fp8_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv) {
  using C = Fp8Cfg<D, MHA>;
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
  int4* list = reinterpret_cast<int4*>(smem + C::kListOffset);  // the same, of the item's pages
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
    const uint64_t pol = l2_evict_first_policy();
    const int my_w = lane & 3;  // consumer warp this lane feeds
    const bool issuer = lane < C::kIssueLanes;
    int wc = 0;           // stages issued so far to warp my_w
    bool failed = false;  // a lane gave up waiting for a free slot
    for (int k = 0;; ++k) {
      int item = 0, n = 0, b = 0, kvh = 0, first = 0, unit = 0;
      while (true) {
        if (lane == 0) item = static_cast<int>(atomicAdd(a.work_counter, 1u));
        item = __shfl_sync(0xffffffffu, item, 0);
        if (item >= a.n_items) {
          item = -1;
          n = 0;
          break;
        }
        const int chunk = item % a.n_chunks;
        unit = item / a.n_chunks;
        kvh = unit % a.Hkv;
        b = unit / a.Hkv;
        first = chunk * a.pages_per_chunk;
        const bool empty_seq = a.lens != nullptr && a.lens[b] <= 0;  // nothing to attend
        if constexpr (SPARSE) {
          if (unit_flags) {
            int rdy = 1;
            if (lane == 0) rdy = flag_wait_bounded(a.unit_ready + unit, a.wait_limit_ns, abort_flag);
            if (!__shfl_sync(0xffffffffu, rdy, 0)) {
              if (lane == 0 && *abort_flag == 0) {
                set_status(a.status, kStatusTimeout);
                *abort_flag = 1;
              }
              item = -1;  // stop: publish the end of work
              n = 0;
              break;
            }
          }
          n = max(0, min(__ldcg(a.union_count + unit) - first, a.pages_per_chunk));
        } else {
          const int Pb = static_cast<int>(ceil_div(seq_len_of(a.lens, b, a.N), kPage));
          n = max(0, min(Pb - first, a.pages_per_chunk));
        }
        if (empty_seq) n = 0;
        if (n == 0 && !whole) continue;  // no partial is read for it
        break;
      }
      const int slot = k & 1;
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
        desc[slot].item = item;
        desc[slot].n_pages = n;
        mbar_arrive(dfull0 + 8 * slot);  // release: consumers see the descriptor
      }
      if (item < 0) break;
      const float* ks = a.k8.scale + kvh * a.k8.sh;
      const float* vs = a.v8.scale + kvh * a.v8.sh;
      bool lok = true;
      for (int l0 = 0; l0 < n && lok; l0 += kListPages) {
        // The pages of this part of the item, with their scales and blocks:
        // one round of loads for all of them, while the ring still holds the
        // previous item's pages.
        const int ln = min(kListPages, n - l0);
        __syncwarp();
        for (int j = lane; j < ln; j += 32) {
          int page = first + l0 + j, mask = 0xff;
          if constexpr (SPARSE) {
            const int2 e = __ldcg(a.union_list + static_cast<int64_t>(unit) * a.union_stride +
                                  first + l0 + j);
            page = e.x;
            mask = e.y;
          }
          int64_t ko, vo;
          if (a.bt != nullptr) {
            // An entry outside [0, num_blocks) is clamped into it, so no copy
            // leaves the pool, and reported as a failed check.
            const int raw = a.bt[b * a.bts + page];
            if (raw < 0 || raw >= a.nblocks) set_status(a.status, kStatusCheck);
            const int blk = min(max(raw, 0), a.nblocks - 1);
            blocks[j] = blk;
            ko = blk * a.k8.sb;
            vo = blk * a.v8.sb;
          } else {
            ko = b * a.k8.sb + page;
            vo = b * a.v8.sb + page;
          }
          list[j] = make_int4(page, mask, __float_as_int(ks[ko]), __float_as_int(vs[vo]));
        }
        __syncwarp();
        for (int j0 = 0; j0 < ln; j0 += C::kIssueLanes * kQ) {
          const int j = j0 + lane * kQ;  // first page of this lane's stage
          if (issuer && j < ln) {
            const int c = wc + (j / kQ >> 2);            // (a list is a whole number of rounds)
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
              mbar_arrive_expect_tx(full0 + 8 * s, cnt * C::kSlotBytes);
#pragma unroll
              for (int t = 0; t < kQ; ++t) {
                if (t < cnt) {
                  // {channel, token, -, kv head, batch} of the cache, or
                  // {channel, token in block, -, kv head, block} of a pool
                  const uint32_t dst = sbase + s * C::kStageBytes + t * C::kSlotBytes;
                  const int y = a.bt != nullptr ? 0 : list[j + t].x * kPage;
                  const int z = a.bt != nullptr ? blocks[j + t] : b;
                  tma_load_5d_hint(dst, &mk, full0 + 8 * s, 0, y, 0, kvh, z, pol);
                  tma_load_5d_hint(dst + C::kTileBytes, &mv, full0 + 8 * s, 0, y, 0, kvh, z, pol);
                }
              }
            }
          }
          lok = __all_sync(0xffffffffu, lok);
          if (!lok) break;
        }
        const int nq = static_cast<int>(ceil_div(ln, kQ));  // stages of this part
        wc += nq > my_w ? (nq - my_w + 3) >> 2 : 0;
      }
      if (!__all_sync(0xffffffffu, lok)) {
        failed = true;
        break;
      }
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
    if (lane == 0) {
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
  const bool head_ok = MHA || g < a.G;
  const int mtx = lane >> 3, mrow = lane & 7;
  // Channel of output tile cn, column 2 t4 + e.
  auto out_channel = [t4](int cn, int e) { return 16 * (cn >> 1) + 4 * t4 + 2 * e + (cn & 1); };
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

    // The query's A fragments: k-step c of lane (g, t4) is channels
    // 16 c + 4 t4 .. + 3 of head g (row 8 + g is unused), in fp16.
    uint32_t qa[D / 16][2];
    float qscale = a.scale_log2;
    {
      const uint16_t* qrow = static_cast<const uint16_t*>(a.q) + b * a.q_sb +
                             static_cast<int64_t>(kvh * a.G + (head_ok && !MHA ? g : 0)) * a.q_sh +
                             4 * t4;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint2 w = head_ok ? *reinterpret_cast<const uint2*>(qrow + 16 * c) : make_uint2(0u, 0u);
        qa[c][0] = w.x;
        qa[c][1] = w.y;
      }
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
        qscale *= __int_as_float((127 - up) << 23);
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qa[c][i] = pack2<true>(lo16<false>(qa[c][i]) * f, hi16<false>(qa[c][i]) * f);
      }
    }
    float m_run = -INFINITY, mv_run = -INFINITY, r_run = 0.f, l_run = 0.f;
    constexpr int kAccTiles = MHA ? D / 16 : D / 8;
    float acc[kAccTiles][4];
#pragma unroll
    for (int cn = 0; cn < kAccTiles; ++cn) acc[cn][0] = acc[cn][1] = acc[cn][2] = acc[cn][3] = 0.f;

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

      if constexpr (MHA) {
        // S = K q, the query in every column: lane (g, t4) gets the scores of
        // tokens g (d[0]) and g + 8 (d[2]) of both pages and keeps one of the
        // 32: token g + 8 (t4 & 1) of page t4 >> 1.
        float sc[kQ][4];
#pragma unroll
        for (int t = 0; t < kQ; ++t) {
          sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
          if (t < cnt) {
#pragma unroll
            for (int c = 0; c < D / 16; c += 2) {
              uint32_t r[4];  // [chunk c, c + 1][tokens 0-7, 8-15]
              ldsm_x4(code_addr<D>(st + t * C::kSlotBytes, 8 * (mtx & 1) + mrow, c + (mtx >> 1)),
                      r[0], r[1], r[2], r[3]);
#pragma unroll
              for (int i = 0; i < 2; ++i)
                mma16816<true>(sc[t], e4m3_lo2(r[2 * i]), e4m3_lo2(r[2 * i + 1]),
                               e4m3_hi2(r[2 * i]), e4m3_hi2(r[2 * i + 1]), qa[c + i][0],
                               qa[c + i][1]);
            }
          }
        }
        const int4 meta = stage_meta[s * kQ + (t4 >> 1)];
        const bool mine = (t4 >> 1) < cnt;
        const int in_page = g + 8 * (t4 & 1);
        const int sl = SPARSE ? a.sub_log2 : 0;
        const bool on = !SPARSE || ((meta.y >> (sl ? in_page >> (4 - sl) : 0)) & 1);
        const bool past = mine && meta.x * kPage + in_page >= Nb;
        const float raw = (t4 & 2) ? ((t4 & 1) ? sc[1][2] : sc[1][0])
                                   : ((t4 & 1) ? sc[0][2] : sc[0][0]);
        const float sv = mine && on && !past ? raw * (qscale * __int_as_float(meta.z)) : -INFINITY;
        // vs = 2^ve * vf (a scale below 2^-126 counts as 0)
        const uint32_t vb = static_cast<uint32_t>(meta.w);
        const int ex = (vb >> 23) & 0xff;
        const float ve = static_cast<float>(ex - 127);
        const float vf = ex == 0 ? 0.f : __uint_as_float((vb & 0x807fffffu) | 0x3f800000u);
        const float m_new = fmaxf(m_run, warp_max(sv));
        const float mv_new = fmaxf(mv_run, warp_max(sv + ve));
        const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
        const float r_new = (m_new == -INFINITY) ? 0.f : ceilf(mv_new - m_new);
        const float x = sv - m_use;
        const float down = m_run - m_use;
        l_run = l_run * exp2_fast(down) + exp2_fast(x);  // (this lane's tokens)
        if (m_new != m_run || r_new != r_run) {          // warp-uniform
          const float alpha = exp2_fast(down + (r_run - r_new));
#pragma unroll
          for (int cn = 0; cn < kAccTiles; ++cn) {
            acc[cn][0] *= alpha;
            acc[cn][1] *= alpha;
            acc[cn][2] *= alpha;
            acc[cn][3] *= alpha;
          }
        }
        m_run = m_new;
        mv_run = mv_new;
        r_run = r_new;
        if (__any_sync(0xffffffffu, past)) {
          // Slots past the sequence's end hold anything: zero those V codes
          // (their weights are 0, but 0 * NaN is not).
          for (int t = 0; t < cnt; ++t) {
            const int nt = min(kPage, Nb - stage_meta[s * kQ + t].x * kPage);
            uint8_t* vt = smem + s * C::kStageBytes + t * C::kSlotBytes + C::kTileBytes;
            for (int i = lane; i < (kPage - nt) * (D / 16); i += 32)
              *reinterpret_cast<uint4*>(vt + nt * D + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          // (before the slot goes back to the copy engine)
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        // The weight as two fp16 halves, hi below lo.  O^T += V^T P: B holds the
        // hi halves in even columns and the lo halves in odd ones (columns 0 and
        // 1 are read at the end).
        const float w = exp2_fast(x + (ve - r_run)) * vf;
        const __half wh = __float2half_rn(w);
        const __half2 w2 = __halves2half2(wh, __float2half_rn(w - __half2float(wh)));
        const uint32_t wp = *reinterpret_cast<const uint32_t*>(&w2);
        const uint32_t pick = (g & 1) ? 0x7632u : 0x5410u;
#pragma unroll
        for (int t = 0; t < kQ; ++t) {
          // tokens 2 t4, 2 t4 + 1 (b0) and 2 t4 + 8, 2 t4 + 9 (b1) of page t
          const int src = 8 * t4 + 2 * t;
          const uint32_t w0 = __shfl_sync(0xffffffffu, wp, src);
          const uint32_t w1 = __shfl_sync(0xffffffffu, wp, src + 4);
          const uint32_t w8 = __shfl_sync(0xffffffffu, wp, src + 1);
          const uint32_t w9 = __shfl_sync(0xffffffffu, wp, src + 5);
          if (t < cnt) {
            const uint32_t b0 = __byte_perm(w0, w1, pick), b1 = __byte_perm(w8, w9, pick);
            const uint32_t vt = st + t * C::kSlotBytes + C::kTileBytes;
#pragma unroll
            for (int c = 0; c < D / 16; c += 2) {
              uint32_t r[4];  // [chunk c, c + 1][tokens 0-7, 8-15]
              ldsm_x4_trans(code_addr<D>(vt, 8 * (mtx & 1) + mrow, c + (mtx >> 1)), r[0], r[1],
                            r[2], r[3]);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                // rows: the even (g) and the odd (g + 8) channels of the chunk
                const uint32_t y0 = __byte_perm(r[2 * i], 0u, 0x3120);
                const uint32_t y8 = __byte_perm(r[2 * i + 1], 0u, 0x3120);
                mma16816<true>(acc[c + i], e4m3_lo2(y0), e4m3_hi2(y0), e4m3_lo2(y8), e4m3_hi2(y8),
                               b0, b1);
              }
            }
          }
        }
      } else {
      // S = Q K^T: sc[t][h][e] = score of head g, page t's token 8 h + 2 t4 + e.
      float sc[kQ][2][4];
#pragma unroll
      for (int t = 0; t < kQ; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) sc[t][h][0] = sc[t][h][1] = sc[t][h][2] = sc[t][h][3] = 0.f;
        if (t < cnt) {
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t r[4];  // [chunk c, c + 1][tokens 0-7, 8-15]
            ldsm_x4(code_addr<D>(st + t * C::kSlotBytes, 8 * (mtx & 1) + mrow, c + (mtx >> 1)),
                    r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                mma16816<true>(sc[t][h], qa[c + i][0], 0u, qa[c + i][1], 0u, e4m3_lo2(r[2 * i + h]),
                               e4m3_hi2(r[2 * i + h]));
          }
        }
      }

      // Scores in log2 units, masked; the two running maxima.  Token t of a
      // page counts for head g if bit (g << sub_log2) + (t >> (4 - sub_log2))
      // of its mask is set.
      const int sl = SPARSE ? a.sub_log2 : 0;
      float sv[kQ][4], ve[kQ], vf[kQ];
      float pmax = -INFINITY, vmax = -INFINITY;
#pragma unroll
      for (int t = 0; t < kQ; ++t) {
        const int4 meta = t < cnt ? stage_meta[s * kQ + t] : make_int4(0, 0, 0, 0);
        const uint32_t hmask = static_cast<uint32_t>(meta.y);
        const uint32_t hbits =
            head_ok ? (hmask >> ((g << sl) + (sl == 2 ? (t4 >> 1) : 0))) : 0u;
        const bool on_lo = hbits & 1u, on_hi = (hbits >> sl) & 1u;
        const float f = qscale * __int_as_float(meta.z);
        // vs = 2^ve * vf (a scale below 2^-126 counts as 0)
        const uint32_t vb = static_cast<uint32_t>(meta.w);
        const int ex = (vb >> 23) & 0xff;
        ve[t] = static_cast<float>(ex - 127);
        vf[t] = ex == 0 ? 0.f : __uint_as_float((vb & 0x807fffffu) | 0x3f800000u);
        float tmax = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = meta.x * kPage + 8 * (e >> 1) + 2 * t4 + (e & 1);
          const bool on = e < 2 ? on_lo : on_hi;
          sv[t][e] = (on && tok < Nb) ? sc[t][e >> 1][e & 1] * f : -INFINITY;
          tmax = fmaxf(tmax, sv[t][e]);
        }
        pmax = fmaxf(pmax, tmax);
        vmax = fmaxf(vmax, tmax + ve[t]);
      }
      pmax = fmaxf(pmax, __shfl_xor_sync(0xffffffffu, pmax, 1));
      vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 1));
      pmax = fmaxf(pmax, __shfl_xor_sync(0xffffffffu, pmax, 2));
      vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 2));
      const float m_new = fmaxf(m_run, pmax), mv_new = fmaxf(mv_run, vmax);
      // (mv is -inf exactly when m is: no token yet)
      const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
      const float r_new = (m_new == -INFINITY) ? 0.f : ceilf(mv_new - m_new);
      float psum = 0.f;
#pragma unroll
      for (int t = 0; t < kQ; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sv[t][e] -= m_use;
          psum += exp2_fast(sv[t][e]);
        }
      const float down = m_run - m_use;
      l_run = l_run * exp2_fast(down) + psum;
      if (__any_sync(0xffffffffu, m_new != m_run || r_new != r_run)) {
        const float alpha = exp2_fast(down + (r_run - r_new));
#pragma unroll
        for (int cn = 0; cn < D / 8; ++cn) {
          acc[cn][0] *= alpha;
          acc[cn][1] *= alpha;
          acc[cn][2] *= alpha;
          acc[cn][3] *= alpha;
        }
      }
      m_run = m_new;
      mv_run = mv_new;
      r_run = r_new;

      // O += P V, with P = hi + lo (A rows 0-7 and 8-15).
#pragma unroll
      for (int t = 0; t < kQ; ++t) {
        if (t < cnt) {
          const uint32_t vb = st + t * C::kSlotBytes + C::kTileBytes;
          const int page = stage_meta[s * kQ + t].x;
          if ((page + 1) * kPage > Nb) {
            // Slots past the sequence's end hold anything: zero those V codes
            // (their weights are 0, but 0 * NaN is not).
            const int nt = Nb - page * kPage;
            uint8_t* vt = smem + s * C::kStageBytes + t * C::kSlotBytes + C::kTileBytes;
            for (int i = lane; i < (kPage - nt) * (D / 16); i += 32)
              *reinterpret_cast<uint4*>(vt + nt * D + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            // (before the slot goes back to the copy engine)
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          const float shift = ve[t] - r_run;
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = exp2_fast(sv[t][e] + shift) * vf[t];
          uint32_t a0, a1, a2, a3;
          split_pair<true>(w[0], w[1], a0, a1);
          split_pair<true>(w[2], w[3], a2, a3);
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t r[4];  // [chunk c, c + 1][tokens 0-7, 8-15]
            ldsm_x4_trans(code_addr<D>(vb, 8 * (mtx & 1) + mrow, c + (mtx >> 1)), r[0], r[1], r[2],
                          r[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // bytes (token 2 t4: even, odd; token 2 t4 + 1: even, odd channel)
              // to (even, even; odd, odd)
              const uint32_t x = __byte_perm(r[2 * i], 0u, 0x3120);
              const uint32_t y = __byte_perm(r[2 * i + 1], 0u, 0x3120);
              mma16816<true>(acc[2 * (c + i)], a0, a1, a2, a3, e4m3_lo2(x), e4m3_lo2(y));
              mma16816<true>(acc[2 * (c + i) + 1], a0, a1, a2, a3, e4m3_hi2(x), e4m3_hi2(y));
            }
          }
        }
      }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * s);
    }

    if constexpr (MHA) {
#pragma unroll
      for (int o = 1; o < 32; o *= 2) l_run += __shfl_xor_sync(0xffffffffu, l_run, o);
      if (consumers_any(aborted)) return;
      // Lanes (g, 0): channels 16 c + 2 g (d[0] + d[1]) and + 1 (d[2] + d[3]).
      // Warps 1-3 hand their states to warp 0, which merges them with its own
      // (ascending warp order) and writes the item's partial.
      if (warp > 0) {
        float* r = mrg + (warp - 1) * C::kMergeRow;
        if (lane == 0) {
          r[D] = m_run;
          r[D + 1] = l_run;
          r[D + 2] = r_run;
        }
        if (t4 == 0) {
#pragma unroll
          for (int cn = 0; cn < kAccTiles; ++cn) {
            r[16 * cn + 2 * g] = acc[cn][0] + acc[cn][1];
            r[16 * cn + 2 * g + 1] = acc[cn][2] + acc[cn][3];
          }
        }
      }
      consumers_sync();
      if (warp == 0) {
        float M = m_run;
#pragma unroll
        for (int w = 1; w < kConsumerWarps; ++w) M = fmaxf(M, mrg[(w - 1) * C::kMergeRow + D]);
        // f: 2^(m - M + r), the weight of a warp's o
        float f[kConsumerWarps];
        f[0] = (m_run == -INFINITY) ? 0.f : exp2f((m_run - M) + r_run);
        float L = (m_run == -INFINITY) ? 0.f : exp2f(m_run - M) * l_run;
#pragma unroll
        for (int w = 1; w < kConsumerWarps; ++w) {
          const float* r = mrg + (w - 1) * C::kMergeRow;
          f[w] = (r[D] == -INFINITY) ? 0.f : exp2f((r[D] - M) + r[D + 2]);
          L += (r[D] == -INFINITY) ? 0.f : exp2f(r[D] - M) * r[D + 1];
        }
        const int64_t pi = (static_cast<int64_t>(b) * a.Hq + kvh) * a.n_chunks + chunk;
        float* po = a.part_o + pi * D;
        const int64_t oo = b * a.o_sb + kvh * a.o_sh;
        if (t4 == 0) {
#pragma unroll
          for (int cn = 0; cn < kAccTiles; ++cn) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c = 16 * cn + 2 * g + e;
              float O = f[0] * (acc[cn][2 * e] + acc[cn][2 * e + 1]);
#pragma unroll
              for (int w = 1; w < kConsumerWarps; ++w) O += f[w] * mrg[(w - 1) * C::kMergeRow + c];
              if (whole)
                store_out(a.out, a.out_dtype, oo + c, L > 0.f ? O / L : 0.f);  // (no token: 0)
              else
                po[c] = O;
            }
          }
        }
        if (lane == 0 && !whole) {
          a.part_ml[2 * pi] = M;
          a.part_ml[2 * pi + 1] = L;
        }
      }
    } else {
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
    l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);

    // Warps 1-3 hand their states to warp 0, which merges them with its own
    // (ascending warp order) and writes the item's partial.
    if (consumers_any(aborted)) return;
    if (warp > 0) {
      float* r = mrg + ((warp - 1) * 8 + g) * C::kMergeRow;
      if (t4 == 0) {
        r[D] = m_run;
        r[D + 1] = l_run;
        r[D + 2] = r_run;
      }
#pragma unroll
      for (int cn = 0; cn < D / 8; ++cn) {
        r[out_channel(cn, 0)] = acc[cn][0] + acc[cn][2];
        r[out_channel(cn, 1)] = acc[cn][1] + acc[cn][3];
      }
    }
    consumers_sync();
    if (warp == 0 && head_ok) {
      float M = m_run;
#pragma unroll
      for (int w = 1; w < kConsumerWarps; ++w)
        M = fmaxf(M, mrg[((w - 1) * 8 + g) * C::kMergeRow + D]);
      // f: 2^(m - M + r), the weight of a warp's o
      float f[kConsumerWarps];
      f[0] = (m_run == -INFINITY) ? 0.f : exp2f((m_run - M) + r_run);
      float L = (m_run == -INFINITY) ? 0.f : exp2f(m_run - M) * l_run;
#pragma unroll
      for (int w = 1; w < kConsumerWarps; ++w) {
        const float* r = mrg + ((w - 1) * 8 + g) * C::kMergeRow;
        f[w] = (r[D] == -INFINITY) ? 0.f : exp2f((r[D] - M) + r[D + 2]);
        L += (r[D] == -INFINITY) ? 0.f : exp2f(r[D] - M) * r[D + 1];
      }
      const int64_t pi = (static_cast<int64_t>(b) * a.Hq + kvh * a.G + g) * a.n_chunks + chunk;
      float* po = a.part_o + pi * D;
      const int64_t oo = b * a.o_sb + (kvh * a.G + g) * a.o_sh;
#pragma unroll
      for (int cn = 0; cn < D / 8; ++cn) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = out_channel(cn, e);
          float O = f[0] * (acc[cn][e] + acc[cn][2 + e]);
#pragma unroll
          for (int w = 1; w < kConsumerWarps; ++w)
            O += f[w] * mrg[((w - 1) * 8 + g) * C::kMergeRow + c];
          if (whole)
            store_out(a.out, a.out_dtype, oo + c, L > 0.f ? O / L : 0.f);  // (no token: 0)
          else
            po[c] = O;
        }
      }
      if (t4 == 0 && !whole) {
        a.part_ml[2 * pi] = M;
        a.part_ml[2 * pi + 1] = L;
      }
    }
    }
    consumers_sync();  // merge area free again; the descriptor slot was read by all
    if (threadIdx.x == 0) mbar_arrive(dempty0 + 8 * slot);
  }
}

// Resident CTAs per SM of one instantiation, at most Fp8Cfg::kCtas; computed once.
template <int D, bool F16, bool SPARSE, bool MHA>
cudaError_t ctas_per_sm_t(int* out) {
  using C = Fp8Cfg<D, MHA>;
  static int cached = 0;  // benign race: every thread computes the same value
  if (cached > 0) {
    *out = cached;
    return cudaSuccess;
  }
  auto kern = attn_fp8_kernel<D, F16, SPARSE, MHA>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  int n = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kAttnThreads, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  if (n < 1) return cudaErrorInvalidConfiguration;
  cached = n < C::kCtas ? n : C::kCtas;
  *out = cached;
  return cudaSuccess;
}

template <int D, bool F16, bool SPARSE, bool MHA>
cudaError_t launch_t(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int num_sms,
                     cudaStream_t s) {
  int per_sm = 0;
  const cudaError_t e = ctas_per_sm_t<D, F16, SPARSE, MHA>(&per_sm);
  if (e != cudaSuccess) return e;
  const int64_t want = static_cast<int64_t>(num_sms) * per_sm;
  const int grid = static_cast<int>(a.n_items < want ? a.n_items : want);
  return launch_pdl(attn_fp8_kernel<D, F16, SPARSE, MHA>, dim3(grid), dim3(kAttnThreads),
                    Fp8Cfg<D, MHA>::kSmemBytes, s, a, mk, mv);
}

// One call of f.template run<D, F16, SPARSE, MHA>() for the run-time values.
template <typename F>
cudaError_t dispatch(int d, bool f16, bool sparse, bool mha, const F& f) {
  const int key = (d == 128 ? 8 : 0) + (f16 ? 4 : 0) + (sparse ? 2 : 0) + (mha ? 1 : 0);
  switch (key) {
    case 0: return f.template run<64, false, false, false>();
    case 1: return f.template run<64, false, false, true>();
    case 2: return f.template run<64, false, true, false>();
    case 3: return f.template run<64, false, true, true>();
    case 4: return f.template run<64, true, false, false>();
    case 5: return f.template run<64, true, false, true>();
    case 6: return f.template run<64, true, true, false>();
    case 7: return f.template run<64, true, true, true>();
    case 8: return f.template run<128, false, false, false>();
    case 9: return f.template run<128, false, false, true>();
    case 10: return f.template run<128, false, true, false>();
    case 11: return f.template run<128, false, true, true>();
    case 12: return f.template run<128, true, false, false>();
    case 13: return f.template run<128, true, false, true>();
    case 14: return f.template run<128, true, true, false>();
    default: return f.template run<128, true, true, true>();
  }
}

struct Launch {
  const AttnArgs& a;
  const CUtensorMap &mk, &mv;
  int num_sms;
  cudaStream_t s;
  template <int D, bool F16, bool SPARSE, bool MHA>
  cudaError_t run() const {
    return launch_t<D, F16, SPARSE, MHA>(a, mk, mv, num_sms, s);
  }
};
struct Ctas {
  int* out;
  template <int D, bool F16, bool SPARSE, bool MHA>
  cudaError_t run() const {
    return ctas_per_sm_t<D, F16, SPARSE, MHA>(out);
  }
};

}  // namespace

cudaError_t launch_attn_fp8(int d, bool f16, bool sparse, const AttnArgs& a, const CUtensorMap& mk,
                            const CUtensorMap& mv, int num_sms, cudaStream_t s) {
  // one query head per kv head: the single-head layout
  return dispatch(d, f16, sparse, a.G == 1, Launch{a, mk, mv, num_sms, s});
}

cudaError_t attn_fp8_ctas_per_sm(int d, bool f16, bool sparse, int* out) {
  return dispatch(d, f16, sparse, false, Ctas{out});
}

}  // namespace dkv
