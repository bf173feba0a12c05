// pages.cu -- the blocks of paged caches: rows of a block table that continue, fork,
// grow and end (fork), and a pool whose blocks in use move to its front (compact).
//
// Everything is whole numbers and copies, so results are exact, and they do not depend
// on the order in which CTAs run: blocks are taken in ascending order by prefix sums,
// and counts of references change by integer atomics.
//
// fork, two kernels.  fork_plan_kernel: CTA 0 finds each parent's lowest child (which
// keeps a last page that is not whole), counts the pages that every row takes, and
// lists the lowest free blocks; the other CTAs, one a row, keep a copy of the table --
// rows are replaced in place while others still read them -- and check the entries
// that will be continued.  fork_apply_kernel: writes the rows, the reference counts of
// entries that change, and copies the last pages.  A plan that fails leaves a flag that
// the second kernel reads first, so a call changes everything or nothing.
//
// compact, three kernels: counts of blocks in use per chunk; ranks of the moves' ends
// (the k-th block in use at or past n goes to the k-th free one below n, n the number
// in use); the copies, 16 KB an item, and the table's new names.
//
// Measured on a GB300: a step of 64 beams over 32K-token contexts (two pools, 8 KB a block)
// 9.5 us, of four beams 8 us beside the caller's own work: two launches, each a chain of
// four to six dependent loads (parents - lengths - table - counts; plan - table - blocks).
// A gigabyte pool half in use compacted (268 MB moved) 91 us, 81 of them the copies at 6.6
// TB/s both ways (99 with 4096 counts a CTA in the ranks' kernel), 7 MB 10 us.

#include "dkv_device.cuh"
#include "dkv_kernels.h"
#include "pages.h"

namespace dkv {
namespace {

constexpr int kPlanThreads = 1024, kThreads = 256;
constexpr int kFail = 16, kExit = 17;  // words of the workspace header, 0 between calls

__device__ __forceinline__ int4 ld4(const int32_t* p) {
  return *reinterpret_cast<const int4*>(p);
}

// Exclusive prefix sum of v over the CTA; *total receives the sum.
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += up;
  }
  __syncthreads();  // the sums of an earlier scan have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < THREADS / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += up;
    }
    if (lane < THREADS / 32) warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[THREADS / 32 - 1];
  return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

__device__ __forceinline__ int pages_of(int64_t tokens, int block) {
  return static_cast<int>((tokens + block - 1) / block);
}

__device__ void plan_rows(const ForkArgs& a, int* first, int* sums) {
  const PagesArgs& g = a.g;
  const int tid = threadIdx.x;
  const int64_t room = static_cast<int64_t>(g.cols) * g.block;
  bool bad = false;
  for (int b = tid; b < g.rows; b += kPlanThreads) first[b] = g.rows;
  __syncthreads();
  for (int b = tid; b < g.rows; b += kPlanThreads) {
    const int p = a.parents != nullptr ? a.parents[b] : b;
    if (p < -1 || p >= g.rows)
      bad = true;
    else if (p >= 0)
      atomicMin(&first[p], b);
  }
  __syncthreads();
  int need = 0;
  for (int b0 = 0; b0 < g.rows; b0 += kPlanThreads) {
    const int b = b0 + tid;
    RowPlan r{-1, 0, 0, 0, 0, 0, {0, 0}};
    if (b < g.rows) {
      const int p = a.parents != nullptr ? a.parents[b] : b;
      const int64_t kept = p >= 0 && p < g.rows ? a.lens[p] : 0;
      const int64_t fresh = a.news != nullptr ? a.news[b] : 0;
      if (kept < 0 || fresh < 0 || kept + fresh > room) {
        bad = true;
      } else {
        r.parent = p;
        r.whole = static_cast<int>(kept / g.block);
        r.pages = pages_of(kept, g.block);
        r.end = pages_of(kept + fresh, g.block);
        if (r.pages > r.whole) {
          const int last = g.table[p * g.ts + r.whole];
          if (last < 0 || last >= g.nb)
            bad = true;
          else
            r.copied = first[p] != b || g.refs[last] > 1;
        }
      }
    }
    int total;
    const int mine = r.end - r.pages + r.copied;
    r.fresh = need + block_scan<kPlanThreads>(mine, sums, &total);
    // (a table of more entries than 2^31 is refused, so the sum cannot wrap)
    need += total;
    if (b < g.rows) a.plan[b] = r;
  }
  // the lowest free blocks, 8 counts a thread at a time
  int found = 0;
  for (int64_t i0 = 0; i0 < g.nb && found < need; i0 += 8 * kPlanThreads) {
    const int64_t i = i0 + 8 * tid;
    uint32_t free = 0;
    if (i + 8 <= g.nb) {
      const int4 u = ld4(g.refs + i), v = ld4(g.refs + i + 4);
      free = (u.x == 0) | (u.y == 0) << 1 | (u.z == 0) << 2 | (u.w == 0) << 3 | (v.x == 0) << 4 |
             (v.y == 0) << 5 | (v.z == 0) << 6 | (v.w == 0) << 7;
    } else {
      for (int k = 0; k < 8 && i + k < g.nb; ++k) free |= (g.refs[i + k] == 0) << k;
    }
    int total;
    int at = found + block_scan<kPlanThreads>(__popc(free), sums, &total);
    for (; free != 0 && at < need; free &= free - 1)
      a.taken[at++] = static_cast<int32_t>(i) + __ffs(free) - 1;
    found += total;
  }
  bad |= found < need;
  if (__syncthreads_or(bad) && tid == 0) {
    g.status[kFail] = 1;
    set_status(g.status, kStatusCheck);
  }
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkArgs a) {
  extern __shared__ int first[];  // [rows], CTA 0
  __shared__ int sums[32];
  griddep_launch_dependents();
  griddep_wait();
  const PagesArgs& g = a.g;
  if (blockIdx.x == 0) {
    plan_rows(a, first, sums);
    return;
  }
  const int row = blockIdx.x - 1;
  bool child = a.parents == nullptr;
  if (!child)
    for (int b = threadIdx.x; b < g.rows; b += kPlanThreads) child |= a.parents[b] == row;
  child = __syncthreads_or(child);
  // (a length below 0 or past the table is CTA 0's to report)
  const int64_t len = child ? a.lens[row] : 0;
  const int pages = static_cast<int>(min(static_cast<int64_t>(g.cols),
                                         (max(len, int64_t{0}) + g.block - 1) / g.block));
  bool bad = false;
  for (int j = threadIdx.x; j < g.cols; j += kPlanThreads) {
    const int e = g.table[row * g.ts + j];
    a.snap[static_cast<int64_t>(row) * g.cols + j] = e;
    bad |= j < pages && (e < 0 || e >= g.nb);
  }
  if (bad) {
    g.status[kFail] = 1;
    set_status(g.status, kStatusCheck);
  }
}

// Copies n bytes of block src to block dst of a pool, from byte `at` on, a CTA's part
// of a step at a time: `step` bytes from one turn of a thread to its next.
template <typename V>
__device__ __forceinline__ void copy_piece(const PoolView& pool, int src, int dst, int64_t at,
                                           int64_t n, int64_t step) {
  const V* from = reinterpret_cast<const V*>(pool.p + src * pool.stride + at);
  V* to = reinterpret_cast<V*>(pool.p + dst * pool.stride + at);
  const int64_t count = n / static_cast<int64_t>(sizeof(V)), by = step / static_cast<int64_t>(sizeof(V));
  int64_t i = threadIdx.x;
  for (; i + 3 * by < count; i += 4 * by) {
    const V x = from[i], y = from[i + by], z = from[i + 2 * by], w = from[i + 3 * by];
    to[i] = x, to[i + by] = y, to[i + 2 * by] = z, to[i + 3 * by] = w;
  }
  for (; i < count; i += by) to[i] = from[i];
}

__global__ void __launch_bounds__(kThreads) fork_apply_kernel(const ForkArgs a) {
  __shared__ int fail;
  griddep_launch_dependents();
  griddep_wait();
  const PagesArgs& g = a.g;
  if (threadIdx.x == 0) fail = *reinterpret_cast<volatile uint32_t*>(g.status + kFail) != 0;
  __syncthreads();
  const int b = blockIdx.y, slice = blockIdx.x;
  if (!fail) {
    const RowPlan r = a.plan[b];
    const int32_t* was = a.snap + static_cast<int64_t>(b) * g.cols;
    const int32_t* from = a.snap + static_cast<int64_t>(max(r.parent, 0)) * g.cols;
    for (int j = slice * kThreads + threadIdx.x; j < g.cols; j += a.slices * kThreads) {
      const int old = was[j];
      int now = -1;
      if (j < r.whole || (j < r.pages && !r.copied))
        now = from[j];
      else if (j < r.end)
        now = a.taken[r.fresh + j - r.pages + r.copied];
      if (now == old) continue;
      g.table[b * g.ts + j] = now;
      if (old >= 0 && old < g.nb) atomicSub(g.refs + old, 1);
      if (now >= 0) atomicAdd(g.refs + now, 1);
    }
    if (r.copied) {
      const int src = from[r.whole], dst = a.taken[r.fresh];
      // 16 bytes a thread of every slice in turn
      for (int i = 0; i < g.npools; ++i) {
        const PoolView& pool = g.pool[i];
        const int64_t unit = kThreads * (pool.wide ? 16 : 4);
        if (slice * unit >= pool.bytes) continue;
        if (pool.wide)
          copy_piece<uint4>(pool, src, dst, slice * unit, pool.bytes - slice * unit,
                            a.slices * unit);
        else
          copy_piece<uint32_t>(pool, src, dst, slice * unit, pool.bytes - slice * unit,
                               a.slices * unit);
      }
    }
  }
  // the last CTA leaves the header as it was
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(g.status + kExit, 1u) == gridDim.x * gridDim.y - 1) {
    g.status[kFail] = 0;
    g.status[kExit] = 0;
  }
}

// ------------------------------------------------------------------- compact
constexpr int kPer = kCompactChunk / kThreads;  // counts a thread
static_assert(kPer == 4, "a vector a thread");

// The thread's four counts from index `at` on; past the end -1.
__device__ __forceinline__ int4 four_refs(const PagesArgs& g, int64_t at) {
  if (at + 4 <= g.nb) return ld4(g.refs + at);
  int4 r = make_int4(-1, -1, -1, -1);
  if (at < g.nb) r.x = g.refs[at];
  if (at + 1 < g.nb) r.y = g.refs[at + 1];
  if (at + 2 < g.nb) r.z = g.refs[at + 2];
  return r;
}
__device__ __forceinline__ int live_of(const int4& r) {
  return (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
}

__global__ void __launch_bounds__(kThreads) compact_count_kernel(const CompactArgs a) {
  __shared__ int sums[32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kCompactChunk + threadIdx.x * kPer;
  int total;
  block_scan<kThreads>(live_of(four_refs(a.g, at)), sums, &total);
  if (threadIdx.x == 0) a.counts[blockIdx.x] = total;
}

// Sums of x and y over the CTA.
__device__ __forceinline__ int2 block_sum2(int x, int y, int2* warp_sums) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
  }
  if (threadIdx.x % 32 == 0) warp_sums[threadIdx.x / 32] = make_int2(x, y);
  __syncthreads();
  int2 s = make_int2(0, 0);
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s.x += warp_sums[i].x, s.y += warp_sums[i].y;
  return s;
}

__global__ void __launch_bounds__(kThreads) compact_rank_kernel(const CompactArgs a) {
  __shared__ int sums[32];
  __shared__ int2 pairs[2][kThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const PagesArgs& g = a.g;
  const int tid = threadIdx.x, chunk = blockIdx.x, chunks = gridDim.x;
  const int64_t at = static_cast<int64_t>(chunk) * kCompactChunk + tid * kPer;
  const int4 refs = four_refs(g, at);  // (before anything is written)
  int part = 0, all = 0;
  for (int c = tid; c < chunks; c += kThreads) {
    const int x = a.counts[c];
    all += x;
    if (c < chunk) part += x;
  }
  const int2 s = block_sum2(part, all, pairs[0]);
  const int before = s.x, n = s.y;
  // blocks in use below n: whole chunks, and part of the one that n lies in
  int below = 0;
  for (int c = tid; c < n / kCompactChunk; c += kThreads) below += a.counts[c];
  const int64_t edge = static_cast<int64_t>(n / kCompactChunk) * kCompactChunk + tid * kPer;
  if (edge < n) {
    const int4 r = four_refs(g, edge);
    below += (r.x > 0) + (edge + 1 < n && r.y > 0) + (edge + 2 < n && r.z > 0) +
             (edge + 3 < n && r.w > 0);
  }
  const int kept = block_sum2(below, 0, pairs[1]).x;
  if (chunk == 0 && tid == 0) {
    a.totals[0] = n;
    a.totals[1] = n - kept;
  }
  int unused;
  int rank = before + block_scan<kThreads>(live_of(refs), sums, &unused);
  const int count[4] = {refs.x, refs.y, refs.z, refs.w};
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t i = at + k;
    if (i >= g.nb) break;
    const bool on = count[k] > 0;
    if (i < n) {
      a.map[i] = on ? static_cast<int32_t>(i) : -1;
      if (on)
        a.refs_out[i] = count[k];
      else
        a.dst[i - rank] = static_cast<int32_t>(i);  // (free blocks before i)
    } else {
      a.rank[i] = on ? rank - kept : -1;
      if (on) {
        a.src[rank - kept] = static_cast<int32_t>(i);
        a.count[rank - kept] = count[k];
      } else {
        a.map[i] = -1;
      }
      a.refs_out[i] = 0;
    }
    rank += on;
  }
}

__global__ void __launch_bounds__(kThreads) compact_move_kernel(const CompactArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const PagesArgs& g = a.g;
  const int n = a.totals[0], moves = a.totals[1];
  const int64_t work = static_cast<int64_t>(moves) * a.items;
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int m = static_cast<int>(w / a.items);
    int piece = static_cast<int>(w % a.items);
    const int src = a.src[m], dst = a.dst[m];
    for (int i = 0; i < g.npools; ++i) {
      const PoolView& pool = g.pool[i];
      const int pieces = static_cast<int>((pool.bytes + kCompactPiece - 1) / kCompactPiece);
      if (piece < pieces) {
        const int64_t at = static_cast<int64_t>(piece) * kCompactPiece;
        const int64_t len = min(static_cast<int64_t>(kCompactPiece), pool.bytes - at);
        if (pool.wide)
          copy_piece<uint4>(pool, src, dst, at, len, kThreads * 16);
        else
          copy_piece<uint32_t>(pool, src, dst, at, len, kThreads * 4);
        break;
      }
      piece -= pieces;
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  for (int64_t m = id; m < moves; m += step) {
    a.map[a.src[m]] = a.dst[m];
    a.refs_out[a.dst[m]] = a.count[m];
  }
  const int64_t entries = static_cast<int64_t>(g.rows) * g.cols;
  for (int64_t i = id; i < entries; i += step) {
    const int64_t row = i / g.cols, j = i % g.cols;
    const int e = g.table[row * g.ts + j];
    int to = -1;
    if (e >= 0 && e < n && e < g.nb) {
      to = a.map[e];
    } else if (e >= n && e < g.nb) {
      const int m = a.rank[e];
      if (m >= 0) to = a.dst[m];
    }
    a.table_out[row * a.ts_out + j] = to;
  }
}

}  // namespace

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(int) * static_cast<size_t>(a.g.rows);
  if (smem > 48 * 1024) {
    // (an attribute of the device that is current: set on every such call)
    const cudaError_t e = cudaFuncSetAttribute(
        fork_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMaxTableRows);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e =
      launch_pdl(fork_plan_kernel, dim3(1 + a.g.rows), dim3(kPlanThreads), smem, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(fork_apply_kernel, dim3(a.slices, a.g.rows), dim3(kThreads), 0, s, a);
}

cudaError_t launch_compact(const CompactArgs& a, int num_sms, cudaStream_t s) {
  const unsigned chunks = static_cast<unsigned>(ceil_div(a.g.nb, kCompactChunk));
  cudaError_t e = launch_pdl(compact_count_kernel, dim3(chunks), dim3(kThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(compact_rank_kernel, dim3(chunks), dim3(kThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(compact_move_kernel, dim3(8 * num_sms), dim3(kThreads), 0, s, a);
}

}  // namespace dkv
