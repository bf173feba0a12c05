// append.cu -- appending new tokens' keys and values to a KV cache, with the
// position rotation of keys and queries applied on the way.
//
// Sequence b's n new tokens take the positions p = N_b - n .. N_b - 1.  With a
// rotary width r, channels (x_a, x_b) of pair i < r / 2 -- (i, i + r/2), or
// (2 i, 2 i + 1) interleaved -- of a key or query become
//   y_a = x_a cos(p, i) - x_b sin(p, i),   y_b = x_b cos(p, i) + x_a sin(p, i),
// each product, sum and difference rounded to fp32, the result once to its
// 16-bit type (or to e4m3).  Other channels and the values are copied.
//
// An 8-bit cache keeps one scale per 16-token block and kv head,
//   s = 2^e, e = the smallest exponent with amax <= 448 * 2^e,
// clamped into the range where code * s is exact in the cache's 16-bit type;
// code = e4m3(y / s), rounded to nearest even, saturated.  A power of two makes
// y / s exact and raising s later nearly so: older codes of a block whose scale
// rises are stored again as e4m3(code * s_old / s), which rounds only values
// that become subnormal.  A block's scale never falls while it holds tokens;
// its first token sets it anew.
//
// Two kernels.  append_token_kernel: d/16 threads a token and head, 16
// channels (two 16-byte vectors, the two halves of 8 rotation pairs) each;
// nothing is shared between tokens, so it serves the single-token call -- where
// the d/16 threads of an 8-bit cache agree on the scale by shuffles -- and short
// appends into a 16-bit cache.  append_block_kernel: a CTA of d threads takes a
// touched block and four heads at a time, a thread per token and 16 channels of
// each; the blocks' amax are reduced through shared memory while the rotated
// values wait in registers, so they are read and rotated once, and the heads
// share the token's angles.  Its CTAs are persistent and count the blocks that
// the sequences touch, so a ragged batch costs nothing for what it lacks.
//
// Measured on a GB300 (copy rate 6.79 TB/s), 32 query / 8 kv heads, d = 128:
// 8 prompts of 8K tokens into an 8-bit cache 231 us (6.4 TB/s), ragged 137 us
// (6.3), into a 16-bit one 269 us (6.0).  The ragged ones took 248 us with one
// head a CTA, 166 with four, 152 with persistent CTAs that rotated twice to save
// registers.  One token of 64 sequences (16-bit) takes 2.0 us, of 16 sequences
// (8-bit) 2.2 us where no scale rises: the latency of the launch and of the
// dependent loads length -> block table -> scale.  Where one rises, the older rows
// of its block are stored again one after the other: 0.3 us more for one row, 1.8
// for 7, 3.8 for 15 (16 sequences; 4.0 of 64), and a batch takes as long as its
// fullest such block.

#include "dkv_device.cuh"
#include "dkv_kernels.h"
#include "rope.cuh"

namespace dkv {
namespace {

constexpr int kTokenThreads = 256;

// Sequence b's new tokens: positions [start, start + n).  Lengths that do not
// fit the cache, the table of angles or the rows given leave the sequence
// alone and are reported as a failed check.
struct NewTokens {
  int start, n;
};
__device__ __forceinline__ NewTokens new_tokens(const AppendArgs& a, int b) {
  const int len = a.lens != nullptr ? a.lens[b] : a.N;
  int n = a.news != nullptr ? a.news[b] : a.T;
  if (len <= 0 || n == 0) return {0, 0};  // an unused batch entry, or nothing new
  if (n < 0 || n > a.T || n > len || len > a.N || (a.r > 0 && len > a.rope_len)) {
    set_status(a.status, kStatusCheck);
    return {0, 0};
  }
  return {len - n, n};
}

// The scale a block needs for values of magnitude up to amax (its bits).
__device__ __forceinline__ float scale_for(uint32_t amax_bits, int e_lo, int e_hi) {
  // amax = 2^k * f: 448 = 1.75 * 2^8, so e = k - 8, or k - 7 when f > 1.75
  const int k = static_cast<int>(amax_bits >> 23) - 127;
  const int e = k - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __int_as_float((127 + min(max(e, e_lo), e_hi)) << 23);
}

// Four values as e4m3 codes (nearest even, saturated), the first in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x4(float x0, float x1, float x2, float x3) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
  return make_float2(lo16<true>(h), hi16<true>(h));
}

// Division by s: for a power of two the exact product with 1 / s.
struct Divider {
  float s, inv;
  bool pow2;
  __device__ __forceinline__ explicit Divider(float s_) : s(s_) {
    pow2 = (__float_as_uint(s_) & 0x7fffffu) == 0u;
    inv = __fdiv_rn(1.f, s_);
  }
};

// (Out of line: only a scale that this file did not write needs it.)
__device__ __noinline__ float divide(float x, float s) { return __fdiv_rn(x, s); }

// The thread's 16 channels as codes.
__device__ __forceinline__ void store_codes(uint8_t* row, Chunks c, const Divider& by,
                                            const float (&x)[16]) {
  float y[16];
  if (by.pow2) {  // (one branch for all 16)
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(x[i], by.inv);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = divide(x[i], by.s);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *reinterpret_cast<uint2*>(row + (h ? c.c2 : c.c1)) =
        make_uint2(to_e4m3x4(y[8 * h], y[8 * h + 1], y[8 * h + 2], y[8 * h + 3]),
                   to_e4m3x4(y[8 * h + 4], y[8 * h + 5], y[8 * h + 6], y[8 * h + 7]));
}

// Codes stored under the scale s_old, stored again under by.s.
__device__ __forceinline__ void rescale_codes(uint8_t* row, Chunks c, float s_old,
                                              const Divider& by) {
  float x[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint2 w = *reinterpret_cast<const uint2*>(row + (h ? c.c2 : c.c1));
    const uint32_t v[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = from_e4m3x2(v[i]);
      x[8 * h + 2 * i] = __fmul_rn(f.x, s_old);
      x[8 * h + 2 * i + 1] = __fmul_rn(f.y, s_old);
    }
  }
  store_codes(row, c, by, x);
}

__device__ __forceinline__ uint32_t amax_bits(const float (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
  return __float_as_uint(m);
}

// Where page `page` of sequence b lies in a cache: the index that its block
// stride multiplies and the element offset of its first token within.  -1 in
// `blk`: the table names no block of the pool (reported; nothing is written).
struct PageAt {
  int64_t blk, tok;
};
__device__ __forceinline__ PageAt page_at(const AppendArgs& a, int b, int page, int d) {
  if (a.bt == nullptr) return {b, static_cast<int64_t>(page) * kPage * d};
  const int blk = a.bt[b * a.bts + page];
  if (blk < 0 || blk >= a.nblocks) {
    set_status(a.status, kStatusCheck);
    return {-1, 0};
  }
  return {blk, 0};
}
__device__ __forceinline__ float* scale_at(const AppendArgs& a, const AppendCache& c, PageAt at,
                                           int page, int h) {
  return c.scale + at.blk * c.ssb + h * c.ssh + (a.bt == nullptr ? page : 0);
}

template <int D, bool F16, bool EIGHT, bool IL>
__global__ void __launch_bounds__(kTokenThreads) append_token_kernel(const AppendArgs a) {
  constexpr int L = D / 16;  // threads of a token and head
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t idx = blockIdx.x * kTokenThreads + threadIdx.x;
  const int b = blockIdx.y;
  const int j = idx % L;
  const uint32_t heads = 2 * a.Hkv + a.Hq;
  const uint32_t row = idx / L;
  const int t = static_cast<int>(row / heads);
  const int hx = static_cast<int>(row % heads);
  const NewTokens nt = new_tokens(a, b);
  const bool on = t < nt.n;  // (8-bit: every lane stays for the shuffles)
  if (!EIGHT && !on) return;
  const int pos = nt.start + t;
  const bool is_q = hx >= 2 * a.Hkv, is_v = !is_q && hx >= a.Hkv;
  const int h = is_q ? hx - 2 * a.Hkv : (is_v ? hx - a.Hkv : hx);
  const bool rotated = !is_v && 16 * j < a.r;
  const Chunks c = chunks_of<IL>(j, a.r, rotated);
  float x[16] = {};
  if (on) {
    const AppendRows& src = is_q ? a.q : (is_v ? a.v : a.k);
    widen<F16>(load_raw(src.p + b * src.sb + t * src.st + h * src.sh, c), x);
    if (rotated) rotate16<IL>(angles_of(a.cos, a.sin, a.r, pos, j), x);
    if (is_q) store16<F16>(a.q_out + b * a.o_sb + t * a.o_st + h * a.o_sh, c, x);
  }
  const AppendCache& cache = is_v ? a.V : a.K;
  const int page = pos / kPage, slot = pos % kPage;
  PageAt at{-1, 0};
  if (on && !is_q) at = page_at(a, b, page, D);
  if constexpr (!EIGHT) {
    if (at.blk >= 0)
      store16<F16>(static_cast<uint16_t*>(cache.p) + at.blk * cache.sb + h * cache.sh + at.tok +
                       slot * D,
                   c, x);
  } else {
    uint32_t m = amax_bits(x);
#pragma unroll
    for (int o = 1; o < L; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool put = at.blk >= 0;  // (the L lanes of a row agree on it)
    float* sp = put ? scale_at(a, cache, at, page, h) : nullptr;
    const float old = put && slot > 0 ? *sp : 0.f;
    __syncwarp();  // every lane of the row has read the old scale
    if (put) {
      const float s = fmaxf(scale_for(m, a.e_lo, a.e_hi), old);
      const Divider by(s);
      uint8_t* rows = static_cast<uint8_t*>(cache.p) + at.blk * cache.sb + h * cache.sh + at.tok;
      if (s > old)
        for (int i = 0; i < slot; ++i) rescale_codes(rows + i * D, c, old, by);
      store_codes(rows + slot * D, c, by, x);
      if (j == 0 && s != old) *sp = s;
    }
  }
}

constexpr int kHeads = 4;      // heads of a block kernel's work item
constexpr int kMaxSeqs = 128;  // sequences whose touched pages are counted first
// CTAs of the persistent grid on an SM: 128 registers a thread, or 102.
template <int D, bool EIGHT>
constexpr int block_ctas() {
  return (EIGHT ? 4 : 5) * (128 / D);
}

template <int D, bool F16, bool EIGHT, bool IL>
__global__ void __launch_bounds__(D, block_ctas<D, EIGHT>()) append_block_kernel(const AppendArgs a) {
  constexpr int L = D / 16, kWarps = D / 32;
  __shared__ uint32_t warp_amax[2][kWarps][kHeads];
  __shared__ int page_end[kMaxSeqs];  // pages that sequences 0 .. b touch
  __shared__ NewTokens seqs[kMaxSeqs];
  griddep_launch_dependents();
  griddep_wait();
  // Work items: (sequence, touched page, four heads of k, v or q), heads fastest.
  // Up to kMaxSeqs sequences, only the pages they touch are counted.
  const bool counted = a.B <= kMaxSeqs;
  const uint32_t kv_groups = (a.Hkv + kHeads - 1) / kHeads;
  const uint32_t groups = 2 * kv_groups + (a.Hq + kHeads - 1) / kHeads;
  const int lane = threadIdx.x % 32;
  uint32_t n_items = static_cast<uint32_t>(a.B) * a.pages * groups;
  if (counted) {
    if (threadIdx.x < 32) {
      int sum = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        int c = 0;
        if (b < a.B) {
          const NewTokens nt = new_tokens(a, b);
          seqs[b] = nt;
          if (nt.n > 0) c = (nt.start + nt.n - 1) / kPage - nt.start / kPage + 1;
        }
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int up = __shfl_up_sync(0xffffffffu, c, o);
          if (lane >= o) c += up;
        }
        if (b < a.B) page_end[b] = sum + c;
        sum += __shfl_sync(0xffffffffu, c, 31);
      }
    }
    __syncthreads();
    n_items = static_cast<uint32_t>(page_end[a.B - 1]) * groups;
  }
  const int j = threadIdx.x % L, i = threadIdx.x / L;
  int turn = 0;
  for (uint32_t item = blockIdx.x; item < n_items; item += gridDim.x) {
    const uint32_t gx = item % groups;
    int y = static_cast<int>(item / groups), b;
    NewTokens nt;
    if (counted) {  // the first sequence that ends past the page
      b = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32)
        b += __popc(__ballot_sync(0xffffffffu, b0 + lane < a.B && page_end[b0 + lane] <= y));
      if (b > 0) y -= page_end[b - 1];
      nt = seqs[b];
    } else {
      b = y / a.pages;
      y %= a.pages;
      nt = new_tokens(a, b);
    }
    const int page = nt.start / kPage + y;
    // no token of this page (compared as pages: a page's tokens may pass 2^31)
    if (nt.n == 0 || page > (nt.start + nt.n - 1) / kPage) continue;
    const int pos = page * kPage + i, t = pos - nt.start;
    const bool on = t >= 0 && t < nt.n;
    const bool is_q = gx >= 2 * kv_groups, is_v = !is_q && gx >= kv_groups;
    const int h0 =
        static_cast<int>(is_q ? gx - 2 * kv_groups : (is_v ? gx - kv_groups : gx)) * kHeads;
    const int nh = min(kHeads, (is_q ? a.Hq : a.Hkv) - h0);
    const bool rotated = !is_v && 16 * j < a.r;
    const Chunks c = chunks_of<IL>(j, a.r, rotated);
    const AppendRows& src = is_q ? a.q : (is_v ? a.v : a.k);
    Raw raw[kHeads] = {};
    Angles ang;
    if (on) {
      const uint16_t* row = src.p + b * src.sb + t * src.st + h0 * src.sh;
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h < nh) raw[h] = load_raw(row + h * src.sh, c);
      if (rotated) ang = angles_of(a.cos, a.sin, a.r, pos, j);
    }
    const AppendCache& cache = is_v ? a.V : a.K;
    PageAt at{-1, 0};
    if (!is_q) at = page_at(a, b, page, D);
    if (is_q || (!EIGHT && at.blk >= 0)) {  // 16-bit rows
      uint16_t* out = is_q ? a.q_out + b * a.o_sb + t * a.o_st + h0 * a.o_sh
                           : static_cast<uint16_t*>(cache.p) + at.blk * cache.sb + h0 * cache.sh +
                                 at.tok + i * D;
      const int64_t osh = is_q ? a.o_sh : cache.sh;
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        if (!on || h >= nh) break;
        float x[16];
        widen<F16>(raw[h], x);
        if (rotated) rotate16<IL>(ang, x);
        store16<F16>(out + h * osh, c, x);
      }
      continue;
    }
    if (!EIGHT || at.blk < 0) continue;
    float* sp = scale_at(a, cache, at, page, h0);
    const int kept = max(0, nt.start - page * kPage);  // tokens the block held before
    float old[kHeads], x[kHeads][16];
    turn ^= 1;
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      old[h] = kept > 0 && h < nh ? sp[h * cache.ssh] : 0.f;
      widen<F16>(raw[h], x[h]);
      if (rotated) rotate16<IL>(ang, x[h]);
      const uint32_t wm = __reduce_max_sync(0xffffffffu, on ? amax_bits(x[h]) : 0u);
      if (lane == 0) warp_amax[turn][threadIdx.x / 32][h] = wm;
    }
    // Every thread has read the old scales; the other turn's maxima are free once
    // all have passed this barrier again.
    __syncthreads();
    uint8_t* rows =
        static_cast<uint8_t*>(cache.p) + at.blk * cache.sb + h0 * cache.sh + at.tok + i * D;
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (h >= nh) break;
      uint32_t m = warp_amax[turn][0][h];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = max(m, warp_amax[turn][w][h]);
      const float s = fmaxf(scale_for(m, a.e_lo, a.e_hi), old[h]);
      const Divider by(s);
      uint8_t* row = rows + h * cache.sh;
      if (on) {
        store_codes(row, c, by, x[h]);
      } else if (i < kept && s > old[h]) {
        rescale_codes(row, c, old[h], by);
      }
      if (threadIdx.x == 0 && s != old[h]) sp[h * cache.ssh] = s;
    }
  }
}

template <int D, bool F16, bool IL>
cudaError_t launch_t(bool eight, const AppendArgs& a, int num_sms, cudaStream_t s) {
  const uint32_t heads = 2 * a.Hkv + a.Hq;
  // Into a 16-bit cache, a thread a row segment while all of them are resident at
  // once (2048 a SM) or there are few tokens a sequence, which fill the blocks that
  // the persistent kernel goes by only in part; us here against that kernel's (32 /
  // 8 heads, d = 128): 1 sequence of 512 tokens 3.1 / 4.0, 8 of 64 3.0 / 4.0, 64 of 4
  // 2.6 / 4.2, 64 of 16 4.6 / 5.6, 128 of 8 4.7 / 7.5, 512 of 8 17.3 / 23.8, 1024 of
  // 1 5.1 / 20.3.  They meet at 16 tokens in large batches (256 17.1 / 17.4, 512 37.7
  // / 36.5, 1024 73.2 / 68.6); past it 256 of 32 36.2 / 33.6, 8 prompts of 8K 302 /
  // 270.
  const int64_t threads = static_cast<int64_t>(a.B) * a.T * heads * (D / 16);
  const bool by_token = eight ? a.T == 1 : a.T <= 16 || threads <= num_sms * 2048;
  if (!by_token) {
    const int64_t groups = 2 * ceil_div(a.Hkv, kHeads) + ceil_div(a.Hq, kHeads);
    const int64_t items = static_cast<int64_t>(a.B) * a.pages * groups;
    const int64_t most = static_cast<int64_t>(num_sms) *
                         (eight ? block_ctas<D, true>() : block_ctas<D, false>());
    const dim3 grid(static_cast<unsigned>(items < most ? items : most));
    return eight ? launch_pdl(append_block_kernel<D, F16, true, IL>, grid, dim3(D), 0, s, a)
                 : launch_pdl(append_block_kernel<D, F16, false, IL>, grid, dim3(D), 0, s, a);
  }
  const dim3 grid(static_cast<unsigned>(
                      ceil_div(static_cast<int64_t>(a.T) * heads * (D / 16), kTokenThreads)),
                  a.B);
  return eight ? launch_pdl(append_token_kernel<D, F16, true, IL>, grid, dim3(kTokenThreads), 0, s, a)
               : launch_pdl(append_token_kernel<D, F16, false, IL>, grid, dim3(kTokenThreads), 0, s,
                            a);
}

}  // namespace

cudaError_t launch_append(int d, bool f16, bool eight, bool interleaved, const AppendArgs& a,
                          int num_sms, cudaStream_t s) {
  if (d == 128) {
    if (f16) return interleaved ? launch_t<128, true, true>(eight, a, num_sms, s)
                                : launch_t<128, true, false>(eight, a, num_sms, s);
    return interleaved ? launch_t<128, false, true>(eight, a, num_sms, s)
                       : launch_t<128, false, false>(eight, a, num_sms, s);
  }
  if (f16) return interleaved ? launch_t<64, true, true>(eight, a, num_sms, s)
                              : launch_t<64, true, false>(eight, a, num_sms, s);
  return interleaved ? launch_t<64, false, true>(eight, a, num_sms, s)
                     : launch_t<64, false, false>(eight, a, num_sms, s);
}

}  // namespace dkv
