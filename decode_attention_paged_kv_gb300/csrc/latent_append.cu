// latent_append.cu -- new tokens into a latent cache: the latent vector normalised, the
// shared key and the queries' rotary parts rotated by the token's position.
//
//   latent_i = c_i * rsqrt(mean(c^2) + eps) * w_i      (fp32, rounded once)
//   y_a = x_a cos - x_b sin,  y_b = x_b cos + x_a sin  (as in rope.cuh)
//
// A warp takes a token: the latent vector, dc / 32 channels a lane, the sum of squares by
// shuffles, and up to 40 rows of 64 rotary channels, four lanes each, the token's angles
// in registers.  All loads of a warp (5 KB at 32 heads) are under way at once, which is
// what a prompt is bound by; a decode step with more heads has further warps for them.
//
// Measured on a GB300, 32 heads, dc = 512: 8 ragged prompts of up to 8K tokens 55 to 87 us over
// six draws of lengths, 5.0 to 5.8 TB/s by their tokens (the first, 55 us: 88 with six warps a
// token, each one load deep): 100 registers leave two CTAs a multiprocessor, and a warp has
// nothing of a next token under way while it computes and stores one; one token of 64 sequences 2.9 us,
// the latency of the launch and of the loads lengths - rows, table - stores.

#include "dkv_device.cuh"
#include "dkv_kernels.h"
#include "latent.h"
#include "rope.cuh"

namespace dkv {
namespace {

constexpr int kThreads = 256;
constexpr int kTurns = 5;                // rotary rows of a lane
constexpr int kRowsPerWarp = 8 * kTurns;  // rotary rows of a warp

struct Fresh {
  int start, n;
};
// Sequence b's new tokens: positions [start, start + n).  Lengths that do not fit leave
// the sequence alone and are reported.
__device__ __forceinline__ Fresh fresh_tokens(const LatentAppendArgs& a, int b) {
  const int len = a.lens != nullptr ? a.lens[b] : a.cache.N;
  const int n = a.news != nullptr ? a.news[b] : a.T;
  if (len <= 0 || n == 0) return {0, 0};
  if (n < 0 || n > a.T || n > len || len > a.cache.N || (a.rope_len > 0 && len > a.rope_len)) {
    set_status(a.status, kStatusCheck);
    return {0, 0};
  }
  return {len - n, n};
}

// The cache row of position pos of sequence b, or nullptr (reported): the table names no
// block of the pool.
__device__ __forceinline__ uint16_t* row_of(const LatentAppendArgs& a, int b, int pos) {
  const LatentView& c = a.cache;
  if (c.block == 0) return c.p + b * c.sb + pos * c.st;
  const int blk = c.bt[b * c.bts + pos / c.block];
  if (blk < 0 || blk >= c.nblocks) {
    set_status(a.status, kStatusCheck);
    return nullptr;
  }
  return c.p + blk * c.sb + (pos % c.block) * c.st;
}

template <int DC, bool F16, bool IL>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const LatentAppendArgs a) {
  constexpr int V = DC / 256;  // vectors of 8 channels a lane
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x % 32;
  const int b = blockIdx.y;
  // units of a token: its latent vector with its first rotary rows (the key's is row 0),
  // then further rows
  const uint32_t units = (a.H + 1 + kRowsPerWarp - 1) / kRowsPerWarp;
  const uint32_t w = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int t = static_cast<int>(w / units), u = static_cast<int>(w % units);
  const Fresh nt = fresh_tokens(a, b);
  if (t >= nt.n) return;
  const int pos = nt.start + t;
  const int j = lane % 4;
  const bool rotated = a.rope_len > 0;
  const Chunks ch = chunks_of<IL>(j, kLatentRope, rotated);
  // everything that is read
  uint4 raw[V], wt[V];
  if (u == 0) {
    const uint16_t* src = a.c + b * a.c_sb + t * a.c_st;
#pragma unroll
    for (int i = 0; i < V; ++i) raw[i] = *reinterpret_cast<const uint4*>(src + 8 * (lane + 32 * i));
  }
  Raw rope[kTurns];
  const int row0 = u * kRowsPerWarp + lane / 4;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int h = row0 + 8 * i - 1;  // -1: the key
    if (h < a.H)
      rope[i] = load_raw(h < 0 ? a.k + b * a.k_sb + t * a.k_st
                               : a.q + b * a.q_sb + t * a.q_st + h * a.q_sh,
                         ch);
  }
  Angles ang;
  if (rotated) ang = angles_of(a.cos, a.sin, kLatentRope, pos, j);
  uint16_t* row = nullptr;
  if (u == 0) {
    row = row_of(a, b, pos);
    if (a.norm != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        wt[i] = __ldg(reinterpret_cast<const uint4*>(a.norm + 8 * (lane + 32 * i)));
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float lo = lo16<F16>(x[k]), hi = hi16<F16>(x[k]);
          sum = fmaf(lo, lo, fmaf(hi, hi, sum));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      // (a square root and a division, each rounded once: rsqrtf is off by two steps)
      const float r = 1.f / sqrtf(sum * (1.f / DC) + a.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        const uint32_t y[4] = {wt[i].x, wt[i].y, wt[i].z, wt[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = pack2<F16>(lo16<F16>(x[k]) * r * lo16<F16>(y[k]),
                            hi16<F16>(x[k]) * r * hi16<F16>(y[k]));
        raw[i] = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
    if (row != nullptr) {
#pragma unroll
      for (int i = 0; i < V; ++i) *reinterpret_cast<uint4*>(row + 8 * (lane + 32 * i)) = raw[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int h = row0 + 8 * i - 1;
    if (h >= a.H || (h < 0 && row == nullptr)) continue;
    float x[16];
    widen<F16>(rope[i], x);
    if (rotated) rotate16<IL>(ang, x);
    store16<F16>(h < 0 ? row + DC : a.q_out + b * a.o_sb + t * a.o_st + h * a.o_sh, ch, x);
  }
}

template <int DC, bool F16, bool IL>
cudaError_t launch_t(const LatentAppendArgs& a, cudaStream_t s) {
  const int64_t units = ceil_div(a.H + 1, kRowsPerWarp);
  const dim3 grid(static_cast<unsigned>(ceil_div(a.T * units, kThreads / 32)), a.B);
  return launch_pdl(latent_append_kernel<DC, F16, IL>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_latent_append(int dc, bool f16, bool interleaved, const LatentAppendArgs& a,
                                 cudaStream_t s) {
  if (dc == 512) {
    if (f16) return interleaved ? launch_t<512, true, true>(a, s) : launch_t<512, true, false>(a, s);
    return interleaved ? launch_t<512, false, true>(a, s) : launch_t<512, false, false>(a, s);
  }
  if (f16) return interleaved ? launch_t<256, true, true>(a, s) : launch_t<256, true, false>(a, s);
  return interleaved ? launch_t<256, false, true>(a, s) : launch_t<256, false, false>(a, s);
}

}  // namespace dkv
