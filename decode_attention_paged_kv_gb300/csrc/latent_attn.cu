// latent_attn.cu -- attention of new tokens over a latent cache, the simplest form: a CTA
// a row (sequence, new token, head), a warp a cache token at a time, one pass with the
// running maximum and sum.

#include "dkv_device.cuh"
#include "dkv_kernels.h"
#include "latent.h"

namespace dkv {
namespace {

constexpr int kWarps = 8;

template <int DC, bool F16>
__global__ void __launch_bounds__(32 * kWarps) latent_attn_kernel(const LatentAttnArgs a) {
  constexpr int V = DC / 64;  // pairs of channels a lane
  __shared__ float part[kWarps][DC];
  __shared__ float stat[kWarps][2];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int t = blockIdx.x / a.H, h = blockIdx.x % a.H, b = blockIdx.y;
  const LatentView& c = a.cache;
  const int len = a.lens != nullptr ? min(a.lens[b], c.N) : c.N;
  const int n = a.news != nullptr ? min(max(a.news[b], 0), a.T) : a.T;
  if (t >= n) return;
  const int seen = len - n + t + 1;
  const uint32_t* ql = reinterpret_cast<const uint32_t*>(a.ql + b * a.ql_sb + t * a.ql_st + h * a.ql_sh);
  const uint32_t* qr = reinterpret_cast<const uint32_t*>(a.qr + b * a.qr_sb + t * a.qr_st + h * a.qr_sh);
  uint32_t q[V];
#pragma unroll
  for (int i = 0; i < V; ++i) q[i] = ql[lane + 32 * i];
  const uint32_t qk = qr[lane];
  float o[2 * V] = {}, m = -INFINITY, l = 0.f;
  for (int j = warp; j < seen; j += kWarps) {
    const uint16_t* row = c.p + b * c.sb + j * c.st;
    if (c.block > 0) {
      int blk = c.bt[b * c.bts + j / c.block];
      if (blk < 0 || blk >= c.nblocks) {
        set_status(a.status, kStatusCheck);
        blk = min(max(blk, 0), c.nblocks - 1);
      }
      row = c.p + blk * c.sb + (j % c.block) * c.st;
    }
    const uint32_t* x = reinterpret_cast<const uint32_t*>(row);
    uint32_t v[V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = x[lane + 32 * i];
      s = fmaf(lo16<F16>(q[i]), lo16<F16>(v[i]), fmaf(hi16<F16>(q[i]), hi16<F16>(v[i]), s));
    }
    const uint32_t k = x[DC / 2 + lane];
    s = fmaf(lo16<F16>(qk), lo16<F16>(k), fmaf(hi16<F16>(qk), hi16<F16>(k), s));
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    const float now = fmaxf(m, s), f = exp2f(m - now), p = exp2f(s - now);
    m = now;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      o[2 * i] = o[2 * i] * f + p * lo16<F16>(v[i]);
      o[2 * i + 1] = o[2 * i + 1] * f + p * hi16<F16>(v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    part[warp][2 * (lane + 32 * i)] = o[2 * i];
    part[warp][2 * (lane + 32 * i) + 1] = o[2 * i + 1];
  }
  if (lane == 0) stat[warp][0] = m, stat[warp][1] = l;
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w][0]);
  for (int w = 0; w < kWarps; ++w)
    if (stat[w][1] > 0.f) sum += stat[w][1] * exp2f(stat[w][0] - top);
  for (int i = threadIdx.x; i < DC; i += 32 * kWarps) {
    float y = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (stat[w][1] > 0.f) y += part[w][i] * exp2f(stat[w][0] - top);
    y = sum > 0.f ? y / sum : 0.f;
    const int64_t at = b * a.o_sb + t * a.o_st + h * a.o_sh + i;
    if (a.out_dtype == 2)
      static_cast<float*>(a.out)[at] = y;
    else if (a.out_dtype == 1)
      static_cast<__half*>(a.out)[at] = __float2half_rn(y);
    else
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
  }
}

}  // namespace

cudaError_t launch_latent_attn(int dc, bool f16, const LatentAttnArgs& a, cudaStream_t s) {
  const dim3 grid(a.T * a.H, a.B), block(32 * kWarps);
  if (dc == 512)
    return f16 ? launch_pdl(latent_attn_kernel<512, true>, grid, block, 0, s, a)
               : launch_pdl(latent_attn_kernel<512, false>, grid, block, 0, s, a);
  return f16 ? launch_pdl(latent_attn_kernel<256, true>, grid, block, 0, s, a)
             : launch_pdl(latent_attn_kernel<256, false>, grid, block, 0, s, a);
}

}  // namespace dkv
