// prompt_attn.cu -- attention of prompts with expanded keys and values, the simplest
// form: a CTA a row (query, head), a warp a key at a time, one pass with the running
// maximum and sum.

#include "dkv_device.cuh"
#include "dkv_kernels.h"
#include "latent.h"

namespace dkv {
namespace {

constexpr int kWarps = 8;

template <int DN, bool F16>
__global__ void __launch_bounds__(32 * kWarps) prompt_attn_kernel(const PromptArgs a) {
  constexpr int V = DN / 64;
  __shared__ float part[kWarps][DN];
  __shared__ float stat[kWarps][2];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int i = blockIdx.x, h = blockIdx.y;
  // the sequence that query row i belongs to
  int b = -1;
  for (int s = 0; s < a.B; ++s) {
    const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k) {
      set_status(a.status, kStatusCheck);
      continue;
    }
    if (i >= q0 && i < q1) {
      b = s;
      break;
    }
  }
  if (b < 0) return;
  const int nq = a.cu_q[b + 1] - a.cu_q[b], k0 = a.cu_k[b], nk = a.cu_k[b + 1] - k0;
  const int seen = a.causal ? nk - nq + (i - a.cu_q[b]) + 1 : nk;
  const uint32_t* qn = reinterpret_cast<const uint32_t*>(a.qn + i * a.qn_st + h * a.qn_sh);
  const uint32_t* qr = reinterpret_cast<const uint32_t*>(a.qr + i * a.qr_st + h * a.qr_sh);
  uint32_t q[V];
#pragma unroll
  for (int d = 0; d < V; ++d) q[d] = qn[lane + 32 * d];
  const uint32_t qk = qr[lane];
  float o[2 * V] = {}, m = -INFINITY, l = 0.f;
  for (int j = warp; j < seen; j += kWarps) {
    const uint32_t* kn =
        reinterpret_cast<const uint32_t*>(a.kn + static_cast<int64_t>(k0 + j) * a.kn_st + h * a.kn_sh);
    const uint32_t* kr =
        reinterpret_cast<const uint32_t*>(a.kr + static_cast<int64_t>(k0 + j) * a.kr_st);
    const uint32_t* vv =
        reinterpret_cast<const uint32_t*>(a.v + static_cast<int64_t>(k0 + j) * a.v_st + h * a.v_sh);
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < V; ++d) {
      const uint32_t k = kn[lane + 32 * d];
      s = fmaf(lo16<F16>(q[d]), lo16<F16>(k), fmaf(hi16<F16>(q[d]), hi16<F16>(k), s));
    }
    const uint32_t k = kr[lane];
    s = fmaf(lo16<F16>(qk), lo16<F16>(k), fmaf(hi16<F16>(qk), hi16<F16>(k), s));
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    const float now = fmaxf(m, s), f = exp2f(m - now), p = exp2f(s - now);
    m = now;
    l = l * f + p;
#pragma unroll
    for (int d = 0; d < V; ++d) {
      const uint32_t v = vv[lane + 32 * d];
      o[2 * d] = o[2 * d] * f + p * lo16<F16>(v);
      o[2 * d + 1] = o[2 * d + 1] * f + p * hi16<F16>(v);
    }
  }
#pragma unroll
  for (int d = 0; d < V; ++d) {
    part[warp][2 * (lane + 32 * d)] = o[2 * d];
    part[warp][2 * (lane + 32 * d) + 1] = o[2 * d + 1];
  }
  if (lane == 0) stat[warp][0] = m, stat[warp][1] = l;
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w][0]);
  for (int w = 0; w < kWarps; ++w)
    if (stat[w][1] > 0.f) sum += stat[w][1] * exp2f(stat[w][0] - top);
  for (int d = threadIdx.x; d < DN; d += 32 * kWarps) {
    float y = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (stat[w][1] > 0.f) y += part[w][d] * exp2f(stat[w][0] - top);
    y = sum > 0.f ? y / sum : 0.f;
    const int64_t at = i * a.o_st + h * a.o_sh + d;
    if (a.out_dtype == 2)
      static_cast<float*>(a.out)[at] = y;
    else if (a.out_dtype == 1)
      static_cast<__half*>(a.out)[at] = __float2half_rn(y);
    else
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
  }
}

}  // namespace

cudaError_t launch_prompt_attn(int dn, bool f16, const PromptArgs& a, cudaStream_t s) {
  const dim3 grid(a.total_q, a.H), block(32 * kWarps);
  if (dn == 128)
    return f16 ? launch_pdl(prompt_attn_kernel<128, true>, grid, block, 0, s, a)
               : launch_pdl(prompt_attn_kernel<128, false>, grid, block, 0, s, a);
  return f16 ? launch_pdl(prompt_attn_kernel<64, true>, grid, block, 0, s, a)
             : launch_pdl(prompt_attn_kernel<64, false>, grid, block, 0, s, a);
}

}  // namespace dkv
