// meta_fp8.cu -- page metadata of an 8-bit KV cache (e4m3 codes, one scale per
// 16-token block and kv head): channel-wise min m_j / max M_j of each page's
// keys, in the cache's 16-bit type.
//
// A block's scale s >= 0 is common to its keys, so min and max are taken over
// the codes (as fp16 pairs, exact) and multiplied by s once per block; pages of
// 32 or 64 tokens join their blocks in fp32.  Powers of two give the exact min
// and max; another scale's products are rounded outward (m down, M up), which
// keeps the bound scores upper bounds.  One thread owns 16 channels (one 16-byte
// vector a token) of a page with the page's 16 rows in flight together: bound by
// HBM, 24 instructions a vector.  Measured on a GB300 (copy rate 6.79 TB/s), 16 x
// 8 kv heads of 32K tokens, d = 128: 104 us (6.4 TB/s) with five CTAs of 128
// threads an SM; two of 256 threads 121 us, four with eight rows in flight
// 135 us.

#include "dkv_device.cuh"
#include "dkv_kernels.h"

namespace dkv {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ __half2 codes2(uint32_t w) {  // the low half's two codes
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return *reinterpret_cast<const __half2*>(&r);
}

// Two values rounded down (UP: up) to a packed 16-bit pair.
template <bool F16, bool UP>
__device__ __forceinline__ uint32_t pack_outward(float lo, float hi) {
  if constexpr (F16) {
    const __half a = UP ? __float2half_ru(lo) : __float2half_rd(lo);
    const __half b = UP ? __float2half_ru(hi) : __float2half_rd(hi);
    return static_cast<uint32_t>(__half_as_ushort(a)) |
           (static_cast<uint32_t>(__half_as_ushort(b)) << 16);
  } else {
    const __nv_bfloat16 a = UP ? __float2bfloat16_ru(lo) : __float2bfloat16_rd(lo);
    const __nv_bfloat16 b = UP ? __float2bfloat16_ru(hi) : __float2bfloat16_rd(hi);
    return static_cast<uint32_t>(__bfloat16_as_ushort(a)) |
           (static_cast<uint32_t>(__bfloat16_as_ushort(b)) << 16);
  }
}

// MULTI: pages of several blocks (S > 16).
template <int D, bool F16, bool MULTI>
__global__ void __launch_bounds__(kThreads, MULTI ? 3 : 5) meta_fp8_kernel(const MetaFp8Args a) {
  constexpr int kVec = D / 16;  // 16-byte vectors per row
  griddep_launch_dependents();
  griddep_wait();
  // every page, or those that an append changed
  const int pages = a.fresh.slots > 0 ? a.fresh.slots : a.P;
  const int64_t total = static_cast<int64_t>(a.B) * a.Hkv * pages * kVec;
  for (int64_t idx = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; idx < total;
       idx += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int v = static_cast<int>(idx % kVec);
    const int64_t bh = idx / kVec / pages;
    const int h = static_cast<int>(bh % a.Hkv);
    const int b = static_cast<int>(bh / a.Hkv);
    const int Nb = seq_len_of(a.lens, b, a.N);
    const int page = static_cast<int>(idx / kVec % pages) +
                     (a.fresh.slots > 0 ? first_new_page(a.fresh, b, Nb, a.S) : 0);
    // past a shorter sequence, or an empty one: not written
    if (page > page_of(Nb - 1, a.S) || (a.lens != nullptr && a.lens[b] <= 0)) continue;
    const int t0 = page * a.S;  // a metadata page of S tokens
    const int nt = min(a.S, Nb - t0);
    float mn[16], mx[16];
    if constexpr (MULTI) {
#pragma unroll
      for (int i = 0; i < 16; ++i) mn[i] = INFINITY, mx[i] = -INFINITY;
    }
#pragma unroll 1
    for (int c0 = 0; c0 < (MULTI ? nt : 1); c0 += kPage) {
      const int cp = (t0 + c0) / kPage;  // cache page
      const int ntc = min(kPage, nt - c0);
      int64_t at, so;
      if (a.bt != nullptr) {  // the page's pool block (clamped)
        const int64_t blk = min(max(a.bt[b * a.bts + cp], 0), a.nblocks - 1);
        at = blk * a.sb + static_cast<int64_t>((t0 + c0) % kPage) * D;
        so = blk * a.scale.sb;
      } else {
        at = b * a.sb + static_cast<int64_t>(t0 + c0) * D;
        so = b * a.scale.sb + cp;
      }
      const uint8_t* src = a.codes + at + h * a.sh + 16 * v;
      const float s = a.scale.scale[so + h * a.scale.sh];
      __half2 lo[8], hi[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        lo[u] = __half2half2(__ushort_as_half(0x7c00));  // +inf
        hi[u] = __half2half2(__ushort_as_half(0xfc00));  // -inf
      }
      uint4 x[kPage];
#pragma unroll
      for (int t = 0; t < kPage; ++t)
        if (t < ntc) x[t] = __ldcs(reinterpret_cast<const uint4*>(src + t * D));
#pragma unroll
      for (int t = 0; t < kPage; ++t) {
        if (t < ntc) {
          const uint32_t w[4] = {x[t].x, x[t].y, x[t].z, x[t].w};
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const __half2 y = codes2(w[u / 2] >> (16 * (u & 1)));
            lo[u] = __hmin2(lo[u], y);
            hi[u] = __hmax2(hi[u], y);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float m0 = __fmul_rd(__low2float(lo[u]), s), m1 = __fmul_rd(__high2float(lo[u]), s);
        const float M0 = __fmul_ru(__low2float(hi[u]), s), M1 = __fmul_ru(__high2float(hi[u]), s);
        mn[2 * u] = MULTI ? fminf(mn[2 * u], m0) : m0;
        mn[2 * u + 1] = MULTI ? fminf(mn[2 * u + 1], m1) : m1;
        mx[2 * u] = MULTI ? fmaxf(mx[2 * u], M0) : M0;
        mx[2 * u + 1] = MULTI ? fmaxf(mx[2 * u + 1], M1) : M1;
      }
    }
    const int64_t o = (bh * a.P + page) * D + 16 * v;
    uint4* omin = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.meta_min) + o);
    uint4* omax = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.meta_max) + o);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* m = mn + 8 * i;
      const float* M = mx + 8 * i;
      omin[i] = make_uint4(pack_outward<F16, false>(m[0], m[1]), pack_outward<F16, false>(m[2], m[3]),
                           pack_outward<F16, false>(m[4], m[5]), pack_outward<F16, false>(m[6], m[7]));
      omax[i] = make_uint4(pack_outward<F16, true>(M[0], M[1]), pack_outward<F16, true>(M[2], M[3]),
                           pack_outward<F16, true>(M[4], M[5]), pack_outward<F16, true>(M[6], M[7]));
    }
  }
}

template <bool MULTI>
cudaError_t launch_t(int d, bool f16, const MetaFp8Args& a, dim3 grid, cudaStream_t s) {
  const dim3 block(kThreads);
  if (d == 128)
    return f16 ? launch_pdl(meta_fp8_kernel<128, true, MULTI>, grid, block, 0, s, a)
               : launch_pdl(meta_fp8_kernel<128, false, MULTI>, grid, block, 0, s, a);
  return f16 ? launch_pdl(meta_fp8_kernel<64, true, MULTI>, grid, block, 0, s, a)
             : launch_pdl(meta_fp8_kernel<64, false, MULTI>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_meta_fp8(int d, bool f16, const MetaFp8Args& a, cudaStream_t s) {
  const int64_t work =
      static_cast<int64_t>(a.B) * a.Hkv * (a.fresh.slots > 0 ? a.fresh.slots : a.P) * (d / 16);
  const int64_t blocks = ceil_div(work, kThreads);
  const dim3 grid(static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30)));
  return a.S > kPage ? launch_t<true>(d, f16, a, grid, s) : launch_t<false>(d, f16, a, grid, s);
}

}  // namespace dkv
