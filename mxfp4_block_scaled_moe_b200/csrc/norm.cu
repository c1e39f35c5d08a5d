// Residual addition, root-mean-square norm and the 8-bit cast in one pass over the rows:
//   h = bf16(x + residual)          (h = x without a residual; written to sum_out)
//   r = 1 / sqrt(sum(h^2) / H + eps)
//   y = bf16(h w r),   q = e4m3(h w f)
// with f = r / s for a static scale s, or f = 448 / max|h w| and the token's scale
// s_t = r max|h w| / 448 written out (1 for a row of zeros). The sum of squares, the
// maximum, r and the products are fp32; h is rounded to bf16 before the norm because
// that is the residual stream that later layers read, and y / q are the only other
// roundings. h w is formed once and multiplied by the row's factor, so a row needs one
// reduction (sum and maximum together) and no division per element.
//
// Bound by HBM: a row is read once, held packed in registers (16 bytes per vector of 8)
// across the reduction, and every output is written once.
//
// One CTA per row, or one warp per row for many short rows; the rule and what it measured
// stand at launch_rmsnorm. 4096 x 2880 with a residual and a static scale (82.6 MB): 15.8 us,
// 5.2 TB/s; 16384 x 2880 to bf16 (377 MB): 58.8 us, 6.4 TB/s. CTAs that walk the rows with the next
// one's loads in flight were no faster (17.5 and 69 us).
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "launchers.h"

namespace mxmoe {
namespace {

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t add_bf16(uint32_t a, uint32_t b) {
  return pack_bf16(bf_lo(a) + bf_lo(b), bf_hi(a) + bf_hi(b));
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// (sum, max) over the row's threads; every thread gets both.
template <bool kWarp>
__device__ __forceinline__ float2 row_reduce(float s, float m, float2* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if (kWarp) return make_float2(s, m);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(s, m);
  __syncthreads();
  const int l = threadIdx.x & 31;
  const float2 v = l < warps ? buf[l] : make_float2(0.f, 0.f);
  s = v.x;
  m = v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  return make_float2(s, m);
}

// The thread's products v = h w and its share of sum(h^2) and max|v|. kScaled: h times `by`
// throughout, and the products times `up`, which the smaller of either factor takes: products below
// 2^-96 times 2^96 then stay in range whatever the factors (a zero by a weight of 2^32 first of all).
template <int kVec, bool kMax, bool kScaled>
__device__ __forceinline__ void row_stats(const uint4 (&h)[kVec], const uint4 (&w)[kVec], float by, float up,
                                          float (&v)[kVec][8], float& s, float& m) {
  s = 0.f;
  m = 0.f;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const uint32_t hu[4] = {h[j].x, h[j].y, h[j].z, h[j].w}, wu[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = bf_lo(hu[i]), b = bf_hi(hu[i]), wa = bf_lo(wu[i]), wb = bf_hi(wu[i]);
      if (kScaled) {
        a *= by;
        b *= by;
      }
      s = fmaf(a, a, s);
      s = fmaf(b, b, s);
      if (kScaled) {
        (fabsf(a) < fabsf(wa) ? a : wa) *= up;
        (fabsf(b) < fabsf(wb) ? b : wb) *= up;
      }
      v[j][2 * i] = a * wa;
      v[j][2 * i + 1] = b * wb;
      if (kMax) m = fmaxf(m, fmaxf(fabsf(v[j][2 * i]), fabsf(v[j][2 * i + 1])));
    }
  }
}

// kToken: one scale per token. kWarp: a warp per row (blockDim.x / 32 rows per CTA), else a CTA per row.
template <int kVec, bool kWarp, bool kToken>
__global__ void __launch_bounds__(kWarp ? 128 : 512) rmsnorm_kernel(NormArgs p) {
  __shared__ float2 buf[2][16];
  const int lanes = kWarp ? 32 : blockDim.x;
  const int tid = kWarp ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t t = kWarp ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  griddep_launch_dependents();
  griddep_wait();
  if (kWarp && t >= p.T) return;
  const int nv = p.H >> 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint4* x = reinterpret_cast<const uint4*>(p.x + t * p.ldx);
  const uint4* wp = reinterpret_cast<const uint4*>(p.weight);
  uint4 h[kVec], w[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) h[j] = tid + j * lanes < nv ? __ldcs(x + tid + j * lanes) : zero;
  if (p.residual) {
    const uint4* res = reinterpret_cast<const uint4*>(p.residual + t * p.ldr);
    uint4 r[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) r[j] = tid + j * lanes < nv ? __ldcs(res + tid + j * lanes) : zero;
#pragma unroll
    for (int j = 0; j < kVec; ++j) w[j] = tid + j * lanes < nv ? __ldg(wp + tid + j * lanes) : zero;
    uint4* so = reinterpret_cast<uint4*>(p.sum_out + t * p.H);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      h[j] = make_uint4(add_bf16(h[j].x, r[j].x), add_bf16(h[j].y, r[j].y), add_bf16(h[j].z, r[j].z),
                        add_bf16(h[j].w, r[j].w));
      if (tid + j * lanes < nv) so[tid + j * lanes] = h[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) w[j] = tid + j * lanes < nv ? __ldg(wp + tid + j * lanes) : zero;
  }

  float v[kVec][8], s, m, up = 1.0f, eps = p.eps;
  row_stats<kVec, kToken, false>(h, w, 1.0f, 1.0f, v, s, m);
  float2 st = row_reduce<kWarp>(s, m, buf[0]);
  // Powers of two that keep rare rows inside fp32: squares past its range (|h| above about
  // 2^63; eps is then below half an ulp of the mean), and products too small to divide by.
  const bool big = !(st.x <= FLT_MAX), small = kToken && st.y < 0x1p-96f;
  if (big || small) {
    if (big) eps = 0.f;
    if (small) up = 0x1p96f;
    row_stats<kVec, kToken, true>(h, w, big ? 0x1p-96f : 1.0f, up, v, s, m);
    st = row_reduce<kWarp>(s, m, buf[1]);
  }
  const float r = rsqrtf(fmaf(st.x, 1.0f / static_cast<float>(p.H), eps));
  const float f = r / up;
  float fq = f;
  if (kToken) {
    if (st.y > 0.f) fq = 448.0f / st.y;
    if (tid == 0) p.q_scale[t] = st.y > 0.f ? f * st.y / 448.0f : 1.0f;
  } else if (p.q) {
    fq = f / p.s;
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    if (tid + j * lanes >= nv) break;
    const float(&a)[8] = v[j];
    if (p.y)
      reinterpret_cast<uint4*>(p.y + t * p.H)[tid + j * lanes] =
          make_uint4(pack_bf16(a[0] * f, a[1] * f), pack_bf16(a[2] * f, a[3] * f), pack_bf16(a[4] * f, a[5] * f),
                     pack_bf16(a[6] * f, a[7] * f));
    if (p.q)
      reinterpret_cast<uint2*>(p.q + t * p.H)[tid + j * lanes] =
          make_uint2(pack_e4m3(a[0] * fq, a[1] * fq, a[2] * fq, a[3] * fq),
                     pack_e4m3(a[4] * fq, a[5] * fq, a[6] * fq, a[7] * fq));
  }
}

template <int kVec, bool kWarp>
cudaError_t launch_variant(const NormArgs& p, unsigned grid, int threads, cudaStream_t st) {
  return p.q_scale ? launch_early(rmsnorm_kernel<kVec, kWarp, true>, dim3(grid), threads, 0, 0, st, p)
                   : launch_early(rmsnorm_kernel<kVec, kWarp, false>, dim3(grid), threads, 0, 0, st, p);
}

}  // namespace

// Few rows (fewer than four for every SM): one vector a thread, the shortest chain. Many rows:
// four 16-byte loads in flight a thread, so two vectors with a residual and four without;
// rows of up to 512 values then take a warp each. On a B200 at 4096 x 2880 with a residual,
// one vector against two: 17.1 / 15.8 us (static scale), 19.2 / 17.8 us (token scale). At 9973 x 4096
// without one, one / two / four vectors: 36.9 / 29.4 / 27.5 us. At 16000 x 512 with one, a warp per
// row 12.4 us, a CTA 17.8 us.
//
// Longer rows hold more a thread: two vectors up to 8192 values, four up to 16384, eight above. 4096 rows
// with a residual, static and token scales: H = 8192 38 and 43 us (6.1 and 5.5 TB/s), 16384 73 and
// 107, 32768 185 and 224 (5.1 and 4.2 TB/s); one row of 32768 4.8 and 7.6. Token scales keep the
// products beside the row: at eight vectors that is past the 128 registers of 512 threads, and 352
// bytes a thread spill.
cudaError_t launch_rmsnorm(const NormArgs& p, int sms, cudaStream_t st) {
  const int nv = p.H / 8;
  const bool many = p.T >= 4 * sms;
  if (many && nv <= 64) {
    const unsigned grid = static_cast<unsigned>(cdiv(p.T, 4));
    return nv <= 32 ? launch_variant<1, true>(p, grid, 128, st) : launch_variant<2, true>(p, grid, 128, st);
  }
  const unsigned grid = static_cast<unsigned>(p.T);
  const auto threads = [nv](int vec) { return static_cast<int>(32 * cdiv(nv, 32 * vec)); };
  if (!many && nv <= 512) return launch_variant<1, false>(p, grid, threads(1), st);
  if (nv <= 1024 && (p.residual || nv > 512 || !many)) return launch_variant<2, false>(p, grid, threads(2), st);
  if (nv <= 2048) return launch_variant<4, false>(p, grid, threads(4), st);
  return launch_variant<8, false>(p, grid, threads(8), st);
}

}  // namespace mxmoe
