// Append to a paged MXFP4 key/value cache: row t of k and v, (Hkv, D) bf16, is quantized along
// D and written at slot slots[t] (page slot / page_size, place slot % page_size). The blocks
// are those of mxfp4_quantize, bit for bit: scale byte max(0, exponent of amax - 2), each value
// times 2^-e to the nearest e2m1 value, ties to the even code (the conversion instruction's
// own rounding), magnitudes past 6 saturating, the sign bit kept; a NaN counts as a zero of its sign.
//
// Cache layout: blocks (page, head, place, D/2), scales (page, head, place, D/32): a head's
// places in a page are one contiguous run, which is what the attention kernel streams.
//
// Bound by HBM for long batches and by the launch for decode steps. A thread holds 8
// consecutive values of k and of v (one 16-byte load each), four threads a 32-value block, so
// a block's largest magnitude is two shuffles; it writes 4 bytes of codes. In long batches a
// warp takes neighbouring tokens of one head, whose places (and scale bytes) lie side by side
// in a page, and a thread two pieces at a time.
#include <algorithm>

#include <cuda_fp4.h>

#include "common.cuh"
#include "launchers.h"

namespace mxmoe {
namespace {

constexpr int kThreads = 128;

// largest magnitude of a block, as bf16 bits: their order is the values' order, and NaN's lie above
__device__ __forceinline__ uint32_t largest(const uint4& u) {
  uint32_t top = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  return max(top >> 16, top & 0xFFFFu);
}

__device__ __forceinline__ uint32_t without_nan(uint32_t u) {
  return u & ~(__vcmpgtu2(u & 0x7FFF7FFFu, 0x7F807F80u) & 0x7FFF7FFFu);
}

// eight values of a block whose largest magnitude is `top`
__device__ __forceinline__ void quantize8(const uint4& v, uint32_t top, uint32_t& codes, uint32_t& scale) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  scale = static_cast<uint32_t>(max(0, static_cast<int>(top >> 7) - 2));
  const float inv = __uint_as_float((254u - scale) << 23);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp4x2(make_float2(__uint_as_float(u[i] << 16) * inv, __uint_as_float(u[i] & 0xFFFF0000u) * inv),
                                    __NV_E2M1, cudaRoundNearest);
  codes = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

// A CTA takes 2^shift tokens: pieces in the order (head, token, piece of the row). kVecs: 8-value
// pieces of a row (a multiple of 4), 0 where only the call knows it.
template <int kVecs>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(KvAppendArgs p, int shift) {
  const int row_vecs = kVecs ? kVecs : p.D >> 3;
  const int D = 8 * row_vecs;
  const int units = (p.Hkv * row_vecs) << shift;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) << shift;
  constexpr int kAtOnce = 2;
  griddep_launch_dependents();
  griddep_wait();
  for (int first = threadIdx.x; first - static_cast<int>(threadIdx.x) < units; first += kAtOnce * kThreads) {
    int64_t slot[kAtOnce];
    uint4 k[kAtOnce], v[kAtOnce];
    int h[kAtOnce], piece[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int i = first + j * kThreads;
      const int row = i / row_vecs;
      piece[j] = i - row * row_vecs;
      h[j] = row >> shift;
      const int64_t t = t0 + (row & ((1 << shift) - 1));
      slot[j] = -1;
      k[j] = v[j] = make_uint4(0, 0, 0, 0);
      if (i < units && t < p.T) {
        const int at = h[j] * D + 8 * piece[j];
        slot[j] = __ldg(p.slots + t);
        k[j] = __ldcs(reinterpret_cast<const uint4*>(p.k + t * p.ldk + at));
        v[j] = __ldcs(reinterpret_cast<const uint4*>(p.v + t * p.ldv + at));
      }
    }
    uint32_t k_top[kAtOnce], v_top[kAtOnce], most = 0;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      k_top[j] = largest(k[j]);
      v_top[j] = largest(v[j]);
      most = max(most, max(k_top[j], v_top[j]));
    }
    if (__any_sync(0xffffffffu, most > 0x7F80u)) {
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        k[j] = make_uint4(without_nan(k[j].x), without_nan(k[j].y), without_nan(k[j].z), without_nan(k[j].w));
        v[j] = make_uint4(without_nan(v[j].x), without_nan(v[j].y), without_nan(v[j].z), without_nan(v[j].w));
        k_top[j] = largest(k[j]);
        v_top[j] = largest(v[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      uint32_t kc, ks, vc, vs;
      quantize8(k[j], k_top[j], kc, ks);
      quantize8(v[j], v_top[j], vc, vs);
      if (slot[j] < 0) continue;            // a padded row, or no row at all
      if (slot[j] >= p.num_slots) {
        set_device_error(p.err, MXMOE_EDEVICE);
        continue;
      }
      const int page = static_cast<int>(slot[j] >> p.page_shift);   // below 2^31: num_pages is
      const int place = static_cast<int>(slot[j]) & ((1 << p.page_shift) - 1);
      const int64_t row = static_cast<int64_t>(page) * (p.Hkv << p.page_shift) + ((h[j] << p.page_shift) + place);
      *reinterpret_cast<uint32_t*>(p.k_blocks + row * (D >> 1) + 4 * piece[j]) = kc;
      *reinterpret_cast<uint32_t*>(p.v_blocks + row * (D >> 1) + 4 * piece[j]) = vc;
      if ((piece[j] & 3) == 0) {
        p.k_scales[row * (D >> 5) + (piece[j] >> 2)] = static_cast<uint8_t>(ks);
        p.v_scales[row * (D >> 5) + (piece[j] >> 2)] = static_cast<uint8_t>(vs);
      }
    }
  }
}

}  // namespace

// Tokens per CTA: as many as give each of its threads its two pieces, fewer where that would leave
// SMs idle. 16384 tokens of 8 heads of 64 (42.5 MB), slices of a fused projection: 9.9 us, 4.3 TB/s;
// 1024 tokens 2.8. Launch, first loads and tail are that 2.8 of it; in the rest (5.6 TB/s) the SMs issue in
// 0.66 of the cycles. With 256 threads a CTA 10.4 and 3.5, 512 11.1 and 4.8, 64 11.0 and 2.9; one piece a
// thread 10.9 and 2.2, four 10.4 and 3.6.
cudaError_t launch_kv_append(const KvAppendArgs& p, int sms, cudaStream_t st) {
  const int vecs = p.Hkv * (p.D / 8);
  int shift = 0;
  while ((vecs << shift) < 2 * kThreads && (static_cast<int64_t>(p.T) >> (shift + 1)) >= 2 * sms) ++shift;
  const unsigned grid = static_cast<unsigned>(cdiv(p.T, static_cast<int64_t>(1) << shift));
  const auto kernel = p.D == 64 ? kv_append_kernel<8> : p.D == 128 ? kv_append_kernel<16> : kv_append_kernel<0>;
  return launch_early(kernel, dim3(grid), kThreads, 0, 0, st, p, shift);
}

}  // namespace mxmoe
