// Append to a paged MXFP4 key/value cache: row t of k and v, (Hkv, D) bf16, is quantized along
// D and written at slot slots[t] (page slot / page_size, place slot % page_size). The blocks
// are those of mxfp4_quantize, bit for bit: scale byte max(0, exponent of amax - 2), each value
// times 2^-e to the nearest e2m1 value, ties to the even code (the conversion instruction's
// own rounding), magnitudes past 6 saturating, the sign bit kept.
//
// Cache layout: blocks (page, head, place, D/2), scales (page, head, place, D/32): a head's
// places in a page are one contiguous run, which is what the attention kernel streams.
//
// Bound by HBM for long batches and by the launch for decode steps. A thread holds 8
// consecutive values of k and of v (one 16-byte load each), four threads a 32-value block, so
// a block's largest magnitude is two shuffles; it writes 4 bytes of codes.
#include <algorithm>

#include <cuda_fp4.h>

#include "common.cuh"
#include "launchers.h"

namespace mxmoe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void quantize8(const uint4& v, uint32_t& codes, uint32_t& scale) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = 0;   // largest magnitude, as bf16 bits: their order is the values' order
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max((u[i] << 16) & 0x7FFF0000u, u[i] & 0x7FFF0000u));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  scale = static_cast<uint32_t>(max(0, static_cast<int>(top >> 23) - 2));
  const float inv = __uint_as_float((254u - scale) << 23);
  codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2(__uint_as_float(u[i] << 16) * inv, __uint_as_float(u[i] & 0xFFFF0000u) * inv);
    codes |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest)) << (8 * i);
  }
}

__global__ void __launch_bounds__(kThreads) kv_append_kernel(KvAppendArgs p, int per_block) {
  const int vecs = p.Hkv * (p.D >> 3);   // 8-value pieces of a token's row, a multiple of 4
  const int row_vecs = p.D >> 3;
  const int units = per_block * vecs;
  for (int first = 0; first < units; first += kThreads) {
    const int i = first + threadIdx.x;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * per_block + i / vecs;
    const bool live = i < units && t < p.T;
    const int vec = i % vecs;
    int64_t slot = -1;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (live) {
      slot = __ldg(p.slots + t);
      k = __ldcs(reinterpret_cast<const uint4*>(p.k + t * p.ldk) + vec);
      v = __ldcs(reinterpret_cast<const uint4*>(p.v + t * p.ldv) + vec);
    }
    uint32_t kc, ks, vc, vs;
    quantize8(k, kc, ks);
    quantize8(v, vc, vs);
    if (slot < 0) continue;               // a padded row, or no row at all
    if (slot >= p.num_slots) {
      set_device_error(p.err, MXMOE_EDEVICE);
      continue;
    }
    const int h = vec / row_vecs, piece = vec % row_vecs;
    const int64_t page = slot >> p.page_shift, place = slot & ((1 << p.page_shift) - 1);
    const int64_t row = ((page * p.Hkv + h) << p.page_shift) + place;
    *reinterpret_cast<uint32_t*>(p.k_blocks + row * (p.D >> 1) + 4 * piece) = kc;
    *reinterpret_cast<uint32_t*>(p.v_blocks + row * (p.D >> 1) + 4 * piece) = vc;
    if ((piece & 3) == 0) {
      p.k_scales[row * (p.D >> 5) + (piece >> 2)] = static_cast<uint8_t>(ks);
      p.v_scales[row * (p.D >> 5) + (piece >> 2)] = static_cast<uint8_t>(vs);
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& p, cudaStream_t st) {
  const int vecs = p.Hkv * (p.D / 8);
  const int per_block = std::max(1, kThreads / vecs);
  kv_append_kernel<<<static_cast<unsigned>(cdiv(p.T, per_block)), kThreads, 0, st>>>(p, per_block);
  return cudaGetLastError();
}

}  // namespace mxmoe
