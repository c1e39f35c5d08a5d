// Attention of a few queries per sequence over the paged MXFP4 cache (kv_append.cu's layout):
//   o = sum_j e^{z_j - m} v_j / (sum_j e^{z_j - m} + e^{sink - m}),  z_j = scale q.k_j,
// over the keys j that a query sees (causal from the sequence's end, an optional sliding
// window), for grouped-query heads: the G query heads of a key/value head and the Lq queries
// of a sequence are R = G Lq rows that read the same keys.
//
// Bound by HBM (0.53 bytes a value) with the expansion of 4-bit codes close behind, so codes
// are expanded once, in registers, straight into matrix-instruction operands:
//  - S^T = K Q^T by m16n8k16 (f16 operands, fp32 sums): 16 keys by 8 rows. Eight rows are what
//    a group of 8 heads gives one query, so no tensor work is wasted on padding; tcgen05's
//    64/128-row tiles would be mostly padding and would need the codes expanded through
//    shared memory. A key's e2m1 codes are exact in f16; its block scale multiplies the fp32
//    block sum instead of 32 values. Queries enter as f16 after an exact power-of-two shift
//    per row and 32-value block (largest magnitude to [2^14, 2^15): bf16's 8 bits survive down
//    to 2^-29 of the block's largest).
//  - O^T += V^T P^T: the value scales multiply the weights, p 2^(e_j - E + 15), where E is the
//    largest value exponent seen so far in that 32-value block; the weights are then rounded
//    to f16 (11 bits; absolute floor 2^-40 of the largest scale). Maximum, sum, and all
//    accumulators are fp32.
// Row maxima, sums and E stay with the warp and its accumulators are rescaled only in units
// where one of them grows.
//
// Work split: 32-key units of all (sequence, key/value head, row tile) items in one line; each
// CTA takes an equal run of them whatever the sequences' lengths (the lengths are on the
// device, so every CTA finds its run by itself), its warps take units in turn through private
// cp.async rings, without barriers between them, and join at an item's end. An item that ends
// up in several CTAs leaves fp32 partials in the caller's workspace, joined in CTA order by a
// second small kernel: nothing in the result depends on timing, and no counter outlives a call.
#include <algorithm>

#include "common.cuh"
#include "launchers.h"

namespace mxmoe {
namespace kva {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 32;          // keys per unit
constexpr int kMinUnits = 8;       // least units of a CTA's run: one per warp
constexpr int kCombineThreads = 256;

template <int D, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kBlocks = D / 32;               // MXFP4 blocks of a row
  static constexpr int kRowBytes = D / 2;
  static constexpr int kKV = kUnit * kRowBytes;        // bytes of a unit's keys (or values)
  static constexpr int kSc = kUnit * kBlocks;          // their scales
  static constexpr int kStageBytes = 2 * kKV + 2 * kSc + 16;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kJoinBytes = 2 * kWarps * kRows * 32 * 4;   // two 32-column slabs of every warp's rows
  static constexpr int kSmem = kWarps * kStages * kStageBytes + kJoinBytes;
};

// ------------------------------------------------------------------ small pieces ---
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// the four f16 pairs of a word of eight e2m1 codes, byte by byte (low nibble in the low half)
__device__ __forceinline__ void expand(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// e8m0 byte to fp32 (255 reads as infinity, 0 as 2^-127)
__device__ __forceinline__ float scale_f32(uint32_t byte) { return __uint_as_float(max(byte << 23, 0x00400000u)); }

// ------------------------------------------------------------------- work line -----
__device__ __forceinline__ int seq_len(const KvAttentionArgs& p, int b) {
  const int n = __ldg(p.seq_lens + b);
  const int64_t cap = static_cast<int64_t>(p.max_pages) << p.page_shift;
  if (n > cap) {   // more keys than the table has pages for
    set_device_error(p.err, MXMOE_EDEVICE);
    return static_cast<int>(cap);
  }
  return max(n, 0);
}

// first key of a sequence's units: the first that its first query sees, rounded down to a unit
__device__ __forceinline__ int first_key(const KvAttentionArgs& p, int len) {
  return p.window > 0 ? max(0, len - p.Lq + 1 - p.window) & ~(kUnit - 1) : 0;
}

__device__ __forceinline__ int units_of(const KvAttentionArgs& p, int len) {
  return max(1, (len - first_key(p, len) + kUnit - 1) / kUnit);   // an empty sequence still writes its zeros
}

// Position in the line of units: item j (key/value head and row tile) of sequence b.
struct Cursor {
  int b, j, len, first, units;
  int64_t start;   // of the item
  __device__ void load(const KvAttentionArgs& p) {
    len = seq_len(p, b);
    first = first_key(p, len);
    units = units_of(p, len);
  }
  __device__ void next(const KvAttentionArgs& p, int per_seq) {
    start += units;
    if (++j == per_seq) {
      j = 0;
      if (++b < p.B) load(p);
    }
  }
};

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += buf[w];
  __syncthreads();
  return v;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, (D == 64 || NT == 1) ? 2 : 1) kv_attention_kernel(const KvAttentionArgs p) {
  using S = Shape<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 s_ml[kWarps][S::kRows];
  __shared__ int64_t s_sum[kWarps];
  __shared__ int s_b;
  __shared__ int64_t s_base;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int per_seq = p.Hkv * p.RT;
  griddep_launch_dependents();   // the joining kernel may take its places; it waits for this one's end

  // ---- this CTA's run of units [t0, t1) of n ----
  int64_t mine = 0;
  for (int b = threadIdx.x; b < p.B; b += kThreads) mine += units_of(p, seq_len(p, b));
  const int64_t n = block_sum(mine, s_sum) * per_seq;
  const int64_t per = max(static_cast<int64_t>(kMinUnits), (n + gridDim.x - 1) / gridDim.x);
  const int64_t t0 = per * blockIdx.x, t1 = min(n, t0 + per);
  if (t0 >= n) return;
  {
    int64_t base = 0;   // units before this chunk of sequences
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      const int64_t u = b < p.B ? static_cast<int64_t>(units_of(p, seq_len(p, b))) * per_seq : 0;
      int64_t pre = u;   // inclusive over the warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += x;
      }
      if (lane == 31) s_sum[warp] = pre;
      __syncthreads();
      int64_t all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) pre += s_sum[w];
        all += s_sum[w];
      }
      const int64_t from = base + pre - u;
      if (u > 0 && from <= t0 && t0 < from + u) {
        s_b = b;
        s_base = from;
      }
      base += all;
      __syncthreads();
      if (t0 < base) break;
    }
  }
  Cursor cur;
  cur.b = s_b;
  cur.load(p);
  cur.j = static_cast<int>((t0 - s_base) / cur.units);
  cur.start = s_base + static_cast<int64_t>(cur.j) * cur.units;

  // ---- this warp's ring of units ----
  uint8_t* ring = smem + warp * S::kStages * S::kStageBytes;
  const uint32_t ring_u32 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  float* join = reinterpret_cast<float*>(smem + kWarps * S::kStages * S::kStageBytes);

  Cursor in = cur;           // of the next unit to load
  int64_t in_unit = t0 + warp;
  int pid0 = 0, pid1 = 0, in_key = 0;
  bool in_load0 = false, in_load1 = false;
  // looks up the pages of unit in_unit (16 keys from each: a page holds 16 keys or more)
  auto look = [&]() {
    if (in_unit >= t1) return;
    while (in_unit >= in.start + in.units) in.next(p, per_seq);
    in_key = in.first + kUnit * static_cast<int>(in_unit - in.start);
    const int lo = p.window > 0 ? max(0, in.len - p.Lq + 1 - p.window) : 0;   // keys that no query sees need no page
    in_load0 = in_key < in.len && in_key + 16 > lo;
    in_load1 = in_key + 16 < in.len && in_key + 32 > lo;
    const int32_t* row = p.block_table + static_cast<int64_t>(in.b) * p.max_pages;
    if (in_load0) pid0 = __ldg(row + (in_key >> p.page_shift));
    if (in_load1) pid1 = __ldg(row + ((in_key + 16) >> p.page_shift));
  };
  auto issue = [&](int stage) {
    if (in_unit < t1) {
      const uint32_t dst = ring_u32 + stage * S::kStageBytes;
      const bool ok0 = in_load0 && static_cast<uint32_t>(pid0) < static_cast<uint32_t>(p.num_pages);
      const bool ok1 = in_load1 && static_cast<uint32_t>(pid1) < static_cast<uint32_t>(p.num_pages);
      if (lane == 0) {
        if (ok0 != in_load0 || ok1 != in_load1) set_device_error(p.err, MXMOE_EDEVICE);   // a page outside the cache
        *reinterpret_cast<int*>(ring + stage * S::kStageBytes + 2 * S::kKV + 2 * S::kSc) = (ok0 ? 1 : 0) | (ok1 ? 2 : 0);
      }
      const int h = in.j / p.RT;
      const int in_page = in_key & ((1 << p.page_shift) - 1);
      const int in_page1 = (in_key + 16) & ((1 << p.page_shift) - 1);
      // cache rows of the unit's first and second 16 keys
      const int64_t r0 = ((static_cast<int64_t>(pid0) * p.Hkv + h) << p.page_shift) + in_page;
      const int64_t r1 = ((static_cast<int64_t>(pid1) * p.Hkv + h) << p.page_shift) + in_page1 - 16;
      constexpr int kChunks = S::kRowBytes / 16;   // 16-byte chunks of a row, one MXFP4 block each
#pragma unroll
      for (int i = 0; i < S::kKV / 512; ++i) {
        const int c = 32 * i + lane, key = c / kChunks, blk = c % kChunks;
        const bool second = key >= 16;
        if (second ? ok1 : ok0) {
          const int64_t off = ((second ? r1 : r0) + key) * S::kRowBytes + 16 * blk;
          // a row's chunks are permuted so that the eight rows of an operand load fall in
          // different banks
          const int sw = kChunks == 2 ? blk ^ ((key >> 2) & 1) : blk ^ ((key >> 1) & 3);
          const uint32_t at = dst + key * S::kRowBytes + 16 * sw;
          cp_async16(at, p.k_blocks + off);
          cp_async16(at + S::kKV, p.v_blocks + off);
        }
      }
      constexpr int kScChunks = S::kSc / 16, kScKeys = kUnit / kScChunks;   // keys of a 16-byte chunk of scales
      if (lane < 2 * kScChunks) {
        const bool val = lane >= kScChunks;
        const int key = (lane % kScChunks) * kScKeys;
        const bool second = key >= 16;
        if (second ? ok1 : ok0)
          cp_async16(dst + 2 * S::kKV + lane * 16,
                     (val ? p.v_scales : p.k_scales) + ((second ? r1 : r0) + key) * S::kBlocks);
      }
      in_unit += kWarps;
    }
    cp_async_commit();
    look();
  };
  look();
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) issue(s);

  int stage = 0, piece = 0;
  for (int64_t at = t0; at < t1; ++piece) {
    // ---- one item: rows, queries ----
    const int64_t item_end = cur.start + cur.units, end = min(t1, item_end);
    const int h = cur.j / p.RT, rt = cur.j % p.RT;
    const int len = cur.len;
    const int row0 = rt * S::kRows;
    uint32_t qf[NT][S::kBlocks][4];
    float qs[NT][S::kBlocks][2];          // of rows 2t, 2t + 1: score scale in base 2, undoing the f16 shift
    int hi[NT][2], lo[NT][2];             // keys [lo, hi) that those rows see
    int full_lo = 0, full_hi = 0x7FFFFFFF, seen_lo = 0x7FFFFFFF, seen_hi = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = row0 + 8 * i + g;
      const bool real = r < p.R;
      const int qi = real ? r / p.G : 0, hd = h * p.G + (real ? r % p.G : 0);
      const uint16_t* src = p.q + (static_cast<int64_t>(cur.b) * p.Lq + qi) * p.q_stride + static_cast<int64_t>(hd) * D;
#pragma unroll
      for (int k = 0; k < S::kBlocks; ++k) {
        const uint4 u = real ? __ldg(reinterpret_cast<const uint4*>(src + 32 * k + 8 * t)) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t top = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) top = max(top, max((w[x] << 16) & 0x7FFF0000u, w[x] & 0x7FFF0000u));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(14 - exponent) and its inverse, both normal fp32
        const int ex = min(max(static_cast<int>(top >> 23), 16), 254);
        const float up = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          qf[i][k][x] = pack_f16(__uint_as_float(w[x] << 16) * up, __uint_as_float(w[x] & 0xFFFF0000u) * up);
        qs[i][k][0] = __shfl_sync(0xffffffffu, down, 8 * t) * p.scale_log2;
        qs[i][k][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4) * p.scale_log2;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rr = row0 + 8 * i + 2 * t + x;
        hi[i][x] = rr < p.R ? len - p.Lq + rr / p.G + 1 : 0;
        lo[i][x] = p.window > 0 ? hi[i][x] - p.window : 0;
      }
    }
    {
      const int q_first = row0 / p.G, q_last = min(row0 + S::kRows, p.R) - 1;
      const int hi_first = len - p.Lq + q_first + 1, hi_last = len - p.Lq + q_last / p.G + 1;
      full_hi = hi_first;
      seen_hi = max(hi_last, 0);
      full_lo = p.window > 0 ? max(0, hi_last - p.window) : 0;
      seen_lo = p.window > 0 ? max(0, hi_first - p.window) : 0;
    }

    float o[NT][S::kBlocks][2][4];
    float m[NT][2], l[NT][2];
    int E[S::kBlocks];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int k = 0; k < S::kBlocks; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][k][0][x] = o[i][k][1][x] = 0.f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < S::kBlocks; ++k) E[k] = 0;

    // ---- its units that fall to this warp ----
    const int skip = static_cast<int>((at - t0) % kWarps);
    for (int64_t u = at + (warp - skip + kWarps) % kWarps; u < end; u += kWarps) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      const int next = stage + S::kStages - 1;
      issue(next >= S::kStages ? next - S::kStages : next);
      const uint8_t* sk = ring + stage * S::kStageBytes;
      const uint8_t* sv = sk + S::kKV;
      const uint8_t* ssk = sv + S::kKV;
      const uint8_t* ssv = ssk + S::kSc;
      const int pages = *reinterpret_cast<const int*>(ssv + S::kSc);
      const int key0 = cur.first + kUnit * static_cast<int>(u - cur.start);
      stage = stage + 1 == S::kStages ? 0 : stage + 1;

      // scores, base 2
      float s[NT][2][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int ka = 16 * half + g, kb = ka + 8;
        uint32_t sca, scb;
        if constexpr (S::kBlocks == 2) {
          sca = *reinterpret_cast<const uint16_t*>(ssk + 2 * ka);
          scb = *reinterpret_cast<const uint16_t*>(ssk + 2 * kb);
        } else {
          sca = *reinterpret_cast<const uint32_t*>(ssk + 4 * ka);
          scb = *reinterpret_cast<const uint32_t*>(ssk + 4 * kb);
        }
#pragma unroll
        for (int k = 0; k < S::kBlocks; ++k) {
          const int swa = S::kBlocks == 2 ? k ^ ((ka >> 2) & 1) : k ^ ((ka >> 1) & 3);
          const int swb = S::kBlocks == 2 ? k ^ ((kb >> 2) & 1) : k ^ ((kb >> 1) & 3);
          uint32_t a[4], b[4];
          expand(*reinterpret_cast<const uint32_t*>(sk + ka * S::kRowBytes + 16 * swa + 4 * t), a);
          expand(*reinterpret_cast<const uint32_t*>(sk + kb * S::kRowBytes + 16 * swb + 4 * t), b);
          const float fa = scale_f32((sca >> (8 * k)) & 0xFFu), fb = scale_f32((scb >> (8 * k)) & 0xFFu);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(c, a[0], b[0], a[1], b[1], qf[i][k][0], qf[i][k][1]);
            mma_f16(c, a[2], b[2], a[3], b[3], qf[i][k][2], qf[i][k][3]);
            if (k == 0) {
              s[i][half][0] = c[0] * (fa * qs[i][k][0]);
              s[i][half][1] = c[1] * (fa * qs[i][k][1]);
              s[i][half][2] = c[2] * (fb * qs[i][k][0]);
              s[i][half][3] = c[3] * (fb * qs[i][k][1]);
            } else {
              s[i][half][0] = fmaf(c[0], fa * qs[i][k][0], s[i][half][0]);
              s[i][half][1] = fmaf(c[1], fa * qs[i][k][1], s[i][half][1]);
              s[i][half][2] = fmaf(c[2], fb * qs[i][k][0], s[i][half][2]);
              s[i][half][3] = fmaf(c[3], fb * qs[i][k][1], s[i][half][3]);
            }
          }
        }
      }
      // the lane's key's value scales (0 for a key that no row sees: what lies there does not count)
      uint32_t ev;
      if constexpr (S::kBlocks == 2) ev = *reinterpret_cast<const uint16_t*>(ssv + 2 * lane);
      else ev = *reinterpret_cast<const uint32_t*>(ssv + 4 * lane);
      const bool edge = pages != 3 || key0 < full_lo || key0 + kUnit > full_hi;
      if (edge) {
        const int key = key0 + lane;
        if (key < seen_lo || key >= seen_hi || !((pages >> (lane >> 4)) & 1)) ev = 0;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int kk = key0 + 16 * half + g + 8 * (x >> 1);
#pragma unroll
            for (int i = 0; i < NT; ++i)
              if (kk < lo[i][x & 1] || kk >= hi[i][x & 1] || !((pages >> half) & 1)) s[i][half][x] = -INFINITY;
          }
      }
      // does a maximum grow?
      float mx[NT][2];
      bool grows = false;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[i][x] = fmaxf(fmaxf(s[i][0][x], s[i][0][x + 2]), fmaxf(s[i][1][x], s[i][1][x + 2]));
          grows |= mx[i][x] > m[i][x];
        }
#pragma unroll
      for (int k = 0; k < S::kBlocks; ++k) grows |= static_cast<int>((ev >> (8 * k)) & 0xFFu) > E[k];
      if (__any_sync(0xffffffffu, grows)) {
        int dE[S::kBlocks];
#pragma unroll
        for (int k = 0; k < S::kBlocks; ++k) {
          const int e = max(E[k], static_cast<int>(__reduce_max_sync(0xffffffffu, (ev >> (8 * k)) & 0xFFu)));
          dE[k] = E[k] - e;
          E[k] = e;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float v = mx[i][x];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float nm = fmaxf(m[i][x], v);
            const float d = nm == -INFINITY ? 0.f : m[i][x] - nm;   // nothing seen yet: all zero anyway
            m[i][x] = nm;
            l[i][x] *= ex2(d);
#pragma unroll
            for (int k = 0; k < S::kBlocks; ++k) {
              const float f = ex2(d + static_cast<float>(dE[k]));
              o[i][k][0][x] *= f;
              o[i][k][0][x + 2] *= f;
              o[i][k][1][x] *= f;
              o[i][k][1][x + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float base = m[i][x] == -INFINITY ? 0.f : m[i][x];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            s[i][half][x] = ex2(s[i][half][x] - base);
            s[i][half][x + 2] = ex2(s[i][half][x + 2] - base);
            l[i][x] += s[i][half][x] + s[i][half][x + 2];
          }
        }
      // O^T += V^T P^T
      const uint32_t pick = g < 4 ? 0x5410u : 0x7632u;   // which half of a code word the lane's four columns are in
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t eva, evb;   // value scales of keys g and g + 8
        if constexpr (S::kBlocks == 2) {
          eva = *reinterpret_cast<const uint16_t*>(ssv + 2 * (16 * half + g));
          evb = *reinterpret_cast<const uint16_t*>(ssv + 2 * (16 * half + g + 8));
        } else {
          eva = *reinterpret_cast<const uint32_t*>(ssv + 4 * (16 * half + g));
          evb = *reinterpret_cast<const uint32_t*>(ssv + 4 * (16 * half + g + 8));
        }
        const int v0 = 16 * half + 2 * t;   // the lane's keys v0, v0 + 1, v0 + 8, v0 + 9
#pragma unroll
        for (int k = 0; k < S::kBlocks; ++k) {
          // 2^(15 + e - E) in [0, 2^15]; a masked key's scale may be anything, its weight is 0
          const int da = static_cast<int>((eva >> (8 * k)) & 0xFFu) - E[k] + 142;
          const int db = static_cast<int>((evb >> (8 * k)) & 0xFFu) - E[k] + 142;
          const float fa = __uint_as_float(static_cast<uint32_t>(min(max(da, 0), 142)) << 23);
          const float fb = __uint_as_float(static_cast<uint32_t>(min(max(db, 0), 142)) << 23);
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = v0 + (x & 1) + 8 * (x >> 1);
            const int sw = S::kBlocks == 2 ? k ^ ((key >> 2) & 1) : k ^ ((key >> 1) & 3);
            w[x] = *reinterpret_cast<const uint32_t*>(sv + key * S::kRowBytes + 16 * sw + 4 * (g & 3));
          }
          // pair the keys' codes of one column in a byte: columns 0, 2 in `even`, 1, 3 in `odd`;
          // bytes 0, 1 of keys (v0, v0 + 1), bytes 2, 3 of keys (v0 + 8, v0 + 9)
          const uint32_t first = __byte_perm(w[0], w[2], pick), second = __byte_perm(w[1], w[3], pick);
          const uint32_t even = (first & 0x0F0F0F0Fu) | ((second << 4) & 0xF0F0F0F0u);
          const uint32_t odd = ((first >> 4) & 0x0F0F0F0Fu) | (second & 0xF0F0F0F0u);
          uint32_t ae[4], ao[4];
          expand(even, ae);
          expand(odd, ao);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const uint32_t b0 = transpose8x8(pack_f16(s[i][half][0] * fa, s[i][half][1] * fa));
            const uint32_t b1 = transpose8x8(pack_f16(s[i][half][2] * fb, s[i][half][3] * fb));
            mma_f16(o[i][k][0], ae[0], ao[0], ae[2], ao[2], b0, b1);
            mma_f16(o[i][k][1], ae[1], ao[1], ae[3], ao[3], b0, b1);
          }
        }
      }
      __syncwarp();
    }

    // ---- join the warps ----
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float v = l[i][x];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        if (g == 0) s_ml[warp][8 * i + 2 * t + x] = make_float2(m[i][x], v);
      }
    __syncthreads();
    const bool whole = cur.start >= t0 && item_end <= t1;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (piece > 0 ? 1 : 0);
    // the thread's output rows: (threadIdx / 32) + 8 i
    float inv[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = warp + 8 * i, row = row0 + r;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][r].x);
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += s_ml[w][r].y * ex2(s_ml[w][r].x - base);
      inv[i] = 1.f;
      if (whole) {
        if (p.sinks && row < p.R) sum += ex2(__ldg(p.sinks + h * p.G + row % p.G) * 1.44269504088896f - base);
        inv[i] = sum > 0.f ? 1.f / sum : 0.f;
      } else if (lane == 0) {
        p.part_ml[slot * S::kRows + r] = make_float2(top, sum);
      }
    }
    float f[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 8 * i + 2 * t + x;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][r].x);
        f[i][x] = top == -INFINITY ? -INFINITY : m[i][x] - top;
      }
#pragma unroll
    for (int k = 0; k < S::kBlocks; ++k) {
      float* slab = join + (k & 1) * (kWarps * S::kRows * 32);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float mul = ex2(f[i][x] + static_cast<float>(E[k] - 142));
          *reinterpret_cast<float4*>(slab + (warp * S::kRows + 8 * i + 2 * t + x) * 32 + 8 * (g & 3) + 4 * (g >> 2)) =
              make_float4(o[i][k][0][x] * mul, o[i][k][0][x + 2] * mul, o[i][k][1][x] * mul, o[i][k][1][x + 2] * mul);
        }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int r = warp + 8 * i, row = row0 + r;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += slab[(w * S::kRows + r) * 32 + lane];
        if (!whole) {
          p.part[(slot * S::kRows + r) * D + 32 * k + lane] = v;
        } else if (row < p.R) {
          const int64_t tok = static_cast<int64_t>(cur.b) * p.Lq + row / p.G;
          p.out[(tok * p.Hkv * p.G + h * p.G + row % p.G) * D + 32 * k + lane] = f32_to_bf16_bits_rn(v * inv[i]);
        }
      }
    }
    // the item's first CTA says where its parts lie (slot, first and last CTA); -1: no parts
    if (threadIdx.x == 0 && cur.start >= t0) {
      const int64_t item = static_cast<int64_t>(cur.b) * per_seq + cur.j;
      p.desc[item] = whole ? make_int4(-1, 0, 0, 0)
                           : make_int4(static_cast<int>(slot), static_cast<int>(blockIdx.x),
                                       static_cast<int>((item_end - 1) / per), 0);
    }
    at = end;
    if (at == item_end && at < t1) cur.next(p, per_seq);
  }
  cp_async_wait<0>();
}

// Joins the parts of the items that several CTAs shared, in CTA order.
template <int D, int NT>
__global__ void __launch_bounds__(kCombineThreads) kv_attention_join_kernel(const KvAttentionArgs p) {
  using S = Shape<D, NT>;
  griddep_wait();
  const int per_seq = p.Hkv * p.RT;
  constexpr int kLanes = D / 4;                               // threads of a row, four columns each
  constexpr int kPass = kCombineThreads / kLanes;             // rows at a time
  const int64_t items = static_cast<int64_t>(p.B) * per_seq;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int4 d = p.desc[item];
    if (d.x < 0) continue;
    const int b = static_cast<int>(item / per_seq), j = static_cast<int>(item % per_seq);
    const int h = j / p.RT, row0 = (j % p.RT) * S::kRows;
    for (int r = threadIdx.x / kLanes; r < S::kRows; r += kPass) {
      const int row = row0 + r, c = 4 * (threadIdx.x % kLanes);
      if (row >= p.R) break;
      float top = -INFINITY;
      for (int cta = d.y; cta <= d.z; ++cta) {
        const int64_t slot = cta == d.y ? d.x : 2 * static_cast<int64_t>(cta);
        top = fmaxf(top, p.part_ml[slot * S::kRows + r].x);
      }
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int cta = d.y; cta <= d.z; ++cta) {
        const int64_t slot = cta == d.y ? d.x : 2 * static_cast<int64_t>(cta);
        const float2 ml = p.part_ml[slot * S::kRows + r];
        const float4 x = *reinterpret_cast<const float4*>(p.part + (slot * S::kRows + r) * D + c);
        const float f = ex2(ml.x - base);
        sum = fmaf(f, ml.y, sum);
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
      }
      if (p.sinks) sum += ex2(__ldg(p.sinks + h * p.G + row % p.G) * 1.44269504088896f - base);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const int64_t tok = static_cast<int64_t>(b) * p.Lq + row / p.G;
      const uint32_t lo = f32_to_bf16_bits_rn(v.x * inv) | (static_cast<uint32_t>(f32_to_bf16_bits_rn(v.y * inv)) << 16);
      const uint32_t hi = f32_to_bf16_bits_rn(v.z * inv) | (static_cast<uint32_t>(f32_to_bf16_bits_rn(v.w * inv)) << 16);
      *reinterpret_cast<uint2*>(p.out + (tok * p.Hkv * p.G + h * p.G + row % p.G) * D + c) = make_uint2(lo, hi);
    }
  }
}

}  // namespace kva

namespace {

int tiles_n(int R) { return R > 8 ? 2 : 1; }   // 8-row tiles of an item

struct Layout {
  size_t desc, ml, part, bytes;
};

Layout layout(int64_t items, int R, int D, int sms) {
  const size_t rows = static_cast<size_t>(2) * (2 * sms) * 8 * tiles_n(R);   // two slots of every CTA
  Layout l;
  l.desc = 0;
  l.ml = (items * sizeof(int4) + 255) & ~static_cast<size_t>(255);
  l.part = l.ml + ((rows * sizeof(float2) + 255) & ~static_cast<size_t>(255));
  l.bytes = l.part + rows * D * sizeof(float);
  return l;
}

template <int D, int NT>
cudaError_t launch(KvAttentionArgs p, int sms, cudaStream_t st) {
  using namespace kva;
  using S = Shape<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = sms * ((D == 64 || NT == 1) ? 2 : 1);
  kv_attention_kernel<D, NT><<<grid, kThreads, S::kSmem, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int64_t items = static_cast<int64_t>(p.B) * p.Hkv * p.RT;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(items, 8 * sms)));
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_attention_join_kernel<D, NT>, p);
}

}  // namespace

size_t kv_attention_workspace(int B, int Lq, int Hq, int Hkv, int D, int sms) {
  const int R = Hq / Hkv * Lq;
  return layout(static_cast<int64_t>(B) * Hkv * cdiv(R, 8 * tiles_n(R)), R, D, sms).bytes;
}

cudaError_t launch_kv_attention(KvAttentionArgs p, void* workspace, int sms, cudaStream_t st) {
  const int nt = tiles_n(p.R);
  p.RT = static_cast<int>(cdiv(p.R, 8 * nt));
  const Layout l = layout(static_cast<int64_t>(p.B) * p.Hkv * p.RT, p.R, p.D, sms);
  char* base = static_cast<char*>(workspace);
  p.desc = reinterpret_cast<int4*>(base + l.desc);
  p.part_ml = reinterpret_cast<float2*>(base + l.ml);
  p.part = reinterpret_cast<float*>(base + l.part);
  if (p.D == 64) return nt == 1 ? launch<64, 1>(p, sms, st) : launch<64, 2>(p, sms, st);
  return nt == 1 ? launch<128, 1>(p, sms, st) : launch<128, 2>(p, sms, st);
}

}  // namespace mxmoe
