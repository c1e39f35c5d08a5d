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
//    per row (largest magnitude to [2^14, 2^15): bf16's 8 bits survive down to 2^-29 of the
//    row's largest, some of them to 2^-39).
//  - O^T += V^T P^T: the value scales multiply the weights, p 2^(e_j - E + 15), where E is the
//    largest value exponent seen so far in that 32-value block; the weights are then rounded
//    to f16 (11 bits; absolute floor 2^-40 of the largest scale). Maximum, sum, and all
//    accumulators are fp32. The rows of a tile share E. Where they belong to queries that see
//    different keys, only keys that all of them see set it, and one that some see and that lies
//    above it (an infinite value behind another query's mask, first of all) is added in fp32
//    beside the matrix products: no query's precision hangs on a key that it does not see.
// Row maxima, sums and E stay with the warp and its accumulators are rescaled only in units
// where one of them grows.
//
// Work split: units of 64 (or 32) keys of all (sequence, key/value head, row tile) items in one
// line; every warp of the grid takes an equal run of them whatever the sequences' lengths (the
// lengths are on the device, so each CTA finds its warps' runs by itself) and streams it
// through a private cp.async ring, without a barrier after the start. A warp writes the items
// that lie wholly in its run; of the others it leaves fp32 partials in the caller's workspace,
// joined in run order by a second small kernel. Items of a few units (a short window) stay in
// one CTA. Nothing in the result depends on timing, and no counter outlives a call.
//
// Measured on a B200 (calls in a row, of the bytes that must be read): 64 sequences of 500 to 8192
// keys, 64 heads over 8 of 64 (154 MB): 46 us, 3.3 TB/s; 3 sequences of up to 131072 keys, 2 queries
// each, 32 heads over 8 of 128 (318 MB): 84 us (up to 91 in long loops, where the power cap lowers the
// clock), 3.8 TB/s; one query over a window of 128: 5.8 us (4.8 in a graph). Of the first, about 9 us
// are launches, the start's chain of loads (lengths, table, keys) and the joining kernel. The products
// are paced by the integer pipe (code expansion, 64 lanes a cycle: half of the cycles), the matrix
// instructions, which on this part take issue slots from it (an m16n8k16 between such instructions
// costs about 5 cycles beyond its own 8), and by latency: twelve warps issue in half of the cycles, and
// more do not fit the registers. Many queries a sequence read and expand every key again for each 16
// rows: 128 queries of 64 heads over 8 of 64 take 111 us over 8192 keys and 361 over 32768 (154 and
// 190 TF/s).
#include <algorithm>

#include "common.cuh"
#include "launchers.h"

namespace mxmoe {
namespace kva {

constexpr int kJoinThreads = 256;

// Keys of a sequence: positions a unit and a warp's lanes past its end, or a window before it, stay in 32 bits.
constexpr int64_t kMaxKeys = 1 << 30;

// A unit is 64 keys of 64 values or 32 of 128, 4 KB of codes: what a step's products, scores and
// weights leave room for in registers. (32 keys of 64 values: 16 rows 47.8 us against 45.2.)
constexpr int unit_keys(int D) { return D == 64 ? 64 : 32; }

// One CTA per SM. Twelve warps leave each 168 registers; sixteen (two CTAs, 128 registers) spilled or
// kept fewer products in flight: 32 sequences of up to 4096 keys, 64 heads over 8 of 64: 32.3 us
// against 30.8; 32 heads over 8 of 128: 43.6 against 40.9. 16 rows of 128 columns need more: eight
// warps 65.3 us, twelve 73.1.
constexpr int warps(int D, int nt) { return D == 128 && nt == 2 ? 8 : 12; }

template <int D, int NT>
struct Shape {
  static constexpr int kWarps = warps(D, NT), kThreads = 32 * kWarps;
  static constexpr int kUnit = unit_keys(D);
  static constexpr int kTiles = kUnit / 16;
  static constexpr int kRows = 8 * NT;
  static constexpr int kBlocks = D / 32;               // MXFP4 blocks of a row
  static constexpr int kRowBytes = D / 2;
  static constexpr int kKV = kUnit * kRowBytes;        // bytes of a unit's keys (or values)
  static constexpr int kSc = kUnit * kBlocks;          // their scales
  static constexpr int kStageBytes = 2 * kKV + 2 * kSc + 16;
  static constexpr int kStages = 3;
  static constexpr int kFactors = 2 * kBlocks * kUnit * 4;   // a unit's scales as fp32, keys' and values'
  static constexpr int kSmem = kWarps * (kStages * kStageBytes + kFactors);
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
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  return make_float2(__half2float(__ushort_as_half(static_cast<unsigned short>(v))),
                     __half2float(__ushort_as_half(static_cast<unsigned short>(v >> 16))));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(const uint8_t* at) { return *reinterpret_cast<const uint32_t*>(at); }
// the scale bytes of a key's blocks (2 or 4 of them), at `at`
template <int kBlocks>
__device__ __forceinline__ uint32_t lds_scales(const uint8_t* at) {
  if constexpr (kBlocks == 4) return lds32(at);
  return *reinterpret_cast<const uint16_t*>(at);
}
// Four 8 x 16-byte matrices whose rows lie at the lanes' addresses (lanes 8 i .. 8 i + 7: matrix
// i). Plain: r[i] is word t of row g. Transposed: the 16-bit elements g of rows 2t (low) and
// 2t + 1.
__device__ __forceinline__ void ldmatrix(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// byte k of a word as the exponent field of an fp32: 2^(byte - 127). As a key's factor byte 0 reads as
// zero: its block's values are below 2^-124.
__device__ __forceinline__ uint32_t exponent_of(uint32_t word, int k) {
  return (k < 3 ? word << (23 - 8 * k) : word >> 1) & 0x7F800000u;
}

// An item's sums carry 2^(15 + 127 - E), E the largest value scale byte of the block: times 2^-15 (and
// the row's 1 / l) they are at most a value, and times 2^(E - 127) then the outputs. In one factor
// 2^(E - 142) would be below the normal numbers for E < 16, and lost.
constexpr float kUndo = 0x1p-15f;
// 2^(e - 127) of an fp32's exponent field; the least, 2^-127, is a subnormal
__device__ __forceinline__ float power_of(int field) { return __int_as_float(max(field, 1 << 22)); }

// 2^(15 + e - E) of exponent fields, zero below the normal numbers. (A key above E gives nothing of use;
// its place is written anew.)
__device__ __forceinline__ float weight_factor(uint32_t e, int E) {
  return __int_as_float(max(static_cast<int>(e - static_cast<uint32_t>(E) + (142u << 23)), 0));
}

// 2^d, which may lie outside of fp32, as two finite factors: a zero stays a zero
struct Power2 {
  float a, b;
  __device__ __forceinline__ explicit Power2(int d)
      : a(ex2(static_cast<float>(min(d >> 1, 127)))), b(ex2(static_cast<float>(min(d - (d >> 1), 127)))) {}
};

// r / G for the rows of an item: r G < 2^32, so the rounded-up reciprocal is exact
__device__ __forceinline__ int query_of(const KvAttentionArgs& p, int r) {
  return p.G == 1 ? r : static_cast<int>(__umulhi(static_cast<uint32_t>(r), p.g_reciprocal));
}

// ------------------------------------------------------------------- work line -----
__device__ __forceinline__ int seq_len(const KvAttentionArgs& p, int b) {
  const int n = __ldg(p.seq_lens + b);
  const int64_t cap = min(static_cast<int64_t>(p.max_pages) << p.page_shift, kMaxKeys);
  if (n > cap) {   // more keys than the table has pages for, or than the arithmetic on keys takes
    set_device_error(p.err, MXMOE_EDEVICE);
    return static_cast<int>(cap);
  }
  return max(n, 0);
}

// the first key that a sequence's first query sees
__device__ __forceinline__ int first_seen(const KvAttentionArgs& p, int len) {
  return p.window > 0 ? max(0, len - p.Lq + 1 - p.window) : 0;
}

template <int kUnit>
__device__ __forceinline__ int units_of(const KvAttentionArgs& p, int len) {
  const int first = first_seen(p, len) & ~(kUnit - 1);
  return max(1, (len - first + kUnit - 1) / kUnit);   // an empty sequence still writes its zeros
}

// Position in the line of units, counted from the warp's run: an item (key/value head h, row
// tile rt of sequence b), the unit behind its last and the key that unit 0 of the run would
// start at if it were the item's.
template <int kUnit>
struct Cursor {
  int b, h, rt, len, end, key0;
  __device__ void open(const KvAttentionArgs& p, int start) {   // b, h, rt set; the item starts at unit `start`
    len = seq_len(p, b);
    const int first = first_seen(p, len) & ~(kUnit - 1);
    end = start + max(1, (len - first + kUnit - 1) / kUnit);
    key0 = first - kUnit * start;
  }
  // one item shared by `ways` warps: this one takes every ways-th unit from `way` on
  __device__ void share(int way, int ways) {
    end = (end - way + ways - 1) / ways;   // 0 for a way past the last unit (end + ways - 1 - way >= 0)
    key0 += kUnit * way;
  }
  __device__ int key(const KvAttentionArgs& p, int unit) const { return key0 + p.unit_step * unit; }
  __device__ void next(const KvAttentionArgs& p) {
    if (++rt == p.RT) {
      rt = 0;
      if (++h == p.Hkv) {
        h = 0;
        if (++b == p.B) return;
      }
    }
    open(p, end);
  }
};

// Run number `run` of `runs` equal ones of a line of n units: its units [t0, t0 + count).
struct Run {
  int per, t0, count;
};
template <int kUnit>
__device__ __forceinline__ Run run_of(int n, int runs, int run) {
  Run r;
  r.per = max(64 / kUnit, n / runs + (n % runs ? 1 : 0));   // 64 keys at least
  r.t0 = static_cast<int>(min(static_cast<int64_t>(n), static_cast<int64_t>(r.per) * run));
  r.count = min(r.per, n - r.t0);
  return r;
}

// Opens the item of sequence b that holds its unit `into`; returns where the item starts, counted
// from that unit (0 or before it).
template <int kUnit>
__device__ __forceinline__ int open_at(const KvAttentionArgs& p, Cursor<kUnit>& c, int b, int into) {
  c.b = b;
  const int units = units_of<kUnit>(p, seq_len(p, b)), j = into / units;
  c.h = p.RT == 1 ? j : j / p.RT;
  c.rt = p.RT == 1 ? 0 : j % p.RT;
  const int start = j * units - into;
  c.open(p, start);
  return start;
}

// kMulti: a row tile may hold rows of several queries. Calls without such tiles take a kernel of their own,
// because what E needs here shows in the loop's schedule: 32 sequences of two queries 54.1 us instead of
// 52.1, 3 long ones of D = 128 83.9 instead of 79.7. (Taking such a part anew, query by query: 88.2.)
template <int D, int NT, bool kMulti>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1) kv_attention_kernel(const KvAttentionArgs p) {
  using S = Shape<D, NT>;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_sum[kWarps];
  __shared__ int s_pre[kThreads];
  __shared__ int s_per[kWarps];   // a run's units; each warp's own word
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int per_seq = p.Hkv * p.RT;
  griddep_launch_dependents();   // the joining kernel may take its places; it waits for this one's end
  griddep_wait();

  // ---- this warp's run: `count` units from `cur` on, whose item may have begun before it ----
  // neighbouring runs go to different SMs, so that a short line still uses all of them
  const int run = warp * gridDim.x + blockIdx.x, runs = gridDim.x * kWarps;
  int count = 0, start = 0;   // start: of the run's first item, in the run
  Cursor<S::kUnit> cur;
  cur.b = -1;
  if (p.whole > 1) {   // at most one item for each group of so many warps
    const int ways = p.whole, way = warp % ways, item = warp / ways * gridDim.x + blockIdx.x;
    if (item >= p.B * per_seq) return;
    cur.b = item / per_seq;
    cur.h = item % per_seq / p.RT;
    cur.rt = item % p.RT;
    cur.open(p, 0);
    cur.share(way, ways);
    count = cur.end;
  } else if (p.whole) {
    const int items = p.B * per_seq, each = (items + runs - 1) / runs;
    const int i0 = run * each, i1 = min(items, i0 + each);
    for (int i = i0 + lane; i < i1; i += 32) count += units_of<S::kUnit>(p, seq_len(p, i / per_seq));
    count = __reduce_add_sync(0xffffffffu, count);
    if (count == 0) return;
    cur.b = i0 / per_seq;
    cur.h = i0 % per_seq / p.RT;
    cur.rt = i0 % p.RT;
    cur.open(p, 0);
  } else if (p.B <= 128) {   // each warp by itself, four sequences a lane
    int pre[4], n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = 32 * i + lane;
      pre[i] = b < p.B ? units_of<S::kUnit>(p, seq_len(p, b)) * per_seq : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (32 * i >= p.B) break;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, pre[i], o);
        if (lane >= o) pre[i] += x;
      }
      pre[i] += n;
      n = __shfl_sync(0xffffffffu, pre[i], 31);
    }
    const Run r = run_of<S::kUnit>(n, runs, run);
    count = r.count;
    if (count == 0) return;
    int before = 0;   // units before the chunk of 32 sequences
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (cur.b >= 0 || 32 * i >= p.B) break;
      const unsigned past = __ballot_sync(0xffffffffu, pre[i] > r.t0);
      if (past) {
        const int at = __ffs(past) - 1;
        const int from = at ? __shfl_sync(0xffffffffu, pre[i], at - 1) : before;
        start = open_at<S::kUnit>(p, cur, 32 * i + at, r.t0 - from);
      }
      before = __shfl_sync(0xffffffffu, pre[i], 31);
    }
    if (lane == 0) s_per[warp] = r.per;
    __syncwarp();
  } else {
    // pass 0 counts the line's units, pass 1 finds the run's first; a batch of one chunk of
    // kThreads sequences needs its prefix sums once
    Run r{};
    for (int pass = p.B > kThreads ? 0 : 1; pass < 2; ++pass) {
      int base = 0;   // units before this chunk of sequences
      for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int pre = b < p.B ? units_of<S::kUnit>(p, seq_len(p, b)) * per_seq : 0;   // inclusive over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane >= o) pre += x;
        }
        __syncthreads();   // s_sum and s_pre of the step before have been read
        if (lane == 31) s_sum[warp] = pre;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) pre += s_sum[w];
          all += s_sum[w];
        }
        s_pre[threadIdx.x] = base + pre;
        __syncthreads();
        if (pass == 0 || p.B <= kThreads) {
          r = run_of<S::kUnit>(base + all, runs, run);
          count = r.count;
        }
        if (pass == 1 && count > 0 && base <= r.t0 && r.t0 < base + all) {
          // the first sequence of the chunk whose units end after t0
#pragma unroll
          for (int i = 0; i < kThreads / 32; ++i) {
            const unsigned past = __ballot_sync(0xffffffffu, s_pre[32 * i + lane] > r.t0);
            if (past && cur.b < 0) {
              const int at = 32 * i + __ffs(past) - 1;
              start = open_at<S::kUnit>(p, cur, b0 + at, r.t0 - (at ? s_pre[at - 1] : base));
            }
          }
        }
        base += all;
      }
    }
    if (count == 0) return;
    if (lane == 0) s_per[warp] = r.per;
    __syncwarp();
  }

  // ---- this warp's ring of units ----
  uint8_t* const ring = smem + warp * (S::kStages * S::kStageBytes + S::kFactors);
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  constexpr int kPages = 2 * S::kKV + 2 * S::kSc;   // offset of a stage's flags: which 16 keys were loaded
  constexpr int kChunks = S::kRowBytes / 16;        // 16-byte chunks of a row, one MXFP4 block each
  constexpr int kLoads = S::kKV / 512 / S::kTiles;  // 16-byte loads a lane makes of 16 keys (or values)
  constexpr int kScChunks = S::kSc / 16;            // 16-byte chunks of a unit's key (or value) scales
  // A row's chunks are permuted so that the eight rows of an operand load fall in different
  // banks; the permutation of a key repeats every 8 keys.
  const uint32_t put = (lane / kChunks) * S::kRowBytes +
                       16 * ((lane % kChunks) ^ (kChunks == 2 ? (lane >> 3) & 1 : (lane >> 3) & 3));
  const int page_rows = p.Hkv << p.page_shift, in_page = (1 << p.page_shift) - 1;
  const bool sc_val = lane >= kScChunks;                            // the lane's chunk of scales
  const int sc_tile = (lane % kScChunks) / (kScChunks / S::kTiles);
  const int sc_off = 16 * (lane % (kScChunks / S::kTiles));

  Cursor<S::kUnit> in = cur;   // of the next unit to load
  int in_unit = 0, pid = 0;    // lane i < kTiles: the page of the unit's i-th 16 keys (a page holds 16 or more)
  bool in_need = false;
  auto look = [&]() {
    if (in_unit >= count) return;
    if (in_unit >= in.end) in.next(p);
    const int key = in.key(p, in_unit) + 16 * lane;
    // keys that no query sees need no page
    in_need = lane < S::kTiles && key < in.len && key + 16 > first_seen(p, in.len);
    if (in_need) pid = __ldg(p.block_table + static_cast<int64_t>(in.b) * p.max_pages + (key >> p.page_shift));
  };
  auto issue = [&](int stage) {
    if (in_unit < count) {
      const uint32_t dst = ring_at + stage * S::kStageBytes;
      const bool ok = in_need && static_cast<uint32_t>(pid) < static_cast<uint32_t>(p.num_pages);
      if (in_need && !ok) set_device_error(p.err, MXMOE_EDEVICE);   // a page outside the cache
      unsigned pages = __ballot_sync(0xffffffffu, ok);
      const int key = in.key(p, in_unit), head = in.h << p.page_shift;
      if (in_page >= S::kUnit - 1) {   // one page holds the unit: its keys are one run
        if (pages) {
          const int page = __shfl_sync(0xffffffffu, pid, __ffs(pages) - 1);
          const int64_t row = static_cast<int64_t>(page) * page_rows + (head + (key & in_page));
          const int64_t off = row * S::kRowBytes + 16 * lane;
#pragma unroll
          for (int x = 0; x < S::kTiles * kLoads; ++x) {
            cp_async16(dst + put + 512 * x, p.k_blocks + off + 512 * x);
            cp_async16(dst + put + 512 * x + S::kKV, p.v_blocks + off + 512 * x);
          }
          if (lane < 2 * kScChunks)
            cp_async16(dst + 2 * S::kKV + 16 * lane,
                       (sc_val ? p.v_scales : p.k_scales) + row * S::kBlocks + 16 * (lane % kScChunks));
          pages = (1u << S::kTiles) - 1;
        }
      } else {
#pragma unroll
        for (int i = 0; i < S::kTiles; ++i) {
          const int page = __shfl_sync(0xffffffffu, pid, i);
          if (!((pages >> i) & 1)) continue;
          const int64_t row = static_cast<int64_t>(page) * page_rows + (head + ((key + 16 * i) & in_page));
          const int64_t off = row * S::kRowBytes + 16 * lane;
#pragma unroll
          for (int x = 0; x < kLoads; ++x) {
            cp_async16(dst + put + 512 * (i * kLoads + x), p.k_blocks + off + 512 * x);
            cp_async16(dst + put + 512 * (i * kLoads + x) + S::kKV, p.v_blocks + off + 512 * x);
          }
        }
        const int page = __shfl_sync(0xffffffffu, pid, sc_tile);
        if (lane < 2 * kScChunks && ((pages >> sc_tile) & 1)) {
          const int64_t row = static_cast<int64_t>(page) * page_rows + (head + ((key + 16 * sc_tile) & in_page));
          cp_async16(dst + 2 * S::kKV + 16 * lane, (sc_val ? p.v_scales : p.k_scales) + row * S::kBlocks + sc_off);
        }
      }
      if (lane == 0) *reinterpret_cast<unsigned*>(ring + stage * S::kStageBytes + kPages) = pages;
      ++in_unit;
    }
    cp_async_commit();
    look();
  };
  // an item's queries, 16 bytes of a row and block a lane; fetched ahead of their use: the first
  // item's beside its first pages, another's while the one before it is written
  uint4 raw[NT][S::kBlocks];
  auto load_q = [&](const Cursor<S::kUnit>& c) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = c.rt * S::kRows + 8 * i + g;
      const bool real = r < p.R;
      const int qi = real ? query_of(p, r) : 0, hd = c.h * p.G + (real ? r - qi * p.G : 0);
      const uint16_t* src = p.q + (static_cast<int64_t>(c.b) * p.Lq + qi) * p.q_stride + static_cast<int64_t>(hd) * D;
#pragma unroll
      for (int k = 0; k < S::kBlocks; ++k)
        raw[i][k] = real ? __ldg(reinterpret_cast<const uint4*>(src + 32 * k + 8 * t)) : make_uint4(0, 0, 0, 0);
    }
  };
  look();
  load_q(cur);
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) issue(s);

  // The lane's row of an operand load of 16 keys and two blocks (matrices: keys 0-7 and 8-15 of
  // the first, of the second), alike for keys and values.
  const uint32_t get = (lane & 15) * S::kRowBytes +
                       16 * ((lane >> 4) ^ (kChunks == 2 ? (lane >> 2) & 1 : (lane >> 1) & 3));
  float* const factors = reinterpret_cast<float*>(ring + S::kStages * S::kStageBytes);   // [key][keys' blocks, values']

  int stage = 0, at = 0;
  do {
    // ---- one item: rows, queries ----
    const int end = min(count, cur.end), from = at;
    const int len = cur.len, h = cur.h, row0 = cur.rt * S::kRows;
    uint32_t qf[NT][S::kBlocks][4];
    float qs[NT][2];                      // of rows 2t, 2t + 1: score scale in base 2, undoing the f16 shift
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < S::kBlocks; ++k) {
        const uint32_t w[4] = {raw[i][k].x, raw[i][k].y, raw[i][k].z, raw[i][k].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) top = max(top, max((w[x] << 16) & 0x7FFF0000u, w[x] & 0x7FFF0000u));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^(14 - exponent) and its inverse, both normal fp32
      const int ex = min(max(static_cast<int>(top >> 23), 16), 254);
      const float up = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23) * p.scale_sign;
      const float down = __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
#pragma unroll
      for (int k = 0; k < S::kBlocks; ++k) {
        const uint32_t w[4] = {raw[i][k].x, raw[i][k].y, raw[i][k].z, raw[i][k].w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
          qf[i][k][x] = pack_f16(__uint_as_float(w[x] << 16) * up, __uint_as_float(w[x] & 0xFFFF0000u) * up);
      }
      // never zero: a masked score's -infinity stays one under it
      qs[i][0] = fmaxf(__shfl_sync(0xffffffffu, down, 8 * t) * p.scale_log2, 0x1p-126f);
      qs[i][1] = fmaxf(__shfl_sync(0xffffffffu, down, 8 * t + 4) * p.scale_log2, 0x1p-126f);
    }
    // keys that some row (seen) and that every row (full) of the tile sees
    const int hi_first = len - p.Lq + query_of(p, row0) + 1;
    const int hi_last = kMulti ? len - p.Lq + query_of(p, min(row0 + S::kRows, p.R) - 1) + 1 : hi_first;
    const int seen_lo = p.window > 0 ? max(0, hi_first - p.window) : 0, seen_hi = max(hi_last, 0);
    const int full_lo = p.window > 0 ? max(0, hi_last - p.window) : 0, full_hi = hi_first;

    float o[NT][S::kBlocks][2][4];
    float m[NT][2], l[NT][2];   // m before the row's factor, so that the largest weight is exactly 1
    int E[S::kBlocks];   // as an fp32's exponent field
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
    unsigned lone = 0;   // blocks whose E is of keys that some queries do not see: no other has come yet

    // ---- its units in this run ----
    for (; at < end; ++at) {
      cp_async_wait<S::kStages - 2>();
      __syncwarp();
      const uint8_t* sk = ring + stage * S::kStageBytes;
      const uint32_t sk_at = ring_at + stage * S::kStageBytes;
      const uint8_t *ssk = sk + 2 * S::kKV, *ssv = ssk + S::kSc;
      // the unit's key codes and scales are on their way while the next unit's copies are issued (each
      // read just before its use: 46.1 and 81.0 us instead of 44.9 and 78.6, 64 heads of 64, 32 of 128)
      uint32_t kw[S::kTiles][S::kBlocks / 2][4];
#pragma unroll
      for (int y = 0; y < S::kTiles; ++y)
#pragma unroll
        for (int k2 = 0; k2 < S::kBlocks; k2 += 2) ldmatrix(sk_at + (get ^ (16 * k2)) + 16 * y * S::kRowBytes, kw[y][k2 / 2]);
      uint32_t sc[S::kUnit / 32], ev[S::kUnit / 32];
#pragma unroll
      for (int e = 0; e < S::kUnit / 32; ++e) {
        sc[e] = lds_scales<S::kBlocks>(ssk + (32 * e + lane) * S::kBlocks);
        ev[e] = lds_scales<S::kBlocks>(ssv + (32 * e + lane) * S::kBlocks);
      }
      {
        const int next = stage + S::kStages - 1;
        issue(next >= S::kStages ? next - S::kStages : next);
      }
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
      const unsigned pages = lds32(sk + kPages);
      const int key0 = cur.key(p, at);

      // The unit's scales as fp32: the keys' own, the values' as weight factors 2^(15 + e - E). A
      // lane takes keys lane (and lane + 32). A key that no row sees counts as scale 0: what
      // lies in its place does not matter.
      const bool edge = pages != (1u << S::kTiles) - 1 || key0 < full_lo || key0 + S::kUnit > full_hi || (kMulti && lone);
      // the value scales of one of the lane's keys, 0 if no row sees it
      const auto seen_scales = [&](int e) -> uint32_t {
        const int key = key0 + 32 * e + lane;
        if (key < seen_lo || key >= seen_hi || !((pages >> (2 * e + (lane >> 4))) & 1)) return 0;
        return lds_scales<S::kBlocks>(ssv + (32 * e + lane) * S::kBlocks);
      };
      uint32_t top[S::kBlocks], es[S::kUnit / 32];   // es: the scales that set E, of keys that all queries see
#pragma unroll
      for (int e = 0; e < S::kUnit / 32; ++e) es[e] = ev[e];
      if (edge) {
#pragma unroll
        for (int e = 0; e < S::kUnit / 32; ++e) {
          const int key = key0 + 32 * e + lane;
          if (key < seen_lo || key >= seen_hi || !((pages >> (2 * e + (lane >> 4))) & 1)) ev[e] = 0;
          es[e] = kMulti && (key < full_lo || key >= full_hi) ? 0 : ev[e];
        }
      }
      bool higher = false;
#pragma unroll
      for (int k = 0; k < S::kBlocks; ++k) {
        top[k] = exponent_of(es[0], k);
#pragma unroll
        for (int e = 1; e < S::kUnit / 32; ++e) top[k] = max(top[k], exponent_of(es[e], k));
        higher |= static_cast<int>(top[k]) > E[k];
      }
      if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
        for (int k = 0; k < S::kBlocks; ++k) {
          const int e = max(E[k], static_cast<int>(__reduce_max_sync(0xffffffffu, top[k])));
          const float f = ex2(static_cast<float>((E[k] - e) >> 23));
          E[k] = e;
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              o[i][k][0][x] *= f;
              o[i][k][1][x] *= f;
            }
        }
      }
#pragma unroll
      for (int e = 0; e < S::kUnit / 32; ++e) {
        float f[2 * S::kBlocks];
#pragma unroll
        for (int k = 0; k < S::kBlocks; ++k) {
          f[k] = __uint_as_float(exponent_of(sc[e], k));
          f[S::kBlocks + k] = weight_factor(exponent_of(ev[e], k), E[k]);
        }
#pragma unroll
        for (int k = 0; k < 2 * S::kBlocks; k += 4)
          *reinterpret_cast<float4*>(factors + (32 * e + lane) * 2 * S::kBlocks + k) =
              make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
      }
      __syncwarp();

      // scores, before the row's factor
      f32x2 s[NT][S::kTiles][2];   // keys g, g + 8 of a tile; rows 2t, 2t + 1
#pragma unroll
      for (int y = 0; y < S::kTiles; ++y) {
        const float* fa = factors + (16 * y + g) * 2 * S::kBlocks;
        const float* fb = fa + 8 * 2 * S::kBlocks;
#pragma unroll
        for (int k2 = 0; k2 < S::kBlocks; k2 += 2) {
          const uint32_t(&w)[4] = kw[y][k2 / 2];
          const float2 ka = *reinterpret_cast<const float2*>(fa + k2), kb = *reinterpret_cast<const float2*>(fb + k2);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const int k = k2 + kk;
            uint32_t a[4], b[4];
            expand(w[2 * kk], a);
            expand(w[2 * kk + 1], b);
            const f32x2 f0 = kk ? f32x2_of(ka.y, ka.y) : f32x2_of(ka.x, ka.x), f1 = kk ? f32x2_of(kb.y, kb.y) : f32x2_of(kb.x, kb.x);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              float c[4];
              mma_f16_zero(c, a[0], b[0], a[1], b[1], qf[i][k][0], qf[i][k][1]);
              mma_f16(c, a[2], b[2], a[3], b[3], qf[i][k][2], qf[i][k][3]);
              if (k == 0) {
                s[i][y][0] = mul2(f32x2_of(c[0], c[1]), f0);
                s[i][y][1] = mul2(f32x2_of(c[2], c[3]), f1);
              } else {
                s[i][y][0] = fma2(f32x2_of(c[0], c[1]), f0, s[i][y][0]);
                s[i][y][1] = fma2(f32x2_of(c[2], c[3]), f1, s[i][y][1]);
              }
            }
          }
        }
      }
      bool above = kMulti && lone;   // does a key that only some rows see lie above E?
      if (edge) {
        if (kMulti) {
          uint32_t bound = 0;
#pragma unroll
          for (int k = 0; k < S::kBlocks; ++k) bound |= static_cast<uint32_t>(E[k] >> 23) << (8 * k);
#pragma unroll
          for (int e = 0; e < S::kUnit / 32; ++e) above |= __vmaxu4(seen_scales(e), bound) != bound;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          int hi[2], lo[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int row = row0 + 8 * i + 2 * t + x;
            hi[x] = row < p.R ? len - p.Lq + query_of(p, row) + 1 : 0;
            lo[x] = p.window > 0 ? hi[x] - p.window : 0;
          }
#pragma unroll
          for (int y = 0; y < S::kTiles; ++y)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int key = key0 + 16 * y + 8 * z + g;
              const bool gone = !((pages >> y) & 1);
              s[i][y][z] = f32x2_of(gone || key < lo[0] || key >= hi[0] ? -INFINITY : lo_of(s[i][y][z]),
                                gone || key < lo[1] || key >= hi[1] ? -INFINITY : hi_of(s[i][y][z]));
            }
        }
      }
      // does a maximum grow?
      float mx[NT][2];
      bool grows = false;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        mx[i][0] = fmaxf(lo_of(s[i][0][0]), lo_of(s[i][0][1]));
        mx[i][1] = fmaxf(hi_of(s[i][0][0]), hi_of(s[i][0][1]));
#pragma unroll
        for (int y = 1; y < S::kTiles; ++y) {
          mx[i][0] = fmaxf(mx[i][0], fmaxf(lo_of(s[i][y][0]), lo_of(s[i][y][1])));
          mx[i][1] = fmaxf(mx[i][1], fmaxf(hi_of(s[i][y][0]), hi_of(s[i][y][1])));
        }
        grows |= mx[i][0] > m[i][0] || mx[i][1] > m[i][1];
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float v = mx[i][x];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float nm = fmaxf(m[i][x], v);
            // nothing seen yet: all zero anyway
            const float f = nm == -INFINITY ? 1.f : ex2((m[i][x] - nm) * qs[i][x]);
            m[i][x] = nm;
            l[i][x] *= f;
#pragma unroll
            for (int k = 0; k < S::kBlocks; ++k) {
              o[i][k][0][x] *= f;
              o[i][k][0][x + 2] *= f;
              o[i][k][1][x] *= f;
              o[i][k][1][x + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const f32x2 base = f32x2_of(m[i][0] == -INFINITY ? 0.f : -m[i][0], m[i][1] == -INFINITY ? 0.f : -m[i][1]);
        const f32x2 q2 = f32x2_of(qs[i][0], qs[i][1]);
        f32x2 sum = f32x2_of(l[i][0], l[i][1]);
#pragma unroll
        for (int y = 0; y < S::kTiles; ++y)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const f32x2 e = mul2(add2(s[i][y][z], base), q2);
            s[i][y][z] = f32x2_of(ex2(lo_of(e)), ex2(hi_of(e)));
            sum = add2(sum, s[i][y][z]);
          }
        l[i][0] = lo_of(sum);
        l[i][1] = hi_of(sum);
      }
      if (kMulti && __any_sync(0xffffffffu, above)) {
        // Blocks whose E is of such keys alone take the least of them; a key that all rows see then
        // sets E anew, lower if need be. Keys above E leave the matrix products and are added here.
        unsigned apart[S::kUnit / 32];
        uint32_t out = 0, v[S::kUnit / 32];
#pragma unroll
        for (int e = 0; e < S::kUnit / 32; ++e) v[e] = seen_scales(e);
#pragma unroll
        for (int k = 0; k < S::kBlocks; ++k) {
          uint32_t most = 0, least = 255;
#pragma unroll
          for (int e = 0; e < S::kUnit / 32; ++e) {
            const int key = key0 + 32 * e + lane;
            const uint32_t x = v[e] >> (8 * k) & 255;
            if (key >= full_lo && key < full_hi) most = max(most, x);
            else if (x) least = min(least, x);
          }
          most = __reduce_max_sync(0xffffffffu, most);
          least = __reduce_min_sync(0xffffffffu, least);
          const int was = E[k] >> 23;
          int next = was;
          if ((lone >> k) & 1) {
            next = most ? most : min(static_cast<uint32_t>(was), least);
            if (most) lone &= ~(1u << k);
          } else if (was == 0 && least < 255) {
            next = least;
            lone |= 1u << k;
          }
          const Power2 f(was - next);
          E[k] = next << 23;
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              o[i][k][0][x] = o[i][k][0][x] * f.a * f.b;
              o[i][k][1][x] = o[i][k][1][x] * f.a * f.b;
            }
#pragma unroll
          for (int e = 0; e < S::kUnit / 32; ++e)
            if (static_cast<int>(v[e] >> (8 * k) & 255) > next) out |= 1u << e;
        }
#pragma unroll
        for (int e = 0; e < S::kUnit / 32; ++e) {
          apart[e] = __ballot_sync(0xffffffffu, (out >> e) & 1);
#pragma unroll
          for (int k = 0; k < S::kBlocks; ++k)
            factors[(32 * e + lane) * 2 * S::kBlocks + S::kBlocks + k] =
                (out >> e) & 1 ? 0.f : weight_factor(exponent_of(v[e], k), E[k]);
        }
        __syncwarp();
#pragma unroll
        for (int y = 0; y < S::kTiles; ++y)
#pragma unroll
          for (int z = 0; z < 2; ++z)
            for (unsigned left = (apart[y / 2] >> (16 * (y % 2) + 8 * z)) & 255; left; left &= left - 1) {
              const int gk = __ffs(left) - 1, key = 16 * y + 8 * z + gk;
#pragma unroll
              for (int k = 0; k < S::kBlocks; ++k) {
                const uint32_t codes = *reinterpret_cast<const uint16_t*>(
                    sk + S::kKV + key * S::kRowBytes + 16 * (k ^ (kChunks == 2 ? (gk >> 2) & 1 : (gk >> 1) & 3)) + 2 * g);
                uint32_t c[4];   // the lane's four columns: low and high half of c[0], of c[1]
                expand(codes * 0x10001u, c);   // both halves: nvcc 12.9 makes zeros of a lone 16-bit load's bytes here
                const float2 v0 = unpack_f16(c[0]), v1 = unpack_f16(c[1]);
                const Power2 f(15 + ssv[key * S::kBlocks + k] - (E[k] >> 23));
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const float w = __shfl_sync(0xffffffffu, x ? hi_of(s[i][y][z]) : lo_of(s[i][y][z]), 4 * gk + t) * f.a;
                    o[i][k][0][x] = fmaf(w * v0.x, f.b, o[i][k][0][x]);
                    o[i][k][0][x + 2] = fmaf(w * v0.y, f.b, o[i][k][0][x + 2]);
                    o[i][k][1][x] = fmaf(w * v1.x, f.b, o[i][k][1][x]);
                    o[i][k][1][x + 2] = fmaf(w * v1.y, f.b, o[i][k][1][x + 2]);
                  }
              }
            }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int y = 0; y < S::kTiles; ++y) {
        const float* fa = factors + (16 * y + g) * 2 * S::kBlocks + S::kBlocks;
        const float* fb = fa + 8 * 2 * S::kBlocks;
#pragma unroll
        for (int k2 = 0; k2 < S::kBlocks; k2 += 2) {
          uint32_t w[4];   // [2 kk + z]: columns 4g .. 4g + 3 of keys 8z + 2t (low half), 8z + 2t + 1
          ldmatrix_trans(sk_at + S::kKV + (get ^ (16 * k2)) + 16 * y * S::kRowBytes, w);
          const float2 va = *reinterpret_cast<const float2*>(fa + k2), vb = *reinterpret_cast<const float2*>(fb + k2);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            const int k = k2 + kk;
            // pair the keys' codes of one column in a byte: columns 0, 2 in `even`, 1, 3 in `odd`;
            // bytes 0, 1 of keys (2t, 2t + 1), bytes 2, 3 of keys (2t + 8, 2t + 9)
            const uint32_t first = __byte_perm(w[2 * kk], w[2 * kk + 1], 0x5410);
            const uint32_t second = __byte_perm(w[2 * kk], w[2 * kk + 1], 0x7632);
            const uint32_t even = (first & 0x0F0F0F0Fu) | ((second << 4) & 0xF0F0F0F0u);
            const uint32_t odd = ((first >> 4) & 0x0F0F0F0Fu) | (second & 0xF0F0F0F0u);
            uint32_t ae[4], ao[4];
            expand(even, ae);
            expand(odd, ao);
            const f32x2 f0 = kk ? f32x2_of(va.y, va.y) : f32x2_of(va.x, va.x), f1 = kk ? f32x2_of(vb.y, vb.y) : f32x2_of(vb.x, vb.x);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const f32x2 wa = mul2(s[i][y][0], f0), wb = mul2(s[i][y][1], f1);
              const uint32_t b0 = transpose8x8(pack_f16(lo_of(wa), hi_of(wa)));
              const uint32_t b1 = transpose8x8(pack_f16(lo_of(wb), hi_of(wb)));
              mma_f16(o[i][k][0], ae[0], ao[0], ae[2], ao[2], b0, b1);
              mma_f16(o[i][k][1], ae[1], ao[1], ae[3], ao[3], b0, b1);
            }
          }
        }
      }
      __syncwarp();
    }

    // ---- an item that several warps of the CTA shared ----
    if (p.whole > 1) {
      const int ways = p.whole, way = warp % ways;
      cp_async_wait<0>();
      __syncwarp();
      constexpr int kWarpBytes = S::kStages * S::kStageBytes + S::kFactors;
      float* const mine = reinterpret_cast<float*>(ring);   // the ring is done with: sums [row][D]
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float sum = l[i][x];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          const int r = 8 * i + 2 * t + x;
          if (g == 0) reinterpret_cast<float2*>(factors)[r] = make_float2(m[i][x] * qs[i][x], sum);
#pragma unroll
          for (int k = 0; k < S::kBlocks; ++k) {
            const float f = power_of(E[k]);
            *reinterpret_cast<float4*>(mine + r * D + 32 * k + 4 * g) =
                make_float4(o[i][k][0][x] * kUndo * f, o[i][k][0][x + 2] * kUndo * f, o[i][k][1][x] * kUndo * f,
                            o[i][k][1][x + 2] * kUndo * f);
          }
        }
      asm volatile("bar.sync %0, %1;\n" ::"r"(1 + warp / ways), "r"(32 * ways) : "memory");
      const uint8_t* const all = smem + (warp - way) * kWarpBytes;
      constexpr int kCols = D / 32;   // columns of a lane
      for (int r = way; r < S::kRows && row0 + r < p.R; r += ways) {
        const int row = row0 + r, qi = query_of(p, row), hd = h * p.G + row - qi * p.G;
        float top = -INFINITY;
        for (int w = 0; w < ways; ++w)
          top = fmaxf(top, reinterpret_cast<const float2*>(all + w * kWarpBytes + S::kStages * S::kStageBytes)[r].x);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = p.sinks ? ex2(__ldg(p.sinks + hd) * 1.44269504088896f - base) : 0.f, v[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) v[c] = 0.f;
        for (int w = 0; w < ways; ++w) {
          const float2 ml = reinterpret_cast<const float2*>(all + w * kWarpBytes + S::kStages * S::kStageBytes)[r];
          const float f = ex2(ml.x - base);
          sum = fmaf(f, ml.y, sum);
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            v[c] = fmaf(f, reinterpret_cast<const float*>(all + w * kWarpBytes)[r * D + kCols * lane + c], v[c]);
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        uint16_t* dst = p.out + ((static_cast<int64_t>(cur.b) * p.Lq + qi) * p.Hkv * p.G + hd) * D + kCols * lane;
#pragma unroll
        for (int c = 0; c < kCols; c += 2) *reinterpret_cast<uint32_t*>(dst + c) = pack_bf16(v[c] * inv, v[c + 1] * inv);
      }
      return;
    }

    // ---- the item's end in this run ----
    Cursor<S::kUnit> following = cur;
    if (at == cur.end && at < count) {
      following.next(p);
      load_q(following);
    }
    const bool opened = from > 0 || start == 0;   // the item's first unit is in this run
    const bool whole = opened && cur.end <= count;
    const int64_t slot = 2 * static_cast<int64_t>(run) + (from > 0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float sum = l[i][x];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int r = 8 * i + 2 * t + x, row = row0 + r;
        const int c0 = 4 * g;   // the lane's four columns of a block
        if (row < p.R && whole) {
          const int qi = query_of(p, row), hd = h * p.G + row - qi * p.G;
          const float base = m[i][x] == -INFINITY ? 0.f : m[i][x] * qs[i][x];
          if (p.sinks) sum += ex2(__ldg(p.sinks + hd) * 1.44269504088896f - base);
          const float inv = sum > 0.f ? kUndo / sum : 0.f;
          uint16_t* dst = p.out + ((static_cast<int64_t>(cur.b) * p.Lq + qi) * p.Hkv * p.G + hd) * D + c0;
#pragma unroll
          for (int k = 0; k < S::kBlocks; ++k) {
            const float f = power_of(E[k]);
            *reinterpret_cast<uint2*>(dst + 32 * k) =
                make_uint2(pack_bf16(o[i][k][0][x] * inv * f, o[i][k][0][x + 2] * inv * f),
                           pack_bf16(o[i][k][1][x] * inv * f, o[i][k][1][x + 2] * inv * f));
          }
        } else if (row < p.R) {
          if (g == 0) p.part_ml[slot * S::kRows + r] = make_float2(m[i][x] * qs[i][x], sum);
          float* dst = p.part + (slot * S::kRows + r) * D + c0;
#pragma unroll
          for (int k = 0; k < S::kBlocks; ++k) {
            const float f = power_of(E[k]);
            *reinterpret_cast<float4*>(dst + 32 * k) =
                make_float4(o[i][k][0][x] * kUndo * f, o[i][k][0][x + 2] * kUndo * f, o[i][k][1][x] * kUndo * f,
                            o[i][k][1][x + 2] * kUndo * f);
          }
        }
      }
    // the run that holds the item's first unit says where its parts lie (slot, first and last
    // run); -1: no parts
    if (lane == 0 && opened && !p.whole) {
      const int64_t item = (static_cast<int64_t>(cur.b) * p.Hkv + h) * p.RT + cur.rt;
      p.desc[item] = whole ? make_int4(-1, 0, 0, 0)
                           : make_int4(static_cast<int>(slot), run, run + (cur.end - 1) / s_per[warp], 0);
    }
    cur = following;
  } while (at < count);
  cp_async_wait<0>();
}

// Joins the parts of the items that several runs shared, in an order that the runs fix. One
// CTA takes `rows` rows of an item: with all of them, a warp walks the parts of a row alone;
// with one, the warps share the parts.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) kv_attention_join_kernel(const KvAttentionArgs p, int rows) {
  using S = Shape<D, NT>;
  constexpr int kCols = D / 32;   // columns of a lane
  extern __shared__ __align__(16) uint8_t smem[];   // one-row sets only: a CTA without any fits beside the kernel before
  float(*const s_o)[D] = reinterpret_cast<float(*)[D]>(smem);
  float2* const s_ml = reinterpret_cast<float2*>(smem + kJoinThreads / 32 * D * sizeof(float));
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sets = S::kRows / rows;   // CTAs of an item
  const int64_t item = blockIdx.x / sets;
  const int4 d = p.desc[item];
  if (d.x < 0) return;
  const int per_seq = p.Hkv * p.RT;
  const int b = static_cast<int>(item / per_seq), j = static_cast<int>(item % per_seq);
  const int h = j / p.RT, row0 = (j % p.RT) * S::kRows;
  const int first_row = (blockIdx.x % sets) * rows;
  const bool shared = rows == 1;
  for (int r = shared ? first_row : first_row + warp; r < first_row + rows; r += kJoinThreads / 32) {
    const int row = row0 + r;
    if (row >= p.R) break;
    // the parts of this warp, eight at a time: maxima, sums and columns on their way at once
    const int step = shared ? kJoinThreads / 32 : 1;
    float top = -INFINITY, sum = 0.f, v[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) v[c] = 0.f;
    for (int first = d.y + (shared ? warp : 0); first <= d.z; first += 8 * step) {
      float2 ml[8];
      float x[8][kCols];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int run = first + i * step;
        ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int c = 0; c < kCols; ++c) x[i][c] = 0.f;
        if (run <= d.z) {
          const int64_t at = (run == d.y ? d.x : 2 * static_cast<int64_t>(run)) * S::kRows + r;
          ml[i] = p.part_ml[at];
#pragma unroll
          for (int c = 0; c < kCols; c += 2)
            *reinterpret_cast<float2*>(&x[i][c]) = *reinterpret_cast<const float2*>(p.part + at * D + kCols * lane + c);
        }
      }
      float next = top;
#pragma unroll
      for (int i = 0; i < 8; ++i) next = fmaxf(next, ml[i].x);
      const float base = next == -INFINITY ? 0.f : next, old = ex2(top - base);
      top = next;
      sum *= old;
#pragma unroll
      for (int c = 0; c < kCols; ++c) v[c] *= old;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = ex2(ml[i].x - base);
        sum = fmaf(f, ml[i].y, sum);
#pragma unroll
        for (int c = 0; c < kCols; ++c) v[c] = fmaf(f, x[i][c], v[c]);
      }
    }
    float base = top == -INFINITY ? 0.f : top;
    if (shared) {
#pragma unroll
      for (int c = 0; c < kCols; ++c) s_o[warp][kCols * lane + c] = v[c];
      if (lane == 0) s_ml[warp] = make_float2(top, sum);
      __syncthreads();
      if (warp > 0) return;
      top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kJoinThreads / 32; ++w) top = fmaxf(top, s_ml[w].x);
      base = top == -INFINITY ? 0.f : top;
      sum = 0.f;
#pragma unroll
      for (int c = 0; c < kCols; ++c) v[c] = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinThreads / 32; ++w) {
        const float f = ex2(s_ml[w].x - base);
        sum = fmaf(f, s_ml[w].y, sum);
#pragma unroll
        for (int c = 0; c < kCols; ++c) v[c] = fmaf(f, s_o[w][kCols * lane + c], v[c]);
      }
    }
    const int qi = query_of(p, row), hd = h * p.G + row - qi * p.G;
    if (p.sinks) sum += ex2(__ldg(p.sinks + hd) * 1.44269504088896f - base);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    uint16_t* dst = p.out + ((static_cast<int64_t>(b) * p.Lq + qi) * p.Hkv * p.G + hd) * D + kCols * lane;
#pragma unroll
    for (int c = 0; c < kCols; c += 2) *reinterpret_cast<uint32_t*>(dst + c) = pack_bf16(v[c] * inv, v[c + 1] * inv);
  }
}

}  // namespace kva

namespace {

int tiles_n(int R) { return R > 8 ? 2 : 1; }   // 8-row tiles of an item

struct Layout {
  size_t desc, ml, part, bytes;
};

Layout layout(int64_t items, int R, int D, int sms) {
  const int nt = tiles_n(R);
  const size_t rows = static_cast<size_t>(2) * sms * kva::warps(D, nt) * 8 * nt;   // two slots a run
  Layout l;
  l.desc = 0;
  l.ml = (items * sizeof(int4) + 255) & ~static_cast<size_t>(255);
  l.part = l.ml + ((rows * sizeof(float2) + 255) & ~static_cast<size_t>(255));
  l.bytes = l.part + rows * D * sizeof(float);
  return l;
}

template <int D, int NT, bool kMulti>
cudaError_t launch(KvAttentionArgs p, int sms, cudaStream_t st, int* launches) {
  using namespace kva;
  using S = Shape<D, NT>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(kv_attention_kernel<D, NT, kMulti>, S::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = sms;
  // Items of at most four units (a short window or a short table) stay in one CTA: nothing is left
  // for a second kernel, and no run has to be found. Where that still leaves half of the warps
  // without work, two or four share an item and join through shared memory (a window of 128
  // keys, 8 heads of 64: one sequence 9.0 -> 6.2 us with four; 96 sequences 11.0 us with one, 11.8
  // with two).
  const int64_t keys = static_cast<int64_t>(p.max_pages) << p.page_shift;
  const int64_t reach = p.window > 0 ? std::min<int64_t>(keys, static_cast<int64_t>(p.window) + p.Lq - 1) : keys;
  const int64_t most = cdiv(reach, S::kUnit) + (reach < keys ? 1 : 0);   // units of an item
  p.whole = 0;
  if (most <= 4) {
    const int64_t items = static_cast<int64_t>(p.B) * p.Hkv * p.RT, warps = static_cast<int64_t>(grid) * S::kWarps;
    p.whole = most > 2 && 8 * items <= warps ? 4 : most > 1 && 4 * items <= warps ? 2 : 1;
  }
  p.unit_step = S::kUnit * std::max(p.whole, 1);
  *launches = p.whole ? 1 : 2;
  e = launch_early(kv_attention_kernel<D, NT, kMulti>, dim3(static_cast<unsigned>(grid)), S::kThreads, S::kSmem, 0, st, p);
  if (e != cudaSuccess || p.whole) return e;
  // Few items are cut into many parts each: a CTA per row, its warps over the parts.
  const int64_t items = static_cast<int64_t>(p.B) * p.Hkv * p.RT;
  const int rows = items < 2 * sms ? 1 : S::kRows;
  return launch_early(kv_attention_join_kernel<D, NT>, dim3(static_cast<unsigned>(items * (S::kRows / rows))), kJoinThreads,
                      rows == 1 ? kJoinThreads / 32 * (D + 2) * sizeof(float) : 0, 0, st, p, rows);
}

}  // namespace

size_t kv_attention_workspace(int B, int Lq, int Hq, int Hkv, int D, int sms) {
  const int R = Hq / Hkv * Lq;
  return layout(static_cast<int64_t>(B) * Hkv * cdiv(R, 8 * tiles_n(R)), R, D, sms).bytes;
}

cudaError_t launch_kv_attention(KvAttentionArgs p, void* workspace, int sms, cudaStream_t st, int* launches) {
  const int nt = tiles_n(p.R);
  p.RT = static_cast<int>(cdiv(p.R, 8 * nt));
  p.g_reciprocal = static_cast<uint32_t>(((static_cast<uint64_t>(1) << 32) + p.G - 1) / p.G);   // not used for G = 1
  const Layout l = layout(static_cast<int64_t>(p.B) * p.Hkv * p.RT, p.R, p.D, sms);
  char* base = static_cast<char*>(workspace);
  p.desc = reinterpret_cast<int4*>(base + l.desc);
  p.part_ml = reinterpret_cast<float2*>(base + l.ml);
  p.part = reinterpret_cast<float*>(base + l.part);
  const bool multi = p.Lq > 1 && p.G % (8 * nt) != 0;
  const auto pick = [&](auto one, auto several) { return (multi ? several : one)(p, sms, st, launches); };
  if (p.D == 64) return nt == 1 ? pick(launch<64, 1, false>, launch<64, 1, true>) : pick(launch<64, 2, false>, launch<64, 2, true>);
  return nt == 1 ? pick(launch<128, 1, false>, launch<128, 1, true>) : pick(launch<128, 2, false>, launch<128, 2, true>);
}

}  // namespace mxmoe
