// FP8 E4M3 linear on codes that are already quantized, with the whole tail of an attention
// or MLP projection in its epilogue:
//   out[t, n] = bf16( act( s_x[t] s_w[n] sum_k xq[t, k] wq[n, k] + bias[n] ) + residual[t, n] )
// (s_x one scale or one per token, s_w one or one per output channel; fp32 from the
// accumulator to the one rounding at the end). tcgen05 kind::f8f6f4, fp32 accumulators in
// tensor memory, operands by TMA with 128-byte swizzle, 128 values of K per stage.
//
// Two kernels, by how many tiles there are (launch_fp8_linear_fused):
//  - pair: a persistent CTA pair (cta_group::2) per tile of 256 tokens by 64 to 256 columns. Each
//    CTA loads half of either operand's rows, so that a pair reads 512 rows for 65,536 outputs, a
//    third less from L2 for each product than a 128 x 256 tile of a single CTA. The width is the one
//    whose rounds over the pairs are the shortest. Two accumulator slots: a tile's epilogue overlaps
//    the next tile's products.
//  - split: for few tokens, where the weights' bytes are the bound. Weight rows take the M side
//    (128 a CTA), tokens the N side (16 to 128), and K is cut over a cluster of up to 8 CTAs
//    so that every SM streams weights. The partial sums meet in distributed shared memory,
//    added in rank order: no workspace, no second launch, the same bits each time.
//
// Every mbarrier wait gives up after about a second: the kernel then records MXMOE_ETIMEOUT,
// lets copies in flight land, meets the rest of its cluster, frees its tensor memory and
// returns.
#include <algorithm>
#include <atomic>

#include <cuda.h>

#include "common.cuh"
#include "launchers.h"
#include "tc_common.cuh"
#include "tmap.h"

namespace mxmoe {
namespace linf {

using namespace tc;

constexpr int BK = 128;

// kind::f8f6f4 instruction descriptor: D = F32 (bit 4), A = B = E4M3 (format 0), both K-major,
// N/8 at bits 17..22, M/16 at bits 24..28.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// The issuing warp runs its loop as a whole and predicates these on one elected lane: descriptors and
// addresses then stay in uniform registers, where the instructions take them from. A loop of one
// lane moved all of them over before each MMA (92 cycles an MMA, 200 a commit): 1000 x 8192 -> 256,
// tiles of 64 columns: 20.3 us against 18.2.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}

template <int kGroup>
__device__ __forceinline__ void mma_f8(uint32_t elected, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (kGroup == 1)
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
        " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

// arrive on the barrier once the MMAs issued so far are done
__device__ __forceinline__ void commit(uint32_t elected, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}
// the same on the barrier at this offset in both CTAs of a pair
__device__ __forceinline__ void commit_pair(uint32_t elected, uint64_t* bar) {
  asm volatile(
      "{\n .reg .b16 m;\n .reg .pred e;\n mov.b16 m, 3;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(elected)
      : "memory");
}

// Has the phase completed? Unlike a try_wait, which may hold the warp for microseconds while it has not.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// ------------------------------------------------------------------- cluster -------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
// The cluster's barrier as a meeting only, without release and acquire: what the CTAs tell each other
// goes through mbarriers. (Releasing made it wait for the outputs: half a microsecond a call.)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory"); }
// the address of a shared-memory object of this CTA in the cluster's CTA `rank`
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// copies this CTA's shared memory to another's (16-byte pieces), its bytes counted on a barrier there
__device__ __forceinline__ void send_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}
// Relaxed, since a release would wait for the outputs. What it tells is that this warp has read the accumulator:
// those reads have ended (tcgen05.wait::ld), and the fence before it orders them ahead. No memory
// is handed over, and that is all that the next products' writes to the accumulator rest on.
__device__ __forceinline__ void mbar_arrive_peer(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(addr) : "memory");
}
// mbar_wait with cluster scope: some of the barrier's arrivals come from the other CTA
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  const uint32_t addr = smem_u32(bar);
  const long long t0 = clock64();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort_flag = 1;
      set_device_error(err, MXMOE_ETIMEOUT);
      return false;
    }
  }
}
// a TMA load into this CTA's memory that completes on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tc_ld_32x32b_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// ------------------------------------------------------------------- epilogue ------
__device__ __forceinline__ f32x2 both(float v) { return f32x2_of(v, v); }
__device__ __forceinline__ f32x2 rcp2(f32x2 v) {
  float a, b;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(lo_of(v)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(hi_of(v)));
  return f32x2_of(a, b);
}
__device__ __forceinline__ f32x2 exp2_2(f32x2 v) {
  float a, b;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(lo_of(v)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(hi_of(v)));
  return f32x2_of(a, b);
}

// Activations of two values. GELU is max(v, 0) - |v| erfc(x) / 2 with x = |v| / sqrt(2), and
// erfc(x) / 2 = e^{-x^2} sum_i c_i t^i, t = 1 / (1 + x / 2): the coefficients are half of a
// weighted least-squares fit made for this file, relative error below 1.4e-6 on [0, 10] (scaled
// complementary error functions are smooth in such a t). Beyond |v| = 30 it is 0 in fp32, so |v|
// stops there and infinities pass. 777 x 1024 -> 4096: 12.4 us by single values, 11.3 by pairs; the
// library's erfcf took 21.
template <int kAct>
__device__ __forceinline__ f32x2 activate(f32x2 v) {
  if constexpr (kAct == MXMOE_ACT_SILU)
    return mul2(v, rcp2(add2(exp2_2(mul2(v, both(-1.44269504088896f))), both(1.f))));
  if constexpr (kAct == MXMOE_ACT_GELU) {
    const f32x2 a = f32x2_of(fmaxf(-fabsf(lo_of(v)), -30.f), fmaxf(-fabsf(hi_of(v)), -30.f));   // -|v|
    const f32x2 t = rcp2(fma2(a, both(-0.35355339059327f), both(1.f)));
    const f32x2 e = exp2_2(mul2(mul2(v, v), both(-0.72134752044448f)));
    f32x2 s = both(4.4102016e-02f);
    s = fma2(s, t, both(-1.7836859e-01f));
    s = fma2(s, t, both(1.9461153e-01f));
    s = fma2(s, t, both(1.8945863e-02f));
    s = fma2(s, t, both(1.4075167e-01f));
    s = fma2(s, t, both(1.3879111e-01f));
    s = fma2(s, t, both(1.4116570e-01f));
    return fma2(a, mul2(mul2(s, t), e), f32x2_of(fmaxf(lo_of(v), 0.f), fmaxf(hi_of(v), 0.f)));
  }
  return v;
}

__device__ __forceinline__ uint32_t pack2(f32x2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo_of(v), hi_of(v));
  return *reinterpret_cast<const uint32_t*>(&b);
}

// What eight columns [n, n + 8) share over the tokens: channel scales and bias.
struct Columns {
  f32x2 w[4], b[4];
  __device__ __forceinline__ void load(const LinearFusedArgs& p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = both(p.sw_all);
      b[i] = 0;
    }
    if (p.sw) {
      const ulonglong2 x = __ldg(reinterpret_cast<const ulonglong2*>(p.sw + n)), y = __ldg(reinterpret_cast<const ulonglong2*>(p.sw + n) + 1);
      w[0] = x.x; w[1] = x.y; w[2] = y.x; w[3] = y.y;
    }
    if (p.bias) {
      const ulonglong2 x = __ldg(reinterpret_cast<const ulonglong2*>(p.bias + n)), y = __ldg(reinterpret_cast<const ulonglong2*>(p.bias + n) + 1);
      b[0] = x.x; b[1] = x.y; b[2] = y.x; b[3] = y.y;
    }
  }
};

// Those columns' outputs of a token, from element `at` of the output on, from their sums times the
// token's scale; r: their residual
// (zeros without one, which add nothing but turn a -0 into +0).
template <int kAct>
__device__ __forceinline__ void finish8(const LinearFusedArgs& p, int64_t at, const f32x2 (&acc)[4], const Columns& c,
                                        const uint4& r) {
  const uint32_t ru[4] = {r.x, r.y, r.z, r.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = pack2(add2(activate<kAct>(fma2(acc[i], c.w[i], c.b[i])),
                      f32x2_of(__uint_as_float(ru[i] << 16), __uint_as_float(ru[i] & 0xFFFF0000u))));
  *reinterpret_cast<uint4*>(p.out + at) = make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ uint4 residual8(const LinearFusedArgs& p, int64_t at) {
  return p.residual ? *reinterpret_cast<const uint4*>(p.residual + at) : make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------------- pair ----
namespace pair {
constexpr int BM = 256, kMinBN = 64, kMaxBN = 256;   // of the pair; each CTA loads half of either. Widths are multiples of 32
constexpr int kStages = 3;
constexpr int kSub = 2;                // chunks of BK per stage: eight MMAs to a barrier and a commit
constexpr int kHalf = 128 * BK;        // 16 KB: a CTA's rows of one operand, one chunk
constexpr int kStage = 2 * kSub * kHalf;   // [chunk][x rows, weight rows]
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kTurn = 32 * 32 * 4;      // an epilogue warp's buffer: 32 tokens by 32 columns, fp32
constexpr int kSmemBytes = 1024 + kStages * kStage + kEpiWarps * kTurn + 256;
}  // namespace pair

template <int kAct>
__global__ void __launch_bounds__(pair::kThreads, 1)
fp8_linear_pair_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                       const LinearFusedArgs p, const int bn) {
  using namespace pair;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* turn = smem + kStages * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(turn + kEpiWarps * kTurn);   // the leader's: both CTAs' bytes
  uint64_t* empty = full + kStages;                                     // each CTA's
  uint64_t* acc_full = empty + kStages;                                 // each CTA's
  uint64_t* acc_empty = acc_full + 2;                                   // the leader's: both CTAs' epilogue warps
  volatile int* abort_flag = reinterpret_cast<volatile int*>(acc_empty + 2);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_empty + 2) + 1;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform, and known to be
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_x)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(tmem_holder)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();   // the barriers are fenced above, and nothing else is shared yet
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  griddep_launch_dependents();   // only now: a successor's CTA beside this one must not get the tensor memory first
  griddep_wait();

  const int n_tiles = (p.N + bn - 1) / bn, units = ((p.T + BM - 1) / BM) * n_tiles, nk = (p.K + BK - 1) / BK;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer -----
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = first; u < units && ok; u += step) {
        const int m0 = (u / n_tiles) * BM + 128 * static_cast<int>(rank), n0 = (u % n_tiles) * bn + bn / 2 * static_cast<int>(rank);
        for (int kt = 0; kt < nk; kt += kSub) {
          if (!mbar_wait_cluster(&empty[stage], phase ^ 1, abort_flag, p.err)) { ok = false; break; }
          const uint32_t bar = peer_addr(smem_u32(&full[stage]), 0);
          const int chunks = min(kSub, nk - kt);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], (BM + bn) * BK * chunks);
          for (int c = 0; c < chunks; ++c) {
            uint8_t* dst = smem + stage * kStage + 2 * c * kHalf;
            tma_load_2d_pair(dst, &tmap_x, bar, (kt + c) * BK, m0);
            tma_load_2d_pair(dst + kHalf, &tmap_w, bar, (kt + c) * BK, n0);
          }
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      // the leader's last signals have reached this CTA's barriers before it leaves
      for (int s = 0; s < kStages && ok; ++s) {
        ok = mbar_wait_cluster(&empty[stage], phase ^ 1, abort_flag, p.err);
        if (++stage == kStages) { stage = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------- MMA issuer (the leader's warp) ----
    // What the warp does between MMAs shows, since the tensor pipe takes few ahead: eight MMAs
    // to a stage and a commit, the next stage's barrier looked at between them, descriptors
    // that are one addition. (With four MMAs to a stage and a wait before each, 836 cycles for
    // 128 of K although no stage was late; the MMAs need 512, and this loop takes 525.)
    if (rank == 0) {
      const uint32_t elected = elect_one();
      int stage = 0, it = 0;
      uint32_t phase = 0;
      const uint32_t idesc = idesc_e4m3(BM, bn);
      const uint64_t desc = smem_desc(smem_u32(smem), 16, 1024, 2);
      bool ok = true, ready = false;
      for (int u = first; u < units && ok; u += step, ++it) {
        const int ab = it & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&acc_empty[ab], ((it >> 1) & 1) ^ 1, abort_flag, p.err));
        if (!ok) break;
        const uint32_t dacc = tmem + ab * kMaxBN;
        for (int kt = 0; kt < nk; kt += kSub) {
          if (!ready && !__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag, p.err))) { ok = false; break; }
          tc_fence_after();
          const uint64_t ad = desc + static_cast<uint64_t>(stage * (kStage / 16)), bd = ad + kHalf / 16;
          uint64_t* const done = &empty[stage];
          if (++stage == kStages) { stage = 0; phase ^= 1; }
          const int steps = min(4 * kSub, (p.K - kt * BK) / 32);   // K % 32 == 0: the last stage may hold fewer
#pragma unroll
          for (int kk = 0; kk < 4 * kSub; ++kk) {
            const int at = (kk / 4) * (2 * kHalf / 16) + 2 * (kk % 4);
            if (kk < steps) mma_f8<2>(elected, dacc, ad + at, bd + at, idesc, (kt > 0 || kk > 0) ? 1u : 0u);
            if (kk == 4 * kSub - 3) ready = __all_sync(0xffffffffu, mbar_test(&full[stage], phase));
          }
          commit_pair(elected, done);
        }
        if (!ok) break;
        commit_pair(elected, &acc_full[ab]);
      }
      // the other CTA's last signals have reached this CTA's barriers before it leaves
      for (int j = max(0, it - 2); ok && j < it; ++j)
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&acc_empty[j & 1], (j >> 1) & 1, abort_flag, p.err));
    }
  } else {
    // --------------------------------------------------------------- epilogue -----
    // Tensor memory gives a lane one token's columns; global memory wants a row's columns side by
    // side. Each warp turns 32 x 32 sums through its own buffer (16-byte pieces permuted by
    // the token, so that both sides are free of bank conflicts): then eight tokens' 64 bytes
    // go out (and a residual's come in) per instruction instead of 32 tokens' 16. At 4096 x
    // 2880 -> 5120 the direct stores paced the kernel: 60.1 us against 48.1 without them. Steps of 16
    // columns let twelve or sixteen warps fit, but took 52.1 and 54.4 us (eight 51.6) against 50.4;
    // 16 tokens by 64 columns 53.6.
    const int q = warp & 3;              // tensor-memory lane quarter of this warp
    const int c_split = 32 * ((bn / 32 + 1) / 2);   // four warps take the columns up to it, four the others
    const int c_first = warp < 6 ? 0 : c_split, c_count = warp < 6 ? c_split : bn - c_split;
    ulonglong2* const mine = reinterpret_cast<ulonglong2*>(turn + (warp - 2) * kTurn);
    const int row = lane >> 2, col = 8 * (lane & 3);   // the lane's part of a pass: tokens row + 8 i, columns col ..
    // a 32-column chunk's residual and column constants are fetched a chunk ahead
    const int64_t down = 8 * static_cast<int64_t>(p.N);   // eight tokens further
    const auto fetch = [&](uint4 (&res)[4], int64_t at, int left, bool in) {
#pragma unroll
      for (int i = 0; i < 4; ++i) res[i] = in && 8 * i < left ? residual8(p, at + i * down) : make_uint4(0, 0, 0, 0);
    };
    int it = 0;
    for (int u = first; u < units; u += step, ++it) {
      const int ab = it & 1;
      const int64_t t0 = static_cast<int64_t>(u / n_tiles) * BM + 128 * rank + 32 * q;
      const int n0 = (u % n_tiles) * bn + c_first;
      const float sx = t0 + lane < p.T ? (p.sx ? __ldg(p.sx + t0 + lane) : p.sx_all) : 0.f;
      uint4 res[4], res_ahead[4];
      Columns cols, cols_ahead;
      // the lane's first element, and how many tokens are left from it on
      const int64_t at0 = (t0 + row) * p.N + n0 + col;
      const int left = static_cast<int>(min(static_cast<int64_t>(32), p.T - t0 - row));
      fetch(res, at0, left, n0 + col < p.N);   // N % 8 == 0: a group of 8 columns is wholly in or out
      if (n0 + col < p.N) cols.load(p, n0 + col);
      if (!mbar_wait_cluster(&acc_full[ab], (it >> 1) & 1, abort_flag, p.err)) break;
      __syncwarp();
      tc_fence_after();
      const uint32_t tbase = tmem + ab * kMaxBN + c_first + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 32) {
        if (c0 >= c_count || n0 + c0 >= p.N || t0 >= p.T) break;
        const int n = n0 + c0 + col;
        if (c0 + 32 < c_count) {
          fetch(res_ahead, at0 + c0 + 32, left, n + 32 < p.N);
          if (n + 32 < p.N) cols_ahead.load(p, n + 32);
        }
        uint32_t v[32];
        tc_ld_32x32b_x32(tbase + c0, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const f32x2 x = mul2(f32x2_of(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1])), both(sx));
          const f32x2 y = mul2(f32x2_of(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3])), both(sx));
          mine[8 * lane + (j ^ (lane & 7))] = make_ulonglong2(x, y);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = row + 8 * i;
          const ulonglong2 x = mine[8 * r + ((col / 4) ^ (r & 7))], y = mine[8 * r + ((col / 4 + 1) ^ (r & 7))];
          const f32x2 a[4] = {x.x, x.y, y.x, y.y};
          if (n < p.N && 8 * i < left) finish8<kAct>(p, at0 + c0 + i * down, a, cols, res[i]);
        }
        __syncwarp();
        cols = cols_ahead;
#pragma unroll
        for (int i = 0; i < 4; ++i) res[i] = res_ahead[i];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_peer(peer_addr(smem_u32(&acc_empty[ab]), 0));
    }
  }

  // --------------------------------------------------------------------- teardown ---
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {   // let copies already issued land before the CTA's shared memory goes
    const long long t0 = clock64();
    while (clock64() - t0 < 200000) {
    }
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();      // the other CTA may still signal this one's barriers or read its operands
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512));
  }
}

// ------------------------------------------------------------------------ split ----
namespace split {
constexpr int BM = 128;                // weight rows
constexpr int kThreads = 256;
constexpr int kMaxK = 8;               // CTAs of a cluster
constexpr int kA = BM * BK;
constexpr int kRow = 4 * BM;           // bytes of a token's partial sums
constexpr int stage_bytes(int BN) { return kA + BN * BK; }
constexpr int stages(int BN) { return BN <= 64 ? 8 : 5; }
constexpr int tmem_cols(int BN) { return BN < 32 ? 32 : BN; }
// tokens' sums that a CTA is sent: its share of the tile's tokens from each of the others
constexpr int recv_rows(int BN) {
  int most = 0;
  for (int ks = 2; ks <= kMaxK; ++ks) most = std::max(most, (ks - 1) * ((BN + ks - 1) / ks));
  return most;
}
constexpr int smem_bytes(int BN) { return 1024 + stages(BN) * stage_bytes(BN) + recv_rows(BN) * kRow + 256; }
static_assert(smem_bytes(64) <= 232448 && smem_bytes(128) <= 232448, "shared memory of an SM");
}  // namespace split

// Cluster of ks CTAs: weight rows [128 m, + 128), tokens [BN blockIdx.y, + BN), a K range each.
// Each CTA owns a share of the tile's tokens: the others send it their sums of those, one bulk
// copy each, and it adds them and finishes those outputs. Copies cross the cluster at three times
// the rate of plain loads or stores (26 KB in 0.9 us, 2 us or more), and only the receiver waits:
// 64 x 4096 -> 2880 took 9.6 us with each CTA loading its share between two barriers, 8.7 with
// plain stores, and takes 6.3.
template <int BN, int kAct>
__global__ void __launch_bounds__(split::kThreads, 1)
fp8_linear_split_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                        const LinearFusedArgs p, int ks) {
  using namespace split;
  constexpr int kStages = stages(BN), kStage = stage_bytes(BN);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* recv = smem + kStages * kStage;   // [sending rank, this one left out][share][128 weight rows], fp32
  uint64_t* full = reinterpret_cast<uint64_t*>(recv + recv_rows(BN) * kRow);
  uint64_t* empty = full + kStages;
  uint64_t* done = empty + kStages;
  uint64_t* got = done + 1;                  // the others' sums have arrived
  volatile int* abort_flag = reinterpret_cast<volatile int*>(got + 1);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(got + 1) + 1;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform, and known to be
  const int rank = static_cast<int>(cluster_rank());
  const int m0 = (blockIdx.x / ks) * BM, t0 = blockIdx.y * BN;
  const int nk = (p.K + BK - 1) / BK, k0 = rank * nk / ks, count = (rank + 1) * nk / ks - k0;
  // this CTA's share of the tile's tokens
  const int tokens = min(BN, p.T - t0), share = (tokens + ks - 1) / ks, mine = rank * share;
  const int rows = max(0, min(share, tokens - mine));
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_x)) : "memory");
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(got, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    mbar_arrive_expect_tx(got, (ks - 1) * rows * kRow);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(tmem_holder)),
                 "r"(tmem_cols(BN)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  __syncwarp();
  cluster_arrive();   // this CTA's barriers stand (fenced above): the others may send to it
  uint32_t tmem = 0;
  if (warp == 0) {    // needs no tensor memory: the loads start while it is taken
    asm volatile("bar.arrive 1, %0;\n" ::"n"(kThreads) : "memory");
  } else {
    tc_fence_before();
    asm volatile("bar.sync 1, %0;\n" ::"n"(kThreads) : "memory");
    tc_fence_after();
    tmem = *tmem_holder;
    griddep_launch_dependents();   // only now: a successor's CTA beside this one must not get the tensor memory first
  }
  griddep_wait();

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < count; ++i) {
        const int stage = i % kStages;
        if (i >= kStages && !mbar_wait(&empty[stage], (i / kStages + 1) & 1, abort_flag, p.err)) break;
        mbar_arrive_expect_tx(&full[stage], kStage);
        tma_load_2d(smem + stage * kStage, &tmap_w, &full[stage], (k0 + i) * BK, m0);
        tma_load_2d(smem + stage * kStage + kA, &tmap_x, &full[stage], (k0 + i) * BK, t0);
      }
    }
  } else if (warp == 1) {
    const uint32_t elected = elect_one();
    const uint64_t desc = smem_desc(smem_u32(smem), 16, 1024, 2);
    bool ok = true, ready = false;
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < count; ++i) {
      if (!ready && !__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag, p.err))) { ok = false; break; }
      tc_fence_after();
      const uint64_t ad = desc + static_cast<uint64_t>(stage * (kStage / 16)), bd = ad + kA / 16;
      uint64_t* const freed = &empty[stage];
      if (++stage == kStages) { stage = 0; phase ^= 1; }
      const int steps = min(4, (p.K - (k0 + i) * BK) / 32);   // K % 32 == 0
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk < steps) mma_f8<1>(elected, tmem, ad + 2 * kk, bd + 2 * kk, idesc_e4m3(BM, BN), (i > 0 || kk > 0) ? 1u : 0u);
        if (kk == 2) ready = __all_sync(0xffffffffu, mbar_test(&full[stage], phase));
      }
      if (i + kStages < count) commit(elected, freed);   // only a stage that is loaded again
    }
    if (ok) commit(elected, done);
  }
  __syncwarp();
  // a thread finishes 8 columns, the same for each of its tokens; what they need from global memory is
  // fetched while the products run
  constexpr int kPasses = (BN * BM / 8 + kThreads - 1) / kThreads, kStep = kThreads / (BM / 8);
  const int col = 8 * (threadIdx.x % (BM / 8)), n = m0 + col, row0 = threadIdx.x / (BM / 8);
  const int passes = n < p.N && row0 < rows ? (rows - row0 + kStep - 1) / kStep : 0;
  Columns cols;
  uint4 res[kPasses];
  float sx[kPasses];
  if (passes > 0) cols.load(p, n);
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    if (i < passes) {
      const int64_t t = t0 + mine + row0 + i * kStep;
      res[i] = residual8(p, t * p.N + n);
      sx[i] = p.sx ? __ldg(p.sx + t) : p.sx_all;
    }
  __syncwarp();
  cluster_wait();
  if (warp == 0) griddep_launch_dependents();   // tensor memory was taken before that barrier
  // every stage has been consumed when `done` completes: its memory takes this CTA's sums, fp32
  // [token][128 weight rows]; each share of them is one copy to the share's owner
  float* const sums = reinterpret_cast<float*>(smem);
  if (warp >= 4) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(done, 0, abort_flag, p.err));
    if (ok) {
      tc_fence_after();
      const int q = warp & 3;
      if constexpr (BN >= 32) {
        for (int c0 = 0; c0 < tokens; c0 += 32) {
          uint32_t v[32];
          tc_ld_32x32b_x32(tmem + c0 + (static_cast<uint32_t>(32 * q) << 16), v);
#pragma unroll
          for (int i = 0; i < 32; ++i) sums[(c0 + i) * BM + 32 * q + lane] = __uint_as_float(v[i]);
        }
      } else {
        for (int c0 = 0; c0 < tokens; c0 += 8) {
          uint32_t v[8];
          tc_ld_32x32b_x8(tmem + c0 + (static_cast<uint32_t>(32 * q) << 16), v);
          tc_wait_ld(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) sums[(c0 + i) * BM + 32 * q + lane] = __uint_as_float(v[i]);
        }
      }
      tc_fence_before();
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    }
    asm volatile("bar.sync 2, 128;\n" ::: "memory");
    if (warp == 4 && lane < ks && lane != rank && !*abort_flag) {
      const int n = min(share, tokens - lane * share);
      if (n > 0)
        send_bulk(peer_addr(smem_u32(recv) + (rank < lane ? rank : rank - 1) * share * kRow, lane), sums + lane * share * BM,
                  n * kRow, peer_addr(smem_u32(got), lane));
    }
  }
  __syncthreads();     // this CTA's own sums; the accumulators have been read
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(tmem_cols(BN)));
  }
  const bool whole = mbar_wait_cluster(got, 0, abort_flag, p.err);
  __syncwarp();
  cluster_arrive();   // what was sent to this CTA is here
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    if (whole && i < passes) {
      const int row = row0 + i * kStep, at = 4 * (row * BM + col);
      f32x2 a[4] = {0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < kMaxK; ++r)
        if (r < ks) {              // added in rank order
          const uint8_t* from = (r == rank ? smem + mine * kRow : recv + (r < rank ? r : r - 1) * share * kRow) + at;
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(from), y = *reinterpret_cast<const ulonglong2*>(from + 16);
          a[0] = add2(a[0], x.x); a[1] = add2(a[1], x.y); a[2] = add2(a[2], y.x); a[3] = add2(a[3], y.y);
        }
#pragma unroll
      for (int c = 0; c < 4; ++c) a[c] = mul2(a[c], both(sx[i]));
      finish8<kAct>(p, static_cast<int64_t>(t0 + mine + row) * p.N + n, a, cols, res[i]);
    }
  if (*abort_flag) {   // let copies already issued land before the CTA's shared memory goes
    const long long c0 = clock64();
    while (clock64() - c0 < 200000) {
    }
  }
  __syncwarp();
  cluster_wait();      // what this CTA sent has been received
}

}  // namespace linf

namespace {

// (rows, K) bytes, K-major, box (BK, box_rows), 128-byte swizzle, zero fill outside
bool encode_codes(CUtensorMap* m, const void* base, int64_t rows, int64_t K, uint32_t box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(K)};
  const uint32_t box[2] = {static_cast<uint32_t>(linf::BK), box_rows};
  return tmap_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box);
}

template <int kAct>
cudaError_t launch_pair(const LinearFusedArgs& p, int bn, int sms, cudaStream_t st) {
  using namespace linf;
  CUtensorMap mx, mw;
  if (!encode_codes(&mx, p.xq, p.T, p.K, 128) || !encode_codes(&mw, p.wq, p.N, p.K, bn / 2)) return cudaErrorInvalidValue;
  static SmemLimit limit;
  cudaError_t e = limit.raise(fp8_linear_pair_kernel<kAct>, pair::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t units = cdiv(p.T, pair::BM) * cdiv(p.N, bn);
  const int grid = 2 * static_cast<int>(std::min<int64_t>(units, sms / 2));
  return launch_early(fp8_linear_pair_kernel<kAct>, dim3(static_cast<unsigned>(grid)), pair::kThreads, pair::kSmemBytes, 2,
                      st, mx, mw, p, bn);
}

// Clusters of ks CTAs of the split kernel that the device holds at once: a cluster lies in one
// GPC, so a size that does not divide a GPC's SMs leaves some idle (the activations' kernels
// are alike in registers and shared memory). Asked once per device, tile and size.
template <int BN>
int clusters_at_once(int ks, const cudaLaunchConfig_t& cfg) {
  static std::atomic<int> known[64][linf::split::kMaxK + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][ks].load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  const auto kernel = linf::fp8_linear_split_kernel<BN, MXMOE_ACT_NONE>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, linf::split::smem_bytes(BN)) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[dev][ks].store(n + 1, std::memory_order_relaxed);
  return n;
}

// K ranges of the split kernel: the most whose clusters all run at once.
template <int BN>
int split_ranges(int64_t tiles, int K, int sms) {
  using namespace linf;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(split::kThreads);
  cfg.dynamicSmemBytes = split::smem_bytes(BN);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int ks = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({split::kMaxK, cdiv(K, BK), sms / tiles})));
  for (; ks > 1; --ks) {
    attr[0].val.clusterDim.x = static_cast<unsigned>(ks);
    cfg.gridDim = dim3(static_cast<unsigned>(ks));
    if (tiles <= clusters_at_once<BN>(ks, cfg)) break;
  }
  return ks;
}

template <int BN, int kAct>
cudaError_t launch_split(const LinearFusedArgs& p, int sms, cudaStream_t st) {
  using namespace linf;
  CUtensorMap mx, mw;
  if (!encode_codes(&mx, p.xq, p.T, p.K, BN) || !encode_codes(&mw, p.wq, p.N, p.K, split::BM)) return cudaErrorInvalidValue;
  constexpr int smem = split::smem_bytes(BN);
  static SmemLimit limit;
  cudaError_t e = limit.raise(fp8_linear_split_kernel<BN, kAct>, smem);
  if (e != cudaSuccess) return e;
  const int m_tiles = static_cast<int>(cdiv(p.N, split::BM)), t_tiles = static_cast<int>(cdiv(p.T, BN));
  const int ks = split_ranges<BN>(static_cast<int64_t>(m_tiles) * t_tiles, p.K, sms);
  return launch_early(fp8_linear_split_kernel<BN, kAct>, dim3(static_cast<unsigned>(m_tiles * ks), static_cast<unsigned>(t_tiles)),
                      split::kThreads, smem, ks, st, mw, mx, p, ks);
}

// What either kernel takes for more than 64 tokens, in ns, from what they measured on a B200 at 40
// sizes (65 to 18944 tokens, K 64 to 8192, N 64 to 8192); nk = K / 128 rounded up.
//
// A pair's chunk of K is bound by what one SM draws from L2 (its 128 rows and half of the weights'),
// and more of it the more SMs draw at once; a narrow tile costs more loads for each product but
// fills the last round better. E.g. 4096 x 2880 -> 5120: 256 columns 52.2 us, 224 50.9, 160 59.5;
// 1024 x 2880 -> 5120: 160 19.8, 256 23.3, 64 33.7; 200 x 2880 -> 5120: 96 10.3, 256 13.7; 1000 x 8192 ->
// 256: 64 17.8, 160 19.2, 256 24.6; 777 x 1024 -> 4096: 256 9.6, 128 9.4, 64 11.6. (The model was fitted
// to the kernel before its last epilogue, 5 to 10 % slower throughout.)
int64_t pair_ns(const LinearFusedArgs& p, int bn, int sms) {
  using namespace linf;
  const int64_t nk = cdiv(p.K, BK), pairs = std::max(1, sms / 2);
  const int64_t tiles = cdiv(p.T, pair::BM) * cdiv(p.N, bn), rounds = cdiv(tiles, pairs);
  const int64_t chunk = 235 + 30 * bn / 100 + (10 + 53 * bn / 100) * std::min(tiles, pairs) / pairs;
  return 3200 + 10 * bn + rounds * (500 + std::max<int64_t>(nk * chunk, 1000 + 11 * bn));
}

int pair_width(const LinearFusedArgs& p, int sms) {
  using namespace linf;
  int best = pair::kMaxBN;
  for (int bn = best - 32; bn >= pair::kMinBN; bn -= 32)
    if (pair_ns(p, bn, sms) < pair_ns(p, best, sms)) best = bn;
  return best;
}

// The split kernel's, 128 tokens wide. E.g. (pairs, split) 128 x 512 -> 640: 4.8 us, 6.2; 128 x 1024 ->
// 8192: 6.9, 7.0; 128 x 8192 -> 1024: 17.1, 9.6; 200 x 2880 -> 5120: 10.3, 12.5; 300 x 8192 -> 1024: 17.4,
// 11.0; 300 x 4096 -> 4096: 12.3, 15.1; 4000 x 8192 -> 256: 20.5, 16.4. Up to 64 tokens its tiles are
// narrower and it is the shorter everywhere (64 x 1024 -> 8192: 7.5, 5.5; 64 x 512 -> 640: 4.8, 4.8).
int64_t split_ns(const LinearFusedArgs& p, int sms) {
  using namespace linf;
  const int64_t tiles = cdiv(p.N, split::BM) * cdiv(p.T, 128);
  const int ks = split_ranges<128>(tiles, p.K, sms);
  return cdiv(tiles * ks, sms) * (6000 + 370 * cdiv(p.K, BK) / ks);
}

}  // namespace

int fp8_linear_fused_columns(const LinearFusedArgs& p, int sms) {
  if (p.T <= 64) return 0;
  const int bn = pair_width(p, sms);
  return pair_ns(p, bn, sms) < split_ns(p, sms) ? bn : 0;
}

namespace {

template <int kAct>
cudaError_t launch_act(const LinearFusedArgs& p, int sms, cudaStream_t st) {
  if (const int bn = fp8_linear_fused_columns(p, sms)) return launch_pair<kAct>(p, bn, sms, st);
  if (p.T <= 16) return launch_split<16, kAct>(p, sms, st);
  if (p.T <= 32) return launch_split<32, kAct>(p, sms, st);
  if (p.T <= 64) return launch_split<64, kAct>(p, sms, st);
  return launch_split<128, kAct>(p, sms, st);
}

}  // namespace

cudaError_t launch_fp8_linear_fused(const LinearFusedArgs& p, int sms, cudaStream_t st) {
  if (p.act == MXMOE_ACT_SILU) return launch_act<MXMOE_ACT_SILU>(p, sms, st);
  if (p.act == MXMOE_ACT_GELU) return launch_act<MXMOE_ACT_GELU>(p, sms, st);
  return launch_act<MXMOE_ACT_NONE>(p, sms, st);
}

}  // namespace mxmoe
