// The packed layer with adapters for many tokens, on tcgen05: both directions of
//   forward   out[t, r] = Σ_k X[t, k] Ŵ[r, k]  + Σ_j U[t, j] B[a_t, j, r]
//   backward  out[t, k] = Σ_r dY[t, r] Ŵ[r, k] + Σ_j G[t, j] A[a_t, j, k]
// as D[feature, token] tiles of 256 x BN on CTA pairs (cta_group::2): each CTA makes the weight operand
// of its own 128 features and copies its half of the tokens, so that a stage costs 64 KB of its shared
// memory's bandwidth (MMA reads, copies and stores) instead of the 96 KB that held a single-CTA version
// at about 60 % of the tensor cores' rate.  The weight operand is made from the codes on the way into
// shared memory; the stage's image is the same in both directions (row = weight row, 128 bytes = 64
// columns, 128-byte swizzle), read K-major forward (the contraction runs along the row) and MN-major
// backward (it runs down the rows), so one kernel serves both.
//
//   Forward: the stage holds (c - z), exact in 16 bits; the group's Δ multiplies each 128-column
//   partial sum in fp32 as it is taken out of TMEM, so Ŵ is never rounded.
//   Backward: Δ differs along the contraction, so it has to be in the operand.  Δ (c - z) enters as two
//   16-bit parts, a stage each against the same tokens, and keeps 14 bits of bf16 (16 in the mean) or 19
//   of fp16, far below half a step of dX; as one 16-bit number it made dX 1.41 times as far from the
//   exact sum as its own rounding, for half the products.  (fp16 operands carry a power of two, taken
//   out at the end, that brings the largest Δ of the columns' group to 2^11 and more: with a factor for
//   all layers, small Δ were subnormal and lost their bits.)
//   Adapters: each adapter that occurs among the tile's tokens ("slot") adds one more partial sum,
//   whose operands are the adapter's 16-bit rows and U in two tf32 parts (22 bits), both fp32 in
//   shared memory (kind::tf32); the epilogue adds it to that adapter's tokens only, so one request's
//   non-finite values never reach another's.
//
// Roles (one CTA per SM, persistent over tiles; barriers that the MMAs wait for are the leader's, and
// the other CTA's warps arrive on them remotely):
//   warps 0-7     the weight operand: codes and grid of a unit, shared -> registers -> shared
//   warps 8-15    epilogue: TMEM -> fp32 sums in registers -> out, or a split's partial
//   warp 16       TMA producer of the tokens' operand (BN / 2 rows x 128 bytes per stage)
//   warp 17       MMA issuer (the leader's), owner of TMEM (two partial-sum buffers of BN columns)
//   warp 18       copies of the codes (TMA boxes) and of the grid, some units ahead; 19 idle
// Across the pair the order is the memory model's: every wait acquires in cluster scope, and a weight warp
// releases what it wrote by a cluster-scope fence of shared memory alone before its arrivals (neither costs
// anything measurable; arrivals that release all memory took a stage from 0.53 us to 0.87, and passed on
// by one warp for both stages of a unit the call of 4096 tokens from 445 us to 502).
// The grid is first turned column-major (turn_grid), so that the (Δ, z) of a unit's rows are one
// contiguous copy: read in place they are 128 scattered words per step, and loads of codes and grid
// into the weight warps' registers, though issued two to four stages ahead, took as long as the
// whole stage (0.74 us of 256 tokens; without them 0.45).
// Few tokens: the contraction is split over CTAs and k_lora_join adds the splits and the adapter.
//
// 4096 tokens, 11008 x 4096, rank 64, forward: 368 us (1.00 PFLOP/s of 1.67 measured); 4096 x 11008, rank
// 32, backward: 527 us (0.70 of the formula's operations, 1.40 of the products that the two parts make: the
// tensor cores' sustained rate).  Both run at the power limit.  Of the forward's 375 us before its rows
// were written four features at a time, the adapters' partial sums were 48 us, the output 40, the fp32
// additions of the base partials 40.
#include <algorithm>
#include <type_traits>

#include "lora_rings.h"
#include "lora_util.cuh"
#include "tc_util.cuh"

namespace gptq {

constexpr int LT_THREADS = 640;
constexpr int LT_A_BYTES = 128 * 128;      // weight operand of a stage
constexpr int LT_DELTAS = 8;               // forward: partial sums whose Δ wait in shared memory

template <bool FWD, int BN>
struct LtCfg {
  static constexpr int X_BYTES = BN / 2 * 128;
  static constexpr int STAGE = LT_A_BYTES + X_BYTES;
  static constexpr int NS = BN == 256 ? 6 : 8;
  // a unit of codes and grid: 128 rows x 128 columns forward, 64 rows backward
  static constexpr int C_BYTES = FWD ? 8192 : 4096, G_BYTES = FWD ? 1024 : 512;
  static constexpr int NC = FWD ? kLoraCodeSlotsForward : kLoraCodeSlotsBackward;
  static constexpr int NB = lora_code_barriers(NC);   // their barriers
  static constexpr int SMEM = NS * STAGE + NC * (C_BYTES + G_BYTES) + LT_DELTAS * 128 * 4 + 1024 + 512;
  static constexpr int EBN = BN / 2;       // tokens per epilogue thread
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(NB % 2 == 0 && NB % NC == 0, "a barrier of code units belongs to one group of weight warps");
};

struct LtParams {
  int M;                    // features out
  int T;
  int group_steps;          // groups in 128-column steps; 0: one grid per row
  const float2* grid;       // [n_g, m_pad] (Δ, z), zero behind m
  const uint32_t* group_max;   // [n_g] bits of the largest |Δ| (fp16, backward)
  int m_pad, used;          // its columns, and how many n_g there are
  int mtiles, ttiles, splits;
  int units, per;           // the contraction in 128-column (forward) or 64-row (backward) units of two
                            // stages: in all and per split
  int T_rows;               // rows of one part of the split U
  int rank_chunks;          // 32-rank chunks; 0: no adapter partials (split contraction)
  int R, n;
  const int32_t* adapter;
  const void* w;            // [n, R, M] 16-bit
  const int32_t* slots;     // per token tile: count, then the adapters that occur in it
  void* out;                // [T, M]
  int out_f32, wide_out;    // wide_out: 16-bit, M a multiple of 4, 8-byte aligned
  float* part;              // [splits, T, M] or null
  uint32_t idesc, idesc_tf32;
};

// The group of the columns that start at a multiple of 128 (the second CTA's may lie behind the last:
// they are not stored).
__device__ __forceinline__ int lt_group(const LtParams& p, int column) {
  return p.group_steps ? min(column / 128 / p.group_steps, p.used - 1) : 0;
}
// The power of two that brings the group's largest |Δ| into [2^11, 2^12): |Δ (c - z)| stays below 61441.
// (Only within 2^±100: beyond, fp32 products would leave their own range.)
__device__ __forceinline__ int lt_f16_exponent(const LtParams& p, int column) {
  const int e = (int)(p.group_max[lt_group(p, column)] >> 23) - 127;
  return 11 - min(max(e, -89), 100);
}
__device__ __forceinline__ float lt_power(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ bool lt_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool lt_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// What this warp's lanes wrote to shared memory before a __syncwarp is visible to whoever sees the arrivals
// that follow, in either CTA.
__device__ __forceinline__ void lt_release() {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}
// `count` arrivals on a barrier of either CTA (a shared::cluster address; this CTA's shared::cta
// addresses are among them), after lt_release.
__device__ __forceinline__ void lt_arrive_remote(uint32_t cluster_addr, uint32_t count) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_addr), "r"(count)
               : "memory");
}
// Waits for a phase, suspended in hardware between tries; false after `budget` cycles.
__device__ __forceinline__ bool lt_wait(uint64_t* bar, uint32_t parity, long long budget) {
  if (lt_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (!lt_try(bar, parity))
    if (clock64() - t0 > budget) return false;
  return true;
}
// Two phases at once: both are tried before either is waited for.
__device__ __forceinline__ bool lt_wait2(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1,
                                         long long budget) {
  const bool r0 = lt_try(b0, p0), r1 = lt_try(b1, p1);
  return (r0 || lt_wait(b0, p0, budget)) && (r1 || lt_wait(b1, p1, budget));
}
__device__ __forceinline__ bool lt_wait_warp(uint64_t* bar, uint32_t parity, long long budget) {
  return __all_sync(0xffffffffu, lt_wait(bar, parity, budget));
}

// 8 TMEM columns of this warp's lanes; the registers may be read after lt_tmem_wait8 on them.
__device__ __forceinline__ void lt_tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                 "=r"(v[6]), "=r"(v[7])
               : "r"(taddr));
}
__device__ __forceinline__ void lt_tmem_wait8(uint32_t (&v)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7])
               :
               : "memory");
}
__device__ __forceinline__ uint64_t pack_f32x2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
// (a0, a1) += f · (v0, v1)
__device__ __forceinline__ void fma_f32x2(float& a0, float& a1, uint64_t f, uint32_t v0,
                                          uint32_t v1) {
  asm("{\n\t.reg .b64 a, v;\n\t"
      "mov.b64 a, {%0, %1};\n\t"
      "mov.b64 v, {%3, %4};\n\t"
      "fma.rn.f32x2 a, %2, v, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "l"(f), "r"(v0), "r"(v1));
}

// Two values rounded to the 16-bit type, the first in the low half.
template <bool BF16> __device__ __forceinline__ uint32_t pack16(float a, float b) {
  if (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Δ of a row, and with it (c - z) Δ as a sum of two 16-bit numbers.  With Δ = H + L (each rounded once)
// and H' a little below H, hi = round((c - z) H') is always smaller in magnitude than (c - z) Δ: the
// margin of 5/4 half steps (2^-8 of bf16, 2^-11 of fp16) covers its rounding and that of L.  What is
// left, ((c - z) H - hi) + (c - z) L, has an exact first term (at most 158 units of hi's last place, of
// the 256 that the type holds) and is rounded once, to within 2^-14 of the weight (2^-19 for fp16).  It is
// never zero and never of the other sign unless c = z, so that an infinite gradient stays infinite in
// the sum of both products.
template <bool BF16> struct WeightParts {
  using T2 = typename std::conditional<BF16, __nv_bfloat162, __half2>::type;
  T2 h, l, under;
  __device__ __forceinline__ WeightParts() {}
  __device__ __forceinline__ explicit WeightParts(float d) {
    if constexpr (BF16) {
      const __nv_bfloat16 H = __float2bfloat16_rn(d);
      h = __bfloat162bfloat162(H);
      l = __bfloat162bfloat162(__float2bfloat16_rn(d - __bfloat162float(H)));
      under = __bfloat162bfloat162(__float2bfloat16_rz(d * (1.f - 0x5p-10f)));
    } else {
      const __half H = __float2half_rn(d);
      h = __half2half2(H);
      l = __half2half2(__float2half_rn(d - __half2float(H)));
      under = __half2half2(__float2half_rz(d * (1.f - 0x5p-13f)));
    }
  }
  // v: two values of (c - z), replaced by the high parts
  __device__ __forceinline__ void split(uint32_t& v, uint32_t& low) const {
    const T2 c = *reinterpret_cast<const T2*>(&v);
    const T2 hi = __hmul2(c, under);
    const T2 lo = __hfma2(c, l, __hfma2(c, h, __hneg2(hi)));
    v = *reinterpret_cast<const uint32_t*>(&hi);
    low = *reinterpret_cast<const uint32_t*>(&lo);
  }
};

// A position in a ring of N stages or buffers.
template <int N> struct LtRing {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      phase ^= 1;
    }
  }
};

// One work item of a pair: a tile of features x tokens and a range of the contraction; f0 is this
// CTA's half.
struct LtTile {
  int f0, t0, nt, split, u0, u1;
  __device__ __forceinline__ LtTile(const LtParams& p, int i, int BN, int rank) {
    const int mt = i % p.mtiles, r = i / p.mtiles;
    nt = r % p.ttiles;
    split = r / p.ttiles;
    f0 = mt * 256 + 128 * rank;
    t0 = nt * BN;
    u0 = split * p.per;
    u1 = min(p.units, u0 + p.per);
  }
};

template <bool FWD, int BN, bool BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(LT_THREADS, 1)
    k_lora_tc(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmU,
              const __grid_constant__ CUtensorMap tmC,
              const __grid_constant__ LtParams p, DeviceStatus* st, long long budget) {
  using Cfg = LtCfg<FWD, BN>;
  constexpr int NS = Cfg::NS, EBN = Cfg::EBN, ND = 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int NC = Cfg::NC, NB = Cfg::NB;
  uint8_t* codes = smem + NS * Cfg::STAGE;               // NC units of codes, then of grid
  float2* grids = reinterpret_cast<float2*>(codes + NC * Cfg::C_BYTES);
  float* deltas = reinterpret_cast<float*>(codes + NC * (Cfg::C_BYTES + Cfg::G_BYTES));
  uint64_t* full_x = reinterpret_cast<uint64_t*>(deltas + LT_DELTAS * 128);
  uint64_t* full_a = full_x + NS;
  uint64_t* empty = full_a + NS;
  uint64_t* d_full = empty + NS;
  uint64_t* d_empty = d_full + ND;
  uint64_t* full_c = d_empty + ND;
  uint64_t* empty_c = full_c + NB;
  uint64_t* drain = empty_c + NC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int items = p.mtiles * p.ttiles * p.splits;
  const int rank = (int)tc::cluster_rank(), pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(&full_x[s], 1);
      tc::mbar_init(&full_a[s], 16);   // the weight warps of both CTAs
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < ND; ++b) {
      tc::mbar_init(&d_full[b], 1);
      tc::mbar_init(&d_empty[b], 16);
    }
    for (int b = 0; b < NB; ++b) tc::mbar_init(&full_c[b], 1);
    for (int b = 0; b < NC; ++b) tc::mbar_init(&empty_c[b], 8);
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::mbar_fence_init();
    tc::prefetch_tmap(&tmX);
    tc::prefetch_tmap(&tmU);
    tc::prefetch_tmap(&tmC);
  }
  tc::cluster_sync();   // both CTAs' barriers exist before any remote arrive
  if (warp == 17) tc::tmem_alloc_pair(tmem_slot, ND * BN);
  tc::fence_before_sync();
  tc::cluster_sync();   // TMEM allocated in both before the first MMA
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // The kernel right before (A X or B dY of this call) has itself waited for everything earlier, so X
  // and dY may be read now; only its own results (the grid, slots, the split U) wait for it, in each role.
  // the leader's barriers
  const uint32_t lead_full_x = tc::map_to_rank(full_x, 0), lead_full_a = tc::map_to_rank(full_a, 0);
  const uint32_t lead_d_empty = tc::map_to_rank(d_empty, 0);

  // registers: 640 threads start with 96 (61440; build.py refuses a compilation with fewer);
  // 128 x 40 + 256 x 64 + 256 x 152 = 60416
  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 16 && lane == 0) {
      // -------------------------------------------------------------- tokens' operand
      LtRing<NS> ring;
      int issued = 0;
      bool ok = true, waited = false;
      auto stage = [&](const CUtensorMap* map, int x, int y) {
        if (!ok) return;
        if (!lt_wait(&empty[ring.i], ring.phase ^ 1u, budget)) {
          raise_error(st, GPTQ_ERR_TIMEOUT, 71);
          *abort_flag = 1;
          ok = false;
          return;
        }
        if (rank == 0) tc::mbar_expect_tx(&full_x[ring.i], 2 * Cfg::X_BYTES);   // both CTAs' copies
        tc::tma_load_2d_pair(smem + ring.i * Cfg::STAGE + LT_A_BYTES, map, lead_full_x + 8u * ring.i, x,
                             y + rank * (BN / 2));
        ring.next();
        ++issued;
      };
      for (int i = pair; i < items && ok && !*abort_flag; i += npairs) {
        const LtTile t(p, i, BN, rank);
        for (int k = 2 * t.u0; k < 2 * t.u1 && ok; ++k) stage(&tmX, (FWD ? k : k >> 1) * 64, t.t0);
        if (!p.rank_chunks) continue;
        if (!waited) pdl_wait();   // only now: the tokens' operand is the caller's
        waited = true;
        const int count = p.slots[t.nt * (BN + 1)];
        for (int s = 0; s < count && ok; ++s)
          for (int c = 0; c < 2 * p.rank_chunks && ok; ++c)
            stage(&tmU, (c >> 1) * 32, (c & 1) * p.T_rows + t.t0);
      }
      // every copy has landed before the CTAs may exit: the leader's barriers count both CTAs'
      const int left = rank == 0 ? min(issued, NS) : 0;
      for (int s = 0; s < left; ++s) {
        const int j = issued - left + s;
        if (!lt_wait(&full_x[j % NS], (uint32_t)(j / NS) & 1u, kDrainCycles))
          raise_error(st, GPTQ_ERR_TIMEOUT, 72);
      }
    } else if (warp == 17 && rank == 0) {
      // -------------------------------------------------------------- MMA issuer
      // (the whole warp runs the loop, so that descriptors and addresses stay in uniform registers, and
      // one lane issues)
      uint32_t elected;
      asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                   : "=r"(elected));
      LtRing<NS> ring;
      LtRing<ND> dr;
      bool ok = true, any = false, ready = false;
      pdl_wait();   // the slots
      // The descriptors of stage 0; a stage or a k step on is an addition to the address field (in
      // 16-byte units; shared memory ends below its 14 bits).  Little else may stand between the
      // MMAs: this thread's own instructions are what would hold them up.
      const uint32_t a0 = tc::smem_u32(smem), b0 = a0 + LT_A_BYTES;
      const uint64_t da0 = FWD ? tc::sdesc_sw128(a0, 16, 1024) : tc::sdesc_sw128(a0, 8192, 1024);
      const uint64_t dk0 = tc::sdesc_sw128(a0, 16, 1024), db0 = tc::sdesc_sw128(b0, 16, 1024);
      constexpr uint32_t A_STEP = FWD ? 2 : 128;
      // one partial sum of `stages` stages
      auto partial = [&](int stages, bool tf32) {
        if (!ok) return;
        if (!lt_wait_warp(&d_empty[dr.i], dr.phase ^ 1u, budget)) {
          raise_error(st, GPTQ_ERR_TIMEOUT, 73);
          *abort_flag = 1;
          ok = false;
          return;
        }
        const uint32_t d = tmem + dr.i * BN;
        for (int s = 0; s < stages; ++s) {
          if (!ready && !__all_sync(0xffffffffu, lt_wait2(&full_x[ring.i], ring.phase, &full_a[ring.i],
                                                          ring.phase, budget))) {
            raise_error(st, GPTQ_ERR_TIMEOUT, 74);
            *abort_flag = 1;
            ok = false;
            return;
          }
          tc::fence_after_sync();
          const uint32_t at = ring.i * (Cfg::STAGE / 16);
          const uint64_t db = db0 + at;
          LtRing<NS> next = ring;
          next.next();
          if (tf32) {
            const uint64_t da = dk0 + at;
            if (elected) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_tf32_pair(d, da + 2 * kk, db + 2 * kk, p.idesc_tf32, (s | kk) ? 1u : 0u);
              tc::mma_commit_pair(&empty[ring.i]);
            }
            ready = false;
          } else {
            const uint64_t da = da0 + at;
            if (elected) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_f16_pair(d, da + A_STEP * kk, db + 2 * kk, p.idesc, (s | kk) ? 1u : 0u);
              tc::mma_commit_pair(&empty[ring.i]);
            }
            // the next stage's barriers, while these MMAs are still being worked on
            ready = __all_sync(0xffffffffu, lt_test(&full_x[next.i], next.phase) &&
                                                lt_test(&full_a[next.i], next.phase));
          }
          any = true;
          ring = next;
        }
        if (elected) tc::mma_commit_pair(&d_full[dr.i]);
        dr.next();
      };
      for (int i = pair; i < items && ok && !*abort_flag; i += npairs) {
        const LtTile t(p, i, BN, rank);
        const int count = p.rank_chunks ? p.slots[t.nt * (BN + 1)] : 0;   // on its way meanwhile
        if (FWD)
          for (int u = t.u0; u < t.u1 && ok; ++u) partial(2, false);
        else
          partial(2 * (t.u1 - t.u0), false);
        for (int s = 0; s < count && ok; ++s) partial(2 * p.rank_chunks, true);
      }
      // every MMA has completed before TMEM is freed
      if (any) {
        if (elected) tc::mma_commit_pair(drain);
        if (!lt_wait(drain, 0, kDrainCycles)) raise_error(st, GPTQ_ERR_TIMEOUT, 75);
      }
    } else if (warp == 18 && lane == 0) {
      // -------------------------------------------------------------- codes and grid
      LtRing<NC> ring;   // the slots
      LtRing<NB> bar;    // and their barriers
      int issued = 0;
      bool ok = true;
      pdl_wait();   // the grid
      for (int i = pair; i < items && ok && !*abort_flag; i += npairs) {
        const LtTile t(p, i, BN, rank);
        for (int u = t.u0; u < t.u1; ++u) {
          if (!lt_wait(&empty_c[ring.i], ring.phase ^ 1u, budget)) {
            raise_error(st, GPTQ_ERR_TIMEOUT, 79);
            *abort_flag = 1;
            ok = false;
            break;
          }
          const int g = lt_group(p, FWD ? 128 * u : t.f0);
          const int row = FWD ? t.f0 : 64 * u;
          tc::mbar_expect_tx(&full_c[bar.i], Cfg::C_BYTES + Cfg::G_BYTES);
          tc::tma_load_2d(codes + ring.i * Cfg::C_BYTES, &tmC, &full_c[bar.i],
                          FWD ? 16 * u : t.f0 / 8, row);
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
              "[%3];" ::"r"(tc::smem_u32(grids) + ring.i * Cfg::G_BYTES),
              "l"(p.grid + (long long)g * p.m_pad + row), "r"(Cfg::G_BYTES),
              "r"(tc::smem_u32(&full_c[bar.i]))
              : "memory");
          ring.next();
          bar.next();
          ++issued;
        }
      }
      const int left = min(issued, NB);
      for (int s = 0; s < left; ++s) {
        const int j = issued - left + s;
        if (!lt_wait(&full_c[j % NB], (uint32_t)(j / NB) & 1u, kDrainCycles))
          raise_error(st, GPTQ_ERR_TIMEOUT, 80);
      }
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ---------------------------------------------------------------- weight operand
    const int tid = threadIdx.x;
    LtRing<NS> ring;
    LtRing<NB> cring;   // the units' barriers; their slots are cring.i % NC
    bool ok = true;
    pdl_wait();   // the slots
    // A thread's piece is 16 bytes (32 codes) of a row: eight lanes with the same piece of eight rows
    // read eight different 16-byte columns of the 64-byte-swizzled codes, and store to eight
    // different ones of the 128-byte-swizzled operand.  Forward: 128 rows x 128 columns at a time,
    // two stages (pieces 0, 1 and 2, 3).  Backward: 64 rows x 128 columns, the two parts of a weight in two
    // stages.
    // The units alternate between two groups of four warps, so that one's waits and fences overlap the
    // other's arithmetic; each arrives for two on the barriers, which count eight warps.  (The stages need
    // no barriers of their own per group: MMAs complete in order, and a warp that has seen a stage within
    // the last ring released finds no barrier two phases behind.)
    const int group = warp >> 2, q = (tid >> 3) & 3, brow = (tid & 7) + 8 * (warp & 3);
    constexpr int PIECES = FWD ? 4 : 2;
    uint32_t pc = 0;   // partial sums so far
    int turn = 0;      // whose unit it is
    for (int i = pair; i < items && ok && !*abort_flag; i += npairs) {
      const LtTile t(p, i, BN, rank);
      // An adapter's rows go from global memory into registers (thread = feature and half of a chunk's
      // 32 ranks) while the stage before them still waits for its place.
      const int32_t* slots = p.slots + t.nt * (BN + 1);
      const int fr = tid & 127, jh = tid >> 7, f = t.f0 + fr;
      const int chunks = p.rank_chunks ? slots[0] * p.rank_chunks : 0;
      const float scale = FWD || BF16 ? 1.f : lt_power(lt_f16_exponent(p, t.f0));
      uint16_t next[16];
      auto fetch = [&](int q) {
        const int j0 = 32 * (q % p.rank_chunks) + 16 * jh;
        const uint16_t* w = (const uint16_t*)p.w + (long long)slots[1 + q / p.rank_chunks] * p.R * p.M + f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          next[j] = f < p.M && j0 + j < p.R ? w[(long long)(j0 + j) * p.M] : (uint16_t)0;
      };
      for (int k = t.u0; k < t.u1; ++k) {
        LtRing<NS> second = ring;
        second.next();
        const bool mine = turn == group;
        turn ^= 1;
        if (!mine) {
          ring.next();
          ring.next();
          cring.next();
          ++pc;
          continue;
        }
        if (!__all_sync(0xffffffffu,
                        lt_wait(&full_c[cring.i], cring.phase, budget) &&
                            lt_wait2(&empty[ring.i], ring.phase ^ 1u, &empty[second.i], second.phase ^ 1u,
                                     budget))) {
          raise_error(st, GPTQ_ERR_TIMEOUT, 76);
          *abort_flag = 1;
          ok = false;
          break;
        }
        const int slot = cring.i < NC ? cring.i : cring.i - NC;
        uint8_t* dst = smem + (FWD && q >= 2 ? second.i : ring.i) * Cfg::STAGE;
#pragma unroll
        for (int h0 = 0; h0 < PIECES; h0 += 2) {
          uint4 code[2];
          float2 dz[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = brow + 32 * (h0 + h);
            code[h] = *reinterpret_cast<const uint4*>(codes + slot * Cfg::C_BYTES + row * 64 +
                                                      ((q ^ ((row >> 1) & 3)) << 4));
            dz[h] = grids[slot * (Cfg::G_BYTES / 8) + row];
            // the partial that last used this slot of deltas has been taken out: its MMAs' successors,
            // two partials on, have released the stages that were just waited for
            if (FWD && q == 0) deltas[(pc % LT_DELTAS) * 128 + row] = dz[h].x;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t zz = zero_pair<BF16>((int)dz[h].y);
            const uint32_t words[4] = {code[h].x, code[h].y, code[h].z, code[h].w};
            WeightParts<BF16> parts;
            if (!FWD) parts = WeightParts<BF16>(BF16 ? dz[h].x : dz[h].x * scale);
            const int row = brow + 32 * (h0 + h);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t v[4];
              centered8<BF16>(words[w], zz, v);
              const int chunk = 4 * (q & 1) + w;
              const int at = (FWD ? 0 : (q >> 1) * 8192) + row * 128 + ((chunk ^ (row & 7)) << 4);
              if (!FWD) {
                uint32_t low[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) parts.split(v[e], low[e]);
                *reinterpret_cast<uint4*>(smem + second.i * Cfg::STAGE + at) =
                    make_uint4(low[0], low[1], low[2], low[3]);
              }
              *reinterpret_cast<uint4*>(dst + at) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          lt_release();
          lt_arrive_remote(lead_full_a + 8u * ring.i, 2);
          lt_arrive_remote(lead_full_a + 8u * second.i, 2);
          lt_arrive_remote(tc::smem_u32(&empty_c[slot]), 2);
        }
        ring.next();
        ring.next();
        cring.next();
        ++pc;
      }
      if (chunks) fetch(0);   // (inside the loop above its registers cost the units more than they gain)
      for (int q = 0; q < chunks && ok; ++q) {
        if (q % p.rank_chunks == 0) ++pc;
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = next[2 * j] | ((uint32_t)next[2 * j + 1] << 16);
        if (q + 1 < chunks) fetch(q + 1);
        for (int half = 0; half < 2; ++half) {   // against U's high and low parts
          if (!lt_wait_warp(&empty[ring.i], ring.phase ^ 1u, budget)) {
            raise_error(st, GPTQ_ERR_TIMEOUT, 77);
            *abort_flag = 1;
            ok = false;
            break;
          }
          uint8_t* dst = smem + ring.i * Cfg::STAGE + fr * 128;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = pair_f32<BF16>(v[2 * e]), b = pair_f32<BF16>(v[2 * e + 1]);
            *reinterpret_cast<float4*>(dst + (((4 * jh + e) ^ (fr & 7)) << 4)) =
                make_float4(a.x, a.y, b.x, b.y);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            lt_release();
            lt_arrive_remote(lead_full_a + 8u * ring.i, 1);
          }
          ring.next();
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    // ---------------------------------------------------------------- epilogue
    const int half = (warp - 8) >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + half * EBN;
    LtRing<ND> dr;
    uint32_t pc = 0;
    bool ok = true;
    pdl_wait();   // the slots
    pdl_release();
    for (int i = pair; i < items && ok && !*abort_flag; i += npairs) {
      const LtTile t(p, i, BN, rank);
      const int f = t.f0 + r, tok = t.t0 + half * EBN;
      // the tile's slots and this half's adapters are on their way while the base partials come in
      const int32_t* slots = p.slots + t.nt * (BN + 1);
      const int count = p.rank_chunks ? slots[0] : 0;
      int ids[EBN / 32];
#pragma unroll
      for (int c = 0; c < EBN / 32; ++c)
        ids[c] = count && tok + 32 * c + lane < p.T ? p.adapter[tok + 32 * c + lane] : -1;
      float acc[EBN];
#pragma unroll
      for (int e = 0; e < EBN; ++e) acc[e] = 0.f;
      const float unscale = FWD || BF16 ? 1.f : lt_power(-lt_f16_exponent(p, t.f0));
      // acc += factor · the next partial sum; in a forward base partial the factor is the row's Δ.
      // Eight columns are on their way from TMEM while eight are added.
      auto take = [&](bool scaled, const uint32_t* mask) {
        if (!ok) return;
        if (!lt_wait_warp(&d_full[dr.i], dr.phase, budget)) {
          raise_error(st, GPTQ_ERR_TIMEOUT, 78);
          *abort_flag = 1;
          ok = false;
          return;
        }
        tc::fence_after_sync();
        const float factor = scaled ? deltas[(pc % LT_DELTAS) * 128 + r]
                                    : (FWD || BF16 || mask ? 1.f : unscale);
        const uint64_t ff = pack_f32x2(factor, factor);
        uint32_t v[2][8];
        const uint32_t base = lane_base + dr.i * BN;
        lt_tmem_ld8(base, v[0]);
#pragma unroll
        for (int c = 0; c < EBN / 8; ++c) {
          lt_tmem_wait8(v[c & 1]);
          if (c + 1 < EBN / 8) lt_tmem_ld8(base + (c + 1) * 8, v[(c + 1) & 1]);
          if (mask) {   // an adapter's partial: its own tokens only
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if ((mask[c >> 2] >> (8 * (c & 3) + e)) & 1u)
                acc[c * 8 + e] += __uint_as_float(v[c & 1][e]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; e += 2)
              fma_f32x2(acc[c * 8 + e], acc[c * 8 + e + 1], ff, v[c & 1][e], v[c & 1][e + 1]);
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_remote_relaxed(lead_d_empty + 8u * dr.i);
        dr.next();
        ++pc;
      };
      if (FWD)
        for (int u = t.u0; u < t.u1 && ok; ++u) take(true, nullptr);
      else
        take(false, nullptr);
      for (int s = 0; s < count && ok; ++s) {
        const int a = slots[1 + s];
        uint32_t mask[EBN / 32];
#pragma unroll
        for (int c = 0; c < EBN / 32; ++c) mask[c] = __ballot_sync(0xffffffffu, ids[c] == a);
        take(false, mask);
      }
      if (!ok) continue;
      if (p.wide_out) {
        // 16-bit rows that can be written four features at a time: two exchanges turn four tokens of one
        // feature per lane into four features of one token (a 16-bit store per token and lane took 4 us
        // of a tile's 38)
        using T16 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
        const bool odd = lane & 1, upper = lane & 2;
        uint2* o = reinterpret_cast<uint2*>((T16*)p.out + (long long)(tok + (lane & 3)) * p.M + (f & ~3));
        const long long step = p.M;   // four tokens on, in units of four values
#pragma unroll
        for (int e = 0; e < EBN; e += 4) {
          const uint32_t p0 = pack16<BF16>(acc[e], acc[e + 1]), p1 = pack16<BF16>(acc[e + 2], acc[e + 3]);
          const uint32_t o0 = __shfl_xor_sync(0xffffffffu, p0, 1), o1 = __shfl_xor_sync(0xffffffffu, p1, 1);
          // features 2 k, 2 k + 1 of tokens e + odd and e + 2 + odd
          const uint32_t w0 = odd ? __byte_perm(o0, p0, 0x7632) : __byte_perm(p0, o0, 0x5410);
          const uint32_t w1 = odd ? __byte_perm(o1, p1, 0x7632) : __byte_perm(p1, o1, 0x5410);
          const uint32_t r2 = __shfl_xor_sync(0xffffffffu, upper ? w0 : w1, 2);
          if (tok + e + (lane & 3) < p.T && f < p.M) *o = upper ? make_uint2(r2, w1) : make_uint2(w0, r2);
          o += step;
        }
        continue;
      }
      if (f >= p.M) continue;
      if (p.part) {
        float* o = p.part + ((long long)t.split * p.T + tok) * p.M + f;
#pragma unroll
        for (int e = 0; e < EBN; ++e)
          if (tok + e < p.T) o[(long long)e * p.M] = acc[e];
      } else if (p.out_f32) {
        float* o = (float*)p.out + (long long)tok * p.M + f;
#pragma unroll
        for (int e = 0; e < EBN; ++e)
          if (tok + e < p.T) o[(long long)e * p.M] = acc[e];
      } else {
        using T16 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
        T16* o = (T16*)p.out + (long long)tok * p.M + f;
#pragma unroll
        for (int e = 0; e < EBN; ++e)
          if (tok + e < p.T) o[(long long)e * p.M] = from_f32<T16>(acc[e]);
      }
    }
  }
  // whoever follows may rely on the kernel before this one being done, too
  pdl_wait();
  __syncwarp();
  tc::fence_before_sync();
  tc::cluster_sync();   // neither CTA frees TMEM or exits while the other still uses its memory
  if (warp == 17) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, ND * BN);
  }
}

// ------------------------------------------------------------------------------------------
// U = s A X (or G = s B dY): 16 or 32 tokens per CTA, the features over its 16 warps (and, for few tokens, over
// a cluster's CTAs) on mma.sync straight from global memory (16 bytes a lane; tokens and adapter rows
// share the tensor instruction's free column order).  It is short and bound by the latency of its loads:
// the warps take two steps of 64 features at once.  Every adapter among the tokens takes a pass over
// the tile's features; a token keeps its own adapter's.  Writes U [T, R], its two tf32 parts
// [2, T_rows, Rp] (zero behind R), the lists of adapters per tile of BN tokens, and the layer's grid
// column-major.
// The tensor cores' own additions round towards zero, so that a long run of them drifts (6.7e-7 of U after
// 768 features): a warp takes LU_RUN features at a time, and the runs' sums meet in IEEE additions.
constexpr int LU_THREADS = 512, LU_WARPS = LU_THREADS / 32, LU_RUN = 512;

struct ShrinkParams {
  const void *x, *w;     // [T, F], [n, R, F]
  int T, F, n, R, Rp, T_rows;
  const int32_t* adapter;
  const float* scaling;
  float* U;              // or null
  float* parts;          // or null
  int32_t* slots;        // or null
  int BN, ttiles;
  int shrink_ctas, cluster;
  // the grid: grid[g, r] = (Δ[r, g], z[r, g]) for g < used, zero for r in [m, m_pad); group_max, where it
  // is given (all zero): the bits of the largest |Δ|; limit > 0: |Δ| must be below it
  const float* scales;
  const int32_t* zeros;
  float2* grid;
  uint32_t* group_max;
  int m, ng, used, m_pad, grid_ctas;
  float limit;
};

// The grid's share of CTA i of grid_ctas: a warp takes 32 rows x 8 groups at a time, a row per lane, whose
// 16 loads are independent (a lane's next groups lie in the same sectors) and whose stores are contiguous
// over the lanes.
__device__ __forceinline__ void turn_grid(const ShrinkParams& p, int i, DeviceStatus* st) {
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  const int across = (p.used + 7) / 8, tasks = across * (p.m_pad / 32);
  bool bad = false;
  for (int k = i * warps + (threadIdx.x >> 5); k < tasks; k += p.grid_ctas * warps) {
    const int g0 = k % across * 8, r = k / across * 32 + lane;
    const long long at = (long long)min(r, p.m - 1) * p.ng + g0;
    float d[8];
    int z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool in = r < p.m && g0 + e < p.used;
      d[e] = in ? p.scales[at + e] : 0.f;
      z[e] = in ? p.zeros[at + e] : 0;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (z[e] < 0 || z[e] > 15) {
        bad = true;
        z[e] = 0;
      }
      bad = bad || (p.limit > 0.f && !(fabsf(d[e]) < p.limit));
      if (g0 + e < p.used) p.grid[(long long)(g0 + e) * p.m_pad + r] = make_float2(d[e], (float)z[e]);
      if (p.group_max) {   // of non-negative floats, NaN above all, as their bits
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(d[e])));
        if (lane == 0 && g0 + e < p.used) atomicMax(&p.group_max[g0 + e], most);
      }
    }
  }
  if (bad) raise_error(st, GPTQ_ERR_ARG, i);
}

__device__ __forceinline__ void write_low_rank(const ShrinkParams& p, int t, int j, float u) {
  if (p.U && j < p.R) p.U[(long long)t * p.R + j] = u;
  if (p.parts) {
    float hi, lo;
    tc::tf32_parts(u, hi, lo);
    p.parts[(long long)t * p.Rp + j] = hi;
    p.parts[((long long)p.T_rows + t) * p.Rp + j] = lo;
  }
}

// The adapters that occur among the BN tokens of tile `nt`, in order of their first token.
__device__ __forceinline__ void list_slots(const ShrinkParams& p, int nt) {
  __shared__ int ids[256];
  __shared__ int counts[8];
  const int tid = threadIdx.x & 255, t = nt * p.BN + tid;   // a second half of the threads does the same
  int a = (tid < p.BN && t < p.T) ? p.adapter[t] : -1;
  if (a < 0 || a >= p.n) a = -1;
  ids[tid] = a;
  __syncthreads();
  bool first = a >= 0;
  for (int i = 0; i < tid && first; ++i) first = ids[i] != a;
  const uint32_t b = __ballot_sync(0xffffffffu, first);
  if ((tid & 31) == 0) counts[tid >> 5] = __popc(b);
  __syncthreads();
  int at = __popc(b & ((1u << (tid & 31)) - 1u)), total = 0;
  for (int i = 0; i < 8; ++i) {
    if (i < (tid >> 5)) at += counts[i];
    total += counts[i];
  }
  int32_t* out = p.slots + nt * (p.BN + 1);
  if (first) out[1 + at] = a;
  if (tid == 0) out[0] = total;
}

// NTL: 8-rank tiles of a pass; MT: 16-token tiles of a CTA (two halve the reads of A where there are tokens
// enough for every SM).  At rank 64, d = 4096, 64 ranks in one pass took 22 us for 1024 tokens, 32 in two
// 26; with two tiles the registers do not hold it (4096 tokens: 58 us, 45 in two passes).
template <bool BF16, int NTL, int MT>
__global__ void __launch_bounds__(LU_THREADS, 1) k_lora_shrink(ShrinkParams p, DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  constexpr int COLS = 8 * NTL, LU_TOKENS = 16 * MT;
  __shared__ float sums[LU_WARPS][16][16 + 1];   // 16 tokens x 16 ranks at a time
  __shared__ float total[LU_TOKENS * COLS];
  const int cl = p.cluster, rank = blockIdx.x % cl;
  if ((int)blockIdx.x >= p.shrink_ctas) {   // whole clusters: no cluster barrier
    const int i = blockIdx.x - p.shrink_ctas;
    if (i < p.ttiles) list_slots(p, i);
    else if (i < p.ttiles + p.grid_ctas) turn_grid(p, i - p.ttiles, st);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int t0 = (int)(blockIdx.x / cl) * LU_TOKENS;
  const int id = lane < LU_TOKENS && t0 + lane < p.T ? adapter_of(p.adapter, t0 + lane, p.n, st) : -1;
  // steps of 64 features, spread over the cluster's CTAs and their warps in contiguous runs
  const int steps = (p.F + 63) / 64, lanes = cl * LU_WARPS, per = (steps + lanes - 1) / lanes;
  const int s0 = min(steps, (rank * LU_WARPS + warp) * per), s1 = min(steps, s0 + per);
  // this lane's token rows g + 8 i (clamped: a token outside is not kept)
  const uint16_t* x[2 * MT];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i)
    x[i] = (const uint16_t*)p.x + (long long)min(t0 + g + 8 * i, p.T - 1) * p.F + 8 * t4;
  uint32_t todo = __ballot_sync(0xffffffffu, id >= 0);
  // zeros: tokens without an adapter, and the ranks behind the last pass
  const int passes = (p.R + COLS - 1) / COLS * COLS;
  if (rank == 0)
    for (int e = threadIdx.x; e < LU_TOKENS * p.Rp; e += LU_THREADS) {
      const int row = e / p.Rp, j = e % p.Rp;
      if (t0 + row < p.T && (j >= passes || !((todo >> row) & 1u))) write_low_rank(p, t0 + row, j, 0.f);
    }
  while (todo) {
    const int a = __shfl_sync(0xffffffffu, id, __ffs(todo) - 1);
    const uint32_t mine = __ballot_sync(0xffffffffu, id == a);
    todo &= ~mine;
    const float scale = p.scaling[a];
    for (int j0 = 0; j0 < p.R; j0 += COLS) {
      // this lane's rank rows j0 + g + 8 n (clamped: what lies behind R is not kept)
      const uint16_t* w[NTL];
#pragma unroll
      for (int nt = 0; nt < NTL; ++nt)
        w[nt] = (const uint16_t*)p.w + ((long long)a * p.R + min(j0 + 8 * nt + g, p.R - 1)) * p.F + 8 * t4;
      constexpr int H = MT == 1 && NTL < 8 ? 4 : 2;   // pieces of 32 features loaded at once
      for (int run = 0; run < per * 64; run += LU_RUN) {
        float acc[MT][NTL][4] = {};
        for (int k0 = s0 * 64 + run; k0 < min(s1 * 64, s0 * 64 + run + LU_RUN); k0 += 32 * H) {
          uint4 xv[H][2 * MT], wv[H][NTL];
          if (k0 + 32 * H <= min(s1 * 64, p.F)) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
#pragma unroll
              for (int i = 0; i < 2 * MT; ++i) xv[h][i] = *reinterpret_cast<const uint4*>(x[i] + k0 + 32 * h);
#pragma unroll
              for (int nt = 0; nt < NTL; ++nt)
                wv[h][nt] = *reinterpret_cast<const uint4*>(w[nt] + k0 + 32 * h);
            }
          } else {
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const int k = k0 + 32 * h;
              const bool in = k < s1 * 64 && k + 8 * t4 < p.F;
              const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int i = 0; i < 2 * MT; ++i) xv[h][i] = in ? *reinterpret_cast<const uint4*>(x[i] + k) : none;
#pragma unroll
              for (int nt = 0; nt < NTL; ++nt)
                wv[h][nt] = in ? *reinterpret_cast<const uint4*>(w[nt] + k) : none;
            }
          }
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int nt = 0; nt < NTL; ++nt) {
                const uint4 &u = xv[h][2 * mt], &v = xv[h][2 * mt + 1], &b = wv[h][nt];
                mma16816<BF16>(acc[mt][nt], u.x, v.x, u.y, v.y, b.x, b.y);
                mma16816<BF16>(acc[mt][nt], u.z, v.z, u.w, v.w, b.z, b.w);
              }
        }
        // join the warps (fixed order), 16 tokens and 16 ranks at a time
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int half = 0; half < NTL / 2; ++half) {
            __syncthreads();
#pragma unroll
            for (int n2 = 0; n2 < 2; ++n2)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                sums[warp][8 * (i >> 1) + g][8 * n2 + 2 * t4 + (i & 1)] = acc[mt][2 * half + n2][i];
            __syncthreads();
            if (threadIdx.x < 256) {
              const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
              float v = 0.f;
#pragma unroll
              for (int k = 0; k < LU_WARPS; ++k) v += sums[k][row][col];
              float& sum = total[(16 * mt + row) * COLS + 16 * half + col];
              sum = run ? sum + v : v;
            }
          }
      }
      if (cl > 1) tc::cluster_sync();
      else __syncthreads();
      // each CTA of the cluster finishes its share of the tokens
      const int rows = LU_TOKENS / cl;
      for (int e = threadIdx.x; e < rows * COLS; e += LU_THREADS) {
        const int row = rank * rows + e / COLS, col = e % COLS, j = j0 + col;
        if (!((mine >> row) & 1u) || j >= p.Rp) continue;
        float v = 0.f;
        for (int c = 0; c < cl; ++c) {
          float u = total[row * COLS + col];
          if (cl > 1)
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(u)
                         : "r"(tc::map_to_rank(&total[row * COLS + col], c))
                         : "memory");
          v += u;
        }
        write_low_rank(p, t0 + row, j, j < p.R ? v * scale : 0.f);
      }
      if (cl > 1) tc::cluster_sync();   // every CTA's sums are read before they are reused
      else __syncthreads();
    }
  }
}

// The two parts, the lists and the grid for a U that another kernel has formed.
__global__ void __launch_bounds__(256) k_lora_parts(ShrinkParams p, const float* __restrict__ U, DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  if ((int)blockIdx.x >= p.shrink_ctas) {
    const int i = blockIdx.x - p.shrink_ctas;
    if (i < p.ttiles) list_slots(p, i);
    else turn_grid(p, i - p.ttiles, st);
    return;
  }
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(e / p.Rp), j = (int)(e % p.Rp);
  if (t < p.T) write_low_rank(p, t, j, j < p.R ? U[(long long)t * p.R + j] : 0.f);
}

// Codes of BITS bits -> 4-bit codes in rows of `wpr4` words (a multiple of 4; zeros behind d): 32
// codes a thread.
template <int BITS>
__global__ void __launch_bounds__(256)
    k_lora_widen(const uint32_t* __restrict__ packed, int wpr, int wpr4, uint32_t* __restrict__ out) {
  pdl_wait();
  pdl_release();
  const int i = blockIdx.x * 256 + threadIdx.x;
  const long long row = blockIdx.y;
  if (4 * i >= wpr4) return;
  const uint32_t* src = packed + row * wpr;
  uint32_t w[BITS], v[4];
#pragma unroll
  for (int k = 0; k < BITS; ++k) w[k] = i * BITS + k < wpr ? src[i * BITS + k] : 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = eight_codes<BITS>(w, k);
  *reinterpret_cast<uint4*>(out + row * wpr4 + 4 * i) = make_uint4(v[0], v[1], v[2], v[3]);
}

// Rows of `cols` 16-bit values -> rows of `ld` (zeros behind), so that they start on 16 bytes.
__global__ void __launch_bounds__(256)
    k_lora_pad(const uint16_t* __restrict__ x, int rows, int cols, int ld, uint16_t* __restrict__ out) {
  pdl_wait();
  pdl_release();
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  if (e >= (long long)rows * ld) return;
  const long long r = e / ld;
  const int k = (int)(e % ld);
  out[e] = k < cols ? x[r * cols + k] : (uint16_t)0;
}

// ------------------------------------------------------------------------------------------
namespace {

PFN_cuTensorMapEncodeTiled_v12000 lt_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* ptr = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
  }();
  return fn;
}

// Boxes of box_rows x (swizzle width) bytes.
bool lt_map(CUtensorMap* map, CUtensorMapDataType dt, int esize, const void* base, long long cols,
            long long rows, int box_rows, int width = 128) {
  auto enc = lt_encode();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(cols * esize)};
  cuuint32_t box[2] = {(cuuint32_t)(width / esize), (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(map, dt, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
long long round_up(long long x, long long a) { return (x + a - 1) / a * a; }

// Tile width and splits of the contraction: the smallest waves x (stages of an item x the cycles of
// a stage + what an item costs besides).  A stage costs about the same whatever the tile's width (the
// MMAs read the weight operand at 32 bytes a cycle, 128 cycles per 16 columns: measured 126 at 128
// tokens, 128 at 256), so 128 tokens are for batches that fit in them; an item costs about 3000 cycles
// besides, a split's sums their traffic.
struct LtPlan { int BN, splits, per; };
LtPlan lt_plan(int M, int T, int units, int num_sms, size_t part_floats) {
  const int BN = T <= 128 ? 128 : 256;
  const long long tiles = ((M + 255) / 256) * (long long)((T + BN - 1) / BN), pairs = num_sms / 2;
  LtPlan best{BN, 1, units};
  double best_cost = 0;
  for (int s = 1; s <= 64 && s <= units; ++s) {
    const int per = (units + s - 1) / s, splits = (units + per - 1) / per;
    if (splits > 1 && (T > 1024 || (size_t)splits * T * M > part_floats)) break;
    const long long waves = (tiles * splits + pairs - 1) / pairs;
    const double cost = waves * ((double)per * 2 * 700 + 3000) +
                        (splits > 1 ? 6000 + splits * (double)T * M * 8 / 3000 : 0);
    if (s == 1 || cost < best_cost) {
      best = {BN, splits, per};
      best_cost = cost;
    }
  }
  return best;
}

template <bool FWD, int BN, bool BF16>
int launch_tc(Ctx* c, const CUtensorMap& mx, const CUtensorMap& mu,
              const CUtensorMap& mc, const LtParams& p) {
  GPTQ_CUDA_CHECK(c, cudaFuncSetAttribute(k_lora_tc<FWD, BN, BF16>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          LtCfg<FWD, BN>::SMEM));
  const int grid = 2 * std::min(c->num_sms / 2, p.mtiles * p.ttiles * p.splits);
  GPTQ_LAUNCH(c, (k_lora_tc<FWD, BN, BF16>), grid, LT_THREADS, LtCfg<FWD, BN>::SMEM, mx, mu, mc, p, c->status,
              kDefaultWaitCycles);   // as every kernel on CTA pairs
  return GPTQ_OK;
}

template <bool FWD>
int launch_tc_any(Ctx* c, int BN, bool bf, const CUtensorMap& mx, const CUtensorMap& mu,
                  const CUtensorMap& mc, const LtParams& p) {
  if (BN == 128) return bf ? launch_tc<FWD, 128, true>(c, mx, mu, mc, p) : launch_tc<FWD, 128, false>(c, mx, mu, mc, p);
  return bf ? launch_tc<FWD, 256, true>(c, mx, mu, mc, p) : launch_tc<FWD, 256, false>(c, mx, mu, mc, p);
}

constexpr size_t kMaxParts = 8;   // splits' partial sums that the asked-for workspace holds

}  // namespace

// Workspace in bytes: U, its parts, the lists, rows that have to be padded, widened codes, splits.
size_t lora_tc_bytes(const LoraLayer& l) {
  const size_t Rp = (size_t)round_up(l.R, 32), T = l.T, F = std::max(l.m, l.d);
  size_t b = 256 * 10;
  b += T * l.R * 4 + 2 * T * Rp * 4;
  b += (T / 64 + 1) * 65 * 4 + (T / 256 + 1) * 257 * 4;
  b += T * round_up(F, 8) * 2;                                  // a padded X or dY
  b += (size_t)l.m * round_up((l.d + 7) / 8, 4) * 4;            // widened codes
  b += (size_t)round_up(l.m, 256) * ((l.d + 127) / 128) * 8;    // the grid, column-major
  b += (size_t)((l.d + 127) / 128) * 4;                         // its largest |Δ|
  if (T <= 1024) b += kMaxParts * T * F * 4;
  return b;
}

// forward: x = X, out = Y, low (may be null) = U;  backward: x = dY, out = dX (or null: only G),
// low = where G goes (not null).
int lora_tc(Ctx* c, const LoraLayer& l, bool forward, const void* x, void* out, bool out_f32,
            float* low, size_t ws_offset) {
  const int K = forward ? l.d : l.m, M = forward ? l.m : l.d;
  const bool bf = l.dtype == GPTQ_BF16;
  const void* w1 = forward ? l.A : l.B;   // contracted with x
  const void* w2 = forward ? l.B : l.A;   // multiplies the low-rank values
  const int Rp = (int)round_up(l.R, 32);
  Carver cv(c);
  cv.off = ws_offset;
  // rows on 16-byte boundaries
  const int ld = (int)round_up(K, 8);
  const bool pad = K % 8 != 0 || !aligned16(x);
  uint16_t* xp = pad ? cv.take<uint16_t>((size_t)l.T * ld) : nullptr;
  const int wpr = (int)(((long long)l.d * l.bits + 31) / 32), wpr4 = (int)round_up((l.d + 7) / 8, 4);
  const bool widen = out && (l.bits != 4 || wpr != wpr4 || !aligned16(l.packed));
  uint32_t* codes = widen ? cv.take<uint32_t>((size_t)l.m * wpr4) : nullptr;
  const int m_pad = (int)round_up(l.m, 256);
  const int used = l.group == -1 ? 1 : (l.d + l.group - 1) / l.group;
  float2* grid2 = out ? cv.take<float2>((size_t)used * m_pad) : nullptr;
  uint32_t* group_max = out && !forward && !bf ? cv.take<uint32_t>(used) : nullptr;
  float* u_tmp = low ? low : cv.take<float>((size_t)l.T * l.R);
  float* parts = cv.take<float>((size_t)2 * l.T * Rp);
  int32_t* slots = cv.take<int32_t>((size_t)(l.T / 64 + 1) * 65 + (size_t)(l.T / 256 + 1) * 257);
  if (!cv.ok())
    GPTQ_SET_ERR(c, GPTQ_ERR_NOMEM, "lora: workspace %zu < %zu bytes", c->ws_bytes, cv.off);
  float* part = cv.take<float>(0);
  // of a workspace larger than asked for no more: the splits, and with them the order of the sums, then
  // follow from the call's sizes alone
  const size_t end = std::min(c->ws_bytes, lora_workspace_bytes(l));
  const size_t part_floats = end > cv.off ? (end - cv.off) / sizeof(float) : 0;

  if (group_max) GPTQ_CUDA_CHECK(c, cudaMemsetAsync(group_max, 0, (size_t)used * 4, c->stream));
  if (widen) {
    // rows in the grid's y: in pieces, should there be more than it holds
    for (int r0 = 0; r0 < l.m; r0 += 65535) {
      const dim3 grid((wpr4 / 4 + 255) / 256, std::min(65535, l.m - r0));
      const uint32_t* src = l.packed + (long long)r0 * wpr;
      uint32_t* dst = codes + (long long)r0 * wpr4;
      switch (l.bits) {
        case 1: GPTQ_LAUNCH(c, k_lora_widen<1>, grid, 256, 0, src, wpr, wpr4, dst); break;
        case 2: GPTQ_LAUNCH(c, k_lora_widen<2>, grid, 256, 0, src, wpr, wpr4, dst); break;
        case 3: GPTQ_LAUNCH(c, k_lora_widen<3>, grid, 256, 0, src, wpr, wpr4, dst); break;
        default: GPTQ_LAUNCH(c, k_lora_widen<4>, grid, 256, 0, src, wpr, wpr4, dst); break;
      }
    }
  }
  if (pad)
    GPTQ_LAUNCH(c, k_lora_pad, (unsigned)(((long long)l.T * ld + 255) / 256), 256, 0,
                (const uint16_t*)x, l.T, K, ld, xp);
  const void* xs = pad ? xp : x;

  const int units = forward ? (K + 127) / 128 : (K + 63) / 64;
  const LtPlan plan = lt_plan(M, l.T, units, c->num_sms, part_floats);
  const bool fused = plan.splits == 1;
  const int ttiles = (l.T + plan.BN - 1) / plan.BN;

  ShrinkParams s{};
  s.x = xs;
  s.w = w1;
  s.T = l.T; s.F = K; s.n = l.n; s.R = l.R; s.Rp = Rp; s.T_rows = l.T;
  s.adapter = l.adapter;
  s.scaling = l.scaling;
  s.parts = fused && out ? parts : nullptr;
  s.slots = slots;
  s.BN = plan.BN;
  s.ttiles = fused && out ? ttiles : 0;
  s.scales = l.scales;
  s.zeros = l.zeros;
  s.grid = grid2;
  s.group_max = group_max;
  s.m = l.m; s.ng = l.ng; s.used = used; s.m_pad = m_pad;
  s.grid_ctas = out ? std::min(64, ((used + 7) / 8 * (m_pad / 32) + 7) / 8) : 0;
  s.limit = !forward && !bf ? 17.f : 0.f;
  // the adapter's rows must be readable in 16-byte pieces; x's are (padded rows are longer than the
  // adapter's, so those go the other way)
  if (K % 8 == 0 && aligned16(w1)) {
    s.U = (low || !fused) ? u_tmp : nullptr;
    const int mt = (l.T + 15) / 16 > c->num_sms ? 2 : 1, tiles = (l.T + 16 * mt - 1) / (16 * mt);
    // few tokens: up to a CTA per SM, and two steps of 64 features at least per warp
    s.cluster = 1;
    while (s.cluster < 8 && 2 * tiles * s.cluster <= c->num_sms && (K + 63) / 64 > 2 * LU_WARPS * s.cluster)
      s.cluster *= 2;
    s.shrink_ctas = tiles * s.cluster;
    const int grid = s.shrink_ctas + (int)round_up(s.ttiles + s.grid_ctas, s.cluster);
    auto pick = [&](auto bf16) {
      constexpr bool B = decltype(bf16)::value;
      if (l.R <= 16) return mt == 1 ? k_lora_shrink<B, 2, 1> : k_lora_shrink<B, 2, 2>;
      if (mt == 2) return k_lora_shrink<B, 4, 2>;
      return l.R <= 32 ? k_lora_shrink<B, 4, 1> : k_lora_shrink<B, 8, 1>;
    };
    auto kernel = bf ? pick(std::true_type{}) : pick(std::false_type{});
    GPTQ_CUDA_CHECK(c, launch_pdl_cluster(c, s.cluster, kernel, dim3(grid), dim3(LU_THREADS), 0, s,
                                          c->status));
  } else {
    const int rc = lora_shrink_any(c, l, x, K, w1, u_tmp);
    if (rc) return rc;
    s.shrink_ctas = s.parts ? (int)(((long long)l.T * Rp + 255) / 256) : 0;
    const int ctas = s.shrink_ctas + s.ttiles + s.grid_ctas;
    if (ctas) GPTQ_LAUNCH(c, k_lora_parts, ctas, 256, 0, s, (const float*)u_tmp, c->status);
  }
  if (!out) return GPTQ_OK;

  CUtensorMap mx, mu, mc;
  if (!lt_map(&mx, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, xs,
              ld, l.T, plan.BN / 2) ||
      !lt_map(&mu, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, parts, Rp, 2LL * l.T, plan.BN / 2) ||
      !lt_map(&mc, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, widen ? codes : l.packed, wpr4, l.m,
              forward ? 128 : 64, 64))
    GPTQ_SET_ERR(c, GPTQ_ERR_CUDA, "lora: tensor map failed");
  LtParams p{};
  p.M = M;
  p.T = l.T;
  p.group_steps = l.group == -1 ? 0 : l.group / 128;
  p.grid = grid2;
  p.group_max = group_max;
  p.m_pad = m_pad;
  p.used = used;
  p.mtiles = (M + 255) / 256;
  p.ttiles = ttiles;
  p.splits = plan.splits;
  p.units = units;
  p.per = plan.per;
  p.T_rows = l.T;
  p.rank_chunks = fused ? Rp / 32 : 0;
  p.R = l.R; p.n = l.n;
  p.adapter = l.adapter;
  p.w = w2;
  p.slots = slots;
  p.out = out;
  p.out_f32 = out_f32;
  p.wide_out = fused && !out_f32 && M % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & 7) == 0;
  p.part = fused ? nullptr : part;
  p.idesc = tc::idesc_f32acc(bf ? 1u : 0u, !forward, false, 256, plan.BN);
  p.idesc_tf32 = tc::idesc_f32acc(2u, false, false, 256, plan.BN);
  const int rc = forward ? launch_tc_any<true>(c, plan.BN, bf, mx, mu, mc, p)
                         : launch_tc_any<false>(c, plan.BN, bf, mx, mu, mc, p);
  if (rc || fused) return rc;
  return lora_join(c, l, part, plan.splits, M, u_tmp, 1, nullptr, w2, out, out_f32, nullptr);
}

}  // namespace gptq
