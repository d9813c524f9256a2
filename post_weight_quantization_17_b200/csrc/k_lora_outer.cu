// The adapters' gradients: out[a, j, f] (+)= Σ_{t: a_t = a} u[t, j] x[t, f], with u = G, x = X for dA
// and u = U, x = dY for dB.
//
// Bound by reading x once (2 T F bytes; the products are 2 T R F).  D[rank, feature] tiles run on
// mma.sync tf32 (16 x 8 x 8): x is exact in tf32, u goes in as two tf32 parts (22 bits), so the sums
// are fp32 sums.  x is read straight into the tensor operand: a lane's 16 bytes are 8 features of
// one token, and tile i of the warp's eight takes feature 8 n + i as its column n, so no
// shared-memory pass is needed.  A CTA covers 128 features and 16 ranks (32 at once need twice the
// registers: 169 us with one CTA per SM, 215 with two and spills, where two passes took 134: 4096 tokens,
// 4 adapters of rank 32 on 4096 x 11008, now 119); its four token warps, and the CTAs of a cluster, take
// the 8-token groups in turn (adapters' runs spread evenly) and are joined in a fixed order in
// (distributed) shared memory.  A cluster takes several adapters one after
// the other (one in turn would leave most CTAs of a large adapter table with nothing to do); those
// without a token are cleared.  Groups without a token of the adapter are skipped; in mixed groups the
// others' rows are replaced by zeros, not multiplied.
#include <algorithm>

#include "lora_util.cuh"
#include "tc_util.cuh"

namespace gptq {

constexpr int LO_THREADS = 256;
constexpr int LO_FEATS = 128, LO_PAD = 68;
constexpr int LO_TOKENS = 8192;   // of a launch: their adapters (16 bits each) are kept in shared memory
constexpr int LO_RANKS = 16;
constexpr int LO_RUN = 4;       // pairs of token groups (16 tokens) that the tensor cores add up by themselves
// the warps' sums [8][16][64 + 4] and the CTA's [16][128]; the adapters' bits and the tokens' adapters
// follow
constexpr int LO_SMEM = (8 * LO_RANKS * LO_PAD + LO_RANKS * LO_FEATS) * 4;
constexpr int lo_smem(int n, int T) { return LO_SMEM + (n + 127) / 128 * 16 + (T + 7) / 8 * 16; }

struct OuterProblem {
  const float* u;          // [T, R]
  const void* x;           // [T, F]
  float* out;              // [n, R, F]
  int F, wide, u_wide;     // x may be read in 16-byte pieces, u in 8-byte ones
};
struct OuterParams {
  OuterProblem two[2];
  int first_ctas;          // CTAs of two[0]
  int T, R, n;
  const int32_t* adapter;
  int accumulate, cluster;
};

__device__ __forceinline__ void mma_tf32_1688(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two groups of 8 tokens of a warp: a lane's 8 features of four of the tokens, and their ranks.
struct OuterGroup {
  uint32_t members;
  uint4 x[2][2];
  float u[2][2][2];
};

template <bool BF16>
__global__ void __launch_bounds__(LO_THREADS, 2) k_lora_outer(const __grid_constant__ OuterParams p, DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  extern __shared__ __align__(16) float lo_smem_[];
  float* sums = lo_smem_;                                   // [8 warps][ranks][64 + 4]
  float* total = lo_smem_ + 8 * LO_RANKS * LO_PAD;          // [ranks][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int wf = warp & 1, wt = warp >> 1;
  const int cl = p.cluster, rank = blockIdx.x % cl;
  const bool second = (int)blockIdx.x >= p.first_ctas;
  const float* pu = second ? p.two[1].u : p.two[0].u;
  const uint16_t* px = (const uint16_t*)(second ? p.two[1].x : p.two[0].x);
  float* const out = second ? p.two[1].out : p.two[0].out;
  const int F = second ? p.two[1].F : p.two[0].F, wide = second ? p.two[1].wide : p.two[0].wide;
  const int u_wide = second ? p.two[1].u_wide : p.two[0].u_wide;
  const int fb = ((int)blockIdx.x - (second ? p.first_ctas : 0)) / cl * LO_FEATS;
  const int f0 = fb + wf * 64, j0 = blockIdx.y * LO_RANKS, f = f0 + 8 * g;
  // the tokens' adapters (0xFFFF: none), and which adapters have tokens
  uint32_t* present = reinterpret_cast<uint32_t*>(total + LO_RANKS * LO_FEATS);
  uint16_t* id_of = reinterpret_cast<uint16_t*>(present + (p.n + 127) / 128 * 4);
  for (int i = threadIdx.x; i < (p.n + 31) / 32; i += LO_THREADS) present[i] = 0;
  const int groups = (p.T + 7) / 8;
  if ((int)threadIdx.x < 8 * groups - p.T) id_of[p.T + threadIdx.x] = 0xFFFF;   // behind the last token
  __syncthreads();
  for (int t = threadIdx.x; t < p.T; t += 8 * LO_THREADS) {
    int id[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) id[i] = t + i * LO_THREADS < p.T ? p.adapter[t + i * LO_THREADS] : -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool one = id[i] >= 0 && id[i] < p.n;
      if (id[i] < -1 || id[i] >= p.n) raise_error(st, GPTQ_ERR_ARG, t + i * LO_THREADS);
      if (t + i * LO_THREADS < p.T) id_of[t + i * LO_THREADS] = one ? (uint16_t)id[i] : (uint16_t)0xFFFF;
      if (one && !((present[id[i] >> 5] >> (id[i] & 31)) & 1u))
        atomicOr(&present[id[i] >> 5], 1u << (id[i] & 31));
    }
  }
  __syncthreads();
  for (int a = blockIdx.z; a < p.n; a += gridDim.z) {
  if (!((present[a >> 5] >> (a & 31)) & 1u)) {   // its gradient is zero
    if (!p.accumulate)
      for (int e = rank * LO_THREADS + threadIdx.x; e < LO_RANKS * LO_FEATS; e += cl * LO_THREADS) {
        const int j = j0 + e / LO_FEATS, ff = fb + e % LO_FEATS;
        if (j < p.R && ff < F) out[((long long)a * p.R + j) * F + ff] = 0.f;
      }
    continue;
  }
  float acc[8][4] = {};
  // this warp's groups: rank * 4 + wt, and every `stride`-th from there, taken in pairs.  `word`: which of
  // 32 pairs, a lane looking at one pair's 16 adapters, have a token of this adapter and are still to come
  // (looking at one pair after the other cost a fourth of the instructions with four adapters).
  const int stride = 4 * cl, start = rank * 4 + wt;
  const uint32_t aa = (uint32_t)a * 0x10001u;
  int next = start;
  uint32_t word = 0;
  // the next pair with a token of the adapter: its members, and its first group i
  auto find = [&](int& i) -> uint32_t {
    while (!word) {
      if (next >= groups) return 0u;
      const int mine = next + lane * 2 * stride;
      uint32_t hit = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (mine + k * stride < groups) {
          const uint4 v = *reinterpret_cast<const uint4*>(id_of + (mine + k * stride) * 8);
          hit |= __vcmpeq2(v.x, aa) | __vcmpeq2(v.y, aa) | __vcmpeq2(v.z, aa) | __vcmpeq2(v.w, aa);
        }
      word = __ballot_sync(0xffffffffu, hit != 0);
      next += 64 * stride;
    }
    i = next + (__ffs(word) - 33) * 2 * stride;
    word &= word - 1;
    const int of = i + ((lane >> 3) & 1) * stride;
    return __ballot_sync(0xffffffffu, lane < 16 && of < groups && id_of[of * 8 + (lane & 7)] == a);
  };
  // this lane's first token, features and ranks, for pairs whose 16 tokens are all the adapter's (features
  // and ranks behind the end are read from before it and not kept); with the general reads alone 15 us
  // more of 114
  const bool plain = wide && u_wide;
  const uint16_t* const x_lane = px + (long long)t4 * F + (plain ? min(f, F - 8) : 0);
  const float* const u_lane = pu + (long long)t4 * p.R + (plain ? min(j0 + 2 * g, p.R - 2) : 0);
  auto fetch = [&](OuterGroup& o, int i, uint32_t members) {
    o.members = members;
    if (!members) return;
    if (plain && members == 0xFFFFu) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const long long t = (i + k * stride) * 8 + 4 * h;
          o.x[k][h] = *reinterpret_cast<const uint4*>(x_lane + t * F);
          const float2 v = *reinterpret_cast<const float2*>(u_lane + t * p.R);
          o.u[k][h][0] = v.x;
          o.u[k][h][1] = v.y;
        }
      return;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r8 = t4 + 4 * h;
        const long long t = (long long)(i + k * stride) * 8 + r8;
        const bool in = (members >> (8 * k + r8)) & 1u;
        o.x[k][h] = make_uint4(0, 0, 0, 0);
        if (in && wide) {
          if (f < F) o.x[k][h] = *reinterpret_cast<const uint4*>(px + t * F + f);
        } else if (in) {
          const uint16_t* src = px + t * F + f;
          uint32_t w[4] = {};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (f + e < F) w[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
          o.x[k][h] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // ranks 2 g, 2 g + 1: the operand's row order is free, so a lane's ranks are adjacent
        const int j = j0 + 2 * g;
        o.u[k][h][0] = o.u[k][h][1] = 0.f;
        if (in && u_wide && j < p.R) {
          const float2 v = *reinterpret_cast<const float2*>(pu + t * p.R + j);
          o.u[k][h][0] = v.x;
          o.u[k][h][1] = v.y;
        } else if (in) {
          if (j < p.R) o.u[k][h][0] = pu[t * p.R + j];
          if (j + 1 < p.R) o.u[k][h][1] = pu[t * p.R + j + 1];
        }
      }
    }
  };
  auto multiply = [&](const OuterGroup& o) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!((o.members >> (8 * k)) & 0xffu)) continue;
      const uint32_t x0[4] = {o.x[k][0].x, o.x[k][0].y, o.x[k][0].z, o.x[k][0].w};
      const uint32_t x1[4] = {o.x[k][1].x, o.x[k][1].y, o.x[k][1].z, o.x[k][1].w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // rows g and g + 8 (ranks 2 g, 2 g + 1) of tokens t4 and t4 + 4
        float h, l;
        tc::tf32_parts(o.u[k][e >> 1][e & 1], h, l);
        hi[e] = __float_as_uint(h);
        lo[e] = __float_as_uint(l);
      }
      // all the high parts, then all the low ones: eight products lie between two of one sum
      float2 b0[4], b1[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        b0[e] = pair_f32<BF16>(x0[e]);
        b1[e] = pair_f32<BF16>(x1[e]);
        mma_tf32_1688(acc[2 * e], hi, __float_as_uint(b0[e].x), __float_as_uint(b1[e].x));
        mma_tf32_1688(acc[2 * e + 1], hi, __float_as_uint(b0[e].y), __float_as_uint(b1[e].y));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        mma_tf32_1688(acc[2 * e], lo, __float_as_uint(b0[e].x), __float_as_uint(b1[e].x));
        mma_tf32_1688(acc[2 * e + 1], lo, __float_as_uint(b0[e].y), __float_as_uint(b1[e].y));
      }
    }
  };
  // The tensor cores' own additions round towards zero, so that a long run of them drifts (2.4e-6 of dA
  // after 36 pairs); LO_RUN pairs on, the sums go to the warp's place in shared memory, by IEEE additions
  // (every 8 pairs 8.9e-7 and 114 us, every 4 6.7e-7 and 116 to 119).
  // Tile i's column n is feature 8 n + i: a lane holds features 16 t4 + (0..7) and + 8.
  float* mine = sums + warp * LO_RANKS * LO_PAD;
  bool fresh = true;
  auto flush = [&] {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float4* dst = reinterpret_cast<float4*>(mine + (2 * g + (c >> 1)) * LO_PAD + 16 * t4 + 8 * (c & 1));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 v = fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : dst[h];
        dst[h] = make_float4(v.x + acc[4 * h][c], v.y + acc[4 * h + 1][c], v.z + acc[4 * h + 2][c],
                             v.w + acc[4 * h + 3][c]);
      }
    }
    fresh = false;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;
  };
  {
    int i = 0, run = 0;
    OuterGroup one, other;
    uint32_t m = find(i);
    fetch(one, i, m);
    while (one.members) {
      m = find(i);
      fetch(other, i, m);
      multiply(one);
      if (!m) break;
      m = find(i);
      fetch(one, i, m);
      multiply(other);
      if ((run += 2) == LO_RUN) {
        flush();
        run = 0;
      }
    }
  }
  flush();
  __syncthreads();
  for (int e = threadIdx.x; e < LO_RANKS * LO_FEATS; e += LO_THREADS) {
    const int j = e / LO_FEATS, ff = e % LO_FEATS;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      s += sums[((2 * w + (ff >> 6)) * LO_RANKS + j) * LO_PAD + (ff & 63)];
    total[e] = s;
  }
  if (cl > 1) tc::cluster_sync();
  else __syncthreads();
  // each CTA of the cluster finishes its share of the tile
  const int share = LO_RANKS * LO_FEATS / cl;
  for (int e = rank * share + threadIdx.x; e < (rank + 1) * share; e += LO_THREADS) {
    const int j = j0 + e / LO_FEATS, ff = fb + e % LO_FEATS;
    float s = 0.f;
    for (int c = 0; c < cl; ++c) {
      float v;
      if (cl > 1)
        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                     : "=f"(v)
                     : "r"(tc::map_to_rank(&total[e], c))
                     : "memory");
      else
        v = total[e];
      s += v;
    }
    if (j < p.R && ff < F) {
      float* o = out + ((long long)a * p.R + j) * F + ff;
      *o = p.accumulate ? *o + s : s;
    }
  }
  if (cl > 1) tc::cluster_sync();   // no CTA leaves, or forms new sums, while its sums are being read
  else __syncthreads();
  }
}

// dA from (G, X) and dB from (U, dY) in one launch (each alone is too short to fill the GPU); either may
// be left out (null).  Batches of more than LO_TOKENS tokens take several, which add up.
int lora_outers(Ctx* c, const LoraLayer& l, const float* G, const void* X, float* dA, const float* U,
                const void* dY, float* dB, int accumulate) {
  const int ranks = (l.R + LO_RANKS - 1) / LO_RANKS;
  const int tiles = (dA ? (l.d + LO_FEATS - 1) / LO_FEATS : 0) + (dB ? (l.m + LO_FEATS - 1) / LO_FEATS : 0);
  auto kernel = l.dtype == GPTQ_BF16 ? k_lora_outer<true> : k_lora_outer<false>;
  for (int t0 = 0; t0 < l.T; t0 += LO_TOKENS) {
    OuterParams p{};
    p.T = std::min(LO_TOKENS, l.T - t0);
    p.R = l.R; p.n = l.n;
    p.adapter = l.adapter + t0;
    p.accumulate = accumulate || t0 > 0;
    // tokens over a cluster until there is a CTA for every SM: joining a cluster costs each adapter some
    // microseconds (clusters of 8 took 272 us where clusters of 2 took 217, at the size above)
    p.cluster = 1;
    while (p.cluster < 8 && p.T > 32 * p.cluster && tiles * ranks * p.cluster < c->num_sms) p.cluster *= 2;
    auto problem = [&](const float* u, const void* x, float* out, int F) {
      const float* ut = u ? u + (size_t)t0 * l.R : nullptr;
      const uint16_t* xt = x ? (const uint16_t*)x + (size_t)t0 * F : nullptr;
      return OuterProblem{ut, xt, out, F, F % 8 == 0 && (reinterpret_cast<uintptr_t>(xt) & 15) == 0,
                          l.R % 2 == 0 && (reinterpret_cast<uintptr_t>(ut) & 7) == 0};
    };
    const int ca = dA ? (l.d + LO_FEATS - 1) / LO_FEATS * p.cluster : 0;
    const int cb = dB ? (l.m + LO_FEATS - 1) / LO_FEATS * p.cluster : 0;
    p.two[0] = problem(G, X, dA, l.d);
    p.two[1] = problem(U, dY, dB, l.m);
    p.first_ctas = ca;
    const dim3 grid(ca + cb, ranks, std::max(1, std::min(l.n, 8 * c->num_sms / ((ca + cb) * ranks))));
    // the kernel's limit, not this call's size: other threads' calls set the same attribute
    GPTQ_CUDA_CHECK(c, cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            lo_smem(kLoraMaxAdapters, LO_TOKENS)));
    GPTQ_CUDA_CHECK(c, launch_pdl_cluster(c, p.cluster, kernel, grid, dim3(LO_THREADS), lo_smem(l.n, p.T), p,
                                          c->status));
  }
  return GPTQ_OK;
}

}  // namespace gptq
