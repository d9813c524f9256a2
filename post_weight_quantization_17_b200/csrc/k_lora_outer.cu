// The adapters' gradients: out[a, j, f] (+)= Σ_{t: a_t = a} u[t, j] x[t, f], with u = G, x = X for dA
// and u = U, x = dY for dB.
//
// Bound by reading x once (2 T F bytes; the products are 2 T R F).  D[rank, feature] tiles run on
// mma.sync tf32 (16 x 8 x 8): x is exact in tf32, u goes in as two tf32 parts (22 bits), so the sums
// are fp32 sums.  x is read straight into the tensor operand: a lane's 16 bytes are 8 features of
// one token, and tile i of the warp's eight takes feature 8 n + i as its column n, so no
// shared-memory pass is needed.  A CTA covers 128 features and 32 ranks; its four token warps, and
// the CTAs of a cluster, take the 8-token groups in turn (adapters' runs spread evenly) and are
// joined in a fixed order in (distributed) shared memory.  A cluster takes several adapters one after
// the other (one in turn would leave most CTAs of a large adapter table with nothing to do); those
// without a token are cleared.  Groups without a token of the adapter are skipped; in mixed groups the
// others' rows are replaced by zeros, not multiplied.
#include <algorithm>

#include "lora_util.cuh"
#include "tc_util.cuh"

namespace gptq {

constexpr int LO_THREADS = 256;
constexpr int LO_FEATS = 128, LO_RANKS = 32, LO_PAD = 68;
constexpr int LO_SMEM = (8 * LO_RANKS * LO_PAD + LO_RANKS * LO_FEATS) * 4;

struct OuterParams {
  const float* u;          // [T, R]
  const void* x;           // [T, F]
  int T, F, R, wide;       // wide: x may be read in 16-byte pieces
  const int32_t* adapter;
  int accumulate, cluster, n;
  float* out;              // [n, R, F]
};

__device__ __forceinline__ void mma_tf32_1688(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF16>
__global__ void __launch_bounds__(LO_THREADS, 2) k_lora_outer(OuterParams p) {
  pdl_wait();
  pdl_release();
  extern __shared__ __align__(16) float lo_smem[];
  float* sums = lo_smem;                                   // [8 warps][32 ranks][64 + 4]
  float* total = lo_smem + 8 * LO_RANKS * LO_PAD;          // [32 ranks][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int wf = warp & 1, wt = warp >> 1;
  const int cl = p.cluster, rank = blockIdx.x % cl;
  const int f0 = (int)(blockIdx.x / cl) * LO_FEATS + wf * 64, j0 = blockIdx.y * LO_RANKS;
  const int f = f0 + 8 * g, fb = (int)(blockIdx.x / cl) * LO_FEATS;
  // which adapters have tokens
  uint32_t* present = reinterpret_cast<uint32_t*>(total + LO_RANKS * LO_FEATS);
  for (int i = threadIdx.x; i < (p.n + 31) / 32; i += LO_THREADS) present[i] = 0;
  __syncthreads();
#pragma unroll 4
  for (int t = threadIdx.x; t < p.T; t += LO_THREADS) {
    const int a = p.adapter[t];
    if (a >= 0 && a < p.n && !((present[a >> 5] >> (a & 31)) & 1u))
      atomicOr(&present[a >> 5], 1u << (a & 31));
  }
  __syncthreads();
  for (int a = blockIdx.z; a < p.n; a += gridDim.z) {
  if (!((present[a >> 5] >> (a & 31)) & 1u)) {   // its gradient is zero
    if (!p.accumulate)
      for (int e = rank * LO_THREADS + threadIdx.x; e < LO_RANKS * LO_FEATS; e += cl * LO_THREADS) {
        const int j = j0 + e / LO_FEATS, ff = fb + e % LO_FEATS;
        if (j < p.R && ff < p.F) p.out[((long long)a * p.R + j) * p.F + ff] = 0.f;
      }
    continue;
  }
  float acc[2][8][4] = {};
  const int groups = (p.T + 7) / 8, stride = 4 * cl;
  for (int i0 = rank * 4 + wt; i0 < groups; i0 += 4 * stride) {
    // the adapters of four 8-token groups
    const int mt = (i0 + (lane >> 3) * stride) * 8 + (lane & 7);
    const uint32_t members = __ballot_sync(0xffffffffu, mt < p.T && p.adapter[mt] == a);
    if (!members) continue;
    uint4 x[4][2];
    float u[4][2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m8 = (members >> (8 * i)) & 0xffu;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = t4 + 4 * h;
        const long long t = (long long)(i0 + i * stride) * 8 + k;
        const bool in = (m8 >> k) & 1u;
        x[i][h] = make_uint4(0, 0, 0, 0);
        if (in && p.wide) {
          if (f < p.F)
            x[i][h] = *reinterpret_cast<const uint4*>((const uint16_t*)p.x + t * p.F + f);
        } else if (in) {
          const uint16_t* src = (const uint16_t*)p.x + t * p.F + f;
          uint32_t w[4] = {};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (f + e < p.F) w[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
          x[i][h] = make_uint4(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {   // ranks g, g + 8, g + 16, g + 24
          const int j = j0 + g + 8 * r;
          u[i][h][r] = (in && j < p.R) ? p.u[t * p.R + j] : 0.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!((members >> (8 * i)) & 0xffu)) continue;
      const uint32_t x0[4] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w};
      const uint32_t x1[4] = {x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (j0 + 16 * m >= p.R) break;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // (rank g, token t4), (g + 8, t4), (g, t4 + 4), (g + 8, t4 + 4)
          const float v = u[i][e >> 1][2 * m + (e & 1)];
          const bool finite = fabsf(v) <= 3.0e38f;   // the split is for finite values
          const float h = finite ? tc::tf32_rna(v) : v;
          hi[e] = __float_as_uint(h);
          lo[e] = finite ? __float_as_uint(tc::tf32_rna(v - h)) : 0u;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 b0 = pair_f32<BF16>(x0[e]), b1 = pair_f32<BF16>(x1[e]);
          mma_tf32_1688(acc[m][2 * e], hi, __float_as_uint(b0.x), __float_as_uint(b1.x));
          mma_tf32_1688(acc[m][2 * e + 1], hi, __float_as_uint(b0.y), __float_as_uint(b1.y));
          mma_tf32_1688(acc[m][2 * e], lo, __float_as_uint(b0.x), __float_as_uint(b1.x));
          mma_tf32_1688(acc[m][2 * e + 1], lo, __float_as_uint(b0.y), __float_as_uint(b1.y));
        }
      }
    }
  }
  // tile i's column n is feature 8 n + i: a lane holds features 16 t4 + (0..7) and + 8
  float* mine = sums + warp * LO_RANKS * LO_PAD;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float4* dst = reinterpret_cast<float4*>(mine + (16 * m + 8 * (c >> 1) + g) * LO_PAD + 16 * t4 +
                                              8 * (c & 1));
      dst[0] = make_float4(acc[m][0][c], acc[m][1][c], acc[m][2][c], acc[m][3][c]);
      dst[1] = make_float4(acc[m][4][c], acc[m][5][c], acc[m][6][c], acc[m][7][c]);
    }
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
    if (j < p.R && ff < p.F) {
      float* o = p.out + ((long long)a * p.R + j) * p.F + ff;
      *o = p.accumulate ? *o + s : s;
    }
  }
  if (cl > 1) tc::cluster_sync();   // no CTA leaves, or forms new sums, while its sums are being read
  else __syncthreads();
  }
}

int lora_outer(Ctx* c, const LoraLayer& l, const float* u, const void* x, int F, int accumulate,
               float* out) {
  OuterParams p{};
  p.u = u;
  p.x = x;
  p.T = l.T; p.F = F; p.R = l.R;
  p.wide = F % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  p.adapter = l.adapter;
  p.accumulate = accumulate;
  p.out = out;
  p.n = l.n;
  p.cluster = 1;
  while (p.cluster < 8 && l.T > 32 * p.cluster) p.cluster *= 2;
  const int gx = (F + LO_FEATS - 1) / LO_FEATS * p.cluster, gy = (l.R + LO_RANKS - 1) / LO_RANKS;
  // two CTAs fit on an SM
  const dim3 grid(gx, gy, std::max(1, std::min(l.n, 2 * c->num_sms / (gx * gy))));
  const int smem = LO_SMEM + (l.n + 31) / 32 * 4;
  auto kernel = l.dtype == GPTQ_BF16 ? k_lora_outer<true> : k_lora_outer<false>;
  GPTQ_CUDA_CHECK(c, cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  GPTQ_CUDA_CHECK(c, launch_pdl_cluster(c, p.cluster, kernel, grid, dim3(LO_THREADS), smem, p));
  return GPTQ_OK;
}

}  // namespace gptq
