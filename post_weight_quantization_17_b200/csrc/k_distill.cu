// Distillation from a teacher's stored top logits.  Per token, with y = z / τ, q = softmax(y) over
// the student's V logits and p_k = exp(v_k / τ - L) over the K stored teacher logits (L: the
// teacher's own log-sum-exp at τ where it was stored, else that of the K kept values):
//   loss = w τ² Σ_k p_k (log p_k - (y_{i_k} - lse)),          lse = log Σ_j exp y_j
//   dz_i = g w τ (M q_i - Σ_{k: i_k = i} p_k),                M = Σ_k p_k
// (g: the token's upstream gradient).
//
// Bound by HBM: the logits are read once and the gradients written once.  A row is split over a
// cluster of CTAs so that each CTA's piece (about 64 KB, three CTAs to an SM) stays in shared
// memory: one bulk copy brings it while the teacher's list is read, the running maximum and sum are
// formed in one pass, the cluster joins them through distributed shared memory, and the gradient is
// formed from the same shared memory.  Several CTAs per SM let one load while another computes (a copy
// in two or four parts, each waited for by itself, was slower: the list, the barriers and the joins are
// what a row costs beyond its elements).  4096 x 128000 bf16 with the gradient: 416 us, 77 % of the copy
// rate; 32 KB parts 460.
// Rows too long for 8 CTAs' shared memory take k_distill_long, which reads them again instead.
#include <algorithm>

#include "kernels.h"
#include "tc_util.cuh"

namespace gptq {

constexpr int DS_THREADS = 256;
constexpr int DS_WARPS = DS_THREADS / 32;
constexpr int DS_PART = 64 * 1024;               // a CTA's part of a row, where rows allow it
constexpr int DS_PART_MAX = 160 * 1024;
constexpr int DS_ENTRY = 12;                     // bytes of shared memory per entry of the list
constexpr float DS_LOG2E = 1.4426950408889634f, DS_LN2 = 0.6931471805599453f;

template <class T> __device__ __forceinline__ T ds_round(float v);
template <> __device__ __forceinline__ float ds_round<float>(float v) { return v; }
template <> __device__ __forceinline__ __half ds_round<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 ds_round<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Sum / maximum over the CTA (every thread gets the result); `red`: 33 floats of shared memory.
__device__ __forceinline__ float ds_block(float v, bool is_max, float* red) {
  const float none = is_max ? -INFINITY : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = is_max ? fmaxf(v, u) : v + u;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < blockDim.x / 32 ? red[threadIdx.x] : none;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v, o);
      v = is_max ? fmaxf(v, u) : v + u;
    }
    if (threadIdx.x == 0) red[32] = v;
  }
  __syncthreads();
  return red[32];
}

// 2^x, within 2 units in the last place and 0 below 2^-126.
__device__ __forceinline__ float ds_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <class T> struct DsVec { static constexpr int N = 16 / sizeof(T); };

template <class T>
__device__ __forceinline__ void ds_unpack(const uint4& v, float (&x)[DsVec<T>::N]);
template <> __device__ __forceinline__ void ds_unpack<float>(const uint4& v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x);
  x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z);
  x[3] = __uint_as_float(v.w);
}
template <> __device__ __forceinline__ void ds_unpack<__half>(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <> __device__ __forceinline__ void ds_unpack<__nv_bfloat16>(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <class T>
__device__ __forceinline__ uint4 ds_pack(const float (&x)[DsVec<T>::N]);
template <> __device__ __forceinline__ uint4 ds_pack<float>(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
}
template <> __device__ __forceinline__ uint4 ds_pack<__half>(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ uint4 ds_pack<__nv_bfloat16>(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two fp32 operations per instruction.
__device__ __forceinline__ uint64_t ds_pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void ds_split(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t ds_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t ds_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t ds_mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// x[e] <- 2^(k x[e] + b) for a vector.
template <int N>
__device__ __forceinline__ void ds_exp2_all(float (&x)[N], uint64_t k, uint64_t b) {
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    ds_split(ds_fma2(ds_pair(x[e], x[e + 1]), k, b), x[e], x[e + 1]);
    x[e] = ds_exp2(x[e]);
    x[e + 1] = ds_exp2(x[e + 1]);
  }
}
// The largest of a vector's values (NaN is passed over).
template <class T> __device__ __forceinline__ float ds_max(const uint4& v);
template <> __device__ __forceinline__ float ds_max<float>(const uint4& v) {
  return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
               fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}
template <> __device__ __forceinline__ float ds_max<__half>(const uint4& v) {
  const __half2* h = reinterpret_cast<const __half2*>(&v);
  const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  return fmaxf(__low2float(m), __high2float(m));
}
template <> __device__ __forceinline__ float ds_max<__nv_bfloat16>(const uint4& v) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
  const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  return fmaxf(__low2float(m), __high2float(m));
}

// A running maximum and the sum of 2^(k x - k max): joins (m2, s2) into (m, s).
__device__ __forceinline__ void ds_join(float& m, float& s, float m2, float s2, float k) {
  const float mm = fmaxf(m, m2);
  // an empty side (maximum -inf) has the sum 0; -inf - (-inf) must not become a factor
  const float a = m == mm ? 1.f : ds_exp2((m - mm) * k), b = m2 == mm ? 1.f : ds_exp2((m2 - mm) * k);
  s = s * a + s2 * b;
  m = mm;
}

// The same over the eight warps' (m, s) in shared memory, or a cluster's: n, a power of two up to 8, of
// them; every lane of the calling warp gets the result.
__device__ __forceinline__ void ds_join_all(const float2* ms, int n, float& m, float& s, float k) {
  const float2 v = ms[threadIdx.x & (n - 1)];
  m = v.x;
  s = v.y;
  for (int o = n >> 1; o; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    ds_join(m, s, m2, s2, k);
  }
}

// The teacher's list of one row in shared memory, and what follows from it.  log p_k is taken relative
// to `base`, the teacher's log-sum-exp or, without one, its largest kept logit, so that it is a
// difference of small numbers: log p_k = (v_k - base) - logs.
struct DsList {
  float *v, *z;   // the teacher's and the student's scaled logits
  int32_t* i;
  float base, logs, mass;   // mass: M
  float cm, c;              // g w tau M, g w tau
  __device__ __forceinline__ DsList(uint8_t* at, int K)
      : v(reinterpret_cast<float*>(at)), z(v + K), i(reinterpret_cast<int32_t*>(z + K)) {}
  __device__ __forceinline__ float logp(int k) const { return (v[k] - base) - logs; }
  __device__ __forceinline__ float p(int k) const { return v[k] == -INFINITY ? 0.f : expf(logp(k)); }
};

// Reads the list; the warp's (base, sum of exp(v - base)) into part[warp].  Called by every thread;
// warps behind the list's end do next to nothing.
template <class T>
__device__ __forceinline__ void ds_read_list(const DistillArgs& p, int t, const T* z, float it,
                                             const DsList& l, float2* part, DeviceStatus* st) {
  const bool given = p.teacher_lse != nullptr;
  float most = given ? p.teacher_lse[t] : -INFINITY, s = 0.f;
  if ((int)(threadIdx.x & ~31u) < p.K) {
    bool bad = false;
    for (int k = threadIdx.x; k < p.K; k += DS_THREADS) {
      int i = p.indices[(long long)t * p.K + k];
      if (i < -1 || i >= p.V) {
        bad = true;
        i = -1;
      }
      const float v = i < 0 ? -INFINITY : p.values[(long long)t * p.K + k] * it;
      l.i[k] = i;
      l.v[k] = v;
      l.z[k] = i < 0 ? 0.f : to_f32<T>(z[i]) * it;
      if (!given) most = fmaxf(most, v);
    }
    if (bad) raise_error(st, GPTQ_ERR_ARG, t);
    if (!given) {
#pragma unroll
      for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    for (int k = threadIdx.x; k < p.K; k += DS_THREADS)
      if (l.v[k] != -INFINITY) s += expf(l.v[k] - most);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(most, s);
}
// After a barrier.  (Without the teacher's log-sum-exp the p_k sum to one.)
__device__ __forceinline__ void ds_join_list(const DistillArgs& p, DsList& l, const float2* part) {
  float s;
  ds_join_all(part, DS_WARPS, l.base, s, DS_LOG2E);
  l.logs = p.teacher_lse ? 0.f : logf(s);
  l.mass = p.teacher_lse || !(s > 0.f) ? s : 1.f;
}
// The loss of the row, by warp 0.
__device__ __forceinline__ float ds_loss(const DistillArgs& p, const DsList& l, float lse) {
  float kl = 0.f;
  for (int k = threadIdx.x; k < p.K; k += 32) {
    const float q = l.p(k);
    if (q != 0.f) kl += q * (l.logp(k) - (l.z[k] - lse));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) kl += __shfl_xor_sync(0xffffffffu, kl, o);
  return kl;
}

// The gradient at the listed entries inside [lo, hi), over what the dense pass wrote there: the
// first listing of an index writes the sum of all its listings, rounded once.  After a barrier that
// follows the dense pass.
template <class T>
__device__ __forceinline__ void ds_listed(const DistillArgs& p, T* dz, const DsList& l, float lse,
                                          long long lo, long long hi) {
  for (int k = threadIdx.x; k < p.K; k += DS_THREADS) {
    const int i = l.i[k];
    if (i < lo || i >= hi) continue;
    bool first = true;
    float sum = 0.f;
    for (int j = 0; j < p.K; ++j)
      if (l.i[j] == i) {
        first = first && j >= k;
        sum += l.p(j);
      }
    if (first) dz[i] = ds_round<T>(fmaf(l.cm, ds_exp2((l.z[k] - lse) * DS_LOG2E), -l.c * sum));
  }
}

__device__ __forceinline__ void ds_store_remote(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// One cluster per token; `part`: 16-byte vectors of the row per CTA.  LOSS: the loss and lse are
// formed (else lse is given); GRAD: the gradient is written.
template <class T, bool LOSS, bool GRAD>
__global__ void __launch_bounds__(DS_THREADS, 3)
    k_distill(DistillArgs p, int part, int log2c, DeviceStatus* st, long long budget) {
  constexpr int N = DsVec<T>::N;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar;
  __shared__ float2 row_part[DS_WARPS], list_part[DS_WARPS], joined[8];
  uint4* row = reinterpret_cast<uint4*>(smem);
  DsList l(smem + (size_t)part * 16, p.K);
  const int C = 1 << log2c;
  const int t = blockIdx.x >> log2c, rank = blockIdx.x & (C - 1);
  const T* z = (const T*)p.logits + (long long)t * p.ld;
  T* dz = GRAD ? (T*)p.dlogits + (long long)t * p.ld_grad : nullptr;
  // the row as `head` scalars, nvec aligned vectors and `tail` scalars
  const int head = min(p.V, (int)((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / (int)sizeof(T));
  const int nvec = (p.V - head) / N, tail0 = head + nvec * N;
  const int v0 = min(nvec, rank * part), nv = min(nvec, v0 + part) - v0;
  if (threadIdx.x == 0) {
    tc::mbar_init(&bar, 1);
    tc::mbar_fence_init();
  }
  if (LOSS && C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  pdl_release();
  const float w = p.weight ? p.weight[t] : 1.f;
  if (w == 0.f) {   // the whole cluster takes this branch
    if (LOSS && rank == 0 && threadIdx.x == 0) {
      p.loss[t] = 0.f;
      p.lse_out[t] = 0.f;
    }
    if (GRAD) {
      const int lo = rank ? head + v0 * N : 0, hi = rank == C - 1 ? p.V : head + (v0 + nv) * N;
      for (int i = lo + threadIdx.x; i < hi; i += DS_THREADS) dz[i] = ds_round<T>(0.f);
    }
    if (LOSS && C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    return;
  }
  __syncthreads();
  if (threadIdx.x == 0 && nv) {
    tc::mbar_expect_tx(&bar, nv * 16);
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            tc::smem_u32(row)),
        "l"(reinterpret_cast<const uint4*>(z + head) + v0), "r"(nv * 16), "r"(tc::smem_u32(&bar))
        : "memory");
  }
  auto landed = [&] {
    if (nv && !tc::mbar_wait(&bar, 0, budget)) {
      raise_error(st, GPTQ_ERR_TIMEOUT, 61);
      tc::mbar_wait(&bar, 0, kDrainCycles);
    }
  };
  // while the row is on its way: the scalars at its ends (rank 0's), and the list
  const float it = 1.f / p.tau, k2 = it * DS_LOG2E;
  int edge = -1;
  if (rank == 0 && (int)threadIdx.x < 32) {
    if ((int)threadIdx.x < head) edge = threadIdx.x;
    if ((int)threadIdx.x >= 16 && tail0 + (int)threadIdx.x - 16 < p.V)
      edge = tail0 + threadIdx.x - 16;
  }
  const float edge_z = edge >= 0 ? to_f32<T>(z[edge]) : -INFINITY;
  ds_read_list<T>(p, t, z, it, l, list_part, st);
  float lse;
  if (LOSS) {
    // an end's own sum: 1, 0 for -inf, NaN for +inf (as inf - inf among the vectors) and NaN (which fmaxf
    // drops from the maximum, not from the sum)
    float m = edge_z, s = edge_z == -INFINITY ? 0.f : edge_z - edge_z + 1.f;
    landed();
    for (int i = threadIdx.x; i < nv; i += 2 * DS_THREADS) {
      const uint4 v0 = row[i];
      const bool two = i + DS_THREADS < nv;
      const uint4 v1 = two ? row[i + DS_THREADS] : v0;
      const float mx = fmaxf(m, fmaxf(ds_max<T>(v0), ds_max<T>(v1)));
      const float mk = mx == -INFINITY ? 0.f : mx * k2;
      if (m != mx) s *= ds_exp2((m - mx) * k2);
      m = mx;
      float x[N];
      ds_unpack<T>(v0, x);
      ds_exp2_all<N>(x, ds_pair(k2, k2), ds_pair(-mk, -mk));
      uint64_t sum = ds_pair(x[0], x[1]);
#pragma unroll
      for (int e = 2; e < N; e += 2) sum = ds_add2(sum, ds_pair(x[e], x[e + 1]));
      if (two) {
        ds_unpack<T>(v1, x);
        ds_exp2_all<N>(x, ds_pair(k2, k2), ds_pair(-mk, -mk));
#pragma unroll
        for (int e = 0; e < N; e += 2) sum = ds_add2(sum, ds_pair(x[e], x[e + 1]));
      }
      float s0, s1;
      ds_split(sum, s0, s1);
      s += s0 + s1;
    }
    // join the threads, then the cluster, both in a fixed order
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      ds_join(m, s, m2, s2, k2);
    }
    if ((threadIdx.x & 31) == 0) row_part[threadIdx.x >> 5] = make_float2(m, s);
    __syncthreads();   // also: the list
    ds_join_all(row_part, DS_WARPS, m, s, k2);
    if (C > 1) {
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // every CTA has started
      if ((int)threadIdx.x < C) {
        const uint32_t to = tc::map_to_rank(&joined[rank], threadIdx.x);
        ds_store_remote(to, m);
        ds_store_remote(to + 4, s);
      }
      tc::cluster_sync();   // also: every listed logit was read before any gradient is written
      ds_join_all(joined, C, m, s, k2);
    }
    lse = fmaf(m, it, logf(s));
  } else {
    lse = p.lse_in[t];
    __syncthreads();   // the list
  }
  ds_join_list(p, l, list_part);
  if (LOSS && !GRAD && rank) return;
  if (LOSS && rank == 0 && threadIdx.x < 32) {
    const float kl = ds_loss(p, l, lse);
    if (threadIdx.x == 0) {
      p.loss[t] = w * p.tau * p.tau * kl;
      p.lse_out[t] = lse;
    }
  }
  if (!GRAD) return;
  l.c = p.dloss[t] * w * p.tau;
  l.cm = l.c * l.mass;
  const float lse2 = lse * DS_LOG2E;
  if (edge >= 0) dz[edge] = ds_round<T>(l.cm * ds_exp2(fmaf(edge_z, k2, -lse2)));
  T* out = dz + head + (long long)v0 * N;
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  const uint64_t kk = ds_pair(k2, k2), off = ds_pair(-lse2, -lse2), cc = ds_pair(l.cm, l.cm);
  if (!LOSS) landed();
#pragma unroll 2
  for (int i = threadIdx.x; i < nv; i += DS_THREADS) {
    float x[N];
    ds_unpack<T>(row[i], x);
    ds_exp2_all<N>(x, kk, off);
#pragma unroll
    for (int e = 0; e < N; e += 2) ds_split(ds_mul2(ds_pair(x[e], x[e + 1]), cc), x[e], x[e + 1]);
    if (wide) {
      reinterpret_cast<uint4*>(out)[i] = ds_pack<T>(x);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) out[(long long)i * N + e] = ds_round<T>(x[e]);
    }
  }
  // The listed entries of this CTA's own part, over what was just written there, by the warps that
  // the list reaches.  Their slots in the row's shared memory, no longer needed, find indices that
  // are listed twice: every listing leaves its number, one of each index's listings finds its own
  // again and writes the sum over all of them (in list order, whichever listing it is).
  const int listers = min(DS_THREADS, (p.K + 31) & ~31);
  if ((int)threadIdx.x >= listers) {
    asm volatile("bar.arrive 1, %0;" ::"n"(DS_THREADS) : "memory");
    return;
  }
  asm volatile("bar.sync 1, %0;" ::"n"(DS_THREADS) : "memory");
  auto sync = [&] { asm volatile("bar.sync 2, %0;" ::"r"(listers) : "memory"); };
  const int lo = head + v0 * N, hi = lo + nv * N;
  uint16_t* tag = reinterpret_cast<uint16_t*>(row);
  constexpr int TS = sizeof(T) / 2;
  for (int k = threadIdx.x; k < p.K; k += DS_THREADS)
    if (l.i[k] >= lo && l.i[k] < hi) tag[(l.i[k] - lo) * TS] = (uint16_t)k;
  sync();
  constexpr int kTwice = 1 << 30;
  for (int k = threadIdx.x; k < p.K; k += DS_THREADS) {
    const int i = l.i[k] & ~kTwice;
    if (l.i[k] < 0 || i < lo || i >= hi) continue;
    const int winner = tag[(i - lo) * TS];
    if (winner != k) atomicOr(&l.i[winner], kTwice);
  }
  sync();
  for (int k = threadIdx.x; k < p.K; k += DS_THREADS) {
    const int i = l.i[k] & ~kTwice;
    if (l.i[k] < 0 || i < lo || i >= hi || tag[(i - lo) * TS] != k) continue;
    float sum;
    if (l.i[k] & kTwice) {
      sum = 0.f;
      for (int j = 0; j < p.K; ++j)
        if (l.i[j] >= 0 && (l.i[j] & ~kTwice) == i) sum += l.p(j);
    } else {
      sum = l.p(k);
    }
    dz[i] = ds_round<T>(fmaf(l.cm, ds_exp2((l.z[k] - lse) * DS_LOG2E), -l.c * sum));
  }
  if (rank == 0) {   // the row's ends
    ds_listed<T>(p, dz, l, lse, 0, head);
    ds_listed<T>(p, dz, l, lse, tail0, p.V);
  }
}

// Rows that do not fit a cluster's shared memory: one CTA per token, which reads them again.
template <class T>
__global__ void __launch_bounds__(DS_THREADS) k_distill_long(DistillArgs p, DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[33];
  __shared__ float2 list_part[DS_WARPS];
  DsList l(smem, p.K);
  const int t = blockIdx.x;
  const T* z = (const T*)p.logits + (long long)t * p.ld;
  const float w = p.weight ? p.weight[t] : 1.f;
  T* dz = p.dlogits ? (T*)p.dlogits + (long long)t * p.ld_grad : nullptr;
  if (w == 0.f) {
    if (threadIdx.x == 0 && p.loss) {
      p.loss[t] = 0.f;
      p.lse_out[t] = 0.f;
    }
    if (dz)
      for (int i = threadIdx.x; i < p.V; i += DS_THREADS) dz[i] = ds_round<T>(0.f);
    return;
  }
  const float it = 1.f / p.tau, k2 = it * DS_LOG2E;
  ds_read_list<T>(p, t, z, it, l, list_part, st);
  float lse;
  if (p.lse_in) {
    lse = p.lse_in[t];
  } else {
    float mx = -INFINITY;
    for (int i = threadIdx.x; i < p.V; i += DS_THREADS) mx = fmaxf(mx, to_f32<T>(z[i]));
    mx = ds_block(mx, true, red);
    const float mk = mx == -INFINITY ? 0.f : mx * k2;
    float s = 0.f;
    for (int i = threadIdx.x; i < p.V; i += DS_THREADS) s += ds_exp2(fmaf(to_f32<T>(z[i]), k2, -mk));
    lse = fmaf(mx, it, logf(ds_block(s, false, red)));
  }
  __syncthreads();   // the list; every listed logit was read before any gradient is written
  ds_join_list(p, l, list_part);
  if (p.loss && threadIdx.x < 32) {
    const float kl = ds_loss(p, l, lse);
    if (threadIdx.x == 0) {
      p.loss[t] = w * p.tau * p.tau * kl;
      p.lse_out[t] = lse;
    }
  }
  if (!dz) return;
  l.c = p.dloss[t] * w * p.tau;
  l.cm = l.c * l.mass;
  for (int i = threadIdx.x; i < p.V; i += DS_THREADS)
    dz[i] = ds_round<T>(l.cm * ds_exp2(fmaf(to_f32<T>(z[i]), k2, -lse * DS_LOG2E)));
  __syncthreads();
  ds_listed<T>(p, dz, l, lse, 0, p.V);
}

namespace {

template <class T, bool LOSS, bool GRAD>
int launch_distill(Ctx* c, const DistillArgs& p, int log2c, int part, size_t smem) {
  // the kernel's limit, not this call's size: the attribute is the device's, and another thread's call may
  // set it between this one's attribute and its launch
  GPTQ_CUDA_CHECK(c, cudaFuncSetAttribute(k_distill<T, LOSS, GRAD>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          DS_PART_MAX + kDistillMaxK * DS_ENTRY));
  GPTQ_CUDA_CHECK(c, launch_pdl_cluster(c, LOSS ? 1 << log2c : 1, k_distill<T, LOSS, GRAD>,
                                        dim3((unsigned)p.T << log2c), dim3(DS_THREADS), smem, p,
                                        part, log2c, c->status, c->timeout_cycles));
  return GPTQ_OK;
}

template <class T>
int distill_as(Ctx* c, const DistillArgs& p) {
  const size_t list = (size_t)p.K * DS_ENTRY;
  const long long nvec = std::max<long long>(1, (long long)p.V / DsVec<T>::N);
  // CTAs per row: parts of at most DS_PART bytes; with few rows more, down to 8 KB parts, so that
  // the SMs share the work (the loss of 5 rows of 32000 fp32 logits: 4.5 us, without 5.1).
  int log2c = 0;
  while (log2c < 3 && (nvec * 16 > (long long)DS_PART << log2c ||
                       (((long long)p.T << log2c) * 2 <= c->num_sms && nvec * 16 > 8192LL << log2c)))
    ++log2c;
  const long long part = (nvec + (1 << log2c) - 1) >> log2c;
  if (part * 16 > DS_PART_MAX || ((long long)p.T << log2c) > INT32_MAX) {
    GPTQ_LAUNCH(c, k_distill_long<T>, p.T, DS_THREADS, list, p, c->status);
    return GPTQ_OK;
  }
  const size_t smem = (size_t)part * 16 + list;
  if (!p.loss) return launch_distill<T, false, true>(c, p, log2c, (int)part, smem);
  if (!p.dlogits) return launch_distill<T, true, false>(c, p, log2c, (int)part, smem);
  return launch_distill<T, true, true>(c, p, log2c, (int)part, smem);
}

}  // namespace

int distill(Ctx* c, const DistillArgs& p) {
  if (p.dtype == GPTQ_BF16) return distill_as<__nv_bfloat16>(c, p);
  if (p.dtype == GPTQ_F16) return distill_as<__half>(c, p);
  return distill_as<float>(c, p);
}

}  // namespace gptq
