// Distillation from a teacher's stored top logits.  Per token, with y = z / τ, q = softmax(y) over
// the student's V logits and p_k = exp(v_k / τ - L) over the K stored teacher logits (L: the
// teacher's own log-sum-exp at τ where it was stored, else that of the K kept values):
//   loss = w τ² Σ_k p_k (log p_k - (y_{i_k} - lse)),          lse = log Σ_j exp y_j
//   dz_i = g w τ (M q_i - Σ_{k: i_k = i} p_k),                M = Σ_k p_k
// (g: the token's upstream gradient).
#include "kernels.h"

namespace gptq {

constexpr int DS_THREADS = 256;

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

// One CTA per token.
template <class T>
__global__ void __launch_bounds__(DS_THREADS) k_distill(DistillArgs p, DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  extern __shared__ char smem[];
  float* pk = reinterpret_cast<float*>(smem);               // teacher's probabilities [K]
  float* zk = pk + p.K;                                     // the student's logits there
  int32_t* ik = reinterpret_cast<int32_t*>(zk + p.K);       // and where (-1: no entry)
  __shared__ float red[33];
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
  const float it = 1.f / p.tau;
  float most = -INFINITY;
  bool bad = false;
  for (int k = threadIdx.x; k < p.K; k += DS_THREADS) {
    int i = p.indices[(long long)t * p.K + k];
    if (i < -1 || i >= p.V) {
      bad = true;
      i = -1;
    }
    ik[k] = i;
    pk[k] = i < 0 ? -INFINITY : p.values[(long long)t * p.K + k] * it;
    zk[k] = i < 0 ? 0.f : to_f32<T>(z[i]) * it;
    most = fmaxf(most, pk[k]);
  }
  if (bad) raise_error(st, GPTQ_ERR_ARG, t);
  float L;
  if (p.teacher_lse) {
    L = p.teacher_lse[t];
  } else {
    most = ds_block(most, true, red);
    float s = 0.f;
    for (int k = threadIdx.x; k < p.K; k += DS_THREADS)
      s += pk[k] == -INFINITY ? 0.f : expf(pk[k] - most);
    L = most + logf(ds_block(s, false, red));
  }
  float lse;
  if (p.lse_in) {
    lse = p.lse_in[t];
  } else {
    float mx = -INFINITY;
    for (int i = threadIdx.x; i < p.V; i += DS_THREADS) mx = fmaxf(mx, to_f32<T>(z[i]));
    mx = ds_block(mx, true, red) * it;
    float s = 0.f;
    for (int i = threadIdx.x; i < p.V; i += DS_THREADS) s += expf(fmaf(to_f32<T>(z[i]), it, -mx));
    lse = mx + logf(ds_block(s, false, red));
  }
  float kl = 0.f, mass = 0.f;
  for (int k = threadIdx.x; k < p.K; k += DS_THREADS) {
    const float lp = pk[k] - L, q = pk[k] == -INFINITY ? 0.f : expf(lp);
    pk[k] = q;
    mass += q;
    if (q != 0.f) kl += q * (lp - (zk[k] - lse));
  }
  mass = ds_block(mass, false, red);
  if (p.loss) {
    kl = ds_block(kl, false, red);
    if (threadIdx.x == 0) {
      p.loss[t] = w * p.tau * p.tau * kl;
      p.lse_out[t] = lse;
    }
  }
  if (!dz) return;
  const float c = p.dloss[t] * w * p.tau, cm = c * mass;
  for (int i = threadIdx.x; i < p.V; i += DS_THREADS)
    dz[i] = ds_round<T>(cm * expf(fmaf(to_f32<T>(z[i]), it, -lse)));
  __syncthreads();
  // the listed entries: the first listing of an index writes the sum of all its listings
  for (int k = threadIdx.x; k < p.K; k += DS_THREADS) {
    if (ik[k] < 0) continue;
    bool first = true;
    float sum = 0.f;
    for (int j = 0; j < p.K; ++j)
      if (ik[j] == ik[k]) {
        if (j < k) first = false;
        sum += pk[j];
      }
    if (first) dz[ik[k]] = ds_round<T>(fmaf(cm, expf(zk[k] - lse), -c * sum));
  }
}

int distill(Ctx* c, const DistillArgs& p) {
  const size_t smem = (size_t)p.K * 12;
  if (p.dtype == GPTQ_BF16)
    GPTQ_LAUNCH(c, k_distill<__nv_bfloat16>, p.T, DS_THREADS, smem, p, c->status);
  else if (p.dtype == GPTQ_F16)
    GPTQ_LAUNCH(c, k_distill<__half>, p.T, DS_THREADS, smem, p, c->status);
  else
    GPTQ_LAUNCH(c, k_distill<float>, p.T, DS_THREADS, smem, p, c->status);
  return GPTQ_OK;
}

}  // namespace gptq
