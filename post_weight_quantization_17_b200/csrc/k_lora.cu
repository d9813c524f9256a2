// The packed layer with low-rank adapters of many requests: token t of a batch belongs to a request
// that uses adapter a_t (or none), and every request shares the one packed projection,
//   U[t]  = s[a_t] A[a_t] X[t]                       (A [n, R, d], s [n])
//   Y[t]  = Ŵ X[t] + B[a_t]ᵀ U[t]                    (B [n, R, m])
// and, for training the adapters on the frozen codes,
//   G[t]  = s[a_t] B[a_t] dY[t]
//   dX[t] = Ŵᵀ dY[t] + A[a_t]ᵀ G[t],   dA[a] = Σ_{t: a_t = a} G[t] X[t]ᵀ,   dB[a] = Σ U[t] dY[t]ᵀ.
// A and B are both rank-major, so the four adapter products are two kinds: a contraction over the
// features (A X, B dY) and a sum over tokens (dA, dB).
//
// The kernels of this file take every format (any code width, group, per-column group ids, fp32
// activations) and run on CUDA cores, all sums in fp32 in a fixed order.
#include <algorithm>

#include "lora_util.cuh"

namespace gptq {

// out[t, j] = s[a] Σ_f x[t, f] w[a, j, f]: one warp per (token, rank index).
template <class TX>
__global__ void __launch_bounds__(256)
    k_lora_shrink_any(const TX* __restrict__ x, int T, int F, const TX* __restrict__ w, int n,
                      int R, const int32_t* __restrict__ adapter, const float* __restrict__ scaling,
                      float* __restrict__ out, DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  const int lane = threadIdx.x & 31;
  const long long e = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (e >= (long long)T * R) return;
  const int t = (int)(e / R), j = (int)(e % R);
  const int a = adapter_of(adapter, t, n, st);
  float s = 0.f;
  if (a >= 0) {
    const TX* xr = x + (long long)t * F;
    const TX* wr = w + ((long long)a * R + j) * F;
    for (int f = lane; f < F; f += 32) s = fmaf(to_f32<TX>(xr[f]), to_f32<TX>(wr[f]), s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= scaling[a];
  }
  if (lane == 0) out[e] = s;
}

struct AnyCodes {
  const uint32_t* packed;
  int wpr, bits, group, ng;
  const int32_t* group_id;
  const float* scales;
  const int32_t* zeros;
};

// Ŵ[r, k] as the quantizer defines it, Δ (c - z) in fp32; *bad: a grid index outside [0, n_g).
__device__ __forceinline__ float any_weight(const AnyCodes& q, long long r, int k, bool* bad) {
  const long long bit = (long long)k * q.bits;
  const uint32_t* row = q.packed + r * q.wpr;
  const int w = (int)(bit >> 5), sh = (int)(bit & 31);
  uint32_t c = row[w] >> sh;
  if (sh + q.bits > 32) c |= row[w + 1] << (32 - sh);
  c &= (1u << q.bits) - 1u;
  int g = q.group_id ? q.group_id[k] : (q.group == -1 ? 0 : k / q.group);
  if (g < 0 || g >= q.ng) {
    *bad = true;
    g = 0;
  }
  return __fmul_rn(q.scales[r * q.ng + g], (float)((int)c - q.zeros[r * q.ng + g]));
}

// Y: 128 rows x 8 tokens per CTA, one row per thread; the token's activations pass through shared
// memory in runs of 32 columns.
template <class TX, class TY>
__global__ void __launch_bounds__(128)
    k_lora_fwd_any(const TX* __restrict__ X, int T, int d, AnyCodes q, int m, int n, int R,
                   const int32_t* __restrict__ adapter, const TX* __restrict__ B,
                   const float* __restrict__ U, TY* __restrict__ Y, DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  __shared__ float xs[32][8];
  const int r = blockIdx.x * 128 + threadIdx.x, t0 = blockIdx.y * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  bool bad = false;
  for (int k0 = 0; k0 < d; k0 += 32) {
    __syncthreads();
    for (int e = threadIdx.x; e < 256; e += 128) {
      const int t = t0 + (e >> 5), k = k0 + (e & 31);
      xs[e & 31][e >> 5] = (t < T && k < d) ? to_f32<TX>(X[(long long)t * d + k]) : 0.f;
    }
    __syncthreads();
    if (r >= m) continue;
    const int nk = min(32, d - k0);
    for (int k = 0; k < nk; ++k) {
      const float w = any_weight(q, r, k0 + k, &bad);
#pragma unroll
      for (int t = 0; t < 8; ++t) acc[t] = fmaf(xs[k][t], w, acc[t]);
    }
  }
  if (bad) raise_error(st, GPTQ_ERR_ARG, r);
  if (r >= m) return;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    if (t0 + t >= T) break;
    const int a = adapter[t0 + t];
    if (a >= 0 && a < n) {
      const TX* b = B + (long long)a * R * m + r;
      const float* u = U + (long long)(t0 + t) * R;
      float s = 0.f;
      for (int j = 0; j < R; ++j) s = fmaf(u[j], to_f32<TX>(b[(long long)j * m]), s);
      acc[t] += s;
    }
    Y[(long long)(t0 + t) * m + r] = from_f32<TY>(acc[t]);
  }
}

// dX: 128 columns x 8 tokens per CTA, one column per thread.
template <class TX>
__global__ void __launch_bounds__(128)
    k_lora_dx_any(const TX* __restrict__ dY, int T, int d, AnyCodes q, int m, int n, int R,
                  const int32_t* __restrict__ adapter, const TX* __restrict__ A,
                  const float* __restrict__ G, TX* __restrict__ dX, DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  __shared__ float ys[32][8];
  const int k = blockIdx.x * 128 + threadIdx.x, t0 = blockIdx.y * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  bool bad = false;
  for (int r0 = 0; r0 < m; r0 += 32) {
    __syncthreads();
    for (int e = threadIdx.x; e < 256; e += 128) {
      const int t = t0 + (e >> 5), r = r0 + (e & 31);
      ys[e & 31][e >> 5] = (t < T && r < m) ? to_f32<TX>(dY[(long long)t * m + r]) : 0.f;
    }
    __syncthreads();
    if (k >= d) continue;
    const int nr = min(32, m - r0);
    for (int r = 0; r < nr; ++r) {
      const float w = any_weight(q, r0 + r, k, &bad);
#pragma unroll
      for (int t = 0; t < 8; ++t) acc[t] = fmaf(ys[r][t], w, acc[t]);
    }
  }
  if (bad) raise_error(st, GPTQ_ERR_ARG, k);
  if (k >= d) return;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    if (t0 + t >= T) break;
    const int a = adapter[t0 + t];
    if (a >= 0 && a < n) {
      const TX* w = A + (long long)a * R * d + k;
      const float* g = G + (long long)(t0 + t) * R;
      float s = 0.f;
      for (int j = 0; j < R; ++j) s = fmaf(g[j], to_f32<TX>(w[(long long)j * d]), s);
      acc[t] += s;
    }
    dX[(long long)(t0 + t) * d + k] = from_f32<TX>(acc[t]);
  }
}

// fp32 x: out[a, j, f] (+)= Σ_{t: a_t = a} u[t, j] x[t, f] for 8 rank indices: one feature per thread.
// A token of another adapter is skipped, not multiplied by zero, so its non-finite values stay out.  (The
// first CTA checks the ids: dB alone needs no other kernel.)
__global__ void __launch_bounds__(128)
    k_lora_outer_f32(const float* __restrict__ u, const float* __restrict__ x, int T, int F, int n, int R,
                     const int32_t* __restrict__ adapter, int accumulate, float* __restrict__ out,
                     DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  const int f = blockIdx.x * 128 + threadIdx.x, j0 = blockIdx.y * 8, a = blockIdx.z;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    for (int t = threadIdx.x; t < T; t += 128) adapter_of(adapter, t, n, st);
  if (f >= F) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int t = 0; t < T; ++t) {
    if (adapter[t] != a) continue;
    const float v = x[(long long)t * F + f];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < R) acc[j] = fmaf(u[(long long)t * R + j0 + j], v, acc[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j0 + j >= R) break;
    float* o = out + ((long long)a * R + j0 + j) * F + f;
    *o = accumulate ? *o + acc[j] : acc[j];
  }
}

// ------------------------------------------------------------------------------------------
namespace {

AnyCodes any_codes(const LoraLayer& l) {
  return {l.packed, (int)(((long long)l.d * l.bits + 31) / 32), l.bits, l.group, l.ng, l.group_id,
          l.scales, l.zeros};
}

template <class TX>
int shrink_any(Ctx* c, const LoraLayer& l, const TX* x, int F, const TX* w, float* out) {
  const long long warps = (long long)l.T * l.R;
  GPTQ_LAUNCH(c, k_lora_shrink_any<TX>, (unsigned)((warps + 7) / 8), 256, 0, x, l.T, F, w, l.n, l.R,
              l.adapter, l.scaling, out, c->status);
  return GPTQ_OK;
}

template <class TX>
int forward_any(Ctx* c, const LoraLayer& l, const TX* X, void* Y, bool y_f32, float* U) {
  int rc = shrink_any<TX>(c, l, X, l.d, (const TX*)l.A, U);
  if (rc) return rc;
  const dim3 grid((l.m + 127) / 128, (l.T + 7) / 8);
  if (y_f32)
    GPTQ_LAUNCH(c, k_lora_fwd_any<TX, float>, grid, 128, 0, X, l.T, l.d, any_codes(l), l.m, l.n,
                l.R, l.adapter, (const TX*)l.B, (const float*)U, (float*)Y, c->status);
  else
    GPTQ_LAUNCH(c, k_lora_fwd_any<TX, TX>, grid, 128, 0, X, l.T, l.d, any_codes(l), l.m, l.n, l.R,
                l.adapter, (const TX*)l.B, (const float*)U, (TX*)Y, c->status);
  return GPTQ_OK;
}

int outer_f32(Ctx* c, const LoraLayer& l, const float* u, const float* x, int F, int accumulate,
              float* out) {
  GPTQ_LAUNCH(c, k_lora_outer_f32, dim3((F + 127) / 128, (l.R + 7) / 8, l.n), 128, 0, u, x, l.T, F,
              l.n, l.R, l.adapter, accumulate, out, c->status);
  return GPTQ_OK;
}

template <class TX>
int dx_any(Ctx* c, const LoraLayer& l, const TX* dY, TX* dX, float* G) {
  int rc = shrink_any<TX>(c, l, dY, l.m, (const TX*)l.B, G);
  if (rc || !dX) return rc;
  GPTQ_LAUNCH(c, k_lora_dx_any<TX>, dim3((l.d + 127) / 128, (l.T + 7) / 8), 128, 0, dY, l.T, l.d,
              any_codes(l), l.m, l.n, l.R, l.adapter, (const TX*)l.A, (const float*)G, dX, c->status);
  return GPTQ_OK;
}

}  // namespace

int lora_shrink_any(Ctx* c, const LoraLayer& l, const void* x, int F, const void* w, float* out) {
  if (l.dtype == GPTQ_BF16)
    return shrink_any<__nv_bfloat16>(c, l, (const __nv_bfloat16*)x, F, (const __nv_bfloat16*)w, out);
  if (l.dtype == GPTQ_F16) return shrink_any<__half>(c, l, (const __half*)x, F, (const __half*)w, out);
  return shrink_any<float>(c, l, (const float*)x, F, (const float*)w, out);
}

// The formats that run on tensor cores: 16-bit activations, codes of 1 to 4 bits, one grid per row
// or per multiple of 128 columns.
static bool lora_tensor_format(const LoraLayer& l) {
  return l.dtype != GPTQ_F32 && l.bits <= 4 && !l.group_id && (l.group == -1 || l.group % 128 == 0);
}

size_t lora_workspace_bytes(const LoraLayer& l) {
  size_t floats = (size_t)l.T * l.R;
  const bool tensor = l.dtype != GPTQ_F32 && l.bits <= 4;
  if (tensor && l.T <= kLoraSmallTokens) floats = std::max(floats, lora_small_floats(l));
  size_t b = 256 * 2 + floats * sizeof(float);
  if (tensor)   // the backward pass keeps G in front
    b = std::max(b, 256 + (size_t)l.T * l.R * sizeof(float) + lora_tc_bytes(l));
  return kStatusBytes + b;
}

int lora_forward(Ctx* c, const LoraLayer& l, const void* X, void* Y, bool y_f32, float* U) {
  Carver cv(c);
  if (lora_tensor_format(l) && lora_small_applies(l, X)) {
    float* ws = cv.take<float>(0);
    // of a workspace larger than asked for no more, so that the splits follow from the call's sizes alone
    const size_t end = std::min(c->ws_bytes, lora_workspace_bytes(l));
    const size_t floats = end > cv.off ? (end - cv.off) / sizeof(float) : 0;
    return lora_forward_small(c, l, X, Y, y_f32, U, ws, floats);
  }
  if (lora_tensor_format(l)) return lora_tc(c, l, true, X, Y, y_f32, U, kStatusBytes);
  float* ws_U = cv.take<float>((size_t)l.T * l.R);
  if (!U) {
    if (!cv.ok())
      GPTQ_SET_ERR(c, GPTQ_ERR_NOMEM, "lora_matmul: workspace %zu < %zu bytes", c->ws_bytes, cv.off);
    U = ws_U;
  }
  if (l.dtype == GPTQ_BF16)
    return forward_any<__nv_bfloat16>(c, l, (const __nv_bfloat16*)X, Y, y_f32, U);
  if (l.dtype == GPTQ_F16) return forward_any<__half>(c, l, (const __half*)X, Y, y_f32, U);
  return forward_any<float>(c, l, (const float*)X, Y, true, U);
}

int lora_backward(Ctx* c, const LoraLayer& l, const void* dY, const void* X, const float* U,
                  void* dX, float* dA, float* dB, int accumulate) {
  Carver cv(c);
  float* G = cv.take<float>((size_t)l.T * l.R);
  if (!cv.ok())
    GPTQ_SET_ERR(c, GPTQ_ERR_NOMEM, "lora_backward: workspace %zu < %zu bytes", c->ws_bytes, cv.off);
  int rc = GPTQ_OK;
  if (dX || dA) {   // G, and dX where it is asked for
    if (lora_tensor_format(l)) rc = lora_tc(c, l, false, dY, dX, false, G, cv.off);
    else if (l.dtype == GPTQ_BF16)
      rc = dx_any(c, l, (const __nv_bfloat16*)dY, (__nv_bfloat16*)dX, G);
    else if (l.dtype == GPTQ_F16) rc = dx_any(c, l, (const __half*)dY, (__half*)dX, G);
    else rc = dx_any(c, l, (const float*)dY, (float*)dX, G);
  }
  if (rc || (!dA && !dB)) return rc;
  if (l.dtype != GPTQ_F32) return lora_outers(c, l, G, X, dA, U, dY, dB, accumulate);
  if (dA && (rc = outer_f32(c, l, G, (const float*)X, l.d, accumulate, dA))) return rc;
  return dB ? outer_f32(c, l, U, (const float*)dY, l.m, accumulate, dB) : GPTQ_OK;
}

}  // namespace gptq
