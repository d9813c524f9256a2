// The packed layer with adapters for a few tokens (decoding): up to 32 tokens at once.
//
// Bound by reading the codes from HBM, so the kernel is built around that stream: every warp reads
// its codes straight into registers, 16 bytes a lane (4 lanes cover the 64 bytes of a row's 128
// 4-bit codes), a step ahead of their use, and multiplies on mma.sync (16 rows x 8 tokens x 16
// columns).  The tensor instruction's column order is free as long as both operands share it, so
// lane t of a row's four holds columns 32 t .. 32 t + 31 of each 128-column step: its codes are one
// 16-byte load, its activations four, and neither passes through shared memory.  (c - z) is exact in
// 16 bits; a step's fp32 sum is scaled by the group's Δ, so Ŵ is never rounded.
//
// A X runs in the same launch, as CTAs of its own (one warp per token, rank index and 4096
// columns); k_lora_join then adds the K splits of the base product in a fixed order, forms
// U = s Σ parts and adds Bᵀ U.  With programmatic launch the join has read its part of B before the
// products end.
#include <algorithm>

#include "lora_util.cuh"

namespace gptq {

constexpr int LS_THREADS = 256;
// 16-row tiles per warp: two halve the reads of X per code; at 32 tokens the registers of their
// sums leave room for one (two spilled).
inline constexpr int ls_row_tiles(int token_tiles) { return token_tiles == 4 ? 1 : 2; }
// rows per CTA: 4 row warps x 2 column warps
constexpr int ls_rows(int token_tiles) { return 64 * ls_row_tiles(token_tiles); }
constexpr int LS_KC = 4096;                    // columns per warp of A X

struct SmallParams {
  const void* X;
  int T, d, m, wpr;
  const uint32_t* packed;
  const float* scales;
  const int32_t* zeros;
  int ng, group_steps;       // 128-column steps per group; 0: one grid per row
  int steps, per, row_ctas;  // steps in all and per split, CTAs along the rows
  int wide;                  // rows of codes may be read in 8- or 16-byte pieces
  float* part;               // [splits, T, m]
  int shrink_ctas, n, R, chunks;
  const int32_t* adapter;
  const void* A;
  float* upart;              // [chunks, T, R]
};

// 16 bytes that are used once.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int BITS>
__device__ __forceinline__ void load_codes(const SmallParams& p, int row, int step, int t4,
                                           uint32_t (&w)[BITS]) {
#pragma unroll
  for (int i = 0; i < BITS; ++i) w[i] = 0;
  const int w0 = (step * 4 + t4) * BITS;
  if (row >= p.m || w0 >= p.wpr) return;
  const uint32_t* src = p.packed + (long long)row * p.wpr + w0;
  if (p.wide && BITS == 4) {
    const uint4 v = ld_stream16(src);
    w[0] = v.x;
    w[1 % BITS] = v.y;
    w[2 % BITS] = v.z;
    w[3 % BITS] = v.w;
  } else if (p.wide && BITS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x;
    w[1 % BITS] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BITS; ++i)
      if (w0 + i < p.wpr) w[i] = src[i];
  }
}

// out[c, t, j] = Σ_{k in chunk c} X[t, k] A[a_t, j, k], one warp each.
template <bool BF16>
__device__ __forceinline__ void small_shrink(const SmallParams& p, DeviceStatus* st) {
  const int lane = threadIdx.x & 31;
  const long long e = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (e >= (long long)p.chunks * p.T * p.R) return;
  const int j = (int)(e % p.R), t = (int)(e / p.R % p.T), c = (int)(e / p.R / p.T);
  const int a = adapter_of(p.adapter, t, p.n, st);
  float s0 = 0.f, s1 = 0.f;
  if (a >= 0) {
    const uint4* x = reinterpret_cast<const uint4*>((const uint16_t*)p.X + (long long)t * p.d);
    const uint4* w = reinterpret_cast<const uint4*>((const uint16_t*)p.A + ((long long)a * p.R + j) * p.d);
    const int v1 = min(p.d, (c + 1) * LS_KC) / 8;
#pragma unroll 4
    for (int v = c * (LS_KC / 8) + lane; v < v1; v += 32) {
      const uint4 xv = x[v], wv = w[v];
      const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w}, ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 xf = pair_f32<BF16>(xs[i]), wf = pair_f32<BF16>(ws[i]);
        s0 = fmaf(xf.x, wf.x, s0);
        s1 = fmaf(xf.y, wf.y, s1);
      }
    }
  }
  float s = s0 + s1;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) p.upart[e] = s;
}

template <int BITS, int NT, bool BF16>
__global__ void __launch_bounds__(LS_THREADS, 2) k_lora_small(SmallParams p, DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  if ((int)blockIdx.x < p.shrink_ctas) {
    small_shrink<BF16>(p, st);
    return;
  }
  constexpr int LS_MT = NT == 4 ? 1 : 2;
  __shared__ float joined[4][32][LS_MT * NT * 4 + 1];
  const int bid = blockIdx.x - p.shrink_ctas;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = warp & 3, wk = warp >> 2, g = lane >> 2, t4 = lane & 3;
  const int row0 = (bid % p.row_ctas) * (64 * LS_MT) + wr * (LS_MT * 16) + g, split = bid / p.row_ctas;
  const int n = min(p.steps, (split + 1) * p.per) - split * p.per;
  const int s0 = split * p.per + (wk ? (n + 1) / 2 : 0), s1 = split * p.per + (wk ? n : (n + 1) / 2);
  float acc[LS_MT][NT][4] = {};
  uint32_t cw[LS_MT][2][BITS];
  float sc[LS_MT][2];
  int zs[LS_MT][2];
  bool bad = false;

  auto fetch = [&](int s) {
    const int gi = p.group_steps ? s / p.group_steps : 0;
#pragma unroll
    for (int mt = 0; mt < LS_MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + 16 * mt + 8 * h;
        load_codes<BITS>(p, row, s, t4, cw[mt][h]);
        const long long at = (long long)min(row, p.m - 1) * p.ng + gi;
        sc[mt][h] = p.scales[at];
        zs[mt][h] = p.zeros[at];
      }
  };
  if (s0 < s1) fetch(s0);
  for (int s = s0; s < s1; ++s) {
    uint32_t cur[LS_MT][2][BITS], zz[LS_MT][2];
    float delta[LS_MT][2];
#pragma unroll
    for (int mt = 0; mt < LS_MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < BITS; ++i) cur[mt][h][i] = cw[mt][h][i];
        delta[mt][h] = sc[mt][h];
        int z = zs[mt][h];
        if (z < 0 || z > 15) {
          bad = true;
          z = 0;
        }
        zz[mt][h] = zero_pair<BF16>(z);
      }
    if (s + 1 < s1) fetch(s + 1);
    float dd[LS_MT][NT][4] = {};
    const int k0 = s * 128 + t4 * 32;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 x[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int t = nt * 8 + g;
        x[nt] = make_uint4(0, 0, 0, 0);
        if (t < p.T && k0 + 8 * q < p.d)
          x[nt] = *reinterpret_cast<const uint4*>((const uint16_t*)p.X + (long long)t * p.d + k0 + 8 * q);
      }
#pragma unroll
      for (int mt = 0; mt < LS_MT; ++mt) {
        uint32_t u[4], v[4];
        centered8<BF16>(eight_codes<BITS>(cur[mt][0], q), zz[mt][0], u);
        centered8<BF16>(eight_codes<BITS>(cur[mt][1], q), zz[mt][1], v);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816<BF16>(dd[mt][nt], u[0], v[0], u[1], v[1], x[nt].x, x[nt].y);
          mma16816<BF16>(dd[mt][nt], u[2], v[2], u[3], v[3], x[nt].z, x[nt].w);
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < LS_MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[mt][nt][i] = fmaf(delta[mt][i >> 1], dd[mt][nt][i], acc[mt][nt][i]);
  }
  if (bad) raise_error(st, GPTQ_ERR_ARG, row0);
  float* mine = joined[wr][lane];
  if (wk == 1) {
#pragma unroll
    for (int mt = 0; mt < LS_MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[(mt * NT + nt) * 4 + i] = acc[mt][nt][i];
  }
  __syncthreads();
  if (wk == 1) return;
  float* out = p.part + (long long)split * p.T * p.m;
#pragma unroll
  for (int mt = 0; mt < LS_MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = row0 + 16 * mt + 8 * (i >> 1), t = nt * 8 + 2 * t4 + (i & 1);
        if (row < p.m && t < p.T)
          out[(long long)t * p.m + row] = acc[mt][nt][i] + mine[(mt * NT + nt) * 4 + i];
      }
}

// out[t, f] = Σ_splits part[s, t, f] + Σ_j U[t, j] w[a_t, j, f], U = scaling Σ_chunks upart.  A
// thread has two features of TOKS tokens, whose loads are independent of one another.
constexpr int LJ_THREADS = 128, LJ_AHEAD = 16;
template <class TX, class TY, int TOKS>
__global__ void __launch_bounds__(LJ_THREADS)
    k_lora_join(const float* __restrict__ part, int splits, int T, int F,
                const float* __restrict__ upart, int chunks, int n, int R,
                const int32_t* __restrict__ adapter, const float* __restrict__ scaling,
                const TX* __restrict__ w, TY* __restrict__ out, float* __restrict__ U) {
  extern __shared__ float us[];   // [TOKS, R]
  const int f = 2 * (blockIdx.x * LJ_THREADS + threadIdx.x), t0 = blockIdx.y * TOKS;
  const bool two = f + 1 < F, pairs = F % 2 == 0;
  // the adapters' first rows, an input, while the products still run
  TX first[TOKS][LJ_AHEAD][2];
  int a[TOKS];
#pragma unroll
  for (int k = 0; k < TOKS; ++k) {
    a[k] = t0 + k < T ? adapter[t0 + k] : -1;
    if (a[k] >= n) a[k] = -1;
  }
  auto row_pair = [&](int k, int j, TX (&v)[2]) {
    const TX* src = w + ((long long)a[k] * R + j) * F + f;
    if (pairs && (reinterpret_cast<uintptr_t>(w) & 3) == 0) {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(src);
      v[0] = reinterpret_cast<const TX*>(&u)[0];
      v[1] = reinterpret_cast<const TX*>(&u)[1];
    } else {
      v[0] = src[0];
      v[1] = src[two ? 1 : 0];
    }
  };
  if (TOKS == 1 && f < F) {
#pragma unroll
    for (int j = 0; j < LJ_AHEAD; ++j)
      if (a[0] >= 0 && j < R) row_pair(0, j, first[0][j]);
  }
  pdl_wait();
  pdl_release();
#pragma unroll
  for (int k = 0; k < TOKS; ++k) {
    if (t0 + k >= T) break;
    const float s = a[k] >= 0 && scaling ? scaling[a[k]] : 1.f;
    for (int j = threadIdx.x; j < R; j += LJ_THREADS) {
      float u = 0.f;
      if (a[k] >= 0) {
        for (int c = 0; c < chunks; ++c) u += upart[((long long)c * T + t0 + k) * R + j];
        u *= s;
      }
      us[k * R + j] = u;
      if (U && blockIdx.x == 0) U[(long long)(t0 + k) * R + j] = u;
    }
  }
  __syncthreads();
  if (f >= F) return;
  float y[TOKS][2];
#pragma unroll
  for (int k = 0; k < TOKS; ++k) y[k][0] = y[k][1] = 0.f;
  for (int s = 0; s < splits; ++s)
#pragma unroll
    for (int k = 0; k < TOKS; ++k) {
      if (t0 + k >= T) break;
      const float* src = part + ((long long)s * T + t0 + k) * F + f;
      if (pairs) {
        const float2 v = *reinterpret_cast<const float2*>(src);
        y[k][0] += v.x;
        y[k][1] += v.y;
      } else {
        y[k][0] += src[0];
        if (two) y[k][1] += src[1];
      }
    }
#pragma unroll
  for (int k = 0; k < TOKS; ++k) {
    if (t0 + k >= T) break;
    if (a[k] >= 0) {
      float v0 = 0.f, v1 = 0.f;
      int j = 0;
      if (TOKS == 1) {
#pragma unroll
        for (int i = 0; i < LJ_AHEAD; ++i)
          if (i < R) {
            v0 = fmaf(us[i], to_f32<TX>(first[0][i][0]), v0);
            v1 = fmaf(us[i], to_f32<TX>(first[0][i][1]), v1);
          }
        j = LJ_AHEAD;
      }
#pragma unroll 8
      for (; j < R; ++j) {
        TX v[2];
        row_pair(k, j, v);
        v0 = fmaf(us[k * R + j], to_f32<TX>(v[0]), v0);
        v1 = fmaf(us[k * R + j], to_f32<TX>(v[1]), v1);
      }
      y[k][0] += v0;
      y[k][1] += v1;
    }
    TY* o = out + (long long)(t0 + k) * F + f;
    if (pairs && (reinterpret_cast<uintptr_t>(out) & (2 * sizeof(TY) - 1)) == 0) {
      struct alignas(2 * sizeof(TY)) Pair { TY v[2]; };
      *reinterpret_cast<Pair*>(o) = Pair{{from_f32<TY>(y[k][0]), from_f32<TY>(y[k][1])}};
    } else {
      o[0] = from_f32<TY>(y[k][0]);
      if (two) o[1] = from_f32<TY>(y[k][1]);
    }
  }
}

int lora_join(Ctx* c, const LoraLayer& l, const float* part, int splits, int F, const float* upart,
              int chunks, const float* scaling, const void* w, void* out, bool out_f32, float* U) {
  // one token per CTA while that leaves few CTAs per SM, four (fewer, longer CTAs) beyond
  const int wide = (F + 2 * LJ_THREADS - 1) / (2 * LJ_THREADS);
  const bool four = (long long)wide * l.T > 16LL * c->num_sms;
  const dim3 grid(wide, four ? (l.T + 3) / 4 : l.T);
  const size_t smem = (size_t)(four ? 4 : 1) * l.R * sizeof(float);
#define GPTQ_JOIN_N(TX, TY, N)                                                                       \
  GPTQ_LAUNCH(c, (k_lora_join<TX, TY, N>), grid, LJ_THREADS, smem, part, splits, l.T, F, upart,      \
              chunks, l.n, l.R, l.adapter, scaling, (const TX*)w, (TY*)out, U)
#define GPTQ_JOIN(TX, TY)                                                                            \
  do {                                                                                               \
    if (four) GPTQ_JOIN_N(TX, TY, 4);                                                                \
    else GPTQ_JOIN_N(TX, TY, 1);                                                                     \
  } while (0)
  if (l.dtype == GPTQ_BF16) {
    if (out_f32) GPTQ_JOIN(__nv_bfloat16, float);
    else GPTQ_JOIN(__nv_bfloat16, __nv_bfloat16);
  } else {
    if (out_f32) GPTQ_JOIN(__half, float);
    else GPTQ_JOIN(__half, __half);
  }
#undef GPTQ_JOIN
#undef GPTQ_JOIN_N
  return GPTQ_OK;
}

namespace {

int token_tiles(int T) { return T <= 8 ? 1 : (T <= 16 ? 2 : 4); }

template <int BITS>
int launch_small(Ctx* c, const SmallParams& p, int grid, bool bf) {
  const int nt = token_tiles(p.T);
#define GPTQ_SMALL(NT)                                                                              \
  do {                                                                                              \
    if (bf) GPTQ_LAUNCH(c, (k_lora_small<BITS, NT, true>), grid, LS_THREADS, 0, p, c->status);      \
    else GPTQ_LAUNCH(c, (k_lora_small<BITS, NT, false>), grid, LS_THREADS, 0, p, c->status);        \
  } while (0)
  if (nt == 1) GPTQ_SMALL(1);
  else if (nt == 2) GPTQ_SMALL(2);
  else GPTQ_SMALL(4);
#undef GPTQ_SMALL
  return GPTQ_OK;
}

int small_chunks(int d) { return (d + LS_KC - 1) / LS_KC; }

// Splits of the columns so that the CTAs (two fit on an SM) fill whole waves: the smallest
// waves x (steps of a warp + 2 for its start).
int small_splits(int m, int d, int T, int num_sms, size_t max_floats) {
  const long long rows = (m + ls_rows(token_tiles(T)) - 1) / ls_rows(token_tiles(T)), steps = (d + 127) / 128, slots = 2LL * num_sms;
  long long best = -1;
  int splits = 1;
  for (int s = 1; s <= 64 && s <= steps; ++s) {
    if (s > 1 && (size_t)s * T * m > max_floats) break;
    const long long per = (steps + s - 1) / s, waves = (rows * ((steps + per - 1) / per) + slots - 1) / slots;
    const long long cost = waves * ((per + 1) / 2 + 2);
    if (best < 0 || cost < best) {
      best = cost;
      splits = (int)((steps + per - 1) / per);
    }
  }
  return splits;
}

}  // namespace

bool lora_small_applies(const LoraLayer& l, const void* X) {
  auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  return l.T <= kLoraSmallTokens && l.d % 8 == 0 && al(X) && al(l.A);
}

// Floats of workspace: U's parts and the splits' (at most 64 of them, and no more than fill two
// waves of CTAs).
size_t lora_small_floats(const LoraLayer& l) {
  const size_t rows = (l.m + 127) / 128;
  const size_t splits = std::min<size_t>(64, std::max<size_t>(1, 512 / rows + 1));
  return (size_t)small_chunks(l.d) * l.T * l.R + 64 + splits * l.T * l.m;
}

int lora_forward_small(Ctx* c, const LoraLayer& l, const void* X, void* Y, bool y_f32, float* U,
                       float* ws, size_t ws_floats) {
  const size_t uf = ((size_t)small_chunks(l.d) * l.T * l.R + 63) / 64 * 64;
  if (uf + (size_t)l.T * l.m > ws_floats)
    GPTQ_SET_ERR(c, GPTQ_ERR_NOMEM, "lora_matmul: workspace %zu bytes is too small", c->ws_bytes);
  SmallParams p{};
  p.X = X;
  p.T = l.T; p.d = l.d; p.m = l.m;
  p.wpr = (int)(((long long)l.d * l.bits + 31) / 32);
  p.packed = l.packed;
  p.scales = l.scales;
  p.zeros = l.zeros;
  p.ng = l.ng;
  p.group_steps = l.group == -1 ? 0 : l.group / 128;
  p.steps = (l.d + 127) / 128;
  const int splits = small_splits(l.m, l.d, l.T, c->num_sms, ws_floats - uf);
  p.per = (p.steps + splits - 1) / splits;
  p.row_ctas = (l.m + ls_rows(token_tiles(l.T)) - 1) / ls_rows(token_tiles(l.T));
  const int piece = l.bits == 4 ? 4 : 2;   // words per load of codes
  p.wide = p.wpr % piece == 0 && (reinterpret_cast<uintptr_t>(l.packed) & (piece * 4 - 1)) == 0;
  p.upart = ws;
  p.part = ws + uf;
  p.n = l.n; p.R = l.R;
  p.chunks = small_chunks(l.d);
  p.adapter = l.adapter;
  p.A = l.A;
  const long long warps = (long long)p.chunks * l.T * l.R;
  p.shrink_ctas = (int)((warps + 7) / 8);
  const int grid = p.shrink_ctas + p.row_ctas * splits;
  const bool bf = l.dtype == GPTQ_BF16;
  int rc;
  switch (l.bits) {
    case 1: rc = launch_small<1>(c, p, grid, bf); break;
    case 2: rc = launch_small<2>(c, p, grid, bf); break;
    case 3: rc = launch_small<3>(c, p, grid, bf); break;
    default: rc = launch_small<4>(c, p, grid, bf); break;
  }
  if (rc) return rc;
  return lora_join(c, l, p.part, splits, l.m, p.upart, p.chunks, l.scaling, l.B, Y, y_f32, U);
}

}  // namespace gptq
