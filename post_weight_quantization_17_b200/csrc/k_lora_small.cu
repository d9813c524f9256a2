// The packed layer with adapters for a few tokens (decoding): up to 32 tokens at once.
//
// Bound by reading the codes from HBM, so the kernel is built around that stream: every lane copies
// its own codes, 16 bytes at a time (4 lanes cover the 64 bytes of a row's 128 4-bit codes), into its
// own slots of a ring in shared memory several steps ahead of their use (no barrier is needed, and
// 128 KB per SM are on their way), and multiplies on mma.sync (16 rows x 8 tokens x 16 columns).  The
// tensor instruction's column order is free as long as both operands share it, so lane t of a row's
// four holds columns 32 t .. 32 t + 31 of each 128-column step: its codes are one 16-byte piece and
// its activations four.  The grid of four steps is read at once, a step to each of the four lanes, and
// passed round by shuffles.  (c - z) is exact in 16 bits; a step's fp32 sum is scaled by the group's
// Δ, so Ŵ is never rounded.
//
// A X runs in the same launch, as CTAs of its own (one warp per token, rank index and 4096
// columns); k_lora_join then adds the K splits of the base product in a fixed order, forms
// U = s Σ parts and adds Bᵀ U.  With programmatic launch the join has read its part of B before the
// products end.
#include <algorithm>

#include "lora_small_x.h"
#include "lora_util.cuh"

namespace gptq {

constexpr int LS_THREADS = 256;
constexpr int LS_MT = 2;                       // 16-row tiles per warp: two halve the reads of X per code
constexpr int LS_ROWS = 4 * LS_MT * 16;        // rows per CTA: 4 row warps x 2 column warps
constexpr int LS_KC = 4096;                    // columns per warp of A X
// Up to 16 tokens two CTAs share an SM (128 registers a thread, 4 steps of codes in each ring); with 24
// or 32 the sums take the registers of one, whose ring is twice as deep.  (One 16-row tile per warp and
// two CTAs: L1 then delivers X twice as often, 8 KB per KB of codes, and 24 tokens of 11008 x 4096 took
// 29 us instead of 21.)
__host__ __device__ constexpr int ls_ctas(int token_tiles) { return token_tiles <= 2 ? 2 : 1; }
__host__ __device__ constexpr int ls_depth(int token_tiles) { return token_tiles <= 2 ? 4 : 8; }
__host__ __device__ constexpr int ls_smem(int token_tiles) { return 8 * ls_depth(token_tiles) * 2 * LS_MT * 512; }

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
  int base_ctas, n, R, chunks;
  int ranks;                 // rank indices per warp of A X
  const int32_t* adapter;
  const void* A;
  float* upart;              // [chunks, T, R]
};

// One piece (32 codes, BITS words) of a row into this lane's slot; with CHECK zeros outside the row.
template <int BITS, bool CHECK>
__device__ __forceinline__ void copy_codes(const SmallParams& p, const uint32_t* src, int words_left,
                                           uint32_t dst) {
  if (p.wide && (BITS == 4 || BITS == 2)) {
    const int n = !CHECK || words_left > 0 ? 4 * BITS : 0;
    if (BITS == 4)
      asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst),
                   "l"(n ? src : p.packed), "r"(n)
                   : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst),
                   "l"(n ? src : p.packed), "r"(n)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < BITS; ++i) {
      const int n = !CHECK || i < words_left ? 4 : 0;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 4 * i),
                   "l"(n ? src + i : p.packed), "r"(n)
                   : "memory");
    }
  }
}

// out[c, t, j] = Σ_{k in chunk c} X[t, k] A[a_t, j, k]: a warp takes a chunk of a token and `ranks` rank
// indices one after the other.
template <bool BF16>
__device__ __forceinline__ void small_shrink(const SmallParams& p, int cta, DeviceStatus* st) {
  const int lane = threadIdx.x & 31, runs = (p.R + p.ranks - 1) / p.ranks;
  const long long e = (long long)cta * 8 + (threadIdx.x >> 5);
  if (e >= (long long)p.chunks * p.T * runs) return;
  const int j0 = (int)(e % runs) * p.ranks, t = (int)(e / runs % p.T), c = (int)(e / runs / p.T);
  const int a = adapter_of(p.adapter, t, p.n, st);
  const uint4* x = reinterpret_cast<const uint4*>((const uint16_t*)p.X + (long long)t * p.d);
  const int v1 = min(p.d, (c + 1) * LS_KC) / 8;
  for (int j = j0; j < min(p.R, j0 + p.ranks); ++j) {
    float s0 = 0.f, s1 = 0.f;
    if (a >= 0) {
      const uint4* w = reinterpret_cast<const uint4*>((const uint16_t*)p.A + ((long long)a * p.R + j) * p.d);
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
    if (lane == 0) p.upart[((long long)c * p.T + t) * p.R + j] = s;
  }
}

template <int BITS, int NT, bool BF16>
__global__ void __launch_bounds__(LS_THREADS, ls_ctas(NT)) k_lora_small(SmallParams p, DeviceStatus* st) {
  pdl_wait();
  pdl_release();
  // the product's CTAs first: those of A X then fill what their wave leaves (put first, they pushed 124 of
  // 288 long CTAs into a second wave: 8 tokens of 12288 x 49152 took 101 us instead of 93)
  if ((int)blockIdx.x >= p.base_ctas) {
    small_shrink<BF16>(p, blockIdx.x - p.base_ctas, st);
    return;
  }
  constexpr int DEPTH = ls_depth(NT), PIECES = 2 * LS_MT;
  extern __shared__ __align__(16) uint8_t ls_smem[];
  const int bid = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = warp & 3, wk = warp >> 2, g = lane >> 2, t4 = lane & 3;
  const int row0 = (bid % p.row_ctas) * LS_ROWS + wr * (LS_MT * 16) + g, split = bid / p.row_ctas;
  const int n = min(p.steps, (split + 1) * p.per) - split * p.per;
  const int s0 = split * p.per + (wk ? (n + 1) / 2 : 0), s1 = split * p.per + (wk ? n : (n + 1) / 2);
  float acc[LS_MT][NT][4] = {};
  bool bad = false;

  // Integer instructions bound this loop once the loads are far enough ahead (ALU pipe 72 % busy at
  // 2.7 TB/s with addresses and checks formed in every step), so pointers move by constants, rows and
  // tokens outside are clamped instead of tested (their results are not stored), and only the last
  // step of a row that is not a multiple of 128 columns is checked.
  // This lane's slots: [DEPTH][PIECES] of 16 bytes, 32 lanes side by side.
  const uint8_t* const slot0 = ls_smem + warp * (DEPTH * PIECES * 512) + lane * 16;
  const uint32_t slot0_u = (uint32_t)__cvta_generic_to_shared(slot0);
  const int ragged = p.d % 128 ? p.steps - 1 : -1;   // the step that ends before its last column
  const uint32_t* csrc[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
    csrc[i] = p.packed + (long long)min(row0 + 8 * i, p.m - 1) * p.wpr + (s0 * 4 + t4) * BITS;
  int ahead = s0, put = 0;   // the next step to copy, and its place
  auto copy_step = [&] {
    if (ahead < s1) {
      if (ahead != ragged) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          copy_codes<BITS, false>(p, csrc[i], 0, slot0_u + (put * PIECES + i) * 512);
      } else {
        const int left = p.wpr - (ahead * 4 + t4) * BITS;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          copy_codes<BITS, true>(p, csrc[i], left, slot0_u + (put * PIECES + i) * 512);
      }
#pragma unroll
      for (int i = 0; i < PIECES; ++i) csrc[i] += 4 * BITS;
    }
    ++ahead;
    put = (put + 1) % DEPTH;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) copy_step();
  // the grid of steps s .. s + 3: lane t of a row's four reads step s + t
  float sc[PIECES];
  uint32_t zs[PIECES];
  auto fetch_grid = [&](int s, float (&d)[PIECES], uint32_t (&zz)[PIECES]) {
    const int gi = p.group_steps ? min(s + t4, p.steps - 1) / p.group_steps : 0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const long long at = (long long)min(row0 + 8 * i, p.m - 1) * p.ng + gi;
      d[i] = p.scales[at];
      zz[i] = (uint32_t)p.zeros[at];
    }
  };
  auto zero_pairs = [&](uint32_t (&zz)[PIECES]) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      if (zz[i] > 15u) {
        bad = true;
        zz[i] = 0;
      }
      zz[i] = zero_pair<BF16>((int)zz[i]);
    }
  };
  if (s0 < s1) fetch_grid(s0, sc, zs);
  const uint4* xrow[NT];   // this lane's columns of its token of every tile
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    xrow[nt] = reinterpret_cast<const uint4*>((const uint16_t*)p.X + (long long)min(nt * 8 + g, p.T - 1) * p.d +
                                              s0 * 128 + t4 * 32);
  // The q-th 8 columns of step s, which is the one that `xrow` points to (q 4 and up: of the next one).
  // Loaded XA pieces ahead: three for 8 tokens, where an L2 round trip is as long as the work on two, one
  // where the registers hold more tokens.
  constexpr int XA = NT == 1 ? 3 : 1, XB = XA + 1;
  auto load_x = [&](int s, int q, uint4 (&x)[NT]) {
    const int at = small_x_piece(p.d, s, q, s1, ragged, t4);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) x[nt] = at >= 0 ? xrow[nt][at] : make_uint4(0, 0, 0, 0);
  };
  uint4 x[XB][NT];
  if (s0 < s1) {
#pragma unroll
    for (int q = 0; q < XA; ++q) load_x(s0, q, x[q]);
  }
  int get = 0;
  for (int sb = s0; sb < s1; sb += 4) {
    float sn[PIECES];
    uint32_t zn[PIECES];
    if (sb + 4 < s1) fetch_grid(sb + 4, sn, zn);
    zero_pairs(zs);
    const int se = min(sb + 4, s1);
    for (int s = sb; s < se; ++s) {
      copy_step();
      asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
      uint32_t cur[PIECES][BITS], zz[PIECES];
      float delta[PIECES];
      const int from = (lane & ~3) | (s - sb);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const uint8_t* slot = slot0 + (get * PIECES + i) * 512;
        if (BITS == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(slot);
          cur[i][0] = v.x;
          cur[i][1 % BITS] = v.y;
          cur[i][2 % BITS] = v.z;
          cur[i][3 % BITS] = v.w;
        } else {
#pragma unroll
          for (int w = 0; w < BITS; ++w) cur[i][w] = reinterpret_cast<const uint32_t*>(slot)[w];
        }
        delta[i] = __shfl_sync(0xffffffffu, sc[i], from);
        zz[i] = __shfl_sync(0xffffffffu, zs[i], from);
      }
      get = (get + 1) % DEPTH;
      float dd[LS_MT][NT][4] = {};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        load_x(s, q + XA, x[(q + XA) % XB]);
        if (q == 3) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) xrow[nt] += 16;
        }
        const uint4 (&xq)[NT] = x[q % XB];
        // Eight tokens: codes two apart make a pair (one byte permute each, from the even and the odd
        // nibbles), and the activations are put in the same order; with more tokens that would cost
        // more than the pairs in column order do.
        uint4 xs[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          xs[nt] = NT == 1 ? make_uint4(__byte_perm(xq[nt].x, xq[nt].y, 0x5410),
                                        __byte_perm(xq[nt].z, xq[nt].w, 0x5410),
                                        __byte_perm(xq[nt].x, xq[nt].y, 0x7632),
                                        __byte_perm(xq[nt].z, xq[nt].w, 0x7632))
                           : xq[nt];
#pragma unroll
        for (int mt = 0; mt < LS_MT; ++mt) {
          uint32_t u[4], v[4];
          if (NT == 1) {
            centered8_even_odd<BF16>(eight_codes<BITS>(cur[2 * mt], q), zz[2 * mt], u);
            centered8_even_odd<BF16>(eight_codes<BITS>(cur[2 * mt + 1], q), zz[2 * mt + 1], v);
          } else {
            centered8<BF16>(eight_codes<BITS>(cur[2 * mt], q), zz[2 * mt], u);
            centered8<BF16>(eight_codes<BITS>(cur[2 * mt + 1], q), zz[2 * mt + 1], v);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816<BF16>(dd[mt][nt], u[0], v[0], u[1], v[1], xs[nt].x, xs[nt].y);
            mma16816<BF16>(dd[mt][nt], u[2], v[2], u[3], v[3], xs[nt].z, xs[nt].w);
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < LS_MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[mt][nt][i] = fmaf(delta[2 * mt + (i >> 1)], dd[mt][nt][i], acc[mt][nt][i]);
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      sc[i] = sn[i];
      zs[i] = zn[i];
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();   // the ring's memory serves the join of the two column warps
  float (*joined)[32][LS_MT * NT * 4 + 1] = reinterpret_cast<float (*)[32][LS_MT * NT * 4 + 1]>(ls_smem);
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

int token_tiles(int T) { return (T + 7) / 8; }

template <int BITS>
int launch_small(Ctx* c, const SmallParams& p, int grid, bool bf) {
  const int nt = token_tiles(p.T);
#define GPTQ_SMALL(NT)                                                                              \
  do {                                                                                              \
    auto kernel = bf ? k_lora_small<BITS, NT, true> : k_lora_small<BITS, NT, false>;                \
    GPTQ_CUDA_CHECK(c, cudaFuncSetAttribute(                                                        \
                           kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ls_smem(NT)));       \
    GPTQ_LAUNCH(c, kernel, grid, LS_THREADS, ls_smem(NT), p, c->status);                                \
  } while (0)
  if (nt == 1) GPTQ_SMALL(1);
  else if (nt == 2) GPTQ_SMALL(2);
  else if (nt == 3) GPTQ_SMALL(3);
  else GPTQ_SMALL(4);
#undef GPTQ_SMALL
  return GPTQ_OK;
}

int small_chunks(int d) { return (d + LS_KC - 1) / LS_KC; }

// Splits of the columns so that the CTAs fill whole waves: the smallest waves x (steps of a warp + 2 for
// its start).  (Those of A X are short and run alongside; counting them in cost 24 tokens of 11008 x 4096
// 25 us instead of 21.)
int small_splits(int m, int d, int T, int num_sms, size_t max_floats) {
  const long long rows = (m + LS_ROWS - 1) / LS_ROWS, steps = (d + 127) / 128, slots = (long long)ls_ctas(token_tiles(T)) * num_sms;
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
  p.n = l.n; p.R = l.R;
  p.chunks = small_chunks(l.d);
  // at most about 128 CTAs of A X, so that they run beside the product's first wave
  const long long parts = (long long)p.chunks * l.T * l.R;
  p.ranks = (int)std::min<long long>(l.R, (parts + 1023) / 1024);
  const long long warps = (long long)p.chunks * l.T * ((l.R + p.ranks - 1) / p.ranks);
  const int splits = small_splits(l.m, l.d, l.T, c->num_sms, ws_floats - uf);
  p.per = (p.steps + splits - 1) / splits;
  p.row_ctas = (l.m + LS_ROWS - 1) / LS_ROWS;
  const int piece = l.bits == 4 ? 4 : 2;   // words per load of codes
  p.wide = p.wpr % piece == 0 && (reinterpret_cast<uintptr_t>(l.packed) & (piece * 4 - 1)) == 0;
  p.upart = ws;
  p.part = ws + uf;
  p.adapter = l.adapter;
  p.A = l.A;
  p.base_ctas = p.row_ctas * splits;
  const int grid = p.base_ctas + (int)((warps + 7) / 8);
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
