// Device pieces shared by the kernels of the packed layer with low-rank adapters.
#pragma once
#include "kernels.h"

namespace gptq {

template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// The adapter of token t; an id outside [-1, n) is reported and counts as none.
__device__ __forceinline__ int adapter_of(const int32_t* adapter, int t, int n, DeviceStatus* st) {
  const int a = adapter[t];
  if (a < -1 || a >= n) {
    raise_error(st, GPTQ_ERR_ARG, t);
    return -1;
  }
  return a;
}

// Eight consecutive BITS-wide codes (the low 8 BITS bits of v) -> one 4-bit code per nibble, in
// order.  Each step doubles the number of fields and moves the upper half of each to its place.
template <int BITS> __device__ __forceinline__ uint32_t expand8(uint32_t v);
template <> __device__ __forceinline__ uint32_t expand8<4>(uint32_t v) { return v; }
template <> __device__ __forceinline__ uint32_t expand8<3>(uint32_t v) {
  v = (v & 0x00000FFFu) | ((v & 0x00FFF000u) << 4);
  v = (v & 0x003F003Fu) | ((v & 0x0FC00FC0u) << 2);
  return (v & 0x07070707u) | ((v & 0x38383838u) << 1);
}
template <> __device__ __forceinline__ uint32_t expand8<2>(uint32_t v) {
  v = (v & 0x000000FFu) | ((v & 0x0000FF00u) << 8);
  v = (v & 0x000F000Fu) | ((v & 0x00F000F0u) << 4);
  return (v & 0x03030303u) | ((v & 0x0C0C0C0Cu) << 2);
}
template <> __device__ __forceinline__ uint32_t expand8<1>(uint32_t v) {
  v = (v & 0x0000000Fu) | ((v & 0x000000F0u) << 12);
  v = (v & 0x00030003u) | ((v & 0x000C000Cu) << 6);
  return (v & 0x01010101u) | ((v & 0x02020202u) << 3);
}
// The q-th eight codes of a run of 32 (BITS words).
template <int BITS> __device__ __forceinline__ uint32_t eight_codes(const uint32_t (&w)[BITS], int q) {
  if (BITS == 4) return w[q];
  const int bit = 8 * BITS * q, i = bit >> 5, s = bit & 31;
  uint32_t v = w[i] >> s;
  if (s + 8 * BITS > 32) v |= w[i + 1 < BITS ? i + 1 : i] << (32 - s);
  return expand8<BITS>(v);
}

// (c - z) of the eight 4-bit codes of a word as four 16-bit pairs in column order, exactly: a code
// OR-ed into the mantissa of 128 (bf16) or 1024 (fp16) is 128 + c, and subtracting 128 + z (`zz`,
// in both halves) is exact for z in 0..15.
template <bool BF16>
__device__ __forceinline__ void centered8(uint32_t word, uint32_t zz, uint32_t (&out)[4]) {
  constexpr uint32_t magic = BF16 ? 0x43004300u : 0x64006400u;
  const uint32_t y = word >> 4;   // code 2p + 1 in the low nibble of byte p
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t t = (__byte_perm(word, y, p | (p << 4) | ((4 + p) << 8) | ((4 + p) << 12)) &
                        0x000F000Fu) | magic;
    if (BF16) {
      const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t),
                                       *reinterpret_cast<const __nv_bfloat162*>(&zz));
      out[p] = *reinterpret_cast<const uint32_t*>(&d);
    } else {
      const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&t),
                                *reinterpret_cast<const __half2*>(&zz));
      out[p] = *reinterpret_cast<const uint32_t*>(&d);
    }
  }
}
// The same in the order (0, 2), (4, 6), (1, 3), (5, 7): the even and the odd nibbles as bytes, to which
// one byte permute each adds the constant high byte.
template <bool BF16>
__device__ __forceinline__ void centered8_even_odd(uint32_t word, uint32_t zz, uint32_t (&out)[4]) {
  constexpr uint32_t high = BF16 ? 0x43434343u : 0x64646464u;
  const uint32_t even = word & 0x0F0F0F0Fu, odd = (word >> 4) & 0x0F0F0F0Fu;
  const uint32_t t[4] = {__byte_perm(even, high, 0x4140), __byte_perm(even, high, 0x4342),
                         __byte_perm(odd, high, 0x4140), __byte_perm(odd, high, 0x4342)};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if (BF16) {
      const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t[p]),
                                       *reinterpret_cast<const __nv_bfloat162*>(&zz));
      out[p] = *reinterpret_cast<const uint32_t*>(&d);
    } else {
      const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&t[p]),
                                *reinterpret_cast<const __half2*>(&zz));
      out[p] = *reinterpret_cast<const uint32_t*>(&d);
    }
  }
}
// 128 + z or 1024 + z in both halves: z in 0..15 sits in the mantissa's last bits (a bf16 in
// [128, 256) steps by 1, an fp16 in [1024, 2048) too).
template <bool BF16> __device__ __forceinline__ uint32_t zero_pair(int z) {
  return (BF16 ? 0x43004300u : 0x64006400u) | (uint32_t)z | ((uint32_t)z << 16);
}

// A 16-bit pair as two floats.
template <bool BF16> __device__ __forceinline__ float2 pair_f32(uint32_t v) {
  if (BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// D += A B: 16 x 8 x 16, 16-bit operands, fp32 sums.
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace gptq
