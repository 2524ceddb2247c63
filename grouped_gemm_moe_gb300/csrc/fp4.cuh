// Microscaled 4-bit floats: the encoding steps shared by the quantizers and the fused
// quantization in the gate/up product's epilogue.
//
// Elements are E2M1 (0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives), two to a byte, the
// even one in the low half. Blocks along K share a scale:
//   block 16: an E4M3 scale s beside a 32-bit factor g of the row (activations) or the
//             matrix (weights); an element stands for q s g;
//   block 32: a power of two 2^X, kept as X + 127; an element stands for q 2^X.
// Ties go to the even code.
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {
namespace fp4 {

constexpr uint32_t kNanE4m3 = 0x7fu;   // the scale of a block that holds Inf or NaN, block 16
constexpr uint32_t kNanE8m0 = 0xffu;   // and block 32
constexpr int kMinRowExp = -100;       // smallest row factor: 2^-100

// 2^n for n in [-126, 127].
__device__ __forceinline__ float two_to(int n) { return __int_as_float((n + 127) << 23); }

// Exponent of the row factor for the row's largest |v| (finite, >= 0): the smallest n with
// max <= 2688 * 2^n (6 times 448), at least kMinRowExp. A power of two, so that s g and with
// it every rounding decision of the codes is exact; 2688 = 1.3125 * 2^11.
__device__ __forceinline__ int row_exponent(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = static_cast<int>(b >> 23) - 127;   // subnormals: -127, below the floor anyway
  const int n = e - 11 + ((b & 0x7fffffu) > 0x280000u ? 1 : 0);
  return n < kMinRowExp ? kMinRowExp : n;
}

// E4M3 byte of a block scale t >= 0 (nearest, ties to even, at most 448) and its value.
__device__ __forceinline__ uint32_t to_e4m3(float t) {
  return static_cast<uint32_t>(__nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ float from_e4m3(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
  return __half2float(__half(h));
}

// Exponent X of a block of 32 with the largest |v| `top` (finite): floor(log2 top) - 2, within
// what 2^X and 2^-X hold; -126 for an all-zero block.
__device__ __forceinline__ int block_exponent(float top) {
  const int X = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 2;
  return X < -126 ? -126 : X;   // at most 125
}

// Eight codes of four pairs of quotients (rounded to nearest, ties to even, at most 6).
__device__ __forceinline__ uint32_t to_e2m1x8(const float_pair p[4]) {
  const float2 a = split_pair(p[0]), b = split_pair(p[1]), c = split_pair(p[2]), d = split_pair(p[3]);
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return w;
}

// 1 / v to a few units of the last place (2^-126 <= v <= 2^126), 0 for v = 0.
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return v > 0.f ? r : 0.f;
}

// E4M3 byte of top / (6 g) for a bf16 value `top` and sixth = fl(1/6) / g, g a power of two.
// The product is off by at most 2^-23 of it; a quotient on a rounding border of E4M3 has five
// significant bits, every other is 2^-8 of it away from one. Rounding to 13 bits restores the
// former and moves none of the latter across.
constexpr float kSixth = 1.f / 6.f;
__device__ __forceinline__ uint32_t scale_byte(float top, float sixth) {
  return to_e4m3(__uint_as_float((__float_as_uint(top * sixth) + 0x400u) & ~0x7ffu));
}

// The quotients v / t of bf16 values v and t = s g (four significant bits) by v * (1/t): that
// product may miss a quotient that lies on a rounding border (a multiple of 1/4, at most 9 in
// size) by 2^-21 of it, while every other quotient is at least 2^-8 of it away from one.
// Adding and subtracting kSnap rounds to multiples of 2^-12, which restores the former and
// moves none of the latter across.
constexpr float kSnap = 2560.f;

// The codes of 16 bf16 values (as pairs) of a block with E4M3 scale byte sb under g.
__device__ __forceinline__ uint2 codes16(const float_pair v[8], uint32_t sb, float g) {
  const float f = reciprocal(from_e4m3(sb) * g);   // 2^-109 to 2^126, or 0
  const float_pair m = make_pair(f, f), c = make_pair(kSnap, kSnap), nc = make_pair(-kSnap, -kSnap);
  float_pair y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = add_pair(fma_pair(v[i], m, c), nc);
  return make_uint2(to_e2m1x8(y), to_e2m1x8(y + 4));
}

// The codes of 16 values of a block of 32 with exponent X (the quotients are exact).
__device__ __forceinline__ uint2 codes32(const float_pair v[8], int X) {
  const float f = two_to(-X);
  const float_pair m = make_pair(f, f);
  float_pair y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = mul_pair(v[i], m);
  return make_uint2(to_e2m1x8(y), to_e2m1x8(y + 4));
}

// Scales as the tensor cores read them: 512-byte atoms of 128 rows x 4 scales, row r's four in
// the word (r % 32) * 4 + r / 32; atoms ordered [row tile][K / (4 block)].
__device__ __forceinline__ int atom_word(int r) { return (r & 31) * 4 + ((r >> 5) & 3); }

// Row tiles of 128 (an upper bound of 2 * sum_e ceil(ceil(n_e / 128) / 2)): expert e's rows
// start at tile 2 P(e), P(e) = sum over earlier experts of ceil(ceil(n / 128) / 2).
inline long long row_tiles(long long M, int E) { return (M + 127) / 128 + 2LL * E; }
inline int k_atoms(int K, int block) { return (K + 4 * block - 1) / (4 * block); }
// Output rows of gate and of up that share a tile (see moe_fp4_pack_scales).
inline int gate_up_half(int I) { return I % 128 == 0 ? 128 : 64; }

}  // namespace fp4
}  // namespace moe
