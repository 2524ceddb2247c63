// Activation checkpoints in 8 bits, and the backward steps that read them.
//
// A block kept for the backward pass holds x, [G | U] and y of its experts.
// Here they are kept as int8 codes with one bf16 scale per 32 consecutive
// elements of a row (8.5 bits an element), and the backward's own steps read the
// codes: the dispatch that makes the experts' X again, the SwiGLU that makes H
// again beside [G | U], and the combine's gradient, which needs y.
//
//   t = max(max |v| over the finite v of the block / 127, 2^-110)
//   s = t rounded up to bf16 (so no code passes 127), r = fl32(1 / s)
//   q = rint(fl32(v r)) in -127 .. 127;   q = -128 for a v that is not finite
//   restored: q s, exact in fp32; NaN for q = -128, so that an overflow in the
//   forward is still seen by whoever checks the gradients for it.
//
// Fixed point and not E4M3: a checkpoint is no operand of a tensor core, and
// within a block of 32 the uniform step of max / 127 leaves about a fifth of
// E4M3's error on values of one spread (0.5 % against 2.6 % of their RMS).
//
// All kernels stream their arrays once and are bound by HBM, with the logic pipe
// (which issues every second cycle) next. The conversions go through the fp32
// significand (add and subtract 1.5 * 2^23, or 2^23 with the code's byte as the
// low bits), which keeps them on the FMA pipes: the conversion instructions run at
// an eighth of that rate and would bound the kernels that write more than they read.
//
// Measured on one GB300, a call of both directions in turn (HBM floor at 6.8 TB/s):
//   rows 16384 x 2048 packed, dispatched to 6 experts each    82 us (80)
//   [G | U] 65536 x 1536 packed, restored with H             112 us (105)
//   combine gradient, 8191 tokens, K = 8, d = 2048            77 us (65): its warps wait for
//       loads first (2.3 of 6.8 cycles an instruction; DRAM 63 % busy), 93 registers a thread
//       leaving 27 % of the warps resident with one slot's loads ahead each
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

int grid_for(long long work, int per_block, int blocks_per_sm) {
  const long long b = (work + per_block - 1) / per_block;
  const long long cap = static_cast<long long>(num_sms()) * blocks_per_sm;
  return static_cast<int>(std::max(1LL, std::min(b, cap)));
}

// The scale of a block whose largest finite magnitude is amax (a bf16 value):
// the smallest bf16 s with 127 s >= amax, at least 2^-110. That is amax / 127
// rounded up: 127 s is exact in fp32, and the truncated product c below is the
// quotient's own bf16 neighbour below it, or the quotient where it is a bf16
// value (another quotient of 8-bit numbers is at least 2^-15 away from one,
// relatively, and the product's error is 2^-23).
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t c = __float_as_uint(amax * (1.f / 127.f)) & 0xffff0000u;
  const bool enough = 127.f * __uint_as_float(c) >= amax;
  return fmaxf(__uint_as_float(enough ? c : c + 0x10000u), 0x1p-110f);
}

// Four codes of four finite values: rint(v r) is the low byte of 1.5 * 2^23 + v r.
__device__ __forceinline__ uint32_t encode4(const float* v, float r) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __float_as_uint(__fadd_rn(__fmul_rn(v[i], r), 12582912.f));
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

// Puts the mark -128 in the place of the values that are not finite.
__device__ __forceinline__ uint32_t mark4(uint32_t codes, const float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!(fabsf(v[i]) < INFINITY)) codes = (codes & ~(0xffu << (8 * i))) | (0x80u << (8 * i));
  return codes;
}

// Codes as code + 128 in 0 .. 255; as floats (exact).
__device__ __forceinline__ uint32_t biased(uint32_t w) { return w ^ 0x80808080u; }
__device__ __forceinline__ void decode4(uint32_t b, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __uint_as_float(__byte_perm(b, 0x4b000000u, 0x7440 | i)) - 8388736.f;   // 2^23 + 128
}

// Codes i and i + 1 of a biased word as a pair of floats (exact).
__device__ __forceinline__ float_pair decode2(uint32_t b, int i) {
  const float_pair v = make_pair(__uint_as_float(__byte_perm(b, 0x4b000000u, 0x7440 | i)),
                                 __uint_as_float(__byte_perm(b, 0x4b000000u, 0x7441 | i)));
  return add_pair(v, make_pair(-8388736.f, -8388736.f));
}

// Nonzero if a biased word holds a mark (a zero byte).
__device__ __forceinline__ uint32_t marks(uint32_t b) { return (b - 0x01010101u) & ~b & 0x80808080u; }

// Eight restored values of two code words.
__device__ __forceinline__ void restore8(uint2 w, float s, float f[8]) {
  const uint32_t a = biased(w.x), b = biased(w.y);
  decode4(a, f);
  decode4(b, f + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= s;
  if (marks(a) | marks(b)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (((i < 4 ? a : b) >> (8 * (i & 3)) & 0xffu) == 0u) f[i] = __uint_as_float(0x7fc00000u);
  }
}

__device__ __forceinline__ uint2 ldg_nc_v2(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ float ldg_scale(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}

// Rows are walked in tiles of whole rows, at most kTileUnits units of 8 elements
// (one row where a row is longer), a block per tile. The row of a unit comes from
// a multiplication by the reciprocal of the units per row, exact because units
// of a tile and units per row are both below 2^16 (a 64-bit division per unit
// took a fifth of these kernels' time); a longer row is a tile of its own.
constexpr int kTileUnits = 2048;

struct Tiles {
  int per_row;        // units of a row
  int rows;           // rows of a tile
  unsigned magic;     // ceil(2^32 / per_row); 0 where per_row is 1 or a tile is one row
  long long total_rows, count;
};

// step: units that a block takes at once. The fewest rows whose units fill the
// block's steps to 15 in 16, or the best filling: short tiles keep the last wave short.
Tiles make_tiles(long long rows, int per_row, int step) {
  Tiles t;
  t.per_row = per_row;
  t.rows = 1;
  double best = 0.0;
  for (int r = 1; r == 1 || r * per_row <= kTileUnits; ++r) {
    const int units = r * per_row;
    const double fill = static_cast<double>(units) / ((units + step - 1) / step * step);
    if (fill > best) {
      best = fill;
      t.rows = r;
    }
    if (fill >= 0.9375) break;
  }
  t.magic = (per_row == 1 || t.rows == 1) ? 0u : 0xffffffffu / per_row + 1u;
  t.total_rows = rows;
  t.count = (rows + t.rows - 1) / t.rows;
  return t;
}

__device__ __forceinline__ void row_of(const Tiles& t, int unit, int& row, int& col) {
  row = t.magic ? static_cast<int>(__umulhi(unit, t.magic)) : t.rows == 1 ? 0 : unit;
  col = unit - row * t.per_row;
}

// A unit is 8 elements; 4 units share a scale. Rows hold nv units and are walked
// as per_row = 4 ceil(nv / 4) so that the 4 lanes of a scale's block stay together
// (lanes past the row's end hold zeros).
constexpr int kPackUnroll = 4;

__device__ __forceinline__ __nv_bfloat162 abs2(uint32_t v) {
  v &= 0x7fff7fffu;
  return *reinterpret_cast<__nv_bfloat162*>(&v);
}

// Codes and scales of a thread's kPackUnroll units. The four lanes of a block of 32
// call it together; put(i, codes, scale) stores unit i.
template <typename Put>
__device__ __forceinline__ void pack_units(const uint4 (&raw)[kPackUnroll], Put put) {
  // The magnitude's maximum over each block, in pairs, NaN and infinity kept.
  float amax[kPackUnroll];
#pragma unroll
  for (int i = 0; i < kPackUnroll; ++i) {
    __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(abs2(raw[i].x), abs2(raw[i].y)),
                                   __hmax2_nan(abs2(raw[i].z), abs2(raw[i].w)));
    m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
    amax[i] = __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
  }
  bool fine = true;
#pragma unroll
  for (int i = 0; i < kPackUnroll; ++i) fine = fine && amax[i] < INFINITY;
  if (!__all_sync(0xffffffffu, fine)) {   // rare: the maximum over the finite values instead
#pragma unroll
    for (int i = 0; i < kPackUnroll; ++i) {
      float f[8], top = 0.f;
      unpack8(raw[i], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fabsf(f[k]) < INFINITY ? fmaxf(top, fabsf(f[k])) : top;
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      amax[i] = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    }
  }
  // Lane l of a block's four works out the scale and reciprocal of unit l.
  static_assert(kPackUnroll == 4, "one unit per lane of a block");
  const int l = threadIdx.x & 3;
  const float mine = l == 0 ? amax[0] : l == 1 ? amax[1] : l == 2 ? amax[2] : amax[3];
  const float my_scale = block_scale(mine);
  const float my_inv = __frcp_rn(my_scale);
#pragma unroll
  for (int i = 0; i < kPackUnroll; ++i) {
    const float r = __shfl_sync(0xffffffffu, my_inv, i, 4);
    const float sc = __shfl_sync(0xffffffffu, my_scale, i, 4);
    float f[8];
    unpack8(raw[i], f);
    uint2 c = make_uint2(encode4(f, r), encode4(f + 4, r));
    if (!fine) c = make_uint2(mark4(c.x, f), mark4(c.y, f + 4));
    put(i, c, static_cast<uint16_t>(__float_as_uint(sc) >> 16));
  }
}

// Rows of whole blocks (N % 32 == 0): units, codes and scales are flat arrays, and
// only the last tile of a call has edges. The row arithmetic and edge checks of
// the other form cost it a quarter of its time, on the logic pipe that both wait for.
__global__ void __launch_bounds__(kThreads)
pack_flat_kernel(const uint4* __restrict__ x, long long total, uint2* __restrict__ q,
                 uint16_t* __restrict__ s) {
  pdl_enter();
  constexpr int kTile = kThreads * kPackUnroll;
  for (long long base = static_cast<long long>(blockIdx.x) * kTile; base < total;
       base += static_cast<long long>(gridDim.x) * kTile) {
    const uint4* xt = x + base + threadIdx.x;
    uint2* qt = q + base + threadIdx.x;
    uint16_t* st = s + base / 4 + threadIdx.x / 4;
    uint4 raw[kPackUnroll];
    const bool lead = (threadIdx.x & 3) == 0;
    if (base + kTile <= total) {
#pragma unroll
      for (int i = 0; i < kPackUnroll; ++i) raw[i] = ldg_nc_v4(xt + i * kThreads);
      pack_units(raw, [&](int i, uint2 c, uint16_t sc) {
        qt[i * kThreads] = c;
        if (lead) st[i * (kThreads / 4)] = sc;
      });
    } else {
      const int left = static_cast<int>(total - base) - static_cast<int>(threadIdx.x);
#pragma unroll
      for (int i = 0; i < kPackUnroll; ++i)
        raw[i] = i * kThreads < left ? ldg_nc_v4(xt + i * kThreads) : make_uint4(0u, 0u, 0u, 0u);
      pack_units(raw, [&](int i, uint2 c, uint16_t sc) {
        if (i * kThreads >= left) return;
        qt[i * kThreads] = c;
        if (lead) st[i * (kThreads / 4)] = sc;
      });
    }
  }
}

__global__ void __launch_bounds__(kThreads)
pack_kernel(const uint4* __restrict__ x, Tiles tl, int nv, uint2* __restrict__ q,
            uint16_t* __restrict__ s) {
  pdl_enter();
  for (long long tile = blockIdx.x; tile < tl.count; tile += gridDim.x) {
    const long long row0 = tile * tl.rows;
    const int rows = static_cast<int>(min(static_cast<long long>(tl.rows), tl.total_rows - row0));
    const int units = rows * tl.per_row;
    for (int u0 = threadIdx.x; u0 - static_cast<int>(threadIdx.x & 31) < units;
         u0 += kThreads * kPackUnroll) {   // whole warps
      uint4 raw[kPackUnroll];
      int row[kPackUnroll], col[kPackUnroll];
#pragma unroll
      for (int i = 0; i < kPackUnroll; ++i) {
        const int u = u0 + i * kThreads;
        row_of(tl, u, row[i], col[i]);
        if (u >= units || col[i] >= nv) row[i] = -1;
        raw[i] = row[i] >= 0 ? ldg_nc_v4(x + (row0 + row[i]) * nv + col[i])
                             : make_uint4(0u, 0u, 0u, 0u);
      }
      pack_units(raw, [&](int i, uint2 c, uint16_t sc) {
        if (row[i] < 0) return;
        q[(row0 + row[i]) * nv + col[i]] = c;
        if ((col[i] & 3) == 0) s[(row0 + row[i]) * (tl.per_row / 4) + col[i] / 4] = sc;
      });
    }
  }
}

// xp[inv_perm[t K + j]] = restored row t, token-major: a row's codes are read
// once and its K copies written.
template <int KMAX>
__global__ void __launch_bounds__(kThreads)
dispatch8_kernel(const uint2* __restrict__ q, const uint16_t* __restrict__ s,
                 const int32_t* __restrict__ inv_perm, int K, Tiles tl, int sb,
                 uint4* __restrict__ xp) {
  pdl_enter();
  const int nv = tl.per_row;
  const long long slots = tl.total_rows * K;
  for (long long tile = blockIdx.x; tile < tl.count; tile += gridDim.x) {
    const long long row0 = tile * tl.rows;
    const int rows = static_cast<int>(min(static_cast<long long>(tl.rows), tl.total_rows - row0));
    const int units = rows * nv;
    for (int u = threadIdx.x; u < units; u += kThreads) {
      int row, c;
      row_of(tl, u, row, c);
      const long long t = row0 + row;
      int32_t pos[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (j < K) pos[j] = inv_perm ? __ldg(inv_perm + t * K + j) : static_cast<int32_t>(t * K + j);
      float f[8];
      restore8(ldg_nc_v2(q + t * nv + c), ldg_scale(s + t * sb + (c >> 2)), f);
      const uint4 v = pack8(f);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (j < K && index_ok(pos[j] >= 0 && pos[j] < slots))
          stg_v4(xp + static_cast<long long>(pos[j]) * nv + c, v);
    }
  }
}

// gu = bf16 of the restored [G | U], h = bf16(silu(G) U) from the restored
// values before that rounding. Units of one half of a row.
constexpr int kSwigluUnroll = 2;

__global__ void __launch_bounds__(kThreads)
swiglu8_kernel(const uint2* __restrict__ q, const uint16_t* __restrict__ s, Tiles tl, int sb,
               uint4* __restrict__ gu, uint4* __restrict__ h) {
  pdl_enter();
  const int nv = tl.per_row;
  for (long long tile = blockIdx.x; tile < tl.count; tile += gridDim.x) {
    const long long row0 = tile * tl.rows;
    const int rows = static_cast<int>(min(static_cast<long long>(tl.rows), tl.total_rows - row0));
    const int units = rows * nv;
    for (int u0 = threadIdx.x; u0 < units; u0 += kThreads * kSwigluUnroll) {
      uint2 wg[kSwigluUnroll], wu[kSwigluUnroll];
      float sg[kSwigluUnroll], su[kSwigluUnroll];
      long long at[kSwigluUnroll];
#pragma unroll
      for (int i = 0; i < kSwigluUnroll; ++i) {
        if (u0 + i * kThreads >= units) break;
        int row, c;
        row_of(tl, u0 + i * kThreads, row, c);
        const long long m = row0 + row;
        at[i] = m * 2 * nv + c;
        wg[i] = ldg_nc_v2(q + at[i]);
        wu[i] = ldg_nc_v2(q + at[i] + nv);
        sg[i] = ldg_scale(s + m * sb + (c >> 2));
        su[i] = ldg_scale(s + m * sb + ((c + nv) >> 2));
      }
#pragma unroll
      for (int i = 0; i < kSwigluUnroll; ++i) {
        if (u0 + i * kThreads >= units) break;
        float g[8], u[8], o[8];
        restore8(wg[i], sg[i], g);
        restore8(wu[i], su[i], u);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = __fdividef(g[k], 1.f + __expf(-g[k])) * u[k];
        stg_v4(gu + at[i], pack8(g));
        stg_v4(gu + at[i] + nv, pack8(u));
        stg_v4(h + row0 * nv + u0 + i * kThreads, pack8(o));
      }
    }
  }
}

// The combine's gradient from y's codes: one warp per token, its dout in
// registers (a chunk of 32 x kCbVecs vectors at a time) while the K slots' codes
// stream past, the next slot's loads ahead of this one's use. dy[p] = bf16(w
// dout), the exact product rounded once; dw = <dout, y[p]> in a fixed order,
// lane j keeping slot j's sum.
constexpr int kCbVecs = 4;
constexpr int kCbWarps = 4;

__global__ void __launch_bounds__(kCbWarps * 32)
combine_backward8_kernel(const uint4* __restrict__ dout, const uint2* __restrict__ q,
                         const uint16_t* __restrict__ s, const float* __restrict__ w,
                         const int32_t* __restrict__ inv_perm, long long T, int K, int nv, int sb,
                         uint4* __restrict__ dy, float* __restrict__ dw) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kCbWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  // lane j: slot j's row and weight
  int my_row = lane < K ? __ldg(inv_perm + t * K + lane) : 0;
  const float my_w = lane < K ? __ldg(w + t * K + lane) : 0.f;
  if (!index_ok(my_row >= 0 && my_row < T * K)) my_row = -1;   // debug builds: skipped, dw 0
  float my_dot = 0.f;
  for (int c0 = lane; c0 - lane < nv; c0 += 32 * kCbVecs) {
    uint2 yv[kCbVecs];
    uint16_t sv[kCbVecs];
    auto load = [&](int j) {
      const long long row = __shfl_sync(0xffffffffu, my_row, j);
#pragma unroll
      for (int u = 0; u < kCbVecs; ++u) {
        const int c = c0 + 32 * u;
        yv[u] = make_uint2(0u, 0u);   // codes of 0
        sv[u] = 0;
        if (c < nv && row >= 0) {
          yv[u] = ldg_nc_v2(q + row * nv + c);
          sv[u] = __ldg(s + row * sb + (c >> 2));
        }
      }
    };
    load(0);
    float fd[kCbVecs][8];
#pragma unroll
    for (int u = 0; u < kCbVecs; ++u) {
      const int c = c0 + 32 * u;
      unpack8(c < nv ? ldg_nc_v4(dout + t * nv + c) : make_uint4(0u, 0u, 0u, 0u), fd[u]);
    }
    for (int j = 0; j < K; ++j) {
      uint2 y[kCbVecs];
      float sc[kCbVecs];
#pragma unroll
      for (int u = 0; u < kCbVecs; ++u) {
        y[u] = yv[u];
        sc[u] = __uint_as_float(static_cast<uint32_t>(sv[u]) << 16);
      }
      if (j + 1 < K) load(j + 1);
      const long long row = __shfl_sync(0xffffffffu, my_row, j);
      const float wj = __shfl_sync(0xffffffffu, my_w, j);
      float dot = 0.f;
#pragma unroll
      for (int u = 0; u < kCbVecs; ++u) {
        const int c = c0 + 32 * u;
        float g[8];
        const uint32_t b0 = biased(y[u].x), b1 = biased(y[u].y);
        float_pair part2 = make_pair(0.f, 0.f);   // over the unit's codes; their one scale
#pragma unroll                                     // multiplies the sum
        for (int k = 0; k < 8; k += 2) {
          part2 = fma_pair(make_pair(fd[u][k], fd[u][k + 1]), decode2(k < 4 ? b0 : b1, k & 3), part2);
          g[k] = mul_bf16_exact(wj, fd[u][k]);
          g[k + 1] = mul_bf16_exact(wj, fd[u][k + 1]);
        }
        const float2 both = split_pair(part2);
        float part = both.x + both.y;
        if (marks(b0) | marks(b1)) part = __uint_as_float(0x7fc00000u);
        dot = fmaf(sc[u], part, dot);
        if (c < nv && row >= 0) stg_v4(dy + row * nv + c, pack8(g));
      }
      dot = warp_sum(dot);
      if (lane == j) my_dot += dot;
    }
  }
  if (lane < K) dw[t * K + lane] = my_dot;
}

int scale_blocks(int nv) { return (nv + 3) / 4; }

}  // namespace
}  // namespace moe

extern "C" int moe_ckpt8_pack(const moe_bf16* x, int M, int N, int8_t* q, moe_bf16* s,
                              void* stream) {
  using namespace moe;
  if (M < 0 || N < 8 || N % 8) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!x || !q || !s) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return MOE_ERR_MISALIGNED;
  const int nv = N / 8;
  cudaStream_t st = as_stream(stream);
  ProfScope prof("ckpt8_pack", st);
  if (N % 32 == 0) {
    const long long total = static_cast<long long>(M) * nv;
    return launch_pdl(pack_flat_kernel, grid_for(total, kThreads * kPackUnroll, 128), kThreads, 0, st,
                      1, reinterpret_cast<const uint4*>(x), total, reinterpret_cast<uint2*>(q),
                      reinterpret_cast<uint16_t*>(s));
  }
  const Tiles tl = make_tiles(M, 4 * scale_blocks(nv), kThreads * kPackUnroll);
  return launch_pdl(pack_kernel, grid_for(tl.count, 1, 128), kThreads, 0, st, 1,
                    reinterpret_cast<const uint4*>(x), tl, nv, reinterpret_cast<uint2*>(q),
                    reinterpret_cast<uint16_t*>(s));
}

extern "C" int moe_ckpt8_dispatch(const int8_t* q, const moe_bf16* s, const int32_t* inv_perm,
                                  int T, int K, int d, moe_bf16* xp, void* stream) {
  using namespace moe;
  if (T < 0 || K < 1 || K > 32 || d < 8 || d % 8) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!q || !s || !xp) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(s) || !aligned16(inv_perm) || !aligned16(xp))
    return MOE_ERR_MISALIGNED;
  if (static_cast<long long>(T) * K > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  const int nv = d / 8;
  const Tiles tl = make_tiles(T, nv, kThreads);
  cudaStream_t st = as_stream(stream);
  ProfScope prof("ckpt8_dispatch", st);
  const int grid = grid_for(tl.count, 1, 128);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, kThreads, 0, st, 1, reinterpret_cast<const uint2*>(q),
                      reinterpret_cast<const uint16_t*>(s), inv_perm, K, tl, scale_blocks(nv),
                      reinterpret_cast<uint4*>(xp));
  };
  if (K <= 2) return go(dispatch8_kernel<2>);
  if (K <= 4) return go(dispatch8_kernel<4>);
  if (K <= 8) return go(dispatch8_kernel<8>);
  if (K <= 16) return go(dispatch8_kernel<16>);
  return go(dispatch8_kernel<32>);
}

extern "C" int moe_ckpt8_swiglu(const int8_t* q, const moe_bf16* s, int M, int I, moe_bf16* gu,
                                moe_bf16* h, void* stream) {
  using namespace moe;
  if (M < 0 || I < 8 || I % 8) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!q || !s || !gu || !h) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(s) || !aligned16(gu) || !aligned16(h)) return MOE_ERR_MISALIGNED;
  const int nv = I / 8;
  const Tiles tl = make_tiles(M, nv, kThreads * kSwigluUnroll);
  cudaStream_t st = as_stream(stream);
  ProfScope prof("ckpt8_swiglu", st);
  return launch_pdl(swiglu8_kernel, grid_for(tl.count, 1, 128), kThreads, 0, st, 1,
                    reinterpret_cast<const uint2*>(q), reinterpret_cast<const uint16_t*>(s), tl,
                    scale_blocks(2 * nv), reinterpret_cast<uint4*>(gu),
                    reinterpret_cast<uint4*>(h));
}

extern "C" int moe_ckpt8_combine_backward(const moe_bf16* dout, const int8_t* q, const moe_bf16* s,
                                          const float* topk_w, const int32_t* inv_perm, int T,
                                          int K, int d, moe_bf16* dy, float* dtopk_w,
                                          void* stream) {
  using namespace moe;
  if (T < 0 || K < 1 || K > 32 || d < 8 || d % 8) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!dout || !q || !s || !topk_w || !inv_perm || !dy || !dtopk_w) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {dout, q, s, topk_w, inv_perm, dy, dtopk_w};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_MISALIGNED;
  if (static_cast<long long>(T) * K > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  const int nv = d / 8;
  cudaStream_t st = as_stream(stream);
  ProfScope prof("ckpt8_combine_backward", st);
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(T) + kCbWarps - 1) / kCbWarps);
  return launch_pdl(combine_backward8_kernel, grid, kCbWarps * 32, 0, st, 1,
                    reinterpret_cast<const uint4*>(dout), reinterpret_cast<const uint2*>(q),
                    reinterpret_cast<const uint16_t*>(s), topk_w, inv_perm,
                    static_cast<long long>(T), K, nv, scale_blocks(nv),
                    reinterpret_cast<uint4*>(dy), dtopk_w);
}

namespace moe {
MOE_DEBUG_STATUS_READER(ckpt8)
}  // namespace moe
