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
// All four kernels stream their arrays once and are bound by HBM. The
// conversions go through the fp32 significand (add and subtract 1.5 * 2^23, or
// 2^23 with the code's byte as the low bits), which keeps them on the FMA pipes:
// the conversion instructions run at an eighth of that rate and would bound the
// kernels that write more than they read.
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

// The scale of a block whose largest finite magnitude is amax.
__device__ __forceinline__ float block_scale(float amax) {
  const float t = fmaxf(__fdiv_rn(amax, 127.f), 0x1p-110f);
  return __uint_as_float((__float_as_uint(t) + 0xffffu) & 0xffff0000u);   // bf16, rounded up
}

// Four codes from four values: rint(v r) as the low byte of 1.5 * 2^23 + v r.
__device__ __forceinline__ uint32_t encode4(const float* v, float r) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float m = __fadd_rn(__fmul_rn(v[i], r), 12582912.f);
    c[i] = (fabsf(v[i]) < INFINITY) ? __float_as_uint(m) : 0x80u;
  }
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

// Four codes as floats (exact); -128 stays -128 here.
__device__ __forceinline__ void decode4(uint32_t w, float* v) {
  w ^= 0x80808080u;   // code + 128 in 0 .. 255
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | i)) - 8388736.f;   // 2^23 + 128
}

// Whether a word holds the code -128 (a byte 0x80).
__device__ __forceinline__ bool has_mark(uint32_t w) {
  return __vcmpeq4(w, 0x80808080u) != 0u;
}

// Eight restored values of two code words.
__device__ __forceinline__ void restore8(uint2 w, float s, float f[8]) {
  decode4(w.x, f);
  decode4(w.y, f + 4);
  const bool marked = has_mark(w.x) || has_mark(w.y);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= s;
  if (marked) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu;
      if (b == 0x80u) f[i] = __uint_as_float(0x7fc00000u);
    }
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

// Unit u of a row: 8 elements; 4 units share a scale. Rows hold nv units and
// are walked as `upr` = 4 ceil(nv / 4) so that the 4 lanes of a scale's block
// stay together (lanes past the row's end hold zeros).
__global__ void __launch_bounds__(kThreads)
pack_kernel(const uint4* __restrict__ x, long long total, int nv, int upr, uint2* __restrict__ q,
            uint16_t* __restrict__ s) {
  pdl_enter();
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  const long long span = (total + 31) / 32 * 32;   // whole warps reach the shuffles
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < span;
       i += stride) {
    const long long row = i / upr;
    const int u = static_cast<int>(i - row * upr);
    const bool live = i < total && u < nv;
    const long long at = row * nv + u;
    float f[8];
    unpack8(live ? ldg_nc_v4(x + at) : make_uint4(0u, 0u, 0u, 0u), f);
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float m = fabsf(f[k]);
      amax = m < INFINITY ? fmaxf(amax, m) : amax;
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float sc = block_scale(amax);
    const float r = __frcp_rn(sc);
    if (live) {
      q[at] = make_uint2(encode4(f, r), encode4(f + 4, r));
      if ((u & 3) == 0)
        s[row * (upr / 4) + u / 4] = static_cast<uint16_t>(__float_as_uint(sc) >> 16);
    }
  }
}

// xp[inv_perm[t K + j]] = restored row t, token-major: a row's codes are read
// once and its K copies written.
template <int KMAX>
__global__ void __launch_bounds__(kThreads)
dispatch8_kernel(const uint2* __restrict__ q, const uint16_t* __restrict__ s,
                 const int32_t* __restrict__ inv_perm, int K, int nv, int sb, long long total,
                 uint4* __restrict__ xp) {
  pdl_enter();
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  const long long rows = (total / nv) * K;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += stride) {
    const long long t = i / nv;
    const int c = static_cast<int>(i - t * nv);
    long long pos[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (j < K) pos[j] = inv_perm ? __ldg(inv_perm + t * K + j) : t * K + j;
    float f[8];
    restore8(ldg_nc_v2(q + i), ldg_scale(s + t * sb + (c >> 2)), f);
    const uint4 v = pack8(f);
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (j < K && index_ok(pos[j] >= 0 && pos[j] < rows)) stg_v4(xp + pos[j] * nv + c, v);
  }
}

// gu = bf16 of the restored [G | U], h = bf16(silu(G) U) from the restored
// values before that rounding. nv: units of one half of a row.
__global__ void __launch_bounds__(kThreads)
swiglu8_kernel(const uint2* __restrict__ q, const uint16_t* __restrict__ s, int nv, int sb,
               long long total, uint4* __restrict__ gu, uint4* __restrict__ h) {
  pdl_enter();
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += stride) {
    const long long m = i / nv;
    const int c = static_cast<int>(i - m * nv);
    const long long at = m * 2 * nv + c;
    const uint2 wg = ldg_nc_v2(q + at), wu = ldg_nc_v2(q + at + nv);
    const float sg = ldg_scale(s + m * sb + (c >> 2)), su = ldg_scale(s + m * sb + ((c + nv) >> 2));
    float g[8], u[8], o[8];
    restore8(wg, sg, g);
    restore8(wu, su, u);
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = __fdividef(g[k], 1.f + __expf(-g[k])) * u[k];
    stg_v4(gu + at, pack8(g));
    stg_v4(gu + at + nv, pack8(u));
    stg_v4(h + i, pack8(o));
  }
}

// The combine's gradient from y's codes: one warp per assignment a = t K + j,
// dy[p] = bf16(w dout) (the exact product rounded once), dw = <dout, y[p]> in
// a fixed order.
constexpr int kCbUnroll = 4;

__global__ void __launch_bounds__(kThreads)
combine_backward8_kernel(const uint4* __restrict__ dout, const uint2* __restrict__ q,
                         const uint16_t* __restrict__ s, const float* __restrict__ w,
                         const int32_t* __restrict__ inv_perm, long long TK, int K, int nv, int sb,
                         uint4* __restrict__ dy, float* __restrict__ dw) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long a = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
       a < TK; a += warps) {
    const uint4* drow = dout + a / K * nv;
    const int pa = __ldg(inv_perm + a);
    if (!index_ok(pa >= 0 && pa < TK)) {
      if (lane == 0) dw[a] = 0.f;
      continue;
    }
    const long long prow = static_cast<long long>(pa) * nv;
    const uint16_t* srow = s + static_cast<long long>(pa) * sb;
    const float wa = __ldg(w + a);
    float dot = 0.f;
    for (int c0 = lane; c0 < nv; c0 += 32 * kCbUnroll) {
      uint4 dv[kCbUnroll];
      uint2 yv[kCbUnroll];
      float sc[kCbUnroll];
#pragma unroll
      for (int u = 0; u < kCbUnroll; ++u) {
        const int c = c0 + 32 * u;
        if (c < nv) {
          dv[u] = ldg_nc_v4(drow + c);
          yv[u] = ldg_nc_v2(q + prow + c);
          sc[u] = ldg_scale(srow + (c >> 2));
        }
      }
#pragma unroll
      for (int u = 0; u < kCbUnroll; ++u) {
        const int c = c0 + 32 * u;
        if (c < nv) {
          float fd[8], fy[8], g[8];
          unpack8(dv[u], fd);
          restore8(yv[u], sc[u], fy);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            dot = fmaf(fd[k], fy[k], dot);
            g[k] = mul_bf16_exact(wa, fd[k]);
          }
          stg_v4(dy + prow + c, pack8(g));
        }
      }
    }
    const float sum = warp_sum(dot);
    if (lane == 0) dw[a] = sum;
  }
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
  const int nv = N / 8, upr = 4 * scale_blocks(nv);
  const long long total = static_cast<long long>(M) * upr;
  cudaStream_t st = as_stream(stream);
  ProfScope prof("ckpt8_pack", st);
  return launch_pdl(pack_kernel, grid_for(total, kThreads, 32), kThreads, 0, st, 1,
                    reinterpret_cast<const uint4*>(x), total, nv, upr, reinterpret_cast<uint2*>(q),
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
  const int nv = d / 8;
  const long long total = static_cast<long long>(T) * nv;
  cudaStream_t st = as_stream(stream);
  ProfScope prof("ckpt8_dispatch", st);
  const int grid = grid_for(total, kThreads, 32);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, kThreads, 0, st, 1, reinterpret_cast<const uint2*>(q),
                      reinterpret_cast<const uint16_t*>(s), inv_perm, K, nv, scale_blocks(nv),
                      total, reinterpret_cast<uint4*>(xp));
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
  const long long total = static_cast<long long>(M) * nv;
  cudaStream_t st = as_stream(stream);
  ProfScope prof("ckpt8_swiglu", st);
  return launch_pdl(swiglu8_kernel, grid_for(total, kThreads, 32), kThreads, 0, st, 1,
                    reinterpret_cast<const uint2*>(q), reinterpret_cast<const uint16_t*>(s), nv,
                    scale_blocks(2 * nv), total, reinterpret_cast<uint4*>(gu),
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
  const long long TK = static_cast<long long>(T) * K;
  if (TK > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  const int nv = d / 8;
  cudaStream_t st = as_stream(stream);
  ProfScope prof("ckpt8_combine_backward", st);
  return launch_pdl(combine_backward8_kernel, grid_for(TK, kThreads / 32, 48), kThreads, 0, st, 1,
                    reinterpret_cast<const uint4*>(dout), reinterpret_cast<const uint2*>(q),
                    reinterpret_cast<const uint16_t*>(s), topk_w, inv_perm, TK, K, nv,
                    scale_blocks(nv), reinterpret_cast<uint4*>(dy), dtopk_w);
}

namespace moe {
MOE_DEBUG_STATUS_READER(ckpt8)
}  // namespace moe
