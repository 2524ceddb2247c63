// Microscaled 4-bit floats: quantizing activations while they are dispatched, reading them
// back, quantizing weights and laying their scales out for the tensor cores.
//
// The format and its rounding are stated in fp4.cuh. For a row of x (bf16):
//   block 16:  g = 2^n, n the smallest with max|x| <= 2688 g (n >= -100);
//              s = E4M3(max_b|x| / (6 g)),  q = E2M1(x / (s g)) (0 where s is 0);
//              a row with Inf or NaN keeps g = NaN, so that its products are NaN;
//   block 32:  X = floor(log2 max_b|x|) - 2 within [-126, 125], q = E2M1(x 2^-X), at most 6;
//              a block with Inf or NaN keeps the scale byte 255, which reads as NaN.
#include "fp4.cuh"

namespace moe {
namespace fp4 {
namespace {

constexpr int kThreads = 256;

// Per-expert first row tile into s_tile[0 .. E] from s_off, by the first warp.
__device__ __forceinline__ void tile_prefix(const int* s_off, int* s_tile, int E) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int base = 0; base <= E; base += 32) {
    const int i = base + lane;
    const int v = (i < E) ? 2 * (((s_off[i + 1] - s_off[i] + 127) / 128 + 1) / 2) : 0;
    int y = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += t;
    }
    if (i <= E) s_tile[i] = carry + y - v;
    carry += __shfl_sync(0xffffffffu, y, 31);
  }
}

// (row tile, row in it) of expert-ordered row p; a row past the last expert: tile -1.
__device__ __forceinline__ int2 place_of(int p, const int* s_off, const int* s_tile, int E) {
  int lo = 0, hi = E - 1;   // largest e with off[e] <= p
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_off[mid] <= p) lo = mid; else hi = mid - 1;
  }
  const int local = p - s_off[lo];
  return p < s_off[E] ? make_int2(s_tile[lo] + local / 128, local & 127) : make_int2(-1, 0);
}

// Running maximum of |bf16| bits (Inf 0x7f80, NaN above it) of a word's two halves, each in its
// own half, and the larger of the two as the bits of a float.
__device__ __forceinline__ uint32_t top2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t top_of(uint32_t m) { return max(m & 0xffff0000u, m << 16); }

// 32 bytes: one access where the address allows it (half as many requests), else two.
__device__ __forceinline__ void load32(const uint4* src, bool wide, uint4& a, uint4& b) {
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(src));
  } else {
    a = ldg_nc_v4(src);
    b = ldg_nc_v4(src + 1);
  }
}
__device__ __forceinline__ void store32(uint4* dst, bool wide, const uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ bool aligned32(const void* p) {   // rows are whole multiples of 128 bytes
  return (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
}

// The largest |v| bits of a unit of 16 elements.
__device__ __forceinline__ uint32_t unit_top(const uint4& a, const uint4& b) {
  const uint32_t m = top2(top2(top2(top2(0u, a.x), a.y), a.z), a.w);
  return top_of(top2(top2(top2(top2(m, b.x), b.y), b.z), b.w));
}

// Codes of a unit and, in the first lane of each scale word's units, the word: four
// consecutive units' scales (block 16) or eight's (block 32, two units to a scale; past the
// row's end threads without a unit give the byte of zeros). g, sixth: the row's factor and
// fl(1/6) / g, fine: the row is finite (block 16). Every lane of the warp calls it.
template <int BLOCK>
__device__ __forceinline__ uint2 encode_unit(const uint4& a, const uint4& b, uint32_t top, float g,
                                             float sixth, bool fine, uint32_t* word) {
  float_pair v[8];
  unpack8(a, v);
  unpack8(b, v + 4);
  uint32_t byte;
  uint2 code;
  if constexpr (BLOCK == 16) {
    byte = fine ? scale_byte(__uint_as_float(top), sixth) : 0u;
    code = fine ? codes16(v, byte, g) : make_uint2(0u, 0u);
  } else {
    const uint32_t both = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const bool ok = both < 0x7f800000u;
    const int X = block_exponent(__uint_as_float(ok ? both : 0u));
    byte = ok ? static_cast<uint32_t>(X + 127) : kNanE8m0;
    code = ok ? codes32(v, X) : make_uint2(0u, 0u);
  }
  constexpr int kStep = BLOCK / 16;
  const uint32_t b1 = __shfl_down_sync(0xffffffffu, byte, kStep);
  const uint32_t b2 = __shfl_down_sync(0xffffffffu, byte, 2 * kStep);
  const uint32_t b3 = __shfl_down_sync(0xffffffffu, byte, 3 * kStep);
  *word = byte | (b1 << 8) | (b2 << 16) | (b3 << 24);
  return code;
}

// Each token's row is quantized once and written to its K rows in expert order (inv_perm
// null: to its own row). HBM-bound: 2 bytes read and K (1/2 + 1/block) written an element.
// Rows of up to 192 units: a warp a row, its elements in registers between the row's maximum
// and the codes (lane l takes units l, l + 32, ...: 32 bytes in, 8 bytes out, without gaps), no
// barrier between rows; warps stay for many rows, so that the expert table is made once a
// CTA. The lanes look the K destinations up side by side, and the scale words, each in a
// sector of its own, are spread over the lanes before they are stored. Those words are what
// keeps wide copies from HBM speed: 32768 x 4096 to 8 experts takes 191 us (floor 129), 134
// without them. Block 16, a warp a row against a CTA of 128 threads a row: 65536 rows to one, 2112 columns
// 72 and 117 us, 2560 79 and 117, 2944 90 and 119, 3584 110 and 122; 16384 to 6, 48 and 55, 56 and
// 56, 63 and 60, 74 and 70; to 8, 59 and 62, 71 and 66, 84 and 74, 94 and 87 (32768 rows of 4096
// to 8: 220 and 191). The crossing lies lower the more copies a row has; 192 units stand for all.
// 98304 rows of 1408 to one: 77 us, 64 threads a row 93.
template <int BLOCK, int BPT>
__global__ void __launch_bounds__(kThreads)
quantize_warp_rows_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ inv_perm,
                          const int32_t* __restrict__ offsets, int E, int T, int K, int M, int d,
                          uint2* __restrict__ q, uint32_t* __restrict__ sf,
                          float* __restrict__ row_scale) {
  extern __shared__ int sm[];
  int* s_off = sm;              // [E + 1]
  int* s_tile = s_off + E + 1;  // [E + 1]
  pdl_enter();
  for (int e = threadIdx.x; e <= E; e += kThreads) s_off[e] = __ldg(offsets + e);
  __syncthreads();
  if (!offsets_in_order(s_off, E, M)) return;   // where a row's scales are follows from them
  if (threadIdx.x < 32) tile_prefix(s_off, s_tile, E);
  __syncthreads();
  constexpr int kPer = BLOCK / 4;              // units of a scale word
  constexpr int kWords = 32 / kPer;            // words of 32 units
  constexpr int kHeld = (BPT * kWords + 31) / 32;
  const bool wide = aligned32(x);
  const int lane = threadIdx.x & 31;
  const int units = d / 16;
  const int ka = (units + kPer - 1) / kPer;
  const unsigned warps = gridDim.x * (kThreads / 32);
  for (unsigned t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < static_cast<unsigned>(T);
       t += warps) {
    uint4 a[BPT], b[BPT];
    const uint4* src = x + static_cast<size_t>(t) * units * 2;
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      const int u = i * 32 + lane;
      a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
      if (u < units) {
        load32(src + 2 * u, wide, a[i], b[i]);
      }
    }
    int p = -1;
    int2 pl = make_int2(-1, 0);
    if (lane < K) {
      p = inv_perm ? __ldg(inv_perm + static_cast<size_t>(t) * K + lane) : static_cast<int>(t);
      if (!index_ok(p >= 0 && p < M)) p = -1;
      if (p >= 0) pl = place_of(p, s_off, s_tile, E);
    }
    uint32_t top[BPT], row_top = 0;
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      top[i] = unit_top(a[i], b[i]);
      row_top = max(row_top, top[i]);
    }
    float g = 1.f, sixth = kSixth;
    bool fine = true;
    if constexpr (BLOCK == 16) {
      row_top = __reduce_max_sync(0xffffffffu, row_top);
      fine = row_top < 0x7f800000u;
      const int n = row_exponent(__uint_as_float(fine ? row_top : 0u));
      g = two_to(n);
      sixth = kSixth * two_to(-n);
      if (p >= 0) row_scale[p] = fine ? g : __uint_as_float(0x7fc00000u);
    }
    uint2 code[BPT];
    uint32_t held[kHeld];   // lane l: words l, l + 32, ...
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      uint32_t word;
      code[i] = encode_unit<BLOCK>(a[i], b[i], top[i], g, sixth, fine, &word);
      const uint32_t w = __shfl_sync(0xffffffffu, word, (lane % kWords) * kPer);
      if ((i * kWords) % 32 == 0 || lane / kWords == (i * kWords) % 32 / kWords)
        held[i * kWords / 32] = w;
    }
    for (int j = 0; j < K; ++j) {
      const int pj = __shfl_sync(0xffffffffu, p, j);
      const int tile = __shfl_sync(0xffffffffu, pl.x, j), row = __shfl_sync(0xffffffffu, pl.y, j);
      if (pj < 0) continue;
      uint2* dst = q + static_cast<size_t>(pj) * units;
#pragma unroll
      for (int i = 0; i < BPT; ++i)
        if (i * 32 + lane < units) dst[i * 32 + lane] = code[i];
      if (tile >= 0) {
        uint32_t* ds = sf + static_cast<size_t>(tile) * ka * 128 + atom_word(row);
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
          if (i * 32 + lane < ka) ds[static_cast<size_t>(i * 32 + lane) * 128] = held[i];
      }
    }
  }
}

// Wider rows: TPR threads a row, BPT units each, the maximum joined in shared memory.
template <int BLOCK, int TPR, int BPT>
__global__ void __launch_bounds__(kThreads)
quantize_rows_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ inv_perm,
                     const int32_t* __restrict__ offsets, int E, int T, int K, int M, int d,
                     uint2* __restrict__ q, uint32_t* __restrict__ sf, float* __restrict__ row_scale) {
  constexpr int kRows = kThreads / TPR;
  extern __shared__ int sm[];
  int* s_off = sm;              // [E + 1]
  int* s_tile = s_off + E + 1;  // [E + 1]
  __shared__ int s_pos[kRows][32];
  __shared__ int2 s_place[kRows][32];
  __shared__ uint32_t s_top[kThreads / 32];
  pdl_enter();
  const int units = d / 16;
  const int sub = threadIdx.x / TPR, lane_r = threadIdx.x % TPR;
  const bool wide = aligned32(x);
  const unsigned t = blockIdx.x * kRows + sub;
  const bool live = t < static_cast<unsigned>(T);
  uint4 a[BPT], b[BPT];
#pragma unroll
  for (int i = 0; i < BPT; ++i) {
    const int u = i * TPR + lane_r;
    a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
    if (live && u < units) {
      const uint4* src = x + (static_cast<size_t>(t) * units + u) * 2;
      load32(src, wide, a[i], b[i]);
    }
  }
  for (int e = threadIdx.x; e <= E; e += kThreads) s_off[e] = __ldg(offsets + e);
  __syncthreads();
  if (!offsets_in_order(s_off, E, M)) return;   // where a row's scales are follows from them
  if (threadIdx.x < 32) tile_prefix(s_off, s_tile, E);
  // the row's largest element, for its factor
  uint32_t top[BPT];
  uint32_t row_top = 0;
#pragma unroll
  for (int i = 0; i < BPT; ++i) {
    top[i] = unit_top(a[i], b[i]);
    row_top = max(row_top, top[i]);
  }
  if constexpr (BLOCK == 16) {
    row_top = __reduce_max_sync(0xffffffffu, row_top);
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = row_top;
  }
  __syncthreads();
  // where the row's copies go
  for (int j = threadIdx.x; j < kRows * K; j += kThreads) {
    const int r = j / K, slot = j - r * K;
    const unsigned tt = blockIdx.x * kRows + r;
    int p = -1;
    if (tt < static_cast<unsigned>(T)) {
      p = inv_perm ? __ldg(inv_perm + static_cast<size_t>(tt) * K + slot) : static_cast<int>(tt);
      if (!index_ok(p >= 0 && p < M)) p = -1;
    }
    s_pos[r][slot] = p;
    s_place[r][slot] = p >= 0 ? place_of(p, s_off, s_tile, E) : make_int2(-1, 0);
  }
  float g = 1.f, sixth = kSixth;
  bool fine = true;
  if constexpr (BLOCK == 16) {
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) row_top = max(row_top, s_top[sub * (TPR / 32) + w]);
    fine = row_top < 0x7f800000u;
    const int n = row_exponent(__uint_as_float(fine ? row_top : 0u));
    g = two_to(n);
    sixth = kSixth * two_to(-n);
  }
  __syncthreads();
  uint2 code[BPT];
  uint32_t word[BPT];
#pragma unroll
  for (int i = 0; i < BPT; ++i) code[i] = encode_unit<BLOCK>(a[i], b[i], top[i], g, sixth, fine, &word[i]);
  constexpr int kPer = BLOCK / 4;   // units of a scale word
  const int ka = (units + kPer - 1) / kPer;
  for (int j = 0; j < K; ++j) {
    const int p = s_pos[sub][j];
    const int2 pl = s_place[sub][j];
    if (p < 0) continue;
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      const int u = i * TPR + lane_r;
      if (u >= units) break;
      q[static_cast<size_t>(p) * units + u] = code[i];
      if (pl.x >= 0 && (u & (kPer - 1)) == 0)
        sf[(static_cast<size_t>(pl.x) * ka + u / kPer) * 128 + atom_word(pl.y)] = word[i];
    }
    if (BLOCK == 16 && lane_r == 0)
      row_scale[p] = fine ? g : __uint_as_float(0x7fc00000u);
  }
}

// Rows back in bf16, a warp a row: lanes take units of 16 elements (8 bytes of codes, one
// scale byte) side by side.
template <int BLOCK>
__global__ void __launch_bounds__(kThreads)
dequantize_rows_kernel(const uint2* __restrict__ q, const uint32_t* __restrict__ sf,
                       const float* __restrict__ row_scale, const int32_t* __restrict__ offsets,
                       int E, int M, int d, uint4* __restrict__ out) {
  extern __shared__ int sm[];
  int* s_off = sm;
  int* s_tile = s_off + E + 1;
  pdl_enter();
  for (int e = threadIdx.x; e <= E; e += kThreads) s_off[e] = __ldg(offsets + e);
  __syncthreads();
  if (!offsets_in_order(s_off, E, M)) return;   // where a row's scales are follows from them
  if (threadIdx.x < 32) tile_prefix(s_off, s_tile, E);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int units = d / 16;
  constexpr int kPer = BLOCK / 4;
  constexpr int kAhead = 4;   // units a lane has in flight
  const bool wide = aligned32(out);
  const int ka = (units + kPer - 1) / kPer;
  const unsigned rows = static_cast<unsigned>(min(s_off[E], M));
  const unsigned warps = gridDim.x * (kThreads / 32);
  for (unsigned p = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); p < rows; p += warps) {
    const int2 pl = place_of(static_cast<int>(p), s_off, s_tile, E);
    const uint32_t* words = sf + static_cast<size_t>(pl.x) * ka * 128 + atom_word(pl.y);
    const uint2* src = q + static_cast<size_t>(p) * units;
    uint4* dst = out + static_cast<size_t>(p) * units * 2;
    const float g = BLOCK == 16 ? __ldg(row_scale + p) : 1.f;
    for (int u0 = lane; u0 < units; u0 += 32 * kAhead) {
      uint2 c[kAhead];
      uint32_t w[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int u = u0 + 32 * i;
        if (u < units) {
          c[i] = __ldg(src + u);
          w[i] = __ldg(words + static_cast<size_t>(u / kPer) * 128);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int u = u0 + 32 * i;
        if (u >= units) break;
        float f;
        if constexpr (BLOCK == 16) {
          f = from_e4m3((w[i] >> (8 * (u & 3))) & 0xffu) * g;
        } else {
          const uint32_t byte = (w[i] >> (8 * ((u >> 1) & 3))) & 0xffu;
          f = byte == kNanE8m0 ? __uint_as_float(0x7fc00000u) : two_to(static_cast<int>(byte) - 127);
        }
        uint32_t o[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const uint32_t byte = ((h < 4 ? c[i].x : c[i].y) >> (8 * (h & 3))) & 0xffu;
          const __half2_raw hr =
              __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
          const float2 v = __half22float2(__half2(hr));
          o[h] = pack_bf16(v.x * f, v.y * f);
        }
        store32(dst + 2 * u, wide, o);
      }
    }
  }
}

// Largest |w| of each expert's matrix, as bits (max is order-free, so the result is the same
// on every run). scale [E] starts at zero.
__global__ void __launch_bounds__(kThreads)
weight_top_kernel(const uint4* __restrict__ w, long long vecs, uint32_t* __restrict__ top) {
  pdl_enter();
  const uint4* base = w + static_cast<size_t>(blockIdx.y) * vecs;
  uint32_t m = 0;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < vecs;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const uint4 v = ldg_nc_v4(base + i);
    m = top2(top2(top2(top2(m, v.x), v.y), v.z), v.w);
  }
  m = __reduce_max_sync(0xffffffffu, top_of(m));
  if ((threadIdx.x & 31) == 0 && m) atomicMax(top + blockIdx.y, m);
}

__global__ void weight_scale_kernel(float* __restrict__ scale, int E) {
  pdl_enter();
  const int e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= E) return;
  const uint32_t top = __float_as_uint(scale[e]);
  scale[e] = top < 0x7f800000u ? two_to(row_exponent(__uint_as_float(top)))
                               : __uint_as_float(0x7fc00000u);
}

// w [E, K, N] bf16 (N contiguous) -> codes [E, N, K/2], scales [E, N, K/BLOCK]. A thread takes
// one output row and 64 K: a warp reads 64 contiguous bytes of each K row and writes 32 bytes
// of codes an output.
template <int BLOCK>
__global__ void __launch_bounds__(128)
quantize_weights_kernel(const __nv_bfloat16* __restrict__ w, int K, int N,
                        const float* __restrict__ scale, uint4* __restrict__ codes,
                        uint8_t* __restrict__ scales) {
  pdl_enter();
  const int nt = (N + 127) / 128, kt = K / 64;
  long long b = blockIdx.x;
  const int n = static_cast<int>(b % nt) * 128 + threadIdx.x;
  b /= nt;
  const int k64 = static_cast<int>(b % kt);
  const int e = static_cast<int>(b / kt);
  if (n >= N) return;
  const __nv_bfloat16* src = w + (static_cast<size_t>(e) * K + static_cast<size_t>(k64) * 64) * N + n;
  float g = 1.f, sixth = kSixth;
  bool fine = true;
  if constexpr (BLOCK == 16) {
    g = scale[e];
    fine = g == g;
    sixth = kSixth * reciprocal(g);   // a power of two: exact
  }
  uint2 c[4];
  uint32_t word = 0, pair_top = 0;
  float_pair prev[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[16];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      f[j] = __bfloat162float(src[static_cast<size_t>(16 * i + j) * N]);
      m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    }
    float_pair v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = make_pair(f[2 * j], f[2 * j + 1]);
    if constexpr (BLOCK == 16) {
      const uint32_t byte = fine ? scale_byte(__uint_as_float(m), sixth) : 0u;
      c[i] = fine ? codes16(v, byte, g) : make_uint2(0u, 0u);
      word |= byte << (8 * i);
    } else if (i & 1) {
      const uint32_t both = max(m, pair_top);
      const bool ok = both < 0x7f800000u;
      const int X = block_exponent(__uint_as_float(ok ? both : 0u));
      c[i - 1] = ok ? codes32(prev, X) : make_uint2(0u, 0u);
      c[i] = ok ? codes32(v, X) : make_uint2(0u, 0u);
      word |= (ok ? static_cast<uint32_t>(X + 127) : kNanE8m0) << (4 * (i - 1));
    } else {
      pair_top = m;
#pragma unroll
      for (int j = 0; j < 8; ++j) prev[j] = v[j];
    }
  }
  const size_t row = static_cast<size_t>(e) * N + n;
  uint4* dst = codes + row * (K / 32) + static_cast<size_t>(k64) * 2;
  dst[0] = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
  dst[1] = make_uint4(c[2].x, c[2].y, c[3].x, c[3].y);
  if constexpr (BLOCK == 16)
    *reinterpret_cast<uint32_t*>(scales + row * (K / 16) + static_cast<size_t>(k64) * 4) = word;
  else
    *reinterpret_cast<uint16_t*>(scales + row * (K / 32) + static_cast<size_t>(k64) * 2) =
        static_cast<uint16_t>(word);
}

// Plain scales [E, N, K/BLOCK] -> atoms [E, tiles, ka, 128 words], a thread a word. One
// matrix: tile i holds rows 128 i .. With a second (gate a, up b): tiles of half a's rows and
// half b's (gate_up_half).
template <int BLOCK>
__global__ void __launch_bounds__(kThreads)
pack_scales_kernel(const uint8_t* __restrict__ a, const uint8_t* __restrict__ b, int N, int K,
                   int half, int tiles, int ka, long long words, uint32_t* __restrict__ sf) {
  pdl_enter();
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= words) return;
  const int w = static_cast<int>(i & 127);
  long long t = i >> 7;
  const int k = static_cast<int>(t % ka);
  t /= ka;
  const int tile = static_cast<int>(t % tiles);
  const int e = static_cast<int>(t / tiles);
  const int r = (w >> 2) + 32 * (w & 3);
  const uint8_t* src = a;
  int row;
  if (!b) {
    row = tile * 128 + r;
  } else if (half == 128) {
    src = (tile & 1) ? b : a;
    row = (tile >> 1) * 128 + r;
  } else {
    src = r < 64 ? a : b;
    row = tile * 64 + (r & 63);
  }
  const int per = K / BLOCK;   // scales of a row: whole words for block 16, half words may end block 32
  uint32_t v = 0;
  if (row < N) {
    const uint8_t* s = src + (static_cast<size_t>(e) * N + row) * per;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (4 * k + j < per) v |= static_cast<uint32_t>(s[4 * k + j]) << (8 * j);
  }
  sf[i] = v;
}

template <int BLOCK, int TPR, int BPT>
int launch_rows(const void* x, const int32_t* inv_perm, const int32_t* offsets, int E, int T, int K,
                int M, int d, void* q, void* sf, float* row_scale, cudaStream_t st, const char* name) {
  constexpr int kRows = kThreads / TPR;
  ProfScope prof(name, st);
  return launch_pdl(quantize_rows_kernel<BLOCK, TPR, BPT>, (static_cast<unsigned>(T) + kRows - 1) / kRows, kThreads,
                    sizeof(int) * 2 * (E + 1), st, 1, static_cast<const uint4*>(x), inv_perm, offsets,
                    E, T, K, M, d, static_cast<uint2*>(q), static_cast<uint32_t*>(sf), row_scale);
}

// CTAs of warps that stay for many rows: as many as eight to an SM.
unsigned row_grid(long long rows) {
  const long long need = (rows + kThreads / 32 - 1) / (kThreads / 32);
  const long long most = 8LL * num_sms();
  return static_cast<unsigned>(need < most ? need : most);
}

template <int BLOCK, int BPT>
int launch_warp_rows(const void* x, const int32_t* inv_perm, const int32_t* offsets, int E, int T,
                     int K, int M, int d, void* q, void* sf, float* row_scale, cudaStream_t st,
                     const char* name) {
  ProfScope prof(name, st);
  return launch_pdl(quantize_warp_rows_kernel<BLOCK, BPT>, row_grid(T), kThreads,
                    sizeof(int) * 2 * (E + 1), st, 1, static_cast<const uint4*>(x), inv_perm, offsets,
                    E, T, K, M, d, static_cast<uint2*>(q), static_cast<uint32_t*>(sf), row_scale);
}

template <int BLOCK>
int launch_rows_for(const void* x, const int32_t* inv_perm, const int32_t* offsets, int E, int T,
                    int K, int M, int d, void* q, void* sf, float* row_scale, cudaStream_t st,
                    const char* name) {
  const int units = d / 16;
#define MOE_ROWS(BPT) \
  return launch_warp_rows<BLOCK, BPT>(x, inv_perm, offsets, E, T, K, M, d, q, sf, row_scale, st, name)
  if (units <= 64) MOE_ROWS(2);
  if (units <= 128) MOE_ROWS(4);
  if (units <= 192) MOE_ROWS(6);
#undef MOE_ROWS
  if (units <= 256)
    return launch_rows<BLOCK, 128, 2>(x, inv_perm, offsets, E, T, K, M, d, q, sf, row_scale, st, name);
  if (units <= 512)
    return launch_rows<BLOCK, kThreads, 2>(x, inv_perm, offsets, E, T, K, M, d, q, sf, row_scale, st,
                                           name);
  return launch_rows<BLOCK, kThreads, 4>(x, inv_perm, offsets, E, T, K, M, d, q, sf, row_scale, st, name);
}

}  // namespace

int launch_quantize(const void* x, const int32_t* inv_perm, const int32_t* offsets, int E, int T,
                    int K, int M, int d, int block, void* q, void* sf, float* row_scale,
                    cudaStream_t st, const char* name) {
  return block == 16 ? launch_rows_for<16>(x, inv_perm, offsets, E, T, K, M, d, q, sf, row_scale, st, name)
                     : launch_rows_for<32>(x, inv_perm, offsets, E, T, K, M, d, q, sf, row_scale, st, name);
}

}  // namespace fp4
}  // namespace moe

extern "C" int moe_fp4_quantize_rows(const moe_bf16* x, const int32_t* inv_perm, int T, int K,
                                     const int32_t* offsets, int E, int d, int block, uint8_t* q,
                                     uint8_t* sf, float* row_scale, void* stream) {
  using namespace moe;
  if (T < 0 || K < 1 || K > 32 || E < 1 || E > 1024 || d < 64 || d % 64 || (block != 16 && block != 32))
    return MOE_ERR_INVALID_ARG;
  if (!inv_perm && K != 1 && T > 0) return MOE_ERR_INVALID_ARG;   // (an empty array may be null)
  const long long M = static_cast<long long>(T) * K;
  if (d > 16384 || M > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!x || !offsets || !q || !sf || (block == 16 && !row_scale)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(offsets) || !aligned16(q) || !aligned16(sf) ||
      (inv_perm && !aligned16(inv_perm)) || (row_scale && !aligned16(row_scale)))
    return MOE_ERR_MISALIGNED;
  return fp4::launch_quantize(x, inv_perm, offsets, E, T, K, static_cast<int>(M), d, block, q, sf,
                              row_scale, as_stream(stream), "fp4_quantize_rows");
}

extern "C" int moe_fp4_dequantize_rows(const uint8_t* q, const uint8_t* sf, const float* row_scale,
                                       const int32_t* offsets, int E, int M, int d, int block,
                                       moe_bf16* out, void* stream) {
  using namespace moe;
  using namespace moe::fp4;
  if (M < 0 || E < 1 || E > 1024 || d < 64 || d % 64 || (block != 16 && block != 32))
    return MOE_ERR_INVALID_ARG;
  if (d > 16384) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!q || !sf || !offsets || !out || (block == 16 && !row_scale)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(sf) || !aligned16(offsets) || !aligned16(out) ||
      (row_scale && !aligned16(row_scale)))
    return MOE_ERR_MISALIGNED;
  cudaStream_t st = as_stream(stream);
  ProfScope prof("fp4_dequantize_rows", st);
  const size_t smem = sizeof(int) * 2 * (E + 1);
  auto go = [&](auto kern) {
    return launch_pdl(kern, static_cast<unsigned>((static_cast<long long>(M) + kThreads / 32 - 1) / (kThreads / 32)),
                      kThreads, smem, st, 1, reinterpret_cast<const uint2*>(q),
                      reinterpret_cast<const uint32_t*>(sf), row_scale, offsets, E, M, d,
                      reinterpret_cast<uint4*>(out));
  };
  return block == 16 ? go(dequantize_rows_kernel<16>) : go(dequantize_rows_kernel<32>);
}

extern "C" int moe_fp4_quantize_weights(const moe_bf16* w, int E, int K, int N, int block,
                                        uint8_t* codes, uint8_t* scales, float* scale, void* stream) {
  using namespace moe;
  using namespace moe::fp4;
  if (E < 1 || K < 64 || K % 64 || N < 8 || N % 8 || (block != 16 && block != 32))
    return MOE_ERR_INVALID_ARG;
  if (!w || !codes || !scales || (block == 16 && !scale)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(codes) || !aligned16(scales) || (scale && !aligned16(scale)))
    return MOE_ERR_MISALIGNED;
  const long long blocks = static_cast<long long>(E) * (K / 64) * ((N + 127) / 128);
  if (E > 65535 || blocks > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = as_stream(stream);
  if (block == 16) {
    const long long vecs = static_cast<long long>(K) * N / 8;
    const cudaError_t err = cudaMemsetAsync(scale, 0, sizeof(float) * E, st);
    if (err != cudaSuccess) {
      set_last_cuda_error(err);
      return MOE_ERR_CUDA;
    }
    long long gx = (vecs + kThreads * 8 - 1) / (kThreads * 8);   // eight vectors a thread
    if (gx > 4096) gx = 4096;
    {
      ProfScope prof("fp4_weight_top", st);
      const int rc = launch_pdl(weight_top_kernel, dim3(static_cast<unsigned>(gx), E), kThreads, 0, st, 1,
                                reinterpret_cast<const uint4*>(w), vecs,
                                reinterpret_cast<uint32_t*>(scale));
      if (rc) return rc;
    }
    ProfScope prof("fp4_weight_scale", st);
    const int rc = launch_pdl(weight_scale_kernel, (E + 127) / 128, 128, 0, st, 1, scale, E);
    if (rc) return rc;
  }
  ProfScope prof("fp4_quantize_weights", st);
  auto go = [&](auto kern) {
    return launch_pdl(kern, static_cast<unsigned>(blocks), 128, 0, st, 1,
                      reinterpret_cast<const __nv_bfloat16*>(w), K, N,
                      static_cast<const float*>(scale), reinterpret_cast<uint4*>(codes), scales);
  };
  return block == 16 ? go(quantize_weights_kernel<16>) : go(quantize_weights_kernel<32>);
}

extern "C" int moe_fp4_pack_scales(const uint8_t* scales_a, const uint8_t* scales_b, int E, int N,
                                   int K, int block, uint8_t* sf, void* stream) {
  using namespace moe;
  using namespace moe::fp4;
  if (E < 1 || K < 64 || K % 64 || N < 8 || N % 8 || (block != 16 && block != 32))
    return MOE_ERR_INVALID_ARG;
  if (scales_b && N % 64) return MOE_ERR_INVALID_ARG;
  if (!scales_a || !sf) return MOE_ERR_INVALID_ARG;
  if (!aligned16(scales_a) || (scales_b && !aligned16(scales_b)) || !aligned16(sf))
    return MOE_ERR_MISALIGNED;
  const int tiles = scales_b ? N / 64 : (N + 127) / 128;
  const int ka = k_atoms(K, block);
  const long long words = static_cast<long long>(E) * tiles * ka * 128;
  const long long blocks = (words + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = as_stream(stream);
  ProfScope prof("fp4_pack_scales", st);
  auto go = [&](auto kern) {
    return launch_pdl(kern, static_cast<unsigned>(blocks), kThreads, 0, st, 1, scales_a, scales_b, N, K,
                      gate_up_half(N), tiles, ka, words, reinterpret_cast<uint32_t*>(sf));
  };
  return block == 16 ? go(pack_scales_kernel<16>) : go(pack_scales_kernel<32>);
}

namespace moe {
MOE_DEBUG_STATUS_READER(fp4)
}  // namespace moe
