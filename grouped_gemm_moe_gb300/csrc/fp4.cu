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

// Largest |bf16| of a word's two, as bits (Inf 0x7f80, NaN above it), kept in the upper half.
__device__ __forceinline__ uint32_t top_bits(uint32_t m, uint32_t w) {
  const uint32_t a = w & 0x7fff0000u, b = (w & 0x00007fffu) << 16;
  return max(m, max(a, b));
}

// One launch quantizes each token's row once and writes it to its K rows in expert order
// (inv_perm null: to its own row). HBM-bound: 2 bytes read and K (1/2 + 1/block) written an
// element. TPR threads take a row (kThreads / TPR rows to a CTA), each BPT units of 16
// elements held in registers between the row's maximum and the codes; consecutive threads
// take consecutive units, so loads are 32 and stores 8 bytes a thread without gaps, and the
// four units of a scale word meet by shuffles.
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
  const unsigned t = blockIdx.x * kRows + sub;
  const bool live = t < static_cast<unsigned>(T);
  uint4 a[BPT], b[BPT];
#pragma unroll
  for (int i = 0; i < BPT; ++i) {
    const int u = i * TPR + lane_r;
    a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
    if (live && u < units) {
      const uint4* src = x + (static_cast<size_t>(t) * units + u) * 2;
      a[i] = ldg_nc_v4(src);
      b[i] = ldg_nc_v4(src + 1);
    }
  }
  for (int e = threadIdx.x; e <= E; e += kThreads) s_off[e] = __ldg(offsets + e);
  __syncthreads();
  if (threadIdx.x < 32) tile_prefix(s_off, s_tile, E);
  // the row's largest element, for its factor
  uint32_t top[BPT];
  uint32_t row_top = 0;
#pragma unroll
  for (int i = 0; i < BPT; ++i) {
    uint32_t m = top_bits(top_bits(0u, a[i].x), a[i].y);
    m = top_bits(top_bits(m, a[i].z), a[i].w);
    m = top_bits(top_bits(m, b[i].x), b[i].y);
    top[i] = top_bits(top_bits(m, b[i].z), b[i].w);
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
  int n = 0;
  bool fine = true;
  if constexpr (BLOCK == 16) {
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) row_top = max(row_top, s_top[sub * (TPR / 32) + w]);
    fine = row_top < 0x7f800000u;
    n = row_exponent(__uint_as_float(fine ? row_top : 0u));
  }
  __syncthreads();
  uint2 code[BPT];
  uint32_t word[BPT];
#pragma unroll
  for (int i = 0; i < BPT; ++i) {
    float_pair v[8];
    unpack8(a[i], v);
    unpack8(b[i], v + 4);
    uint32_t byte;
    if constexpr (BLOCK == 16) {
      byte = fine ? to_e4m3(__fdiv_rn(__uint_as_float(top[i]), 6.f * two_to(n))) : 0u;
      code[i] = fine ? codes16(v, byte, n) : make_uint2(0u, 0u);
      const uint32_t b1 = __shfl_down_sync(0xffffffffu, byte, 1);
      const uint32_t b2 = __shfl_down_sync(0xffffffffu, byte, 2);
      const uint32_t b3 = __shfl_down_sync(0xffffffffu, byte, 3);
      word[i] = byte | (b1 << 8) | (b2 << 16) | (b3 << 24);
    } else {
      const uint32_t both = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      const bool ok = both < 0x7f800000u;
      const int X = block_exponent(__uint_as_float(ok ? both : 0u));
      byte = ok ? static_cast<uint32_t>(X + 127) : kNanE8m0;
      code[i] = ok ? codes32(v, X) : make_uint2(0u, 0u);
      const uint32_t b1 = __shfl_down_sync(0xffffffffu, byte, 2);
      const uint32_t b2 = __shfl_down_sync(0xffffffffu, byte, 4);
      const uint32_t b3 = __shfl_down_sync(0xffffffffu, byte, 6);
      // past the row's end (half an atom): threads without a unit give the byte of zeros
      word[i] = byte | (b1 << 8) | (b2 << 16) | (b3 << 24);
    }
  }
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
      row_scale[p] = fine ? two_to(n) : __uint_as_float(0x7fc00000u);
  }
}

// Rows back in bf16: each thread 16 elements of a row (8 bytes of codes, one scale byte).
template <int BLOCK>
__global__ void __launch_bounds__(kThreads)
dequantize_rows_kernel(const uint2* __restrict__ q, const uint32_t* __restrict__ sf,
                       const float* __restrict__ row_scale, const int32_t* __restrict__ offsets,
                       int E, int M, int d, int rows_per_cta, uint4* __restrict__ out) {
  extern __shared__ int sm[];
  int* s_off = sm;
  int* s_tile = s_off + E + 1;
  pdl_enter();
  for (int e = threadIdx.x; e <= E; e += kThreads) s_off[e] = __ldg(offsets + e);
  __syncthreads();
  if (threadIdx.x < 32) tile_prefix(s_off, s_tile, E);
  __syncthreads();
  const int units = d / 16;
  constexpr int kPer = BLOCK / 4;
  const int ka = (units + kPer - 1) / kPer;
  const long long p0 = static_cast<long long>(blockIdx.x) * rows_per_cta;
  const int rows = static_cast<int>(min(static_cast<long long>(rows_per_cta), M - p0));
  for (int i = threadIdx.x; i < rows * units; i += kThreads) {
    const int r = i / units, u = i - r * units;
    const int p = static_cast<int>(p0) + r;
    const int2 pl = place_of(p, s_off, s_tile, E);
    if (pl.x < 0) continue;
    const uint2 c = q[static_cast<size_t>(p) * units + u];
    const uint32_t word = sf[(static_cast<size_t>(pl.x) * ka + u / kPer) * 128 + atom_word(pl.y)];
    float f;
    if constexpr (BLOCK == 16) {
      f = from_e4m3((word >> (8 * (u & 3))) & 0xffu) * row_scale[p];
    } else {
      const uint32_t byte = (word >> (8 * ((u >> 1) & 3))) & 0xffu;
      f = byte == kNanE8m0 ? __uint_as_float(0x7fc00000u) : two_to(static_cast<int>(byte) - 127);
    }
    uint32_t w[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      const uint32_t byte = ((h < 4 ? c.x : c.y) >> (8 * (h & 3))) & 0xffu;
      const __half2_raw hr = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
      const float2 v = __half22float2(__half2(hr));
      w[h] = pack_bf16(v.x * f, v.y * f);
    }
    uint4* dst = out + (static_cast<size_t>(p) * units + u) * 2;
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
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
    m = top_bits(top_bits(top_bits(top_bits(m, v.x), v.y), v.z), v.w);
  }
  m = __reduce_max_sync(0xffffffffu, m);
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
  int rexp = 0;
  bool fine = true;
  if constexpr (BLOCK == 16) {
    const float g = scale[e];
    fine = g == g;
    rexp = fine ? static_cast<int>(__float_as_uint(g) >> 23) - 127 : 0;
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
      const uint32_t byte = fine ? to_e4m3(__fdiv_rn(__uint_as_float(m), 6.f * two_to(rexp))) : 0u;
      c[i] = fine ? codes16(v, byte, rexp) : make_uint2(0u, 0u);
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
                int M, int d, void* q, void* sf, float* row_scale, cudaStream_t st) {
  constexpr int kRows = kThreads / TPR;
  ProfScope prof("fp4_quantize_rows", st);
  return launch_pdl(quantize_rows_kernel<BLOCK, TPR, BPT>, (static_cast<unsigned>(T) + kRows - 1) / kRows, kThreads,
                    sizeof(int) * 2 * (E + 1), st, 1, static_cast<const uint4*>(x), inv_perm, offsets,
                    E, T, K, M, d, static_cast<uint2*>(q), static_cast<uint32_t*>(sf), row_scale);
}

// Threads a row: the fewest of 32 .. 256 that hold it with two units each, four above d = 8192.
template <int BLOCK>
int launch_rows_for(const void* x, const int32_t* inv_perm, const int32_t* offsets, int E, int T,
                    int K, int M, int d, void* q, void* sf, float* row_scale, cudaStream_t st) {
  const int units = d / 16;
#define MOE_ROWS(TPR, BPT) \
  return launch_rows<BLOCK, TPR, BPT>(x, inv_perm, offsets, E, T, K, M, d, q, sf, row_scale, st)
  if (units <= 64) MOE_ROWS(32, 2);
  if (units <= 128) MOE_ROWS(64, 2);
  if (units <= 256) MOE_ROWS(128, 2);
  if (units <= 512) MOE_ROWS(256, 2);
  MOE_ROWS(256, 4);
#undef MOE_ROWS
}

}  // namespace

int launch_quantize(const void* x, const int32_t* inv_perm, const int32_t* offsets, int E, int T,
                    int K, int M, int d, int block, void* q, void* sf, float* row_scale,
                    cudaStream_t st) {
  return block == 16 ? launch_rows_for<16>(x, inv_perm, offsets, E, T, K, M, d, q, sf, row_scale, st)
                     : launch_rows_for<32>(x, inv_perm, offsets, E, T, K, M, d, q, sf, row_scale, st);
}

}  // namespace fp4
}  // namespace moe

extern "C" int moe_fp4_quantize_rows(const moe_bf16* x, const int32_t* inv_perm, int T, int K,
                                     const int32_t* offsets, int E, int d, int block, uint8_t* q,
                                     uint8_t* sf, float* row_scale, void* stream) {
  using namespace moe;
  if (T < 0 || K < 1 || K > 32 || E < 1 || E > 1024 || d < 64 || d % 64 || (block != 16 && block != 32))
    return MOE_ERR_INVALID_ARG;
  if (!inv_perm && K != 1) return MOE_ERR_INVALID_ARG;
  const long long M = static_cast<long long>(T) * K;
  if (d > 16384 || M > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!x || !offsets || !q || !sf || (block == 16 && !row_scale)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(offsets) || !aligned16(q) || !aligned16(sf) ||
      (inv_perm && !aligned16(inv_perm)) || (row_scale && !aligned16(row_scale)))
    return MOE_ERR_MISALIGNED;
  return fp4::launch_quantize(x, inv_perm, offsets, E, T, K, static_cast<int>(M), d, block, q, sf,
                              row_scale, as_stream(stream));
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
  const int units = d / 16;
  const int rows = units >= 4 * kThreads ? 1 : (4 * kThreads + units - 1) / units;   // about four units a thread
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(M) + rows - 1) / rows);
  cudaStream_t st = as_stream(stream);
  ProfScope prof("fp4_dequantize_rows", st);
  const size_t smem = sizeof(int) * 2 * (E + 1);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, kThreads, smem, st, 1, reinterpret_cast<const uint2*>(q),
                      reinterpret_cast<const uint32_t*>(sf), row_scale, offsets, E, M, d, rows,
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
