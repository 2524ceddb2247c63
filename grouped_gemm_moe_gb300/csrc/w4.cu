// SwiGLU experts on 4-bit weights with group scales, for the few rows per expert
// of a decoding batch, and the quantizer and layout of such weights.
//
//   w = s (q - 8),  q in 0 .. 15, one bf16 scale s per group of 32, 64 or 128
//   consecutive elements along K;  H = bf16(silu(X Wg) * (X Wu)),  Y = bf16(H Wd)
//
// With a few rows per expert the products are bound by reading the weights
// (half a byte each, plus 2 / group), so the design is about a steady weight
// stream. Weights are laid out once in the order the tensor cores take them:
// tiles of 16 outputs x 64 K, 512 bytes, 16 bytes per lane, so one coalesced
// load per warp and tile feeds four m16n8k16 products whose A is the weights
// and whose 8 columns are rows of X. A code becomes the bf16 integer q - 8 in
// registers (exact), so the products run on integers and the scale multiplies
// the fp32 sums of a group: no weight is ever rounded. The lane's 16 elements
// of K are two runs of 8, one in each half of the 64, which is the order the
// rows of X are loaded in 16-byte pieces and keeps groups of 32 apart.
//
// mma.sync and not tcgen05: the A operand is made in registers from 4-bit codes
// and N is 8 to 32; tcgen05 would take it through shared memory or TMEM at
// M = 128 for a product that is bound by HBM either way.
//
// Gate and up share tiles: outputs 0-7 of a tile are eight gate columns, 8-15 the
// same up columns, which puts G and U of one element in one lane.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

#ifndef W4_CUT1
#define W4_CUT1 6
#endif
#ifndef W4_CUT2
#define W4_CUT2 12
#endif
#ifndef W4_STAGES
#define W4_STAGES 4
#endif
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

// ----------------------------------------------------------------- quantizer
// s = max|w| / 7 rounded up to bf16, q = rint(w fl32(1 / s)) + 8 in 1 .. 15. One
// thread per (expert, group, output); a warp reads 32 neighbouring outputs of a
// K row at a time. Runs when weights are loaded, not per token.
__global__ void __launch_bounds__(256)
w4_quantize_kernel(const __nv_bfloat16* __restrict__ w, int K, int N, int group, long long total,
                   uint8_t* __restrict__ codes, uint16_t* __restrict__ scales) {
  pdl_enter();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const int ng = K / group;
  const int n = static_cast<int>(i % N);
  const long long eg = i / N;
  const int gi = static_cast<int>(eg % ng);
  const long long e = eg / ng;
  const __nv_bfloat16* p = w + (e * K + static_cast<long long>(gi) * group) * N + n;
  float amax = 0.f;
  for (int k = 0; k < group; ++k) amax = fmaxf(amax, fabsf(__bfloat162float(p[static_cast<long long>(k) * N])));
  const float t = fmaxf(__fdiv_rn(amax, 7.f), 0x1p-110f);
  const float s = __uint_as_float((__float_as_uint(t) + 0xffffu) & 0xffff0000u);
  const float r = __frcp_rn(s);
  uint32_t* out = reinterpret_cast<uint32_t*>(codes + ((e * N + n) * K + static_cast<long long>(gi) * group) / 2);
  for (int k0 = 0; k0 < group; k0 += 8) {
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float v = __bfloat162float(p[static_cast<long long>(k0 + k) * N]);
      const float q = fminf(fmaxf(rintf(__fmul_rn(v, r)), -7.f), 7.f);
      word |= static_cast<uint32_t>(static_cast<int>(q) + 8) << (4 * k);
    }
    out[k0 / 8] = word;
  }
  scales[(e * N + n) * ng + gi] = static_cast<uint16_t>(__float_as_uint(s) >> 16);
}

// ----------------------------------------------------------------- layout
// The plain row of row `m` (0 .. 15) of tile `i`: outputs 16 i + m, or with gate
// and up in one tile output 8 i + (m & 7) of gate (m < 8) or up.
__device__ __forceinline__ long long plain_row(long long e, int i, int m, int N, bool pair) {
  return pair ? e * N + 8 * i + (m & 7) : e * N + 16 * i + m;
}

// One thread per word of a tile: word j of lane l is row l / 4 (j even) or that + 8
// (odd), k = 32 (j / 2) + 8 (l % 4) + 0 .. 7; nibble n holds k offset 2 n
// (n < 4) or 2 (n - 4) + 1, so word >> 4 n & 0x000f000f is the pair (2 n, 2 n + 1).
__global__ void __launch_bounds__(256)
w4_pack_kernel(const uint8_t* __restrict__ ca, const uint8_t* __restrict__ cb, int N, int K, int nt,
               long long total, uint32_t* __restrict__ tiles) {
  pdl_enter();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const int j = static_cast<int>(i & 3);
  const int l = static_cast<int>(i >> 2 & 31);
  const long long tile = i >> 7;
  const int kt = K / 64;
  const int kb = static_cast<int>(tile % kt);
  const long long et = tile / kt;
  const int it = static_cast<int>(et % nt);
  const long long e = et / nt;
  const int m = (l >> 2) + 8 * (j & 1);
  const uint8_t* src = (cb && m >= 8) ? cb : ca;
  const long long k = 64LL * kb + 32 * (j >> 1) + 8 * (l & 3);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(src + (plain_row(e, it, m, N, cb != nullptr) * K + k) / 2);
  uint32_t o = 0;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const int at = n < 4 ? 2 * n : 2 * (n - 4) + 1;
    o |= (w >> (4 * at) & 15u) << (4 * n);
  }
  tiles[i] = o;
}

// Scales [E][tile][K / group][16], rows m and m + 8 of a tile next to each other.
__global__ void __launch_bounds__(256)
w4_pack_scales_kernel(const uint16_t* __restrict__ sa, const uint16_t* __restrict__ sb, int N,
                      int ng, int nt, long long total, uint16_t* __restrict__ out) {
  pdl_enter();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const int at = static_cast<int>(i & 15);
  const int m = (at >> 1) + 8 * (at & 1);
  const long long g = i >> 4;
  const int gi = static_cast<int>(g % ng);
  const long long et = g / ng;
  const int it = static_cast<int>(et % nt);
  const long long e = et / nt;
  const uint16_t* src = (sb && m >= 8) ? sb : sa;
  out[i] = src[plain_row(e, it, m, N, sb != nullptr) * ng + gi];
}

// ----------------------------------------------------------------- products
// The pair (2 n, 2 n + 1) of a word as bf16 integers q - 8: 0x4300 | q is
// 128 + q, and subtracting 136 is exact.
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int n) {
  uint32_t v = ((w >> (4 * n)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 c = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), c);
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same into a fresh sum.
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Half a tile (32 K): two products per 8 rows of X. FIRST starts the group's
// sums, LAST adds them scaled into acc.
template <int NT, bool FIRST, bool LAST>
__device__ __forceinline__ void half_tile(uint32_t w0, uint32_t w1, const uint4 (&x)[NT],
                                          float (&part)[NT][4], float s0, float s1,
                                          float (&acc)[NT][4]) {
  const uint32_t a0[4] = {pair_of(w0, 0), pair_of(w1, 0), pair_of(w0, 1), pair_of(w1, 1)};
  const uint32_t a1[4] = {pair_of(w0, 2), pair_of(w1, 2), pair_of(w0, 3), pair_of(w1, 3)};
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (FIRST) mma16816_first(part[n], a0, x[n].x, x[n].y);
    else mma16816(part[n], a0, x[n].x, x[n].y);
    mma16816(part[n], a1, x[n].z, x[n].w);
    if (LAST) {
      acc[n][0] = fmaf(s0, part[n][0], acc[n][0]);
      acc[n][1] = fmaf(s0, part[n][1], acc[n][1]);
      acc[n][2] = fmaf(s1, part[n][2], acc[n][2]);
      acc[n][3] = fmaf(s1, part[n][3], acc[n][3]);
    }
  }
}

// Each warp streams its weights through a ring of its own in shared memory: a
// stage is two k-tiles and their scales, every lane copies the 16 bytes per tile
// that it will read itself, a few lanes also the scales. cp.async and not
// registers: 3 KB a warp stay in flight and the accumulators keep the registers.
constexpr int kStages = W4_STAGES;
constexpr int scale_vecs(int group) { return 256 / group; }           // 16-byte pieces a stage
constexpr int stage_vecs(int group) { return 64 + scale_vecs(group); }
constexpr size_t ring_bytes(int group) {
  return sizeof(uint4) * kWarps * kStages * stage_vecs(group);
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// Half h (32 K) of the p-th k-tile of the lane's rows of X.
template <int NT>
__device__ __forceinline__ void load_x(const uint4* const (&xr)[NT], int p, int h, uint4 (&x)[NT]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) x[n] = __ldg(xr[n] + 8 * p + 4 * h);
}

// A warp's weights: `count` k-tiles of one tile of outputs.
template <int GROUP>
struct Stream {
  const uint4* codes;    // this lane's 16 bytes of the next stage to copy
  const uint4* scales;
  uint4* ring;
  uint32_t ring_addr;
  int left;              // k-tiles not yet copied
  int slot;              // stage slot of the next copy

  __device__ __forceinline__ void issue() {
    const int lane = threadIdx.x & 31;
    if (left > 0) {
      const uint32_t to = ring_addr + slot * (16 * stage_vecs(GROUP));
      copy16(to + 16 * lane, codes);
      if (left > 1) copy16(to + 512 + 16 * lane, codes + 32);
      // a last stage of one tile has half the scales (groups of 128 never end so)
      if (lane < scale_vecs(GROUP) && (left > 1 || lane < (scale_vecs(GROUP) + 1) / 2))
        copy16(to + 1024 + 16 * lane, scales + lane);
      codes += 64;
      scales += scale_vecs(GROUP);
      left -= 2;
      slot = slot + 1 == kStages ? 0 : slot + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

// acc[n][.] += the tile's outputs over the stream's k-tiles, for the 8 NT rows of
// X at xr[n] (this lane's share of the first k-tile). With 8 rows X is loaded a
// stage ahead; with more, the registers for that are missing.
template <int NT, int GROUP>
__device__ __forceinline__ void product(Stream<GROUP>& st, int count, const uint4* (&xr)[NT],
                                        float (&acc)[NT][4]) {
  constexpr bool kAhead = NT == 1;
  const int lane = threadIdx.x & 31, g = lane >> 2;
  uint4 nx[2][2][NT];
  if (kAhead) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      if (p < count) {
        load_x<NT>(xr, p, 0, nx[p][0]);
        load_x<NT>(xr, p, 1, nx[p][1]);
      }
  }
  int slot = 0;
  for (int k = 0; k < count; k += 2) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();   // the scales of this stage are there; all lanes are done with the last one
    st.issue();
    const uint4* stage = st.ring + slot * stage_vecs(GROUP);
    slot = slot + 1 == kStages ? 0 : slot + 1;
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(stage + 64) + g;
    uint4 x[2][2][NT];
    if (kAhead) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n) x[p][h][n] = nx[p][h][n];
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (k + 2 + p < count) {
          load_x<NT>(xr, 2 + p, 0, nx[p][0]);
          load_x<NT>(xr, 2 + p, 1, nx[p][1]);
        }
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (k + p >= count) break;
      const uint4 w = stage[32 * p + lane];
      const uint32_t s0 = sc[GROUP == 32 ? 16 * p : GROUP == 64 ? 8 * p : 0];
      const uint32_t s1 = GROUP == 32 ? sc[16 * p + 8] : s0;
      float part[NT][4];
      if (!kAhead) load_x<NT>(xr, p, 0, x[p][0]);
      half_tile<NT, true, GROUP == 32>(w.x, w.y, x[p][0], part, bf16_lo(s0), bf16_hi(s0), acc);
      if (!kAhead) load_x<NT>(xr, p, 1, x[p][1]);
      half_tile<NT, GROUP == 32, true>(w.z, w.w, x[p][1], part, bf16_lo(s1), bf16_hi(s1), acc);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) xr[n] += 16;
  }
}

// The expert of grid row `slot`: the slot-th expert that has rows, or with a grid
// row per expert the expert itself. Returns -1 past the last.
__device__ __forceinline__ int expert_of(const int32_t* offsets, int E, int slot, bool direct) {
  if (direct) return slot;
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int base = 0; base < E; base += 128) {   // 128 experts' offsets in one round trip
    bool any[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = base + 32 * i + lane;
      any[i] = e < E && __ldg(offsets + e + 1) > __ldg(offsets + e);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned m = __ballot_sync(0xffffffffu, any[i]);
      const int n = __popc(m);
      if (before + n > slot) return base + 32 * i + static_cast<int>(__fns(m, 0, slot - before + 1));
      before += n;
    }
  }
  return -1;
}

struct W4Args {
  const uint8_t* x;         // rows of K bf16
  const int32_t* perm;      // GATE_UP: row p of the experts is x[perm[p] / top_k]; null: x[p]
  int top_k;
  const int32_t* offsets;
  const uint4* tiles;
  const uint4* scales;
  __nv_bfloat16* out;       // h [M, I] or y [M, d]
  int E, M, K, N, nt, group;   // nt: tiles of outputs per expert; N: columns of out
  int x_rows;
};

// One pass over a tile's weights for rows [r0, r0 + 8 NT) of the expert's rows
// ending at r1, its K split over S warps of the block.
template <bool GATE_UP, int S, int NT, int GROUP>
__device__ __forceinline__ void pass(const W4Args& A, int e, int it, int ks, int r0, int r1,
                                     uint4* ring) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int kt = A.K / 64;
  const bool live = it < A.nt;
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[n][q] = 0.f;
  if (S > 1) __syncthreads();   // the last pass has read the sums that lie over the rings
  if (live) {
    const long long tile = static_cast<long long>(e) * A.nt + it;
    // whole pairs of k-tiles to each split, so that groups of 128 stay in one
    const int k0 = kt * ks / S & ~1, k1 = ks + 1 == S ? kt : kt * (ks + 1) / S & ~1;
    Stream<GROUP> stream;
    stream.codes = A.tiles + (tile * kt + k0) * 32 + lane;
    stream.scales = A.scales + (tile * (A.K / GROUP) + k0 * 64 / GROUP) * 2;
    stream.ring = ring + warp * kStages * stage_vecs(GROUP);
    stream.ring_addr = static_cast<uint32_t>(__cvta_generic_to_shared(stream.ring));
    stream.left = k1 - k0;
    stream.slot = 0;
    __syncwarp();   // every lane is done with the ring's last use
    for (int p = 0; p + 1 < kStages; ++p) stream.issue();   // before the rows of X are looked up
    const uint4* xr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // past the expert's last row: that row again (the products' columns are
      // apart, and these are not stored)
      int row = min(r0 + 8 * n + g, r1 - 1);
      if (GATE_UP && A.perm) row = __ldg(A.perm + row) / A.top_k;
      if (!index_ok(row >= 0 && row < A.x_rows)) row = 0;
      xr[n] = reinterpret_cast<const uint4*>(A.x) + static_cast<long long>(row) * (A.K / 8) + k0 * 8 + c;
    }
    product<NT, GROUP>(stream, k1 - k0, xr, acc);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  if (S > 1) {
    __syncthreads();   // every warp is done with its ring
    float* red = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) red[(warp * 4 * NT + n * 4 + q) * 32 + lane] = acc[n][q];
    __syncthreads();
    if (ks != 0) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int o = 1; o < S; ++o) acc[n][q] += red[((warp + o) * 4 * NT + n * 4 + q) * 32 + lane];
  }
  if (!live) return;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int p = r0 + 8 * n + 2 * c + q;
      if (p >= r1) continue;
      __nv_bfloat16* row = A.out + static_cast<long long>(p) * A.N;
      if (GATE_UP) {
        const float G = acc[n][q], U = acc[n][q + 2];
        row[8 * it + g] = __float2bfloat16(__fdividef(G, 1.f + __expf(-G)) * U);
      } else {
        row[16 * it + g] = __float2bfloat16(acc[n][q]);
        row[16 * it + g + 8] = __float2bfloat16(acc[n][q + 2]);
      }
    }
  }
}

// NTMAX: the most groups of 8 rows a pass takes (a power of two).
template <bool GATE_UP, int S, int NTMAX, int GROUP>
__global__ void __launch_bounds__(kThreads, NTMAX == 1 ? 3 : 2) w4_kernel(W4Args A) {
  pdl_enter();
  extern __shared__ uint4 ring[];   // [warp][stage][codes, scales]
  const int e = expert_of(A.offsets, A.E, blockIdx.y, gridDim.y == static_cast<unsigned>(A.E));
  if (e < 0) return;
  int r0 = __ldg(A.offsets + e);
  const int r1 = min(__ldg(A.offsets + e + 1), A.M);
  const int warp = threadIdx.x >> 5;
  const int it = blockIdx.x * (kWarps / S) + warp / S, ks = warp % S;
  for (; r0 < r1; r0 += 8 * NTMAX) {
    const int n = r1 - r0;
    if (NTMAX == 1 || n <= 8) pass<GATE_UP, S, 1, GROUP>(A, e, it, ks, r0, r1, ring);
    else if (NTMAX == 2 || n <= 16) pass<GATE_UP, S, 2, GROUP>(A, e, it, ks, r0, r1, ring);
    else pass<GATE_UP, S, 4, GROUP>(A, e, it, ks, r0, r1, ring);
  }
}

template <bool GATE_UP, int NTMAX, int GROUP>
int launch_split(int S, dim3 grid, const W4Args& a, cudaStream_t st) {
  auto go = [&](auto kern) {
#if W4_STAGES > 4
    cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
#endif
    return launch_pdl(kern, grid, kThreads, ring_bytes(GROUP), st, 1, a);
  };
  static_assert(ring_bytes(GROUP) >= sizeof(float) * kWarps * NTMAX * 4 * 32, "sums over the rings");
  if (S == 1) return go(w4_kernel<GATE_UP, 1, NTMAX, GROUP>);
  if (S == 2) return go(w4_kernel<GATE_UP, 2, NTMAX, GROUP>);
  if (S == 4) return go(w4_kernel<GATE_UP, 4, NTMAX, GROUP>);
  return go(w4_kernel<GATE_UP, 8, NTMAX, GROUP>);
}

// most_rows: a bound on the rows of one expert.
template <bool GATE_UP>
int launch_w4(const char* name, const W4Args& a, int most_rows, cudaStream_t st) {
  const int slots = std::min(a.E, a.M);
  // Split K until the launch has about 24 warps per SM, a warp keeping four tiles at least.
  const long long want = static_cast<long long>(num_sms()) * 24;
  const long long tiles = static_cast<long long>(slots) * a.nt;
  int S = 1;
  while (S < 8 && tiles * S < want && a.K / 64 >= 8 * S) S *= 2;
  ProfScope prof(name, st);
  const dim3 grid((a.nt + kWarps / S - 1) / (kWarps / S), slots);
  auto by_group = [&](auto nt) {
    constexpr int N = decltype(nt)::value;
    if (a.group == 32) return launch_split<GATE_UP, N, 32>(S, grid, a, st);
    if (a.group == 64) return launch_split<GATE_UP, N, 64>(S, grid, a, st);
    return launch_split<GATE_UP, N, 128>(S, grid, a, st);
  };
  const int mean = std::min<long long>(most_rows, (a.M + a.E - 1) / a.E);
  if (mean <= W4_CUT1) return by_group(std::integral_constant<int, 1>());
  if (mean <= W4_CUT2) return by_group(std::integral_constant<int, 2>());
  return by_group(std::integral_constant<int, 4>());
}

bool group_ok(int group) { return group == 32 || group == 64 || group == 128; }

}  // namespace
}  // namespace moe

extern "C" int moe_w4_quantize_weights(const moe_bf16* w, int E, int K, int N, int group,
                                       uint8_t* codes, moe_bf16* scales, void* stream) {
  using namespace moe;
  if (E < 1 || K < 64 || N < 1 || !group_ok(group) || K % 64 || K % group)
    return MOE_ERR_INVALID_ARG;
  if (!w || !codes || !scales) return MOE_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(codes) || !aligned16(scales)) return MOE_ERR_MISALIGNED;
  const long long total = static_cast<long long>(E) * (K / group) * N;
  const long long blocks = (total + 255) / 256;
  if (blocks > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = as_stream(stream);
  ProfScope prof("w4_quantize_weights", st);
  return launch_pdl(w4_quantize_kernel, static_cast<unsigned>(blocks), 256, 0, st, 1,
                    reinterpret_cast<const __nv_bfloat16*>(w), K, N, group, total, codes,
                    reinterpret_cast<uint16_t*>(scales));
}

extern "C" int moe_w4_pack_weights(const uint8_t* codes_a, const moe_bf16* scales_a,
                                   const uint8_t* codes_b, const moe_bf16* scales_b, int E, int N,
                                   int K, int group, uint8_t* tiles, moe_bf16* scales,
                                   void* stream) {
  using namespace moe;
  if (E < 1 || K < 64 || N < 1 || !group_ok(group) || K % 64 || K % group ||
      (codes_b == nullptr) != (scales_b == nullptr) || N % (codes_b ? 8 : 16))
    return MOE_ERR_INVALID_ARG;
  if (!codes_a || !scales_a || !tiles || !scales) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {codes_a, scales_a, codes_b, scales_b, tiles, scales};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_MISALIGNED;
  const int nt = codes_b ? N / 8 : N / 16, ng = K / group;
  const long long words = static_cast<long long>(E) * nt * (K / 64) * 128;
  const long long ns = static_cast<long long>(E) * nt * ng * 16;
  if ((words + 255) / 256 > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = as_stream(stream);
  int rc;
  {
    ProfScope prof("w4_pack", st);
    rc = launch_pdl(w4_pack_kernel, static_cast<unsigned>((words + 255) / 256), 256, 0, st, 1,
                    codes_a, codes_b, N, K, nt, words, reinterpret_cast<uint32_t*>(tiles));
  }
  if (rc != MOE_OK) return rc;
  ProfScope prof("w4_pack_scales", st);
  return launch_pdl(w4_pack_scales_kernel, static_cast<unsigned>((ns + 255) / 256), 256, 0, st, 1,
                    reinterpret_cast<const uint16_t*>(scales_a),
                    reinterpret_cast<const uint16_t*>(scales_b), N, ng, nt, ns,
                    reinterpret_cast<uint16_t*>(scales));
}

extern "C" int moe_grouped_ffn_w4(const moe_bf16* x, const int32_t* perm, int T, int K,
                                  const int32_t* offsets, int E, int M, int d, int I,
                                  int group_gu, int group_d, const uint8_t* wgu,
                                  const moe_bf16* wgu_s, const uint8_t* wd, const moe_bf16* wd_s,
                                  moe_bf16* y, moe_bf16* h, void* ws, size_t ws_bytes,
                                  void* stream) {
  using namespace moe;
  if (E < 1 || E > 1024 || M < 0 || T < 0 || K < 1 || !group_ok(group_gu) || !group_ok(group_d) ||
      d < 64 || I < 64 || d % 64 || I % 64 || d % group_gu || I % group_d)
    return MOE_ERR_INVALID_ARG;
  if (perm ? static_cast<long long>(T) * K != M : T != M) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!x || !offsets || !wgu || !wgu_s || !wd || !wd_s || !y || !h) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {x, perm, offsets, wgu, wgu_s, wd, wd_s, y, h, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_MISALIGNED;
  if (!ws || ws_bytes < kWorkspaceHeader) return MOE_ERR_WORKSPACE;
  cudaStream_t st = as_stream(stream);
  W4Args a = {};
  a.x = reinterpret_cast<const uint8_t*>(x);
  a.perm = perm;
  a.top_k = K;
  a.offsets = offsets;
  a.tiles = reinterpret_cast<const uint4*>(wgu);
  a.scales = reinterpret_cast<const uint4*>(wgu_s);
  a.out = reinterpret_cast<__nv_bfloat16*>(h);
  a.E = E;
  a.M = M;
  a.K = d;
  a.N = I;
  a.nt = I / 8;
  a.group = group_gu;
  a.x_rows = T;
  const int rc = launch_w4<true>("w4_gate_up", a, perm ? T : M, st);
  if (rc != MOE_OK) return rc;
  a.x = reinterpret_cast<const uint8_t*>(h);
  a.perm = nullptr;
  a.tiles = reinterpret_cast<const uint4*>(wd);
  a.scales = reinterpret_cast<const uint4*>(wd_s);
  a.out = reinterpret_cast<__nv_bfloat16*>(y);
  a.K = I;
  a.N = d;
  a.nt = d / 16;
  a.group = group_d;
  a.x_rows = M;
  return launch_w4<false>("w4_down", a, perm ? T : M, st);
}

namespace moe {
MOE_DEBUG_STATUS_READER(w4)
}  // namespace moe
