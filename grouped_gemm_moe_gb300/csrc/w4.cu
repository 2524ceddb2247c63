// SwiGLU experts on 4-bit weights with group scales, for the few rows per expert
// of a decoding batch, and the quantizer and layout of such weights.
//
//   w = s (q - 8),  q in 0 .. 15, one bf16 scale s per group of 32, 64 or 128
//   consecutive elements along K;  H = bf16(silu(X Wg) * (X Wu)),  Y = bf16(H Wd)
//
// With a few rows per expert the products are bound by reading the weights
// (half a byte each, plus 2 / group), and next by the instructions that unpack
// them: the logic pipe issues every second cycle, and at HBM speed an SM has 42
// cycles for the 2048 weights of a k-tile. Weights are laid out once in the order
// the tensor cores take them: tiles of 32 outputs x 64 K, 1 KB, twice 16 bytes per
// lane, which feed eight m16n8k16 products whose A is the weights and whose 8
// columns are rows of X. A code becomes the bf16 integer q - 8 in registers (exact:
// two logic instructions and a subtraction a pair), so the products run on integers
// and the scale multiplies fp32 sums of 32 K: no weight is ever rounded. The
// lane's 16 elements of K are two runs of 8, one in each half of the 64, which is
// the order the rows of X are loaded in 16-byte pieces and keeps groups of 32 apart.
//
// H is rounded to bf16 between the products, as by the bf16 experts: it is an output, and
// as the down product's 16-bit operand it takes one MMA a tile. Next to a product of the
// unrounded H that moves y by 1.7e-3 of its norm, as much as y's own rounding does.
//
// mma.sync and not tcgen05: the A operand is made in registers from 4-bit codes
// and N is 8 to 32; tcgen05 would take it through shared memory or TMEM at
// M = 128 for a product that is bound by HBM and by the unpacking either way.
//
// Gate and up share tiles: of each 16 outputs the first eight are gate columns,
// the others the same up columns, which puts G and U of one element in one lane.
//
// Measured on one GB300, both products, device time a call (floor: the weights of
// the experts that have rows at 6.8 TB/s): 128 experts, K 8, d 2048, I 768, group
// 128: 1 token 12 us (2.9), 16 tokens 48 us (30), 64 tokens 65 us (46); 64 experts,
// K 6, d 2048, I 1408, group 64: 16 tokens 50 us (34).
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

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
// The plain row of row m (0 .. 31) of tile i: output 32 i + m, or with gate and
// up in one tile output 16 i + 8 (m / 16) + m % 8 of gate (m % 16 < 8) or up.
__device__ __forceinline__ long long plain_row(long long e, int i, int m, int N, bool pair) {
  return e * N + (pair ? 16 * i + 8 * (m >> 4) + (m & 7) : 32 * i + m);
}

// One thread per word of a tile: word j of lane l's piece h is row 16 h + l / 4
// (j even) or that + 8 (odd), k = 32 (j / 2) + 8 (l % 4) + 0 .. 7; nibble n holds k
// offset 2 n (n < 4) or 2 (n - 4) + 1, so word >> 4 n & 0x000f000f is the pair
// (2 n, 2 n + 1).
__global__ void __launch_bounds__(256)
w4_pack_kernel(const uint8_t* __restrict__ ca, const uint8_t* __restrict__ cb, int N, int K, int nt,
               long long total, uint32_t* __restrict__ tiles) {
  pdl_enter();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const int j = static_cast<int>(i & 3);
  const int l = static_cast<int>(i >> 2 & 31);
  const int h = static_cast<int>(i >> 7 & 1);
  const long long tile = i >> 8;
  const int kt = K / 64;
  const int kb = static_cast<int>(tile % kt);
  const long long et = tile / kt;
  const int it = static_cast<int>(et % nt);
  const long long e = et / nt;
  const int m = 16 * h + (l >> 2) + 8 * (j & 1);
  const uint8_t* src = (cb && (m & 8)) ? cb : ca;
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

// Scales [E][tile][K / group][8][4]: of row r's four, rows r, r + 8, r + 16, r + 24
// of the tile, so that a lane takes its four with one load.
__global__ void __launch_bounds__(256)
w4_pack_scales_kernel(const uint16_t* __restrict__ sa, const uint16_t* __restrict__ sb, int N,
                      int ng, int nt, long long total, uint16_t* __restrict__ out) {
  pdl_enter();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const int m = static_cast<int>(i >> 2 & 7) + 8 * static_cast<int>(i & 3);
  const long long g = i >> 5;
  const int gi = static_cast<int>(g % ng);
  const long long et = g / ng;
  const int it = static_cast<int>(et % nt);
  const long long e = et / nt;
  const uint16_t* src = (sb && (m & 8)) ? sb : sa;
  out[i] = src[plain_row(e, it, m, N, sb != nullptr) * ng + gi];
}

// ----------------------------------------------------------------- products
// The pair (2 n, 2 n + 1) of a word as bf16 integers 128 + q: 0x4300 | q, the
// masking and the joining in one three-input logic instruction (two halve the
// kernels' speed: the logic pipe is what they wait for first).
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int n) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;"   // (a & b) | c
      : "=r"(v) : "r"(w >> (4 * n)), "r"(0x000f000fu), "r"(0x43004300u));
  return v;
}

// The same less 136, exactly q - 8. The subtraction could be left to the fp32 sums
// (start them from -136 sum x): that saves up to 2 % (4 % with groups of 32), but
// the sums would then lose what 136 sum|x| exceeds the result by.
__device__ __forceinline__ uint32_t centred(uint32_t v) {
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

// A product into d from the sums c.
__device__ __forceinline__ void mma16816_from(float (&d)[4], const float (&c)[4],
                                              const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ void add_scaled(float (&acc)[4], float s0, float s1, const float (&p)[4]) {
  acc[0] = fmaf(s0, p[0], acc[0]);
  acc[1] = fmaf(s0, p[1], acc[1]);
  acc[2] = fmaf(s1, p[2], acc[2]);
  acc[3] = fmaf(s1, p[3], acc[3]);
}

// Half a tile (32 K) against 8 NT rows of X, scaled into acc[16 outputs][rows].
// w: the lane's words of rows g and g + 8 in each 16 outputs; sc its four scales.
template <int NT>
__device__ __forceinline__ void half_tile(uint32_t w00, uint32_t w01, uint32_t w10, uint32_t w11,
                                          const uint4 (&x)[NT], uint2 sc, float (&acc)[2][NT][4]) {
  const float s[2][2] = {{bf16_lo(sc.x), bf16_hi(sc.x)}, {bf16_lo(sc.y), bf16_hi(sc.y)}};
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint32_t w0 = m ? w10 : w00, w1 = m ? w11 : w01;
    const uint32_t a0[4] = {centred(pair_of(w0, 0)), centred(pair_of(w1, 0)),
                            centred(pair_of(w0, 1)), centred(pair_of(w1, 1))};
    const uint32_t a1[4] = {centred(pair_of(w0, 2)), centred(pair_of(w1, 2)),
                            centred(pair_of(w0, 3)), centred(pair_of(w1, 3))};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
      float p[4];
      mma16816_from(p, zero, a0, x[n].x, x[n].y);
      mma16816(p, a1, x[n].z, x[n].w);
      add_scaled(acc[m][n], s[m][0], s[m][1], p);
    }
  }
}

// Each warp streams its weights through a ring of its own in shared memory: a
// stage is two k-tiles and their scales, every lane copies the 16-byte pieces that
// it will read itself, some lanes also the scales. cp.async and not registers:
// 4.6 KB a warp stay in flight and the accumulators keep the registers.
constexpr int kStages = 3;
constexpr int kStageTiles = 2;
constexpr int scale_vecs(int group) { return 256 * kStageTiles / group; }   // 16-byte pieces a stage
constexpr int stage_vecs(int group) { return 64 * kStageTiles + scale_vecs(group); }
constexpr size_t ring_bytes(int group) {
  return sizeof(uint4) * kWarps * kStages * stage_vecs(group);
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// A warp's weights: a run of k-tiles of one tile of outputs.
template <int GROUP>
struct Stream {
  const uint4* codes;    // this lane's first piece of the next stage to copy
  const uint4* scales;   // this lane's piece of its scales
  const uint4* ring;
  uint32_t to;           // this lane's place in the slot of the next copy
  int left;              // k-tiles not yet copied
  int slot;

  __device__ __forceinline__ void begin(const uint4* c, const uint4* s, uint4* r, int count) {
    const int lane = threadIdx.x & 31;
    codes = c + lane;
    scales = s + lane;
    ring = r;
    to = static_cast<uint32_t>(__cvta_generic_to_shared(r)) + 16 * lane;
    left = count;
    slot = 0;
  }
  __device__ __forceinline__ void issue() {
    const int lane = threadIdx.x & 31;
    if (left >= kStageTiles) {
#pragma unroll
      for (int p = 0; p < 2 * kStageTiles; ++p) copy16(to + 512 * p, codes + 32 * p);
      if (lane < scale_vecs(GROUP)) copy16(to + 1024 * kStageTiles, scales);
    } else if (left > 0) {   // the rest: fewer tiles and their share of the scales
      for (int p = 0; p < 2 * left; ++p) copy16(to + 512 * p, codes + 32 * p);
      if (lane < scale_vecs(GROUP) * left / kStageTiles) copy16(to + 1024 * kStageTiles, scales);
    }
    codes += 64 * kStageTiles;
    scales += scale_vecs(GROUP);
    left -= kStageTiles;
    const bool wrap = ++slot == kStages;
    to += 16 * stage_vecs(GROUP) - (wrap ? 16 * kStages * stage_vecs(GROUP) : 0);
    slot = wrap ? 0 : slot;
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

// The lane's rows of X in the p-th k-tile: both halves of 32 K.
template <int NT>
__device__ __forceinline__ void load_x(const uint4* const (&xr)[NT], int p, uint4 (&x)[2][NT]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < NT; ++n) x[h][n] = __ldg(xr[n] + 8 * p + 4 * h);
}

// One k-tile: w the lane's first piece of codes, sc its scales of the tile's first group.
template <int NT, int GROUP>
__device__ __forceinline__ void one_tile(const uint4* w, const uint2* sc, const uint4 (&x)[2][NT],
                                         float (&acc)[2][NT][4]) {
  const uint4 a = w[0], b = w[32];
  const uint2 s0 = sc[0], s1 = GROUP == 32 ? sc[8] : s0;
  half_tile<NT>(a.x, a.y, b.x, b.y, x[0], s0, acc);
  half_tile<NT>(a.z, a.w, b.z, b.w, x[1], s1, acc);
}

constexpr int scale_step(int group) { return group == 32 ? 16 : group == 64 ? 8 : 0; }

// acc += the tile's outputs over the stream's `count` k-tiles, for the 8 NT rows of
// X at xr[n] (this lane's share of the first k-tile). With 8 rows X is loaded a
// tile ahead; with more, the registers for that are missing.
template <int NT, int GROUP>
__device__ __forceinline__ void product(Stream<GROUP>& st, int count, const uint4* (&xr)[NT],
                                        float (&acc)[2][NT][4]) {
  static_assert(kStageTiles == 2, "X alternates between two buffers");
  constexpr bool kAhead = NT == 1;
  const int lane = threadIdx.x & 31, g = lane >> 2;
  uint4 x[2][2][NT];   // by the parity of the tile
  if (kAhead) load_x<NT>(xr, 0, x[0]);
  int slot = 0;
  for (; count > 0; count -= kStageTiles) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();   // this stage's scales are there, and all lanes are done with the last stage
    st.issue();
    const uint4* stage = st.ring + slot * stage_vecs(GROUP);
    slot = slot + 1 == kStages ? 0 : slot + 1;
    const uint2* sc = reinterpret_cast<const uint2*>(stage + 64 * kStageTiles) + g;
    if (count > kStageTiles) {   // a whole stage, and more after it
#pragma unroll
      for (int p = 0; p < kStageTiles; ++p) {
        if (kAhead) load_x<NT>(xr, p + 1, x[(p + 1) & 1]);
        else load_x<NT>(xr, p, x[p & 1]);
        one_tile<NT, GROUP>(stage + 64 * p + lane, sc + scale_step(GROUP) * p, x[p & 1], acc);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) xr[n] += 8 * kStageTiles;
    } else {
#pragma unroll
      for (int p = 0; p < kStageTiles; ++p) {
        if (p >= count) break;
        if (!kAhead) load_x<NT>(xr, p, x[p & 1]);
        else if (p + 1 < count) load_x<NT>(xr, p + 1, x[(p + 1) & 1]);
        one_tile<NT, GROUP>(stage + 64 * p + lane, sc + scale_step(GROUP) * p, x[p & 1], acc);
      }
    }
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
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[m][n][q] = 0.f;
  if (S > 1) __syncthreads();   // the last pass has read the sums that lie over the rings
  if (live) {
    const long long tile = static_cast<long long>(e) * A.nt + it;
    // whole pairs of k-tiles to each split, so that groups of 128 stay in one
    const int k0 = kt * ks / S & ~1, k1 = ks + 1 == S ? kt : kt * (ks + 1) / S & ~1;
    Stream<GROUP> stream;
    __syncwarp();   // every lane is done with the ring's last use
    stream.begin(A.tiles + (tile * kt + k0) * 64, A.scales + (tile * (A.K / GROUP) + k0 * 64 / GROUP) * 4,
                 ring + warp * kStages * stage_vecs(GROUP), k1 - k0);
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
    if (k0 < k1) product<NT, GROUP>(stream, k1 - k0, xr, acc);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  if (S > 1) {
    constexpr int kSums = 8 * NT;   // per lane
    __syncthreads();   // every warp is done with its ring
    float* red = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int i = 0; i < kSums; ++i) red[(warp * kSums + i) * 32 + lane] = acc[i / (4 * NT)][i / 4 % NT][i % 4];
    __syncthreads();
    if (ks != 0) return;
#pragma unroll
    for (int i = 0; i < kSums; ++i)
#pragma unroll
      for (int o = 1; o < S; ++o)
        acc[i / (4 * NT)][i / 4 % NT][i % 4] += red[((warp + o) * kSums + i) * 32 + lane];
  }
  if (!live) return;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int p = r0 + 8 * n + 2 * c + q;
      if (p >= r1) continue;
      __nv_bfloat16* row = A.out + static_cast<long long>(p) * A.N;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (GATE_UP) {
          const float G = acc[m][n][q], U = acc[m][n][q + 2];
          row[16 * it + 8 * m + g] = __float2bfloat16(__fdividef(G, 1.f + __expf(-G)) * U);
        } else {
          row[32 * it + 16 * m + g] = __float2bfloat16(acc[m][n][q]);
          row[32 * it + 16 * m + g + 8] = __float2bfloat16(acc[m][n][q + 2]);
        }
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

// ----------------------------------------------------------------- few rows per expert
// The same products for experts of about 8 rows or fewer, as one persistent block
// of 16 warps per SM. An entry is up to 8 rows of one expert, an item one tile of
// 32 outputs for one entry; a block takes a contiguous run of items, the same
// number as every other block, and its warps share that run's k-tiles evenly,
// each a contiguous piece of them. A warp's weight stream so runs on from item to
// item, the rows of X of the block's entries lie in shared memory, and no warp has
// more to do than another, from one token (an item over six warps) to a full batch
// (five items a warp). An item that crosses warps is finished by the warp that has
// its first k-tile, from the other warps' sums in shared memory.

constexpr int kDWarps = 16;
constexpr int kDThreads = kDWarps * 32;
constexpr int kDRows = 32;                      // most rows of X in shared memory
constexpr int kSums = 8;                        // of a lane for one item
constexpr size_t kDecodeSmem = 226 * 1024;

constexpr int row_vecs(int K) { return K / 8 + 4; }   // rows 64 bytes apart modulo 128
constexpr size_t decode_ring_bytes(int group) {
  return sizeof(uint4) * kDWarps * kStages * stage_vecs(group);
}
constexpr size_t decode_row_bytes(int K) { return sizeof(uint4) * row_vecs(K); }
constexpr size_t decode_fixed_bytes(int group, int E) {
  return decode_ring_bytes(group) + sizeof(float) * kDWarps * kSums * 32 +
         sizeof(int) * (2 * (E + 1) + 4 * kDRows + 4);
}
// Rows of X that fit beside the rest, at most kDRows.
int decode_rows(int group, int K, int E) {
  const size_t fixed = decode_fixed_bytes(group, E);
  if (fixed >= kDecodeSmem) return 0;
  return static_cast<int>(std::min<size_t>(kDRows, (kDecodeSmem - fixed) / decode_row_bytes(K)));
}

// The expert of an entry: the last e with first[e] <= entry.
__device__ __forceinline__ int entry_expert(const int* first, int E, int entry) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= entry) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <bool GATE_UP, int GROUP>
__global__ void __launch_bounds__(kDThreads, 1) w4_decode_kernel(W4Args A, int cap) {
  extern __shared__ uint4 smem[];
  uint4* const ring = smem;
  uint4* const panel = ring + decode_ring_bytes(GROUP) / sizeof(uint4);           // [cap] rows
  float* const red = reinterpret_cast<float*>(panel + cap * row_vecs(A.K));       // [warp][kSums][lane]
  int* const offs = reinterpret_cast<int*>(red + kDWarps * kSums * 32);           // [E + 1]
  int* const first = offs + A.E + 1;      // [E + 1] first entry of each expert
  int* const c_expert = first + A.E + 1;  // of each entry at hand: its expert,
  int* const c_row = c_expert + kDRows;   // its first row,
  int* const c_rows = c_row + kDRows;     // its rows,
  int* const c_at = c_rows + kDRows;      // their place in the panel; [count] ends it
  int* const c_end = c_at + kDRows + 1;   // the first item past the entries at hand
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int kt = A.K / 64;
  // The down projection's offsets and weights are older than the launch before
  // it (that launch has waited for all earlier ones), so they are read before the
  // wait for H. No thread leaves without the wait.
  if (GATE_UP) pdl_wait();
  pdl_launch_dependents();
  for (int e = threadIdx.x; e <= A.E; e += kDThreads) offs[e] = min(__ldcg(A.offsets + e), A.M);
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base < A.E; base += 32) {
      const int e = base + lane;
      const int n = e < A.E ? (offs[e + 1] - offs[e] + 7) / 8 : 0;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (e < A.E) first[e] = carry + x - n;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) first[A.E] = carry;
  }
  __syncthreads();
  const long long total = static_cast<long long>(first[A.E]) * A.nt;
  const int end = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
  int c0 = static_cast<int>(total * blockIdx.x / gridDim.x);
  bool waited = GATE_UP;
  Stream<GROUP> stream;
  while (c0 < end) {
    // The entries at hand: from item c0 on, as many as the panel holds rows of.
    const int entry0 = c0 / A.nt;
    if (threadIdx.x == 0) {
      int e = entry_expert(first, A.E, entry0), n = 0, at = 0;
      for (int entry = entry0; n < kDRows && static_cast<long long>(entry) * A.nt < end; ++entry) {
        while (entry >= first[e + 1]) ++e;
        const int row = offs[e] + 8 * (entry - first[e]);
        const int rows = min(offs[e + 1] - row, 8);
        if (at + rows > cap) break;
        c_expert[n] = e;
        c_row[n] = row;
        c_rows[n] = rows;
        c_at[n] = at;
        at += rows;
        ++n;
      }
      c_at[n] = at;
      *c_end = static_cast<int>(min(static_cast<long long>(entry0 + n) * A.nt, static_cast<long long>(end)));
    }
    __syncthreads();
    const int c1 = *c_end;
    const int entries = (c1 - 1) / A.nt - entry0 + 1;
    // This warp's piece of the items' k-tiles (whole pairs, which groups of 128 need).
    const int unit = kt & 1 ? 1 : 2;
    const long long units = static_cast<long long>(c1 - c0) * kt / unit;
    auto piece = [&](int w) { return static_cast<int>(units * w / kDWarps) * unit; };
    const int t0 = piece(warp), t1 = piece(warp + 1);
    int ahead = t0;
    stream.begin(A.tiles, A.scales, ring + warp * kStages * stage_vecs(GROUP), 0);
    auto issue = [&]() {
      if (stream.left <= 0 && ahead < t1) {   // on to the next item's run
        const int i = ahead / kt, k = ahead - i * kt;
        const int entry = (c0 + i) / A.nt;
        const long long tile = static_cast<long long>(c_expert[entry - entry0]) * A.nt + (c0 + i - entry * A.nt);
        stream.codes = A.tiles + (tile * kt + k) * 64 + lane;
        stream.scales = A.scales + (tile * (A.K / GROUP) + k * 64 / GROUP) * 4 + lane;
        stream.left = min(kt - k, t1 - ahead);
        ahead += stream.left;
      }
      stream.issue();
    };
    for (int p = 0; p + 1 < kStages; ++p) issue();
    if (!waited) {
      pdl_wait();
      waited = true;
    }
    // The entries' rows of X, a warp per row.
    const int nv = A.K / 8, rows = c_at[entries];
    for (int j = warp, i = 0; j < rows; j += kDWarps) {
      while (j >= c_at[i + 1]) ++i;
      int row = c_row[i] + j - c_at[i];
      if (GATE_UP && A.perm) row = __ldg(A.perm + row) / A.top_k;
      if (!index_ok(row >= 0 && row < A.x_rows)) row = 0;
      const uint4* from = reinterpret_cast<const uint4*>(A.x) + static_cast<long long>(row) * nv;
      const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(panel + j * row_vecs(A.K)));
      for (int v = lane; v < nv; v += 32) copy16(to + 16 * v, from + v);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    float acc[2][1][4];
    int item = 0, run = 0, k = 0;
    auto finish = [&]() {   // acc is the whole of `item`
      const int entry = (c0 + item) / A.nt, i = entry - entry0;
      const int it = c0 + item - entry * A.nt, n = c_rows[i];
      __nv_bfloat16* const out = A.out + static_cast<long long>(c_row[i]) * A.N;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (2 * c + q >= n) continue;
        __nv_bfloat16* row = out + static_cast<long long>(2 * c + q) * A.N;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (GATE_UP) {
            const float G = acc[m][0][q], U = acc[m][0][q + 2];
            row[16 * it + 8 * m + g] = __float2bfloat16(__fdividef(G, 1.f + __expf(-G)) * U);
          } else {
            row[32 * it + 16 * m + g] = __float2bfloat16(acc[m][0][q]);
            row[32 * it + 16 * m + g + 8] = __float2bfloat16(acc[m][0][q + 2]);
          }
        }
      }
    };
    for (int t = t0; t < t1; t += run) {
      item = t / kt;
      k = t - item * kt;
      run = min(kt - k, t1 - t);
      const int i = (c0 + item) / A.nt - entry0;
      const int row = c_at[i] + min(g, c_rows[i] - 1);   // past the last row: that row
      const uint4* xk = panel + row * row_vecs(A.K) + c + 8 * k;
#pragma unroll
      for (int j = 0; j < kSums; ++j) acc[j / 4][0][j % 4] = 0.f;
      for (int left = run; left > 0; left -= kStageTiles) {
        const int slot = stream.slot + 1 == kStages ? 0 : stream.slot + 1;   // the oldest stage
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();   // its scales are there, and all lanes are done with the last stage
        issue();
        const uint4* stage = stream.ring + slot * stage_vecs(GROUP);
        const uint2* sc = reinterpret_cast<const uint2*>(stage + 64 * kStageTiles) + g;
#pragma unroll
        for (int p = 0; p < kStageTiles; ++p) {
          if (p >= left) break;
          const uint4 a = stage[64 * p + lane], b = stage[64 * p + 32 + lane];
          const uint2 s0 = sc[scale_step(GROUP) * p];
          const uint2 s1 = GROUP == 32 ? sc[scale_step(GROUP) * p + 8] : s0;
          const uint4 x0[1] = {xk[8 * p]}, x1[1] = {xk[8 * p + 4]};
          half_tile<1>(a.x, a.y, b.x, b.y, x0, s0, acc);
          half_tile<1>(a.z, a.w, b.z, b.w, x1, s1, acc);
        }
        xk += 8 * kStageTiles;
      }
      if (k != 0) {   // the end, or the middle, of an item begun by an earlier warp
#pragma unroll
        for (int j = 0; j < kSums; ++j) red[(warp * kSums + j) * 32 + lane] = acc[j / 4][0][j % 4];
      } else if (run == kt) {
        finish();
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (t0 < t1 && k == 0 && run < kt) {   // this warp's last item goes on in the next warps
      int need = kt - run;
      for (int w = warp + 1; need > 0; ++w) {
        const int n = min(need, piece(w + 1) - piece(w));
        if (n > 0) {
#pragma unroll
          for (int j = 0; j < kSums; ++j) acc[j / 4][0][j % 4] += red[(w * kSums + j) * 32 + lane];
        }
        need -= n;
      }
      finish();
    }
    c0 = c1;
    __syncthreads();   // panel, sums and entries are free again
  }
  if (!waited) pdl_wait();
}

template <bool GATE_UP, int S, int NTMAX, int GROUP>
int launch_kernel(dim3 grid, const W4Args& a, cudaStream_t st) {
  static_assert(ring_bytes(GROUP) >= sizeof(float) * kWarps * NTMAX * 8 * 32, "sums over the rings");
  auto kern = w4_kernel<GATE_UP, S, NTMAX, GROUP>;
  static thread_local int configured = -1;   // the device this thread raised the limit on
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured != dev) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(ring_bytes(GROUP)));
    if (e != cudaSuccess) {
      set_last_cuda_error(e);
      return MOE_ERR_CUDA;
    }
    configured = dev;
  }
  return launch_pdl(kern, grid, kThreads, ring_bytes(GROUP), st, 1, a);
}

template <bool GATE_UP, int NTMAX, int GROUP>
int launch_split(int S, dim3 grid, const W4Args& a, cudaStream_t st) {
  if (S == 1) return launch_kernel<GATE_UP, 1, NTMAX, GROUP>(grid, a, st);
  if (S == 2) return launch_kernel<GATE_UP, 2, NTMAX, GROUP>(grid, a, st);
  if (S == 4) return launch_kernel<GATE_UP, 4, NTMAX, GROUP>(grid, a, st);
  return launch_kernel<GATE_UP, 8, NTMAX, GROUP>(grid, a, st);
}

// Launches the persistent kernel with room for `cap` rows of X.
template <bool GATE_UP, int GROUP>
int launch_decode(const W4Args& a, int cap, cudaStream_t st) {
  auto kern = w4_decode_kernel<GATE_UP, GROUP>;
  static thread_local int configured = -1;   // the device this thread raised the limit on
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured != dev) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kDecodeSmem));
    if (e != cudaSuccess) {
      set_last_cuda_error(e);
      return MOE_ERR_CUDA;
    }
    configured = dev;
  }
  const size_t smem = decode_fixed_bytes(GROUP, a.E) + cap * decode_row_bytes(a.K);
  return launch_pdl(kern, num_sms(), kDThreads, smem, st, 1, a, cap);
}

// The persistent kernel is for few rows per expert (mean, rounded up) and enough
// k-tiles to share; its measured times against the other kernel's, both products:
//   1 row   (16 tokens, 128 experts, K 8, d 2048, I 768)    48 : 56 us
//   4 rows  (64 tokens)                                     65 : 81 us
//   8 rows  (128 tokens)                                    87 : 97 us
//   12 rows (192 tokens)                                   116 : 118 us
//   16 rows (256 tokens)                                   143 : 144 us
//   16 rows (256 tokens, 64 experts, K 4, I 1408)          134 : 141 us
//   16 rows (128 tokens, 32 experts, K 4, d 4096, I 2048)  174 : 179 us
//   32 rows (256 tokens)                                   315 : 280 us
// and by the k-tiles of a product at less than 1 row. The gate and up product
// starts behind the kernel's reading of the row counts, the down product does that
// while the first one ends, so they pay from different counts on:
//   gate and up 25 K (2 tokens, 128 experts)    18.0 : 15.8 us
//               33 K (1 token, 32 experts)      21.7 : 20.0 us
//               37 K (3 tokens, 128 experts)    20.8 : 21.8 us
//   down        25 K (4 tokens, 128 experts)    25.5 : 27.3 us
//               33 K (2 tokens, 32 experts)     29.7 : 32.0 us
// A block has to hold an entry's 8 rows of X, which ends the persistent kernel at K = 6400 to
// 6976 (groups of 32 to 128): gate and up of wider models take the other one. Both products,
// 32 experts, K 4, I 2048, floor in brackets: d 6656, 16, 64 and 128 tokens 113 (90), 166 and
// 280 us (99); d 7168 135 (97), 187 and 279 (107); d 8192 140 (103), 216 and 333 (122).
constexpr int kDecodeRows = 16;
constexpr int kGateUpTiles = 36000;
constexpr int kDownTiles = 20000;

// most_rows: a bound on the rows of one expert.
template <bool GATE_UP>
int launch_w4(const char* name, const W4Args& a, int most_rows, cudaStream_t st) {
  const int slots = std::min(a.E, a.M);
  const int mean_rows = std::min(most_rows, (a.M - 1) / a.E + 1);
  const long long entries = a.E + a.M / 8;   // at most
  const int cap = decode_rows(a.group, a.K, a.E);
  const long long k_tiles = static_cast<long long>(slots) * a.nt * (a.K / 64);
  if (mean_rows <= kDecodeRows && k_tiles >= (GATE_UP ? kGateUpTiles : kDownTiles) &&
      cap >= 8 && entries * a.nt * (a.K / 64) < 0x7fffffffLL) {
    ProfScope prof(name, st);
    if (a.group == 32) return launch_decode<GATE_UP, 32>(a, cap, st);
    if (a.group == 64) return launch_decode<GATE_UP, 64>(a, cap, st);
    return launch_decode<GATE_UP, 128>(a, cap, st);
  }
  // Split K until the launch has about 24 warps per SM three times over, a warp
  // keeping four k-tiles at least. Against a third and three times of that, 32 experts,
  // K 4, I 2048: 256 tokens of d 4096 272 us (332, 331), 128 of d 8192 333 (373, 353); a few
  // tokens take the same time (1 of d 8192: 31 us each).
  const long long want = static_cast<long long>(num_sms()) * 72;
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
  // Rows of a pass: the weights are read again for every 8, 16 or 32 rows of an
  // expert, and the wider passes leave room for fewer warps. 128 experts, K 8,
  // d 2048, I 768, with 8, 16 and 32 rows a pass: 4 rows per expert 81, 83 and 85 us,
  // 8 rows 108, 97 and 99 us, 16 rows 170, 144 and 146 us, 24 rows 215, 179 and
  // 175 us, 32 rows 379, 307 and 280 us.
  if (mean_rows <= 6) return by_group(std::integral_constant<int, 1>());
  if (mean_rows <= 16) return by_group(std::integral_constant<int, 2>());
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
      (codes_b == nullptr) != (scales_b == nullptr) || N % (codes_b ? 16 : 32))
    return MOE_ERR_INVALID_ARG;
  if (!codes_a || !scales_a || !tiles || !scales) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {codes_a, scales_a, codes_b, scales_b, tiles, scales};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_MISALIGNED;
  const int nt = codes_b ? N / 16 : N / 32, ng = K / group;
  const long long words = static_cast<long long>(E) * nt * (K / 64) * 256;
  const long long ns = static_cast<long long>(E) * nt * ng * 32;
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
  a.nt = I / 16;
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
  a.nt = d / 32;
  a.group = group_d;
  a.x_rows = M;
  return launch_w4<false>("w4_down", a, perm ? T : M, st);
}

namespace moe {
MOE_DEBUG_STATUS_READER(w4)
}  // namespace moe
