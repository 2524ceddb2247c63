// Products grouped by expert on microscaled 4-bit floats: the plain product Y = X W[e]^T
// and the SwiGLU experts built from it.
//
// Rows of X and outputs of W are E2M1 codes with K contiguous and one scale per 16 (E4M3,
// with a 32-bit factor per row of X and per expert) or per 32 (power of two); see fp4.cuh.
// The tensor cores multiply codes and block scales exactly and sum in fp32
// (tcgen05.mma kind::mxf4nvf4 with four scales per 64 K, kind::mxf4 with two); the 32-bit
// factors multiply the sums so that only a result outside fp32's range leaves it.
//
// Kernel shape: the bf16 kernels' (grouped_gemm.cu): clusters of two CTAs share MMAs of
// M = 256, persistent over a tile list that every CTA derives from the expert offsets, one
// TMA warp, one MMA warp, epilogue warps, every wait bounded. What differs:
//   * a k-block is 256 K (128-byte swizzled rows, as a bf16 k-block of 64), four MMAs of 64 K;
//   * scales come as 512-byte atoms (128 rows x 4 scales), KA per k-block for the CTA's A rows
//     and for each 128 of the pair's B columns, and are copied to TMEM (tcgen05.cp) into one
//     of kRing slots beside the accumulator. A slot is written again only when the MMAs that
//     read it have completed (their stage's empty barrier says so);
//   * one 256 x BN accumulator: eight epilogue warps take it into registers at once (128
//     columns a thread) and hand it back before they work on it, so the next tile's MMAs wait
//     for the TMEM loads only. (Two accumulators of 256 columns leave no TMEM for scales.)
//     The drafter workload's gate and up (262144 rows, d 4096, I 2048): 1.28 ms, 6.9 PFLOP/s.
//     Parts by themselves: MMAs and copies of scales 1.03 ms (8.6 PFLOP/s, the rate of steps of
//     64 K), loads 0.94, both together without the epilogue's work 1.16, MMAs with the epilogue
//     1.13. Its down projection: 0.79 ms, MMAs 0.56, loads 0.46, both 0.60; there the epilogue's
//     bf16 stores count for most (loads and epilogue without MMAs 0.67). So no single part binds:
//     MMAs and loads take nearly as long as each other and slow each other by a seventh, and a
//     tile's epilogue is hidden in part (one accumulator). sm_103a also has steps of 96 K, which
//     these kernels do not use;
//   * the MMA thread is elected (elect_one): with a branch on the lane number the same gate and
//     up took 3.6 ms;
//   * the SwiGLU epilogue quantizes H in registers: codes and scale words leave directly, and
//     H never exists in bf16 unless its rows are to be scaled by their own maximum.
#include "fp4.cuh"
#include "tc.cuh"

namespace moe {
namespace fp4 {

using namespace gemm;   // PTX helpers, tensor maps

int launch_quantize(const void* x, const int32_t* inv_perm, const int32_t* offsets, int E, int T,
                    int K, int M, int d, int block, void* q, void* sf, float* row_scale,
                    cudaStream_t st, const char* name);   // fp4.cu

namespace {

enum Epi : int {
  OUT = 0,   // Y in bf16
  H4 = 1,    // SwiGLU, H quantized
  HB = 2     // SwiGLU, H in bf16
};

constexpr int BM = 128;          // rows of a CTA
constexpr int kThreads = 320;    // TMA warp, MMA warp, eight epilogue warps
constexpr int kRing = 3;         // scale slots in TMEM
constexpr uint32_t kScaleCol = 256;

struct Params {
  const int32_t* offsets;
  int E, M;
  int N;               // outputs (SwiGLU: I, of gate and of up each)
  int k64;             // K / 64
  int n_tiles;         // tiles along N
  int sf_tiles;        // scale tiles of 128 B rows per expert
  const float* row_scale;   // [M] or null
  const float* scale0;      // [E] or null: the matrix's factor (gate's)
  const float* scale1;      // [E] or null: up's, or (OUT) a factor of X's rows per expert
  const float* h_scale;     // [E] or null (H4)
  __nv_bfloat16* out;       // y or h, row length N
  uint8_t* hq;              // H4: codes [M, N / 2]
  uint32_t* hsf;            // H4: scale words
  int h_atoms;              // H4: atoms along H's K
  int* status;
};

struct Tile {
  int e, row0, rows, n0, mg, nt;
};

template <int EPI, int BN>
__device__ __forceinline__ Tile decode(int t, int rank, const Params& p, const int* s_off,
                                       const int* s_mp) {
  Tile tl;
  tl.mg = t / p.n_tiles;
  tl.nt = t - tl.mg * p.n_tiles;
  int lo = 0, hi = p.E - 1;   // largest e with s_mp[e] <= mg
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_mp[mid] <= tl.mg) lo = mid; else hi = mid - 1;
  }
  tl.e = lo;
  tl.row0 = s_off[lo] + (2 * (tl.mg - s_mp[lo]) + rank) * BM;
  tl.rows = min(BM, s_off[lo + 1] - tl.row0);
  tl.n0 = tl.nt * (EPI == OUT ? BN : BN / 2);
  return tl;
}

// fp32 D, E2M1 A and B (K-major), scales E4M3 (block 16) or powers of two, M = 256.
template <int N, int BLOCK>
__host__ __device__ constexpr uint32_t make_idesc_fp4() {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         ((BLOCK == 32 ? 1u : 0u) << 23) | (static_cast<uint32_t>(256 >> 4) << 24);
}

template <int BLOCK>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  if constexpr (BLOCK == 16)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4],"
        " [%5], p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4],"
        " [%5], p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ int exponent_of(float v) {   // of a normal v: floor(log2 |v|)
  return static_cast<int>((__float_as_uint(v) >> 23) & 0xffu) - 127;
}

// a b and a b c stay among the normal numbers.
__device__ __forceinline__ bool product_in_range(float a, float b, float c) {
  const int ab = exponent_of(a) + exponent_of(b);
  return abs(ab) <= 120 && abs(ab + exponent_of(c)) <= 120;
}

// The factors a, b, c of a sum as one to multiply it by after `pre`, a power of two that takes half of
// their exponent, so that neither step leaves fp32's range unless the result does, and a sum of zero
// stays zero. (A sum is 0 or 2^-20 to 2^40 in size.) The mantissas' product is rounded as a b c is.
__device__ __forceinline__ float split_factors(float a, float b, float c, float& pre) {
  pre = 1.f;
  int ea, eb, ec;
  const float m = frexpf(a, &ea) * frexpf(b, &eb) * frexpf(c, &ec);
  if (!(fabsf(m) <= 1.f)) return m;   // Inf or NaN
  const int e = ea + eb + ec;
  const int half = max(-126, min(127, e / 2));
  pre = two_to(half);
  return m * two_to(max(-126, min(127, e - half)));
}

// Output staging: boxes of 32 rows x 64 columns a warp, used in turn.
template <int EPI, int BOXES>
constexpr uint32_t epi_bytes() { return EPI == OUT ? 8u * BOXES * 4096u : 0u; }

template <int EPI, int BLOCK, int BN, int STAGES, int BOXES>
struct Shape {
  static constexpr uint32_t KA = 64 / BLOCK;            // scale atoms of a k-block (256 K)
  static constexpr uint32_t NB = BN / 128;              // B's scale tiles
  static constexpr uint32_t A = BM * 128;
  static constexpr uint32_t B = (BN / 2) * 128;
  static constexpr uint32_t SA = KA * 512;
  static constexpr uint32_t SB = KA * 512 * NB;
  static constexpr uint32_t STAGE = (A + B + SA + SB + 1023) / 1024 * 1024;
  static constexpr uint32_t SLOT = 4 * KA * (1 + NB);   // TMEM columns of a k-block's scales
  // At least 116 KB: a CTA takes all of its SM's TMEM, so two must not share one.
  static constexpr size_t smem(int E) {
    const size_t n = 1024 + STAGES * STAGE + epi_bytes<EPI, BOXES>() + 8 * (2 * STAGES + 3) + 16 +
                     sizeof(int) * 2 * (E + 1) + 16;
    return n < 118784 ? 118784 : n;
  }
  static_assert(kScaleCol + kRing * SLOT <= 512, "scale slots in TMEM");
  static_assert(BN <= static_cast<int>(kScaleCol), "accumulator below the scale slots");
};

template <int EPI, int BLOCK, int BN, int STAGES, int BOXES>
__global__ void __launch_bounds__(kThreads, 1)
fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmSA,
                const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmC,
                const Params p) {
  using S = Shape<EPI, BLOCK, BN, STAGES, BOXES>;
  constexpr uint32_t IDESC = make_idesc_fp4<BN, BLOCK>();

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* epi = smem + STAGES * S::STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(epi + epi_bytes<EPI, BOXES>());
  // bars: full[STAGES] (leader), empty[STAGES], tfull, tempty (leader), drain
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_off = reinterpret_cast<int*>(tmem_slot + 4);
  int* s_mp = s_off + (p.E + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = (rank == 0);
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t bar_base = smem_u32(bars);
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  const uint32_t tfull_bar = bar_base + 8u * (2 * STAGES);
  const uint32_t tempty_bar = bar_base + 8u * (2 * STAGES + 1);
  const uint32_t drain_bar = bar_base + 8u * (2 * STAGES + 2);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(full_bar(s), 1); mbar_init(empty_bar(s), 1); }
    mbar_init(tfull_bar, 1);
    mbar_init(tempty_bar, 16);   // the eight epilogue warps of both CTAs
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (const CUtensorMap* m : {&tmA, &tmB0, &tmB1, &tmSA, &tmSB, &tmC})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  if (warp == 1) {   // one warp in each CTA of the pair allocates collectively
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_wait();   // offsets and operands come from earlier launches
  pdl_launch_dependents();
  // H goes to the workspace
  if (EPI != OUT && blockIdx.x == 0 && threadIdx.x == 0) end_backward_record(p.status);
  for (int e = threadIdx.x; e <= p.E; e += kThreads) s_off[e] = __ldg(p.offsets + e);
  __syncthreads();
  bool offs_ok = true;
#ifdef MOE_DEBUG_CHECKS
  for (int e = threadIdx.x; e < p.E; e += kThreads) offs_ok = offs_ok && s_off[e] <= s_off[e + 1];
  if (threadIdx.x == 0) offs_ok = offs_ok && s_off[0] == 0 && s_off[p.E] <= p.M;
  offs_ok = __syncthreads_and(offs_ok) != 0;
  if (!offs_ok && threadIdx.x == 0) report_status(p.status, MOE_ERR_DEVICE_CHECK);
  index_ok(offs_ok);
#endif
  if (warp == 0) {   // exclusive prefix of per-expert m-tile pairs
    int carry = 0;
    for (int base = 0; base <= p.E; base += 32) {
      const int i = base + lane;
      const int v = (i < p.E) ? ((s_off[i + 1] - s_off[i] + BM - 1) / BM + 1) / 2 : 0;
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (i <= p.E) s_mp[i] = carry + x - v;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // both CTAs' barriers exist before any remote arrive or TMA
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // both CTAs must hold the same TMEM columns for the pair's MMAs; otherwise do nothing
  uint32_t peer_base;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(peer_base)
               : "r"(map_to_rank(smem_u32(tmem_slot), rank ^ 1u))
               : "memory");
  const bool tmem_ok = (peer_base == tmem_base);
  if (!tmem_ok && threadIdx.x == 0) report_status(p.status, MOE_ERR_DEVICE_CHECK);
  const int total = (tmem_ok && offs_ok) ? s_mp[p.E] * p.n_tiles : 0;
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(n_clusters_x());
  const int k_blocks = (p.k64 + 3) / 4;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      unsigned long long issued = 0;   // k-blocks
      bool ok = true;
      const uint32_t full0 = map_to_rank(full_bar(0), 0);   // the leader's
      const CUtensorMap* mb = EPI != OUT && rank ? &tmB1 : &tmB0;
      for (int t = cid; t < total && ok; t += ncl) {
        const Tile tl = decode<EPI, BN>(t, static_cast<int>(rank), p, s_off, s_mp);
        // a follower without rows (the expert's end) loads no A: its rows are not stored
        const int rows1 = leader ? s_off[tl.e + 1] - (tl.row0 + BM) : tl.rows;
        const bool load_a = leader || rows1 > 0;
        const uint32_t bytes = 2 * (S::B + S::SB) + (rows1 > 0 ? 2u : 1u) * (S::A + S::SA);
        const int brow = EPI == OUT ? tl.n0 + static_cast<int>(rank) * (BN / 2) : tl.n0;
        const int a_tile = 2 * tl.mg + static_cast<int>(rank);
        const int b_tile = tl.e * p.sf_tiles + tl.nt * static_cast<int>(S::NB);
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
          if (leader) mbar_expect_tx(full_bar(stage), bytes);   // both CTAs' boxes
          const uint32_t fb = full0 + 8u * stage;
          const uint32_t sa = smem_base + stage * S::STAGE;
          const uint32_t ssa = sa + S::A + S::B;
          const int ka = kb * static_cast<int>(S::KA);
          if (load_a) {
            tma_load_2d_pair(sa, &tmA, fb, kb * 128, tl.row0);
            tma_load_3d_pair(ssa, &tmSA, fb, 0, ka, a_tile);
          }
          tma_load_3d_pair(sa + S::A, mb, fb, kb * 128, brow, tl.e);
          tma_load_3d_pair(ssa + S::SA, &tmSB, fb, 0, ka, b_tile);
          ++issued;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (leader) {
        // the leader's full barriers count both CTAs' loads: wait for the last phases
        for (int s = 0; s < STAGES; ++s) {
          const unsigned long long uses = (issued + STAGES - 1 - s) / STAGES;
          if (!uses) continue;
          const uint32_t par = static_cast<uint32_t>(uses - 1) & 1u;
          const uint64_t t0 = globaltimer();
          while (!mbar_try(full_bar(s), par) && globaltimer() - t0 < kTimeoutNs) {
          }
        }
      } else if (!ok) {
        // loads of this CTA may still be landing after a timeout: give them a moment
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (leader && elect_one()) {
      const int my_tiles = total > cid ? (total - cid + ncl - 1) / ncl : 0;
      // descriptors of stage 0; other addresses are added in units of 16 bytes
      const uint64_t desc_op = smem_desc(smem_base, 16, 1024);
      const uint64_t desc_sf = smem_desc_rows16(smem_base + S::A + S::B);
      int stage = 0, slot_i = 0, old_stage = 0;
      uint32_t phase = 0, old_phase = 0;
      int fresh = kRing;   // scale slots not yet used
      bool ok = true;
      for (int j = 0; j < my_tiles && ok; ++j) {
        for (int kb = 0; kb < k_blocks; ++kb) {
          if (!mbar_wait(full_bar(stage), phase, abort_flag, p.status)) { ok = false; break; }
          // the slot's last readers, the MMAs of kRing blocks ago, have completed
          if (fresh) {
            --fresh;
          } else {
            if (!mbar_wait(empty_bar(old_stage), old_phase, abort_flag, p.status)) { ok = false; break; }
            if (++old_stage == STAGES) { old_stage = 0; old_phase ^= 1u; }
          }
          tc_fence_after();
          const uint32_t slot = tmem_base + kScaleCol + S::SLOT * static_cast<uint32_t>(slot_i);
          const uint64_t sf = desc_sf + static_cast<uint32_t>(stage) * (S::STAGE / 16);
#pragma unroll
          for (uint32_t k = 0; k < S::KA; ++k) tc_cp_pair_32x128(slot + 4 * k, sf + 32 * k);
#pragma unroll
          for (uint32_t b = 0; b < S::NB; ++b)
#pragma unroll
            for (uint32_t k = 0; k < S::KA; ++k)
              tc_cp_pair_32x128(slot + 4 * S::KA + 4 * (k * S::NB + b),
                                sf + S::SA / 16 + 32 * (b * S::KA + k));
          // the accumulator, once the first block's operands and scales are in place
          if (kb == 0) {
            if (!mbar_wait(tempty_bar, static_cast<uint32_t>(j & 1) ^ 1u, abort_flag, p.status)) { ok = false; break; }
            tc_fence_after();
          }
          const uint64_t da = desc_op + static_cast<uint32_t>(stage) * (S::STAGE / 16);
          const int steps = min(4, p.k64 - 4 * kb);
          auto step = [&](uint32_t kk, uint32_t acc) {   // 64 K: 32 bytes of a row
            const uint32_t ka = BLOCK == 16 ? kk : kk / 2;
            const uint32_t id = BLOCK == 16 ? 0u : 2u * (kk & 1);
            mma_fp4<BLOCK>(tmem_base, da + 2 * kk, da + S::A / 16 + 2 * kk,
                           IDESC | (id << 4) | (id << 29), slot + 4 * ka,
                           slot + 4 * S::KA + 4 * S::NB * ka, acc);
          };
          if (steps == 4) {
            step(0, kb != 0);
            step(1, 1);
            step(2, 1);
            step(3, 1);
          } else {
            for (int kk = 0; kk < steps; ++kk) step(kk, (kb | kk) != 0);
          }
          tc_commit_pair_both(empty_bar(stage));
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          if (++slot_i == kRing) slot_i = 0;
        }
        if (!ok) break;
        tc_commit_pair_both(tfull_bar);
      }
      tc_commit_pair_local(drain_bar);
      const uint64_t t0 = globaltimer();
      while (!mbar_try(drain_bar, 0) && globaltimer() - t0 < kTimeoutNs) {
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    // Two warps per 32 rows, each half the columns (SwiGLU: half of gate's and of up's).
    const int q = warp & 3;
    const int hh = (warp - 2) >> 2;
    const int r = q * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    constexpr int W = BN / 2;    // accumulator columns of a thread
    uint32_t box = 0;
    uint32_t phase = 0;
    for (int t = cid; t < total; t += ncl) {
      const Tile tl = decode<EPI, BN>(t, static_cast<int>(rank), p, s_off, s_mp);
      const bool valid = r < tl.rows;
      const size_t grow = static_cast<size_t>(tl.row0 + r);
      float rs = 1.f;
      if (p.row_scale && valid) rs = __ldg(p.row_scale + grow);
      float f0 = p.scale0 ? __ldg(p.scale0 + tl.e) : 1.f;
      float f1 = p.scale1 ? __ldg(p.scale1 + tl.e) : 1.f;
      // OUT: rs f0 f1 for all columns; SwiGLU: rs f0 for gate's, rs f1 for up's
      const bool far = __any_sync(0xffffffffu, EPI == OUT ? !product_in_range(rs, f0, f1)
                                                          : !product_in_range(rs, f0, 1.f) ||
                                                                !product_in_range(rs, f1, 1.f));
      const float hs = EPI == H4 && p.h_scale ? __ldg(p.h_scale + tl.e) : 1.f;
      if (!mbar_wait(tfull_bar, phase, abort_flag, p.status)) break;
      phase ^= 1u;
      tc_fence_after();
      const uint32_t tacc = tmem_base + lane_addr;
      // Factors far from one, which data of usual sizes never meets: half of their exponent is
      // multiplied into the accumulator in place. (Where it does not happen the experts on 98304
      // rows, d 2048, I 1408, take 392 us with these lines and 390 without; with the same on the
      // registers, after the loads, 397.)
      if (far) {
        float pre0, pre1 = 1.f;
        if constexpr (EPI == OUT) {
          f0 = split_factors(rs, f0, f1, pre0);
          f1 = 1.f;
        } else {
          f0 = split_factors(rs, f0, 1.f, pre0);
          f1 = split_factors(rs, f1, 1.f, pre1);
        }
        rs = 1.f;
        __syncwarp();
        // this warp's columns: [hh W, +W); SwiGLU: [hh W/2, +W/2) of gate's half, then of up's
#pragma unroll 1
        for (int c = 0; c < W; c += 16) {
          const bool up = EPI != OUT && c >= W / 2;
          float s[16];
          const uint32_t at = tacc + (EPI == OUT ? hh * W + c : hh * (W / 2) + c + (up ? BN / 2 - W / 2 : 0));
          tmem_ld16(at, s);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] *= up ? pre1 : pre0;
          tmem_st16(at, s);
        }
        tmem_wait_st();
      }
      float v[W];
      {
        float (*chunk)[32] = reinterpret_cast<float (*)[32]>(v);
#pragma unroll
        for (int c = 0; c < W / 32; ++c) {
          // OUT: columns [hh W, +W); SwiGLU: [hh W/2, +W/2) of gate, then of up
          const int col = EPI == OUT ? hh * W + 32 * c
                                     : (2 * c < W / 32 ? 0 : BN / 2 - W / 2) + hh * (W / 2) + 32 * c;
          tmem_ld32(tacc + col, chunk[c]);
        }
        tmem_wait_ld();
      }
      tc_fence_before();
      __syncwarp();
      // relaxed: the barrier orders TMEM reads alone, which have completed; a release would wait
      // for the last tile's stores
      if (lane == 0) mbar_arrive_cluster_relaxed(map_to_rank(tempty_bar, 0));
      // A branch the compiler cannot remove: without one it moves arithmetic of the epilogue above
      // the arrive, which the next tile's MMAs wait for (gate/up 1390 -> 1296 us).
      if (*abort_flag) break;

      if constexpr (EPI == OUT) {
        const float f = rs * f0 * f1;
        const int growq = tl.row0 + q * 32;
        const bool full = (tl.rows - q * 32) >= 32;   // every row of the slice is valid
#pragma unroll
        for (int c64 = 0; c64 < W; c64 += 64) {
          const int col = tl.n0 + hh * W + c64;
          if (col >= p.N) continue;
          uint8_t* st = epi + (static_cast<uint32_t>(warp - 2) * BOXES + box) * 4096;
          if (full) {
            if (lane == 0) bulk_wait_read<BOXES - 1>();   // the store that used this box has read it
            __syncwarp();
          }
#pragma unroll
          for (int sub = 0; sub < 64; sub += 32) {
            float o[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = v[c64 + sub + i] * f;
            if (full) {
              stage_row32(st, lane, sub >> 3, o);
            } else if (valid) {
              uint4* dst = reinterpret_cast<uint4*>(p.out + grow * p.N + col + sub);
#pragma unroll
              for (int jj = 0; jj < 4; ++jj)
                if (col + sub + 8 * jj < p.N) dst[jj] = pack8(&o[8 * jj]);
            }
          }
          if (full) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmC, smem_u32(st), col, growq);
              bulk_commit();
            }
            if (++box == BOXES) box = 0;
          }
        }
      } else {
        constexpr int HW = W / 2;   // H columns of a thread: 64 or 32
        const int col = tl.n0 + hh * HW;
        const float fg = rs * f0, fu = rs * f1;
        float hv[HW];
#pragma unroll
        for (int i = 0; i < HW; ++i) hv[i] = silu_f(v[i] * fg) * (v[HW + i] * fu);
        if constexpr (EPI == HB) {
          if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + grow * p.N + col);
#pragma unroll
            for (int j = 0; j < HW / 8; ++j) dst[j] = pack8(&hv[8 * j]);
          }
        } else {
          uint32_t code[HW / 8];
          uint32_t word = 0;
          const float sixth = kSixth * reciprocal(hs);
#pragma unroll
          for (int b = 0; b < HW / BLOCK; ++b) {
            const float* h = hv + b * BLOCK;
            float top = 0.f, sum = 0.f;   // the sum carries a NaN, which the maximum drops
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) {
              top = fmaxf(top, fabsf(h[i]));
              sum += h[i];
            }
            const bool fine = top < __uint_as_float(0x7f800000u) && sum == sum;
            float inv;
            uint32_t byte;
            if constexpr (BLOCK == 16) {
              byte = fine ? to_e4m3(top * sixth) : kNanE4m3;
              inv = reciprocal(from_e4m3(byte) * hs);
            } else {
              const int X = block_exponent(fine ? top : 0.f);
              byte = fine ? static_cast<uint32_t>(X + 127) : kNanE8m0;
              inv = fine ? two_to(-X) : 0.f;
            }
            word |= byte << (8 * b);
#pragma unroll
            for (int o = 0; o < BLOCK / 8; ++o) {
              float_pair y[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int at = 8 * o + 2 * i;
                y[i] = make_pair(fine ? h[at] * inv : 0.f, fine ? h[at + 1] * inv : 0.f);
              }
              code[b * (BLOCK / 8) + o] = to_e2m1x8(y);
            }
          }
          if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(p.hq + (grow * p.N + col) / 2);
#pragma unroll
            for (int j = 0; j < HW / 32; ++j)
              dst[j] = make_uint4(code[4 * j], code[4 * j + 1], code[4 * j + 2], code[4 * j + 3]);
            const long long tile = 2LL * tl.mg + static_cast<long long>(rank);
            uint32_t* w = p.hsf + (tile * p.h_atoms + col / (4 * BLOCK)) * 128 + atom_word(r);
            constexpr int bytes = HW / BLOCK;   // this thread's scales: 4, 2 or 1
            uint8_t* w8 = reinterpret_cast<uint8_t*>(w) + (col / BLOCK) % 4;
            if constexpr (bytes == 4) *w = word;
            else if constexpr (bytes == 2) *reinterpret_cast<uint16_t*>(w8) = static_cast<uint16_t>(word);
            else *w8 = static_cast<uint8_t>(word);
          }
        }
      }
    }
    if (EPI == OUT && lane == 0) bulk_wait_all();   // stores complete before shared memory is released
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // the leader's MMAs into both TMEMs and all remote arrivals are done
  tc_fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u)
                 : "memory");
  }
}

// ----------------------------------------------------------------- host side
// 3-D map over [outer, rows, inner] of bytes, 128-byte swizzle.
bool make_map3_u8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t outer,
                  uint32_t box_inner, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {inner, rows, outer};
  cuuint64_t strides[2] = {inner, inner * rows};
  cuuint32_t box[3] = {box_inner, box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale atoms [tiles, atoms, 128 words]; boxes of box_tiles x box_atoms atoms, zeros past the end.
bool make_map_scales(CUtensorMap* m, const void* base, uint64_t atoms, uint64_t tiles,
                     uint32_t box_atoms, uint32_t box_tiles) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {128, atoms, tiles};
  cuuint64_t strides[2] = {512, 512 * atoms};
  cuuint32_t box[3] = {128, box_atoms, box_tiles};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operands {
  const void *a, *b0, *b1, *sfa, *sfb;
  int K;
};

// Experts whose tables fit beside five stages and the output staging.
constexpr int kDeepMaxE = 448;

template <int EPI, int BLOCK, int BN, int STAGES, int BOXES, int MAX_E>
int launch_stages(const CUtensorMap& ta, const CUtensorMap& tb0, const CUtensorMap& tb1,
                  const CUtensorMap& tsa, const CUtensorMap& tsb, const CUtensorMap& tc,
                  const Params& p, long long tiles, cudaStream_t st, const char* name) {
  using S = Shape<EPI, BLOCK, BN, STAGES, BOXES>;
  static_assert(S::smem(MAX_E) <= kSmemOptIn, "shared memory");
  static thread_local int configured = -1;
  static thread_local int max_clusters = 0;
  return launch_cluster2(fp4_pair_kernel<EPI, BLOCK, BN, STAGES, BOXES>, kThreads, S::smem(p.E), S::smem(MAX_E),
                         &configured, &max_clusters, tiles,
                         name, st, ta, tb0, tb1, tsa, tsb, tc, p);
}

template <int EPI, int BLOCK, int BN>
int launch_pair(const Operands& o, Params p, cudaStream_t st, const char* name) {
  using S = Shape<EPI, BLOCK, BN, 5, 1>;
  const int per = EPI == OUT ? BN : BN / 2;   // outputs of a tile
  p.n_tiles = (p.N + per - 1) / per;
  p.k64 = o.K / 64;
  p.sf_tiles = EPI == OUT ? (p.N + 127) / 128 : p.N / 64;
  const uint64_t atoms = k_atoms(o.K, BLOCK), kb = o.K / 2;
  CUtensorMap ta, tb0, tb1, tsa, tsb, tc;
  if (!make_map_u8(&ta, o.a, kb, p.M, 128, BM) || !make_map3_u8(&tb0, o.b0, kb, p.N, p.E, 128, BN / 2) ||
      !make_map_scales(&tsa, o.sfa, atoms, row_tiles(p.M, p.E), S::KA, 1) ||
      !make_map_scales(&tsb, o.sfb, atoms, static_cast<uint64_t>(p.E) * p.sf_tiles, S::KA, S::NB))
    return MOE_ERR_CUDA;
  if (EPI == OUT) {
    tb1 = tb0;   // not read
    if (!make_map(&tc, p.out, p.N, p.M, 64, 32)) return MOE_ERR_CUDA;
  } else {
    tc = ta;     // not stored through
    if (!make_map3_u8(&tb1, o.b1, kb, p.N, p.E, 128, BN / 2)) return MOE_ERR_CUDA;
  }
  const long long mt_upper = (static_cast<long long>(p.M) + BM - 1) / BM + p.E;
  const long long tiles = mt_upper * p.n_tiles;
  if constexpr (EPI != OUT) {
    return launch_stages<EPI, BLOCK, BN, 5, 1, 1024>(ta, tb0, tb1, tsa, tsb, tc, p, tiles, st, name);
  } else {
    // Up to four k-blocks a tile (K <= 1024) the stores decide, and a second staging box is worth
    // as much as a fifth stage or more; above, the loads do. 65536 rows, 2048 outputs, two boxes
    // against five stages: K = 512 70 and 72 us, 768 74 and 76, 896 to 1024 79 both, 1088 94 and
    // 85, 1280 99 and 85, 1408 107 and 97; 16 experts, 32768 rows, 4096 outputs cross there too.
    if (p.k64 > 16 && p.E <= kDeepMaxE)
      return launch_stages<EPI, BLOCK, BN, 5, 1, kDeepMaxE>(ta, tb0, tb1, tsa, tsb, tc, p, tiles, st, name);
    return launch_stages<EPI, BLOCK, BN, 4, 2, 1024>(ta, tb0, tb1, tsa, tsb, tc, p, tiles, st, name);
  }
}

template <int EPI, int BLOCK>
int launch_bn(const Operands& o, const Params& p, cudaStream_t st, const char* name) {
  // 256 columns a tile even where 128 leave fewer idle (32766 rows of 2048 to 1400, 640 and 384
  // outputs: 64, 42 and 33 us against 76, 44 and 36). Gate and up as their scales are laid out:
  // 64 + 64 columns where I is 64 more than a multiple of 128; 128 + 128 with a last tile half
  // idle would need another layout of the packed scales and has not been timed.
  const bool wide = EPI == OUT ? p.N > 128 : gate_up_half(p.N) == 128;
  return wide ? launch_pair<EPI, BLOCK, 256>(o, p, st, name) : launch_pair<EPI, BLOCK, 128>(o, p, st, name);
}

template <int EPI>
int launch_block(int block, const Operands& o, const Params& p, cudaStream_t st, const char* name) {
  return block == 16 ? launch_bn<EPI, 16>(o, p, st, name) : launch_bn<EPI, 32>(o, p, st, name);
}

// The FFN's scratch: H's codes and scale atoms, and for rows scaled by their own maximum H in
// bf16 and the row factors.
struct Scratch {
  size_t hq, hsf, h, hrs, total;
};
Scratch ffn_layout(long long M, int E, int I, bool own_rows) {
  auto up = [](size_t b) { return (b + 1023) & ~static_cast<size_t>(1023); };
  Scratch s;
  s.hq = 0;
  s.hsf = up(static_cast<size_t>(M) * (I / 2));
  s.h = s.hsf + up(static_cast<size_t>(row_tiles(M, E)) * k_atoms(I, 16) * 512);
  s.hrs = s.h + (own_rows ? up(static_cast<size_t>(M) * I * 2) : 0);
  s.total = s.hrs + (own_rows ? up(static_cast<size_t>(M) * 4) : 0);
  return s;
}

}  // namespace
}  // namespace fp4

size_t ffn_fp4_scratch(long long M, int E, int I, bool own_rows) {
  return fp4::ffn_layout(M, E, I, own_rows).total;
}

}  // namespace moe

extern "C" int moe_grouped_gemm_fp4(const uint8_t* xq, const uint8_t* xsf, const float* row_scale,
                                    const int32_t* offsets, int E, int M, int K, int N, int block,
                                    const uint8_t* w, const uint8_t* w_sf, const float* w_scale,
                                    moe_bf16* y, void* ws, size_t ws_bytes, void* stream) {
  using namespace moe;
  using namespace moe::fp4;
  if (E < 1 || E > 1024 || M < 0 || K < 64 || K % 64 || N < 8 || N % 8 || (block != 16 && block != 32))
    return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!xq || !xsf || !offsets || !w || !w_sf || !y || (block == 16 && (!row_scale || !w_scale)))
    return MOE_ERR_INVALID_ARG;
  for (const void* ptr : {static_cast<const void*>(xq), static_cast<const void*>(xsf),
                          static_cast<const void*>(row_scale), static_cast<const void*>(offsets),
                          static_cast<const void*>(w), static_cast<const void*>(w_sf),
                          static_cast<const void*>(w_scale), static_cast<const void*>(y)})
    if (!aligned16(ptr)) return MOE_ERR_MISALIGNED;
  if (!ws || ws_bytes < kWorkspaceHeader || !aligned16(ws)) return MOE_ERR_WORKSPACE;
  if (cc_major() < 10) return MOE_ERR_UNSUPPORTED;
  Params p{};
  p.offsets = offsets;
  p.E = E;
  p.M = M;
  p.N = N;
  if (block == 16) {
    p.row_scale = row_scale;
    p.scale0 = w_scale;
  }
  p.out = reinterpret_cast<__nv_bfloat16*>(y);
  p.status = static_cast<int*>(ws);
  return launch_block<OUT>(block, Operands{xq, w, w, xsf, w_sf, K}, p, as_stream(stream), "gemm_fp4");
}

extern "C" int moe_grouped_ffn_fp4(const uint8_t* xq, const uint8_t* xsf, const float* row_scale,
                                   const int32_t* offsets, int E, int M, int d, int I, int block,
                                   const uint8_t* w_gate, const uint8_t* w_up, const uint8_t* wgu_sf,
                                   const float* gate_scale, const float* up_scale,
                                   const uint8_t* w_down, const uint8_t* wd_sf,
                                   const float* down_scale, const float* h_scale, moe_bf16* y,
                                   void* ws, size_t ws_bytes, void* stream) {
  using namespace moe;
  using namespace moe::fp4;
  if (E < 1 || E > 1024 || M < 0 || d < 64 || d % 64 || I < 64 || I % 64 || (block != 16 && block != 32))
    return MOE_ERR_INVALID_ARG;
  if (block == 32 && h_scale) return MOE_ERR_INVALID_ARG;
  if (I > 16384) return MOE_ERR_UNSUPPORTED;   // what moe_fp4_quantize_rows takes
  if (M == 0) return MOE_OK;
  if (!xq || !xsf || !offsets || !w_gate || !w_up || !wgu_sf || !w_down || !wd_sf || !y)
    return MOE_ERR_INVALID_ARG;
  if (block == 16 && (!row_scale || !gate_scale || !up_scale || !down_scale)) return MOE_ERR_INVALID_ARG;
  for (const void* ptr :
       {static_cast<const void*>(xq), static_cast<const void*>(xsf), static_cast<const void*>(row_scale),
        static_cast<const void*>(offsets), static_cast<const void*>(w_gate),
        static_cast<const void*>(w_up), static_cast<const void*>(wgu_sf),
        static_cast<const void*>(gate_scale), static_cast<const void*>(up_scale),
        static_cast<const void*>(w_down), static_cast<const void*>(wd_sf),
        static_cast<const void*>(down_scale), static_cast<const void*>(h_scale),
        static_cast<const void*>(y)})
    if (!aligned16(ptr)) return MOE_ERR_MISALIGNED;
  const bool own_rows = block == 16 && !h_scale;   // H's rows scaled by their own maximum
  const Scratch lay = ffn_layout(M, E, I, own_rows);
  if (!ws || !aligned16(ws) || ws_bytes < kWorkspaceHeader + lay.total) return MOE_ERR_WORKSPACE;
  if (cc_major() < 10) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = as_stream(stream);
  uint8_t* scratch = static_cast<uint8_t*>(ws) + kWorkspaceHeader;
  uint8_t* hq = scratch + lay.hq;
  uint8_t* hsf = scratch + lay.hsf;
  float* hrs = reinterpret_cast<float*>(scratch + lay.hrs);   // own_rows, as the bf16 H
  Params p{};
  p.offsets = offsets;
  p.E = E;
  p.M = M;
  p.N = I;
  if (block == 16) {
    p.row_scale = row_scale;
    p.scale0 = gate_scale;
    p.scale1 = up_scale;
  }
  p.h_scale = h_scale;
  p.out = own_rows ? reinterpret_cast<__nv_bfloat16*>(scratch + lay.h) : nullptr;
  p.hq = hq;
  p.hsf = reinterpret_cast<uint32_t*>(hsf);
  p.h_atoms = k_atoms(I, block);
  p.status = static_cast<int*>(ws);
  const Operands gu{xq, w_gate, w_up, xsf, wgu_sf, d};
  const char* const name = "gemm_gate_up_fp4";
  int rc = own_rows ? launch_bn<HB, 16>(gu, p, st, name) : launch_block<H4>(block, gu, p, st, name);
  if (rc) return rc;
  if (own_rows) {
    rc = launch_quantize(p.out, nullptr, offsets, E, M, 1, M, I, block, hq, hsf, hrs, st, "fp4_quantize_h");
    if (rc) return rc;
  }
  p.N = d;
  p.row_scale = own_rows ? hrs : nullptr;
  p.scale0 = block == 16 ? down_scale : nullptr;
  p.scale1 = h_scale;
  p.h_scale = nullptr;
  p.out = reinterpret_cast<__nv_bfloat16*>(y);
  return launch_block<OUT>(block, Operands{hq, w_down, w_down, hsf, wd_sf, I}, p, st, "gemm_down_fp4");
}

namespace moe {
MOE_DEBUG_STATUS_READER(fp4_gemm)
}  // namespace moe
