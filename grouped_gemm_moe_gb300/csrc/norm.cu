// The RMS norms before and after one MoE block, with the block's combine, gate,
// residual scale and residual add, and their gradients.
//
//   before:  r_t = (mean_c x_tc^2 + eps)^(-1/2),   xn = bf16(x r g)
//   after:   z_t = sum_j w_tj y[inv_perm[t K + j]] + shared_t          (fp32)
//            out = bf16(resid + alpha * gate * (z r g)),  r of z; without a
//            gain the norm is left out: out = bf16(resid + alpha * gate * z)
//   gradients, with xh = x r (zh = z r) and the saved r:
//            before: u = g dxn,  dx = dres + r (u - xh mean_c(u xh)),
//                    dg = sum_t dxn xh
//            after:  dn = alpha gate dout,  u = g dn,
//                    dz = r (u - zh mean_c(u zh)),  dg = sum_t dn zh,
//                    dgate = alpha sum_{t of the gate's row} dout g zh
//                    (summed over the columns too when the gate has one)
//
// Every kernel reads each row once and is bound by HBM. A row group of G
// threads (whole warps) owns one row at a time, V 16-byte vectors per thread,
// so a row is read once and stays in the SM between its sum and its result. Its
// bytes come through a ring in shared memory that every thread fills for itself
// (cp.async; a thread reads only what it copied, so no barrier guards the ring):
// the rows ahead are in flight while this one waits for its sum, at no registers.
// Once the ring kept HBM busy, the instructions per row decided: several vectors
// per thread (fewer threads take part in a row's sum), algebra that shares factors
// over a row or a span, and two-wide fp32 arithmetic. The gradient kernels keep
// column sums (dg, dgate) in registers over a group's contiguous rows, write them
// once to the workspace, and a second launch adds them in a fixed order: no
// atomics, the same bits every run.
//
// Measured on one GB300, device time a call (HBM floor at 6.8 TB/s in brackets):
//   norm_in           32768 x 4096                        82 us (79); 1.9 us for one row
//   norm_out          8192 x 2048, K = 8, channel gate    57 us (54); 3.2 us for 16 rows
//   norm_in_backward  32768 x 4096 with the residual     157 us (158)
//   norm_out_backward 16383 x 2056, gate per 1000 rows    46 us (30): 4 us of it the join
//                     and about 4 more the spans' partial sums; 36 us at 2048 without a gate
//   norm_out_backward 32768 x 4096, no gate, one for the model, one per channel
//                     123, 131 and 127 us (118): a gate of one column sums a span's rows in
//                     one block, on one SM
// Rows above d = 8192 are further from it. The gradients' four vectors a thread spill (160 to
// 650 bytes): 16384 x 8200 with the residual 357 us (158), 290 without gate and 375 with one
// per channel (119); 8192 x 16384 349 (158), 244 and 311 (118).
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxD = 16384;
constexpr int kMaxGradRows = 1 << 30;   // a gradient's row numbers stay in an int, past its last row too

// How rows of nv vectors map to threads: G threads per row group (a multiple of
// 32), `groups` groups per block.
struct RowPlan {
  int G, groups;
  int block() const { return G * groups; }
};

RowPlan plan_rows(int d, int V) {
  const int per = (d / 8 + V - 1) / V;
  RowPlan p;
  p.G = (per + 31) / 32 * 32;
  p.groups = std::max(1, 256 / p.G);
  return p;
}

// Sums over row groups of G threads, in every thread of the group. The blocks
// call sum() in step with a counting `phase`: the two halves of the buffer
// alternate, so one barrier per sum is enough (a half is written again only
// after the next sum's barrier). A group's warps own consecutive floats, padded
// with zeros to whole float4s.
struct GroupSum {
  float* half0;
  int warps4, first, slot;   // float4s of a group, its first one, this warp's float
  __device__ GroupSum(float (&buf)[64], int G, int grp, int lane) : half0(buf) {
    warps4 = (G / 32 + 3) / 4;
    first = grp * warps4;
    slot = first * 4 + lane / 32;
    if (G > 32) {
      if (threadIdx.x < 64) buf[threadIdx.x] = 0.f;
      __syncthreads();
    }
  }
  __device__ __forceinline__ float sum(float v, int G, int phase) const {
    v = warp_sum(v);
    if (G == 32) return v;
    float* half = half0 + (phase & 1) * 32;
    if ((threadIdx.x & 31) == 0) half[slot] = v;
    __syncthreads();
    const float4* h = reinterpret_cast<const float4*>(half) + first;
    float4 a = h[0];
    float s = (a.x + a.y) + (a.z + a.w);
    for (int w = 1; w < warps4; ++w) {
      a = h[w];
      s += (a.x + a.y) + (a.z + a.w);
    }
    return s;
  }
};

// norm_in's ring: 1024 vectors an SM a stage, 48 KB in flight. More in flight is
// slower: 32768 x 4096 takes 82 us so, 88 us with a stage more, 90 us with twice the
// threads (more rows open at once cost HBM more than they hide); less is slower too.
constexpr int kInStages = 4;
constexpr int in_threads(int V) { return 1024 / V; }

__device__ __forceinline__ void load8f(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ void store_pairs(float* to, const float_pair (&v)[4]) {
  ulonglong2* p = reinterpret_cast<ulonglong2*>(to);
  p[0] = make_ulonglong2(v[0], v[1]);
  p[1] = make_ulonglong2(v[2], v[3]);
}

__device__ __forceinline__ void load_pairs(const float* p, float_pair (&f)[4]) {
  const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(p));
  const ulonglong2 b = __ldg(reinterpret_cast<const ulonglong2*>(p) + 1);
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(live ? 16 : 0)
               : "memory");
}

template <int N>
__device__ __forceinline__ void copies_wait() {   // all but the N newest groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// xn = bf16(x r g) over every workers-th row (the SMs read and write one moving
// stretch of memory), kStages - 1 rows on their way in shared memory. Each thread
// reads only the vectors it copied itself, so the ring has no barrier of its own.
template <int V>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512, 1)
norm_in_ring_kernel(const uint4* __restrict__ x, const float* __restrict__ gain, float eps,
                    float inv_d, int T, int chunk, int nv, int G, uint4* __restrict__ xn,
                    float* __restrict__ rstd) {
  pdl_enter();
  constexpr int kStages = kInStages;
  extern __shared__ uint4 ring[];   // [stage][v][thread]
  __shared__ __align__(16) float red[64];
  const int grp = threadIdx.x / G, lane = threadIdx.x - grp * G;
  const GroupSum group(red, G, grp, lane);
  const int workers = gridDim.x * (blockDim.x / G);
  const int worker = blockIdx.x * (blockDim.x / G) + grp;
  bool has[V];
  float g[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    has[v] = lane + v * G < nv;
    if (has[v]) load8f(gain + (lane + v * G) * 8, g[v]);
  }
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  auto slot = [&](int stage, int v) {
    return (stage * V + v) * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
  };
  auto issue = [&](int i) {   // the group's i-th row
    const long long t = worker + static_cast<long long>(i) * workers;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool live = t < T && has[v];
      copy16(base + 16 * slot(i % kStages, v), x + (live ? t * nv + lane + v * G : 0), live);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int st = 0; st + 1 < kStages; ++st) issue(st);
  for (int i = 0; i < chunk; ++i) {   // every group of a block runs every step
    const long long t = worker + static_cast<long long>(i) * workers;
    copies_wait<kStages - 2>();
    issue(i + kStages - 1);   // into the slot of row i - 1, read by now
    float f[V][8], s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      unpack8(ring[slot(i % kStages, v)], f[v]);
#pragma unroll
      for (int q = 0; q < 8; ++q) s = fmaf(f[v][q], f[v][q], s);
    }
    s = group.sum(s, G, i);
    if (t >= T) continue;
    const float r = rsqrtf(s * inv_d + eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!has[v]) break;
#pragma unroll
      for (int q = 0; q < 8; ++q) f[v][q] = f[v][q] * r * g[v][q];
      stg_v4(xn + t * nv + lane + v * G, pack8(f[v]));
    }
    if (lane == 0) rstd[t] = r;
  }
  copies_wait<0>();
}

// xn = bf16(x r g), one row per group, one vector per thread: the fewest steps
// between a row's arrival and its result, for calls with fewer rows than SMs
// can hold.
template <int V>
__global__ void __launch_bounds__(1024, 1)
norm_in_kernel(const uint4* __restrict__ x, const float* __restrict__ gain, float eps, float inv_d,
               int nv, uint4* __restrict__ xn, float* __restrict__ rstd) {
  pdl_enter();
  __shared__ __align__(16) float red[64];
  const int G = blockDim.x;
  const GroupSum group(red, G, 0, threadIdx.x);
  const long long t = blockIdx.x;
  uint4 raw[V];
  float s = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = threadIdx.x + v * G;
    raw[v] = c < nv ? ldg_nc_v4(x + t * nv + c) : make_uint4(0u, 0u, 0u, 0u);
    float f[8];
    unpack8(raw[v], f);
#pragma unroll
    for (int q = 0; q < 8; ++q) s = fmaf(f[q], f[q], s);
  }
  const float r = rsqrtf(group.sum(s, G, 0) * inv_d + eps);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = threadIdx.x + v * G;
    if (c >= nv) break;
    float f[8], g[8];
    unpack8(raw[v], f);
    load8f(gain + c * 8, g);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = f[q] * r * g[q];
    stg_v4(xn + t * nv + c, pack8(f));
  }
  if (threadIdx.x == 0) rstd[t] = r;
}

// Combine, norm, gate, residual, one row per group. The gathered vectors of a
// column are loaded KC at a time before they are added (slot order, fp32), as in
// the combine of this library, and z is never rounded on its way into the norm;
// only the copy saved for the gradient is bf16.
template <int KC, int V>
__global__ void __launch_bounds__(256, 2)
norm_out_kernel(const uint4* __restrict__ y, const float* __restrict__ w,
                const int32_t* __restrict__ inv_perm, int K, const uint4* __restrict__ shared_y,
                const uint4* resid, const float* __restrict__ gain,
                const float* __restrict__ gate, unsigned span, int gate_cols, float scale,
                float eps, float inv_d, int T, int nv, int G, uint4* out,
                uint4* __restrict__ zsum, float* __restrict__ rstd) {
  pdl_enter();
  __shared__ __align__(16) float red[64];
  const int groups = blockDim.x / G;
  const int grp = threadIdx.x / G, lane = threadIdx.x - grp * G;
  const GroupSum group(red, G, grp, lane);
  const long long t = static_cast<long long>(blockIdx.x) * groups + grp;
  const bool live = t < T;
  const long long slots = static_cast<long long>(T) * K;
  float z[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int q = 0; q < 8; ++q) z[v][q] = 0.f;
  if (live) {
    for (int j0 = 0; j0 < K; j0 += KC) {
      int32_t pos[KC];
      float wj[KC];
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const long long a = t * K + j0 + j;
        pos[j] = -1;
        if (j0 + j < K) {
          pos[j] = inv_perm ? __ldg(inv_perm + a) : static_cast<int32_t>(a);
          wj[j] = w ? __ldg(w + a) : 1.f;
          if (!index_ok(pos[j] >= 0 && pos[j] < slots)) pos[j] = 0;
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = lane + v * G;
        if (c >= nv) break;
        uint4 a[KC];
#pragma unroll
        for (int j = 0; j < KC; ++j)
          if (pos[j] >= 0) a[j] = ldg_nc_v4(y + static_cast<long long>(pos[j]) * nv + c);
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          if (pos[j] >= 0) {
            float f[8];
            unpack8(a[j], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) z[v][q] = fmaf(wj[j], f[q], z[v][q]);
          }
        }
      }
    }
  }
  float s = 0.f;
  uint4 res[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = lane + v * G;
    if (!live || c >= nv) break;
    res[v] = *reinterpret_cast<const uint4*>(resid + t * nv + c);   // may be out's own row
    if (shared_y) {
      float f[8];
      unpack8(ldg_nc_v4(shared_y + t * nv + c), f);
#pragma unroll
      for (int q = 0; q < 8; ++q) z[v][q] += f[q];
    }
    if (zsum) stg_v4(zsum + t * nv + c, pack8(z[v]));
#pragma unroll
    for (int q = 0; q < 8; ++q) s = fmaf(z[v][q], z[v][q], s);
  }
  float r = 1.f;
  if (gain) r = rsqrtf(group.sum(s, G, 0) * inv_d + eps);
  if (!live) return;
  if (gain && rstd && lane == 0) rstd[t] = r;
  const float* grow =
      gate ? gate + static_cast<long long>(static_cast<unsigned>(t) / span) * gate_cols : nullptr;
  const bool wide = grow && gate_cols != 1;
  const float m = (grow && !wide) ? scale * __ldg(grow) : scale;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = lane + v * G;
    if (c >= nv) break;
    float f[8], g[8];
    unpack8(res[v], f);
    if (gain) {
      load8f(gain + c * 8, g);
#pragma unroll
      for (int q = 0; q < 8; ++q) z[v][q] = z[v][q] * r * g[q];
    }
    if (wide) {
      load8f(grow + c * 8, g);
#pragma unroll
      for (int q = 0; q < 8; ++q) z[v][q] *= g[q];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = fmaf(m, z[v][q], f[q]);
    stg_v4(out + t * nv + c, pack8(f));
  }
}

// The same over every workers-th row, one vector per thread: while a row is
// combined and normed, the gathered vectors of the next S - 1 rows are on their way
// into the thread's own slots of shared memory. Lane j of each warp looks up
// slot j's row and weight a row before they are needed.
template <int S>
__global__ void __launch_bounds__(1024, 1)
norm_out_ring_kernel(const uint4* __restrict__ y, const float* __restrict__ w,
                     const int32_t* __restrict__ inv_perm, int K,
                     const uint4* __restrict__ shared_y, const uint4* resid,
                     const float* __restrict__ gain, const float* __restrict__ gate, unsigned span,
                     int gate_cols, float scale, float eps, float inv_d, int T, int chunk, int nv,
                     int G, uint4* out, uint4* __restrict__ zsum, float* __restrict__ rstd) {
  pdl_enter();
  extern __shared__ uint4 ring[];   // [stage][K slots, residual, shared][thread]
  __shared__ __align__(16) float red[64];
  const int grp = threadIdx.x / G, lane = threadIdx.x - grp * G;
  const GroupSum group(red, G, grp, lane);
  const int wl = threadIdx.x & 31;
  const long long workers = gridDim.x * (blockDim.x / G);
  const long long worker = blockIdx.x * (blockDim.x / G) + grp;
  const bool has = lane < nv;
  const int arrays = K + 1 + (shared_y ? 1 : 0);
  const long long slots = static_cast<long long>(T) * K;
  float_pair g[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) g[q] = make_pair(1.f, 1.f);
  if (gain && has) load_pairs(gain + lane * 8, g);
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  auto at = [&](int stage, int array) {
    return (stage * arrays + array) * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
  };
  auto look_up = [&](long long t) {   // lane j: the packed row of slot j
    if (t >= T || wl >= K) return 0;
    const long long a = t * K + wl;
    const int p = inv_perm ? __ldg(inv_perm + a) : static_cast<int>(a);
    return index_ok(p >= 0 && p < slots) ? p : 0;
  };
  auto weight = [&](long long t) { return (w && t < T && wl < K) ? __ldg(w + t * K + wl) : 1.f; };
  auto issue = [&](long long t, int stage, int pos) {
    const bool live = t < T && has;
    for (int j = 0; j < K; ++j) {
      const long long p = __shfl_sync(0xffffffffu, pos, j);
      copy16(base + 16 * at(stage, j), y + (live ? p * nv + lane : 0), live);
    }
    const long long own = live ? t * nv + lane : 0;
    copy16(base + 16 * at(stage, K), resid + own, live);
    if (shared_y) copy16(base + 16 * at(stage, K + 1), shared_y + own, live);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int st = 0; st + 1 < S; ++st) issue(worker + st * workers, st, look_up(worker + st * workers));
  int pos = look_up(worker + (S - 1) * workers);
  float wt = weight(worker);
  for (int i = 0; i < chunk; ++i) {   // every group of a block runs every step
    const long long t = worker + i * workers;
    const bool live = t < T;
    copies_wait<S - 2>();
    issue(t + (S - 1) * workers, (i + S - 1) % S, pos);   // the slots of the last row, read by now
    pos = look_up(t + S * workers);
    const float next_wt = weight(t + workers);
    const int stage = i % S;
    float_pair z[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) z[q] = make_pair(0.f, 0.f);
#pragma unroll 4
    for (int j = 0; j < K; ++j) {
      const float wj = __shfl_sync(0xffffffffu, wt, j);
      const float_pair w2 = make_pair(wj, wj);
      float_pair f[4];
      unpack8(ring[at(stage, j)], f);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] = fma_pair(w2, f[q], z[q]);
    }
    if (shared_y) {
      float_pair f[4];
      unpack8(ring[at(stage, K + 1)], f);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] = add_pair(z[q], f[q]);
    }
    const long long own = t * nv + lane;
    if (zsum && live && has) stg_v4(zsum + own, pack8(z));
    float r = 1.f;
    if (gain) {
      float_pair s2 = mul_pair(z[0], z[0]);
#pragma unroll
      for (int q = 1; q < 4; ++q) s2 = fma_pair(z[q], z[q], s2);
      const float2 both = split_pair(s2);
      r = rsqrtf(group.sum(both.x + both.y, G, i) * inv_d + eps);
      if (rstd && live && lane == 0) rstd[t] = r;
    }
    if (live && has) {
      float m = scale * r;
      float_pair f[4], gt[4];
      unpack8(ring[at(stage, K)], f);
      const float* grow =
          gate ? gate + static_cast<long long>(static_cast<unsigned>(t) / span) * gate_cols : nullptr;
      if (grow && gate_cols != 1) {
        load_pairs(grow + lane * 8, gt);
#pragma unroll
        for (int q = 0; q < 4; ++q) z[q] = mul_pair(z[q], gt[q]);
      } else if (grow) {
        m *= __ldg(grow);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] = fma_pair(make_pair(m, m), mul_pair(z[q], g[q]), f[q]);
      stg_v4(out + own, pack8(f));
    }
    wt = next_wt;
  }
  copies_wait<0>();
}

// Shared memory of an SM and what a block of it costs beside its own, for the
// ring kernels' residency.
constexpr int kSmemPerSm = 228 * 1024, kSmemReserved = 1024, kSmemPerBlock = 227 * 1024;

// Row groups of a kernel that walks consecutive rows: `resident` blocks per SM.
struct ChunkPlan {
  int grid, chunk, workers;
};

ChunkPlan plan_chunks(int T, const RowPlan& p, int resident) {
  const long long most = static_cast<long long>(num_sms()) * resident * p.groups;
  ChunkPlan c;
  c.chunk = static_cast<int>(std::max(1LL, (T + most - 1) / most));
  c.workers = (T - 1) / c.chunk + 1;   // T >= 1, up to 2^31 - 1
  c.grid = (c.workers + p.groups - 1) / p.groups;
  return c;
}

// Launches a kernel that takes `smem` bytes of dynamic shared memory; the limit
// is raised once per kernel and device.
template <typename... KArgs, typename... Args>
int launch_big(void (*kern)(KArgs...), int& configured, int grid, int block, size_t smem,
               cudaStream_t st, const Args&... args) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured != dev) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerBlock - 1024);
    if (e != cudaSuccess) {
      set_last_cuda_error(e);
      return MOE_ERR_CUDA;
    }
    configured = dev;
  }
  return launch_pdl(kern, grid, block, smem, st, 1, args...);
}

// norm_in with few rows takes a block per row: 1.9 against 2.1 us for one row of
// d = 4096, 2.4 against 2.7 for 608 rows of 2048; at 1024 rows of 4096 the ring wins
// (4.7 against 5.0 us).
bool few_rows(int T) { return T <= 4 * num_sms(); }

// ----------------------------------------------------------------- gradients
// A row group takes `chunk` consecutive rows. Its column sums go to slot arrays
// of the workspace, [groups][d] each: dgain, and for a gate of d columns the
// spans that cross the group's ends (gate0: a span that began in an earlier
// group, gate1: one that begins here and goes on). A span that lies within one
// group's rows is written to dgate at once.
enum { kGateNone = 0, kGateScalar = 1, kGateVector = 2 };

struct BackwardArgs {
  const uint4* up;        // dxn or dout
  const uint4* x;         // x or the saved z
  const float* rstd;
  const float* gain;
  const float* gate;
  const uint4* dres;      // before the block only, or null
  uint4* dx;
  float* dgate;
  float* part_gain;
  float* part_gate0;
  float* part_gate1;
  float* row_dot;         // per-row gate gradients (gate of one column)
  int T, span, chunk;
  float scale, inv_d;
  int nv, G;
};

// The ring: three stages of two or three arrays with 1024 / V threads an SM, two
// stages and 512 threads with four vectors (d > 8192). 32768 x 4096 with the residual
// takes 156 us so, 161 with four stages, 164 with two.
constexpr int ring_stages(int V) { return V <= 2 ? 3 : 2; }
constexpr int ring_threads(int V) { return V == 1 ? 1024 : 512; }

// With a = dout (or dxn), b = z (or x) and k = gain (times the gate's row and
// scale where the gate has d columns, those being constant over a span), a row
// costs three operations an element before its sum and three after:
//   q = a b,  s = sum_c q k,  mean_c(u xh) = s r sg / d
//   dz = (r sg) k a - (r r mean) b
// where sg is the row's scalar, scale times its one-column gate. The column sums
// are dg += q (r sg), or with a gate of d columns e += q r, from which both
// dgate = scale gain e and dg += scale gate e follow when the span ends.
template <int V, bool RES, bool NORM, int GATE>
__global__ void __launch_bounds__(ring_threads(V), 1) norm_backward_kernel(BackwardArgs A) {
  pdl_enter();
  constexpr int kStages = ring_stages(V), kArrays = RES ? 3 : 2;
  constexpr bool kVec = GATE == kGateVector;
  extern __shared__ uint4 ring[];   // [stage][array][v][thread]
  __shared__ __align__(16) float red[64];
  const int G = A.G, nv = A.nv, nthreads = blockDim.x;
  const int groups = nthreads / G;
  const int grp = threadIdx.x / G, lane = threadIdx.x - grp * G;
  const GroupSum group(red, G, grp, lane);
  const int worker = blockIdx.x * groups + grp;
  const int row0 = min(static_cast<long long>(worker) * A.chunk, static_cast<long long>(A.T));
  const int row1 = min(static_cast<long long>(row0) + A.chunk, static_cast<long long>(A.T));
  bool has[V];
  float_pair k[V][4], dg[V][4], e[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    has[v] = lane + v * G < nv;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      k[v][q] = make_pair(1.f, 1.f);
      dg[v][q] = make_pair(0.f, 0.f);
      e[v][q] = make_pair(0.f, 0.f);
    }
    if (NORM && !kVec && has[v]) load_pairs(A.gain + (lane + v * G) * 8, k[v]);
  }
  // This thread's slots: array and vector at fixed distances, stages `stage_step` apart.
  const int vec_step = nthreads, stage_step = kArrays * V * nthreads;
  const uint4* const mine = ring + threadIdx.x;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + 16 * threadIdx.x;
  long long at = static_cast<long long>(min(row0, A.T - 1)) * nv + lane;   // the next row to copy
  int copied = row0, to = 0;                                               // that row, its stage
  auto issue = [&]() {   // always one group of copies, of nothing past the rows
    const bool live = copied < row1;
    const uint32_t slot = base + 16 * to;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool read = live && has[v];
      const long long from = has[v] ? at + v * G : at;
      copy16(slot + 16 * v * vec_step, A.up + from, read);
      copy16(slot + 16 * (V + v) * vec_step, A.x + from, read);
      if (RES) copy16(slot + 16 * (2 * V + v) * vec_step, A.dres + from, read);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++copied;
    if (copied < row1) at += nv;
    to = to + stage_step == kStages * stage_step ? 0 : to + stage_step;
  };
  auto row_scalars = [&](int t, float& r, float& sg) {
    r = 1.f;
    sg = kVec ? 1.f : A.scale;
    if (t < row1) {
      if (NORM) r = __ldg(A.rstd + t);
      if (GATE == kGateScalar) sg *= __ldg(A.gate + (A.span == 1 ? t : t / A.span));
    }
  };
  if (lane >= nv) at -= lane;   // a thread without a vector copies nothing, from a place that exists
#pragma unroll
  for (int st = 0; st + 1 < kStages; ++st) issue();
  float rs, sg;
  row_scalars(row0, rs, sg);
  int span_id = 0, span_end = -1, stage = 0;
  for (int i = 0; i < A.chunk; ++i) {   // every group of a block runs every step
    const int t = row0 + i;
    const bool live = t < row1;
    copies_wait<kStages - 2>();
    issue();   // into the slots of row t - 1, read by now
    const uint4* const row = mine + stage;
    stage = stage + stage_step == kStages * stage_step ? 0 : stage + stage_step;
    if (kVec && live && t >= span_end) {   // a span begins (or is entered)
      span_id = t / A.span;
      span_end = static_cast<int>(min((span_id + 1LL) * A.span, static_cast<long long>(A.T)));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!has[v]) break;
        const int c = (lane + v * G) * 8;
        float_pair gn[4];
        load_pairs(A.gate + span_id * (nv * 8LL) + c, k[v]);
        if (NORM) load_pairs(A.gain + c, gn);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          k[v][q] = mul_pair(k[v][q], make_pair(A.scale, A.scale));
          if (NORM) k[v][q] = mul_pair(k[v][q], gn[q]);
        }
      }
    }
    float nrs, nsg;
    row_scalars(t + 1, nrs, nsg);
    float_pair a[V][4], b[V][4], s2 = make_pair(0.f, 0.f);
    const float w = rs * (kVec ? 1.f : sg);
    const float_pair w2 = make_pair(w, w);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if ((lane & ~31) + v * G >= nv) break;   // nothing for this warp
      unpack8(row[v * vec_step], a[v]);
      unpack8(row[(V + v) * vec_step], b[v]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float_pair p = mul_pair(a[v][q], b[v][q]);
        if (kVec) e[v][q] = fma_pair(p, w2, e[v][q]);
        else if (NORM) dg[v][q] = fma_pair(p, w2, dg[v][q]);
        s2 = fma_pair(p, k[v][q], s2);
      }
    }
    float s = 0.f;
    if (NORM || GATE == kGateScalar) {
      const float2 both = split_pair(s2);
      s = group.sum(both.x + both.y, G, i);
    }
    if (GATE == kGateScalar && live && lane == 0) A.row_dot[t] = A.scale * rs * s;
    if (live) {
      const float wa = rs * sg, wb = -(rs * rs) * (s * rs * sg * A.inv_d);
      const float_pair wa2 = make_pair(wa, wa), wb2 = make_pair(wb, wb);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!has[v]) break;
        float_pair o[4];
        if (RES) unpack8(row[(2 * V + v) * vec_step], o);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float_pair ka = mul_pair(k[v][q], a[v][q]);
          if (NORM) o[q] = RES ? fma_pair(wb2, b[v][q], o[q]) : mul_pair(wb2, b[v][q]);
          o[q] = (NORM || RES) ? fma_pair(wa2, ka, o[q]) : mul_pair(wa2, ka);
        }
        stg_v4(A.dx + static_cast<long long>(t) * nv + lane + v * G, pack8(o));
      }
    }
    if (kVec && live && (t + 1 == span_end || t + 1 == row1)) {
      const long long begin = static_cast<long long>(span_id) * A.span;
      float* to_row = begin < row0 ? A.part_gate0 + worker * (nv * 8LL)
                      : span_end > row1 ? A.part_gate1 + worker * (nv * 8LL)
                                        : A.dgate + span_id * (nv * 8LL);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!has[v]) break;
        const int c = (lane + v * G) * 8;
        float_pair gn[4], gt[4], o[4];
        if (NORM) {
          load_pairs(A.gain + c, gn);
          load_pairs(A.gate + span_id * (nv * 8LL) + c, gt);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          o[q] = mul_pair(make_pair(A.scale, A.scale), e[v][q]);
          if (NORM) {
            dg[v][q] = fma_pair(gt[q], o[q], dg[v][q]);
            o[q] = mul_pair(gn[q], o[q]);
          }
          e[v][q] = make_pair(0.f, 0.f);
        }
        store_pairs(to_row + c, o);
      }
    }
    rs = nrs;
    sg = nsg;
  }
  copies_wait<0>();
  if (NORM && row0 < A.T) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (has[v]) store_pairs(A.part_gain + worker * (nv * 8LL) + (lane + v * G) * 8, dg[v]);
  }
}

// Joins the groups' column sums: blockIdx.x picks 16 columns, the quads of threads
// (a float4 each) take the groups in turn, eight loads at once, then one fixed
// tree. Task 0 sums dgain; the others stand for the spans (by_span) or for the
// groups, whichever are fewer, and sum the span if it crosses groups (of a group:
// the span that begins in its rows and goes on past them).
template <int THREADS>
__global__ void __launch_bounds__(THREADS)
norm_join_kernel(const float* part_gain, const float* part_gate0, const float* part_gate1, int d,
                 int workers, int chunk, int T, int span, int by_span, int task0,
                 float* dgain, float* dgate) {
  pdl_enter();
  __shared__ float4 acc[THREADS / 32][4];
  const int warp = threadIdx.x >> 5, quad = threadIdx.x & 3;
  const int c = blockIdx.x * 16 + quad * 4;
  const float* first = nullptr;   // a row added to the sum of rows [a, b) of `rest`
  const float* rest = part_gain;
  float* to = dgain;
  int a = 0, b = workers;
  const int task = task0 + blockIdx.y;
  if (task == 0) {
    if (!dgain) return;
  } else {
    const long long k = task - 1;
    const long long s = by_span ? k : min((k + 1) * chunk, static_cast<long long>(T)) - 1;
    const long long id = by_span ? s : s / span;
    const long long begin = id * span, end = min(begin + span, static_cast<long long>(T));
    const int w = static_cast<int>(by_span ? begin / chunk : k);
    const long long row1 = (w + 1LL) * chunk;
    if (begin < static_cast<long long>(w) * chunk || end <= row1) return;
    first = part_gate1 + static_cast<long long>(w) * d;
    rest = part_gate0;
    a = w + 1;
    b = static_cast<int>((end - 1) / chunk) + 1;
    to = dgate + id * d;
  }
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [](float4& x, const float4& y) {
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  };
  if (c < d) {
#pragma unroll 8
    for (int w = a + (threadIdx.x >> 2); w < b; w += THREADS / 4)
      add(s, __ldcg(reinterpret_cast<const float4*>(rest + static_cast<long long>(w) * d + c)));
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1)
    add(s, make_float4(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o),
                       __shfl_xor_sync(0xffffffffu, s.z, o), __shfl_xor_sync(0xffffffffu, s.w, o)));
  if ((threadIdx.x & 31) < 4) acc[warp][quad] = s;
  __syncthreads();
  if (threadIdx.x < 4 && c < d) {
    float4 t = first ? __ldcg(reinterpret_cast<const float4*>(first + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) add(t, acc[w][quad]);
    *reinterpret_cast<float4*>(to + c) = t;
  }
}

// dgate of a gate with one column: the rows of each span added, one block per span.
__global__ void __launch_bounds__(256)
norm_join_rows_kernel(const float* row_dot, long long T, long long span, float* dgate) {
  pdl_enter();
  __shared__ float acc[8];
  const long long begin = blockIdx.x * span;
  const long long end = begin + span < T ? begin + span : T;
  float s = 0.f;
  for (long long t = begin + threadIdx.x; t < end; t += 256) s += __ldcg(row_dot + t);
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) acc[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int w = 0; w < 8; ++w) t += acc[w];
    dgate[blockIdx.x] = t;
  }
}

__global__ void zero_floats_kernel(float* a, long long na, float* b, long long nb) {
  pdl_enter();
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i < na) a[i] = 0.f;
  if (i < nb) b[i] = 0.f;
}

// Groups of the gradient kernels and the rows each takes.
struct BackwardPlan {
  RowPlan rows;
  ChunkPlan chunks;
  int V;
};

BackwardPlan plan_backward(int T, int d, int arrays) {
  BackwardPlan p;
  // 16383 x 2056: 47 us with two vectors a thread, 64 with one (registers spill at 1024 threads)
  p.V = d <= 256 ? 1 : d <= 8192 ? 2 : 4;
  p.rows = plan_rows(d, p.V);
  const int smem = 16 * ring_stages(p.V) * arrays * p.V * p.rows.block();
  const int resident = std::min(ring_threads(p.V) / p.rows.block(),
                                kSmemPerSm / (smem + kSmemReserved));
  p.chunks = plan_chunks(T, p.rows, std::max(1, resident));
  return p;
}

bool norm_shape_ok(int T, int d) { return T >= 0 && d >= 8 && d % 8 == 0; }

template <int V, bool RES, bool NORM, int GATE>
int run_backward(const BackwardPlan& p, const BackwardArgs& a, cudaStream_t st) {
  static thread_local int configured = -1;
  const size_t smem = sizeof(uint4) * ring_stages(V) * (RES ? 3 : 2) * V * p.rows.block();
  return launch_big(norm_backward_kernel<V, RES, NORM, GATE>, configured, p.chunks.grid,
                    p.rows.block(), smem, st, a);
}

template <int V>
int run_backward(const BackwardPlan& p, const BackwardArgs& a, bool norm, int gate,
                 cudaStream_t st) {
  if (a.dres) return run_backward<V, true, true, kGateNone>(p, a, st);
  if (norm) {
    if (gate == kGateNone) return run_backward<V, false, true, kGateNone>(p, a, st);
    if (gate == kGateScalar) return run_backward<V, false, true, kGateScalar>(p, a, st);
    return run_backward<V, false, true, kGateVector>(p, a, st);
  }
  if (gate == kGateNone) return run_backward<V, false, false, kGateNone>(p, a, st);
  if (gate == kGateScalar) return run_backward<V, false, false, kGateScalar>(p, a, st);
  return run_backward<V, false, false, kGateVector>(p, a, st);
}

int launch_backward(const char* name, BackwardArgs a, int T, int d, bool norm, int gate,
                    float* dgain, void* ws, cudaStream_t st) {
  const BackwardPlan p = plan_backward(T, d, a.dres ? 3 : 2);
  float* scratch = reinterpret_cast<float*>(static_cast<char*>(ws) + kWorkspaceHeader);
  const size_t slots = static_cast<size_t>(p.chunks.workers) * d;
  a.part_gain = scratch;
  a.part_gate0 = scratch + slots;
  a.part_gate1 = scratch + 2 * slots;
  const bool direct = gate == kGateScalar && a.span == 1;
  a.row_dot = direct ? a.dgate : scratch + 3 * slots;
  a.T = T;
  a.chunk = p.chunks.chunk;
  a.inv_d = 1.f / static_cast<float>(d);
  a.nv = d / 8;
  a.G = p.rows.G;
  int rc;
  {
    ProfScope prof(name, st);
    rc = p.V == 1   ? run_backward<1>(p, a, norm, gate, st)
         : p.V == 2 ? run_backward<2>(p, a, norm, gate, st)
                    : run_backward<4>(p, a, norm, gate, st);
  }
  if (rc != MOE_OK) return rc;
  if (norm || gate == kGateVector) {
    ProfScope prof("norm_join", st);
    const int spans = gate == kGateVector ? (T - 1) / a.span + 1 : 0;
    const int workers = p.chunks.workers, gates = std::min(spans, workers);
    // Tasks [task0, task0 + tasks), `rows` groups each at most: 256 threads take 512
    // of them in one round of loads, and short rows make more groups than that.
    auto join = [&](int task0, int tasks, int rows) {
      auto go = [&](auto kern, int threads) {
        return launch_pdl(kern, dim3((d + 15) / 16, tasks), threads, 0, st, 1, a.part_gain,
                          a.part_gate0, a.part_gate1, d, workers, p.chunks.chunk, T, a.span,
                          static_cast<int>(spans <= workers), task0, norm ? dgain : nullptr,
                          a.dgate);
      };
      return rows <= 1024 ? go(norm_join_kernel<256>, 256) : go(norm_join_kernel<1024>, 1024);
    };
    const int span_rows = a.span / p.chunks.chunk + 2;
    if (gates == 0 || (workers <= 1024) == (span_rows <= 1024)) {
      rc = join(0, 1 + gates, workers);
    } else {   // many groups, short spans
      rc = norm ? join(0, 1, workers) : MOE_OK;
      if (rc == MOE_OK) rc = join(1, gates, span_rows);
    }
    if (rc != MOE_OK) return rc;
  }
  if (gate == kGateScalar && !direct) {
    ProfScope prof("norm_join_rows", st);
    const int rows = (T - 1) / a.span + 1;
    rc = launch_pdl(norm_join_rows_kernel, static_cast<unsigned>(rows), 256, 0, st, 1, a.row_dot,
                    static_cast<long long>(T), static_cast<long long>(a.span), a.dgate);
  }
  return rc;
}

// A call on no rows: the sums over them are zero.
int zero_sums(float* dgain, long long n_gain, float* dgate, long long n_gate, cudaStream_t st) {
  const long long n = std::max(n_gain, n_gate);
  if (n == 0) return MOE_OK;
  ProfScope prof("norm_zero", st);
  return launch_pdl(zero_floats_kernel, static_cast<unsigned>((n + 255) / 256), 256, 0, st, 1,
                    dgain, n_gain, dgate, n_gate);
}

}  // namespace

size_t norm_backward_workspace(int T, int d) {
  if (!norm_shape_ok(T, d) || d > kMaxD || T > kMaxGradRows) return 0;
  const BackwardPlan p = plan_backward(T, d, 2);   // the most groups
  return kWorkspaceHeader + sizeof(float) * (static_cast<size_t>(p.chunks.workers) * d * 3 + T);
}

}  // namespace moe

extern "C" int moe_norm_in(const moe_bf16* x, const float* gain, int T, int d, float eps,
                           moe_bf16* xn, float* rstd, void* stream) {
  using namespace moe;
  if (!norm_shape_ok(T, d) || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (d > kMaxD) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !gain || !xn || !rstd) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(gain) || !aligned16(xn) || !aligned16(rstd))
    return MOE_ERR_MISALIGNED;
  const int nv = d / 8;
  const float inv_d = 1.f / static_cast<float>(d);
  auto xi = reinterpret_cast<const uint4*>(x);
  auto xo = reinterpret_cast<uint4*>(xn);
  cudaStream_t st = as_stream(stream);
  ProfScope prof("norm_in", st);
  if (few_rows(T)) {
    const int V = d <= 8192 ? 1 : 2;
    auto go = [&](auto kern) {
      return launch_pdl(kern, T, plan_rows(d, V).G, 0, st, 1, xi, gain, eps, inv_d, nv, xo, rstd);
    };
    return V == 1 ? go(norm_in_kernel<1>) : go(norm_in_kernel<2>);
  }
  auto go = [&](auto v) {
    constexpr int V = decltype(v)::value;
    static thread_local int configured = -1;
    const RowPlan p = plan_rows(d, V);
    const ChunkPlan c = plan_chunks(T, p, (in_threads(V) + p.block() - 1) / p.block());
    const size_t smem = sizeof(uint4) * kInStages * V * p.block();
    return launch_big(norm_in_ring_kernel<V>, configured, c.grid, p.block(), smem, st, xi, gain, eps,
                      inv_d, T, c.chunk, nv, p.G, xo, rstd);
  };
  // One warp a row up to d = 1024 (776 columns take 86 us a GB so, 100 us with one
  // vector a thread), then as few threads a row as registers allow (2048: 82 us with
  // four vectors, 86 us with two).
  if (nv <= 32) return go(std::integral_constant<int, 1>());
  if (nv <= 64) return go(std::integral_constant<int, 2>());
  return go(std::integral_constant<int, 4>());
}

extern "C" int moe_norm_in_backward(const moe_bf16* dxn, const moe_bf16* x, const float* gain,
                                    const float* rstd, const moe_bf16* dres, int T, int d,
                                    moe_bf16* dx, float* dgain, void* ws, size_t ws_bytes,
                                    void* stream) {
  using namespace moe;
  if (!norm_shape_ok(T, d)) return MOE_ERR_INVALID_ARG;
  if (d > kMaxD || T > kMaxGradRows) return MOE_ERR_UNSUPPORTED;
  if (!dgain) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dgain)) return MOE_ERR_MISALIGNED;
  cudaStream_t st = as_stream(stream);
  if (T == 0) return zero_sums(dgain, d, nullptr, 0, st);
  if (!dxn || !x || !gain || !rstd || !dx) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dxn) || !aligned16(x) || !aligned16(gain) || !aligned16(rstd) || !aligned16(dx) ||
      (dres && !aligned16(dres)) || !aligned16(ws))
    return MOE_ERR_MISALIGNED;
  if (!ws || ws_bytes < norm_backward_workspace(T, d)) return MOE_ERR_WORKSPACE;
  BackwardArgs a = {};
  a.up = reinterpret_cast<const uint4*>(dxn);
  a.x = reinterpret_cast<const uint4*>(x);
  a.rstd = rstd;
  a.gain = gain;
  a.dres = reinterpret_cast<const uint4*>(dres);
  a.dx = reinterpret_cast<uint4*>(dx);
  a.span = T;
  a.scale = 1.f;
  return launch_backward("norm_in_backward", a, T, d, true, kGateNone, dgain, ws, st);
}

extern "C" int moe_norm_out(const moe_bf16* y, const float* topk_w, const int32_t* inv_perm, int K,
                            const moe_bf16* shared_y, const moe_bf16* resid, const float* gain,
                            const float* gate, int span, int gate_cols, float scale, float eps,
                            int T, int d, moe_bf16* out, moe_bf16* zsum, float* rstd,
                            void* stream) {
  using namespace moe;
  if (!norm_shape_ok(T, d) || K < 1 || K > 32 || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (gate && (span < 1 || (gate_cols != 1 && gate_cols != d))) return MOE_ERR_INVALID_ARG;
  if (d > kMaxD) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(T) * K > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!y || !resid || !out) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {y, topk_w, inv_perm, shared_y, resid, gain, gate, out, zsum, rstd};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_MISALIGNED;
  cudaStream_t st = as_stream(stream);
  ProfScope prof("norm_out", st);
  const int nv = d / 8;
  const float inv_d = 1.f / static_cast<float>(d);
  const unsigned gate_span = gate ? span : 1;
  auto yi = reinterpret_cast<const uint4*>(y), si = reinterpret_cast<const uint4*>(shared_y);
  auto ri = reinterpret_cast<const uint4*>(resid);
  auto oo = reinterpret_cast<uint4*>(out), zo = reinterpret_cast<uint4*>(zsum);
  // A ring of two stages, of four where a row has four arrays at most; without one the
  // gathers stay in registers. The ring is faster where it fits: 8192 x 2048, K 8 57 us
  // against 68, 4096 x 6144, K 8 84 against 113. Its 16 S arrays G bytes pass 226 KB above
  // d = 6400 with K 8 (5632 with shared rows): 4096 x 8192, K 8 130 us (floor 109), with
  // shared rows 157 (118); K 32 at 4096 x 2048 100 (86); 4096 x 16384, K 2 149 (99). Four
  // arrays above d = 7168 take registers too, although two stages would fit and be faster:
  // 8192 x 8192, K 3 176 us against 127, K 2 with shared rows 211 against 122 (118).
  const RowPlan wide = plan_rows(d, 1);
  const int arrays = K + 1 + (shared_y ? 1 : 0);
  const int S = arrays <= 4 ? 4 : 2;
  const size_t smem = sizeof(uint4) * S * arrays * wide.block();
  if (nv <= 1024 && smem <= kSmemPerBlock - 1024) {
    const int resident = std::min<int>(std::max(1, 1024 / wide.block()),
                                       kSmemPerSm / static_cast<int>(smem + kSmemReserved));
    const ChunkPlan c = plan_chunks(T, wide, std::max(1, resident));
    static thread_local int configured[2] = {-1, -1};
    auto go = [&](auto kern) {
      return launch_big(kern, configured[S == 2], c.grid, wide.block(), smem, st, yi, topk_w,
                        inv_perm, K, si, ri, gain, gate, gate_span, gate_cols, scale, eps, inv_d, T,
                        c.chunk, nv, wide.G, oo, zo, rstd);
    };
    return S == 2 ? go(norm_out_ring_kernel<2>) : go(norm_out_ring_kernel<4>);
  }
  const int V = nv <= 1024 ? 4 : 8;   // many slots or long rows: the gathers stay in registers
  const RowPlan p = plan_rows(d, V);
  const unsigned grid = (static_cast<unsigned>(T) + p.groups - 1) / p.groups;
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, p.block(), 0, st, 1, yi, topk_w, inv_perm, K, si, ri, gain, gate,
                      gate_span, gate_cols, scale, eps, inv_d, T, nv, p.G, oo, zo, rstd);
  };
  auto by_k = [&](auto v) {
    constexpr int N = decltype(v)::value;
    if constexpr (N == 8) {   // shorter rows of one slot always fit a ring
      if (K == 1) return go(norm_out_kernel<1, N>);
    }
    if (K <= 2) return go(norm_out_kernel<2, N>);
    if (K <= 4) return go(norm_out_kernel<4, N>);
    return go(norm_out_kernel<8, N>);
  };
  if (V == 4) return by_k(std::integral_constant<int, 4>());
  return by_k(std::integral_constant<int, 8>());
}

extern "C" int moe_norm_out_backward(const moe_bf16* dout, const moe_bf16* zsum, const float* rstd,
                                     const float* gain, const float* gate, int span, int gate_cols,
                                     float scale, int T, int d, moe_bf16* dz, float* dgain,
                                     float* dgate, void* ws, size_t ws_bytes, void* stream) {
  using namespace moe;
  if (!norm_shape_ok(T, d)) return MOE_ERR_INVALID_ARG;
  if (gate && (span < 1 || (gate_cols != 1 && gate_cols != d))) return MOE_ERR_INVALID_ARG;
  if (d > kMaxD || T > kMaxGradRows) return MOE_ERR_UNSUPPORTED;
  if ((gain && !dgain) || (gate && !dgate)) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {dout, zsum, rstd, gain, gate, dz, dgain, dgate, ws};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_ERR_MISALIGNED;
  cudaStream_t st = as_stream(stream);
  if (T == 0) return zero_sums(dgain, gain ? d : 0, nullptr, 0, st);   // no tokens: no gate rows
  if (!dout || !zsum || !dz || (gain && !rstd)) return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < norm_backward_workspace(T, d)) return MOE_ERR_WORKSPACE;
  BackwardArgs a = {};
  a.up = reinterpret_cast<const uint4*>(dout);
  a.x = reinterpret_cast<const uint4*>(zsum);
  a.rstd = rstd;
  a.gain = gain;
  a.gate = gate;
  a.dx = reinterpret_cast<uint4*>(dz);
  a.dgate = dgate;
  a.span = gate ? span : T;
  a.scale = scale;
  const int kind = !gate ? kGateNone : gate_cols == 1 ? kGateScalar : kGateVector;
  return launch_backward("norm_out_backward", a, T, d, gain != nullptr, kind, dgain, ws, st);
}

namespace moe {
MOE_DEBUG_STATUS_READER(norm)
}  // namespace moe
