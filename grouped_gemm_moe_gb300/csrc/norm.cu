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
// threads (whole warps) owns one row at a time, one 16-byte vector per thread
// (V = 1 up to d = 8192, then 2), so a row stays in registers between its
// sum and its result and the sum costs one block barrier (none when G = 32).
// Short rows put several groups in a block. Column sums (dg, dgate) stay in the
// threads' registers over a group's contiguous rows; groups write them once to
// the workspace and a second launch adds them in a fixed order: no atomics, the
// same bits every run.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxD = 16384;
constexpr int kGroupTarget = 256;    // threads of a block of several short-row groups

// How rows of nv vectors map to threads.
struct RowPlan {
  int G;        // threads per row group: a multiple of 32
  int groups;   // row groups per block
  int V;        // vectors per thread
  int block() const { return G * groups; }
};

RowPlan plan_rows(int d) {
  const int nv = d / 8;
  RowPlan p;
  p.V = nv <= 1024 ? 1 : 2;
  const int per = (nv + p.V - 1) / p.V;
  p.G = (per + 31) / 32 * 32;
  p.groups = std::max(1, kGroupTarget / p.G);
  return p;
}

int resident(const RowPlan& p) { return std::max(1, 1024 / p.block()); }

// Sum over the G threads of the caller's row group, in every thread. Blocks call
// it in step; `red` holds 2 x 32 floats per block (the two halves alternate by
// `phase`, so one barrier per call is enough: a half is written again only
// after the next call's barrier).
__device__ __forceinline__ float group_sum(float v, int G, float* red, int phase) {
  v = warp_sum(v);
  if (G == 32) return v;
  float* half = red + (phase & 1) * 32;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) half[warp] = v;
  __syncthreads();
  const int nw = G >> 5, first = warp / nw * nw;
  float s = 0.f;
  for (int w = 0; w < nw; ++w) s += half[first + w];
  return s;
}

// xn = bf16(x r g), rows strided over the grid's groups; the next row's loads
// are issued before this row's sum.
template <int V>
__global__ void __launch_bounds__(1024, 1)
norm_in_kernel(const uint4* __restrict__ x, const float* __restrict__ gain, float eps, float inv_d,
               long long T, int nv, int G, uint4* __restrict__ xn, float* __restrict__ rstd) {
  pdl_enter();
  __shared__ float red[64];
  const int groups = blockDim.x / G;
  const int grp = threadIdx.x / G, lane = threadIdx.x - grp * G;
  const long long stride = static_cast<long long>(gridDim.x) * groups;
  float g[V][8];
  bool has[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = lane + v * G;
    has[v] = c < nv;
#pragma unroll
    for (int q = 0; q < 8; ++q) g[v][q] = has[v] ? __ldg(gain + c * 8 + q) : 0.f;
  }
  uint4 cur[V];
  auto load = [&](long long t, uint4 (&to)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      to[v] = (t < T && has[v]) ? ldg_nc_v4(x + t * nv + lane + v * G) : make_uint4(0u, 0u, 0u, 0u);
  };
  const long long first = static_cast<long long>(blockIdx.x) * groups;
  load(first + grp, cur);
  int phase = 0;
  for (long long t0 = first; t0 < T; t0 += stride, ++phase) {
    const long long t = t0 + grp;
    uint4 next[V];
    load(t + stride, next);
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[8];
      unpack8(cur[v], f);
#pragma unroll
      for (int q = 0; q < 8; ++q) s = fmaf(f[q], f[q], s);
    }
    s = group_sum(s, G, red, phase);
    const float r = rsqrtf(s * inv_d + eps);
    if (t < T) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!has[v]) continue;
        float f[8];
        unpack8(cur[v], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = f[q] * r * g[v][q];
        stg_v4(xn + t * nv + lane + v * G, pack8(f));
      }
      if (lane == 0) rstd[t] = r;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) cur[v] = next[v];
  }
}

// Combine, norm, gate, residual. The gathered vectors of a column are loaded KC at
// a time before they are added (slot order, fp32), as in the combine of this library,
// and z is never rounded on its way into the norm; only the copy saved for the
// gradient is bf16.
template <int KC, int V>
__global__ void __launch_bounds__(1024, 1)
norm_out_kernel(const uint4* __restrict__ y, const float* __restrict__ w,
                const int32_t* __restrict__ inv_perm, int K, const uint4* __restrict__ shared_y,
                const uint4* __restrict__ resid, const float* __restrict__ gain,
                const float* __restrict__ gate, unsigned span, int gate_cols, float scale,
                float eps, float inv_d, long long T, int nv, int G, uint4* __restrict__ out,
                uint4* __restrict__ zsum, float* __restrict__ rstd) {
  pdl_enter();
  __shared__ float red[64];
  const int groups = blockDim.x / G;
  const int grp = threadIdx.x / G, lane = threadIdx.x - grp * G;
  const long long stride = static_cast<long long>(gridDim.x) * groups;
  int phase = 0;
  for (long long t0 = static_cast<long long>(blockIdx.x) * groups; t0 < T; t0 += stride, ++phase) {
    const long long t = t0 + grp;
    const bool live = t < T;
    float z[V][8];
    uint4 res[V];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = lane + v * G;
      const bool has = live && c < nv;
#pragma unroll
      for (int q = 0; q < 8; ++q) z[v][q] = 0.f;
      res[v] = make_uint4(0u, 0u, 0u, 0u);
      if (has) {
        uint4 sh = make_uint4(0u, 0u, 0u, 0u);
        if (shared_y) sh = ldg_nc_v4(shared_y + t * nv + c);
        res[v] = ldg_nc_v4(resid + t * nv + c);
        for (int j0 = 0; j0 < K; j0 += KC) {
          uint4 a[KC];
#pragma unroll
          for (int j = 0; j < KC; ++j) {
            if (j0 + j < K) {
              long long p = inv_perm ? __ldg(inv_perm + t * K + j0 + j) : t * K + j0 + j;
              if (!index_ok(p >= 0 && p < T * K)) p = 0;
              a[j] = ldg_nc_v4(y + p * nv + c);
            }
          }
#pragma unroll
          for (int j = 0; j < KC; ++j) {
            if (j0 + j < K) {
              const float wj = w ? __ldg(w + t * K + j0 + j) : 1.f;
              float f[8];
              unpack8(a[j], f);
#pragma unroll
              for (int q = 0; q < 8; ++q) z[v][q] = fmaf(wj, f[q], z[v][q]);
            }
          }
        }
        if (shared_y) {
          float f[8];
          unpack8(sh, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) z[v][q] += f[q];
        }
        if (zsum) stg_v4(zsum + t * nv + c, pack8(z[v]));
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) s = fmaf(z[v][q], z[v][q], s);
    }
    float r = 1.f;
    if (gain) {
      r = rsqrtf(group_sum(s, G, red, phase) * inv_d + eps);
      if (rstd && live && lane == 0) rstd[t] = r;
    }
    if (!live) continue;
    const float* grow =
        gate ? gate + static_cast<long long>(static_cast<unsigned>(t) / span) * gate_cols : nullptr;
    const float row_scale = (grow && gate_cols == 1) ? scale * __ldg(grow) : scale;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = lane + v * G;
      if (c >= nv) continue;
      float f[8];
      unpack8(res[v], f);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float n = z[v][q] * r;
        if (gain) n *= __ldg(gain + c * 8 + q);
        float m = row_scale;
        if (grow && gate_cols != 1) m *= __ldg(grow + c * 8 + q);
        f[q] = fmaf(m, n, f[q]);
      }
      stg_v4(out + t * nv + c, pack8(f));
    }
  }
}

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
  long long T, span, chunk;
  float scale, inv_d;
  int nv, G;
};

__device__ __forceinline__ void store_cols(float* to, const float (&v)[8]) {
  float4* p = reinterpret_cast<float4*>(to);
  p[0] = make_float4(v[0], v[1], v[2], v[3]);
  p[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <int V, bool NORM, int GATE>
__global__ void __launch_bounds__(1024, 1) norm_backward_kernel(BackwardArgs A) {
  pdl_enter();
  __shared__ float red[64];
  const int G = A.G, nv = A.nv;
  const int groups = blockDim.x / G;
  const int grp = threadIdx.x / G, lane = threadIdx.x - grp * G;
  const long long worker = static_cast<long long>(blockIdx.x) * groups + grp;
  const long long row0 = worker * A.chunk;
  const long long row1 = row0 + A.chunk < A.T ? row0 + A.chunk : A.T;
  float g[V][8], gt[V][8], dg[V][8], dgt[V][8];
  bool has[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = lane + v * G;
    has[v] = c < nv;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      g[v][q] = (NORM && has[v]) ? __ldg(A.gain + c * 8 + q) : 1.f;
      gt[v][q] = 1.f;
      dg[v][q] = 0.f;
      dgt[v][q] = 0.f;
    }
  }
  uint4 cu[V], cx[V], cr[V];
  float rs = 1.f, gs = 1.f;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto load = [&](long long t, uint4 (&u)[V], uint4 (&x)[V], uint4 (&res)[V], float& r, float& gsc) {
    const bool live = t < row1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const long long at = t * nv + lane + v * G;
      u[v] = (live && has[v]) ? ldg_nc_v4(A.up + at) : zero;
      x[v] = (live && has[v]) ? ldg_nc_v4(A.x + at) : zero;
      res[v] = (A.dres && live && has[v]) ? ldg_nc_v4(A.dres + at) : zero;
    }
    r = (NORM && live) ? __ldg(A.rstd + t) : 0.f;
    gsc = (GATE == kGateScalar && live) ? __ldg(A.gate + static_cast<unsigned>(t) / static_cast<unsigned>(A.span)) : 1.f;
  };
  load(row0, cu, cx, cr, rs, gs);
  long long span_id = -1, span_end = 0;
  for (long long i = 0; i < A.chunk; ++i) {   // every group of a block runs every step
    const long long t = row0 + i;
    const bool live = t < row1;
    uint4 nu[V], nx[V], nr[V];
    float nrs, ngs;
    load(t + 1, nu, nx, nr, nrs, ngs);
    if (GATE == kGateVector && live && t >= span_end) {   // a span begins (or is entered)
      span_id = static_cast<unsigned>(t) / static_cast<unsigned>(A.span);
      span_end = (span_id + 1) * A.span;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          gt[v][q] = has[v] ? __ldg(A.gate + span_id * (nv * 8LL) + (lane + v * G) * 8 + q) : 0.f;
    }
    // p = alpha dout (or dxn); n = xh g; s = sum p n (times the gate)
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float fu[8], fx[8];
      unpack8(cu[v], fu);
      unpack8(cx[v], fx);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float p = A.scale * fu[q];
        const float xh = NORM ? fx[q] * rs : fx[q];
        const float pn = p * xh;
        if (NORM) dg[v][q] = fmaf(pn, GATE == kGateVector ? gt[v][q] : gs, dg[v][q]);
        const float pg = pn * g[v][q];
        if (GATE == kGateVector) {
          dgt[v][q] += pg;
          s = fmaf(pg, gt[v][q], s);
        } else {
          s += pg;
        }
      }
    }
    if (NORM || GATE == kGateScalar) s = group_sum(s, G, red, static_cast<int>(i));
    if (GATE == kGateScalar) {
      if (live && lane == 0) A.row_dot[t] = s;
      s *= gs;
    }
    const float mean = s * A.inv_d;
    if (live) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!has[v]) continue;
        float fu[8], fx[8], fr[8];
        unpack8(cu[v], fu);
        unpack8(cx[v], fx);
        unpack8(cr[v], fr);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float dn = A.scale * fu[q] * (GATE == kGateVector ? gt[v][q] : gs);
          if (NORM) {
            const float xh = fx[q] * rs;
            fr[q] = fmaf(rs, fmaf(-xh, mean, g[v][q] * dn), fr[q]);
          } else {
            fr[q] += dn;
          }
        }
        stg_v4(A.dx + t * nv + lane + v * G, pack8(fr));
      }
    }
    if (GATE == kGateVector && live && (t + 1 == span_end || t + 1 == row1)) {
      const long long begin = span_id * A.span;
      const long long end = span_end < A.T ? span_end : A.T;
      float* to = begin < row0 ? A.part_gate0 + worker * (nv * 8LL)
                  : end > row1 ? A.part_gate1 + worker * (nv * 8LL)
                               : A.dgate + span_id * (nv * 8LL);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (has[v]) store_cols(to + (lane + v * G) * 8, dgt[v]);
#pragma unroll
        for (int q = 0; q < 8; ++q) dgt[v][q] = 0.f;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      cu[v] = nu[v];
      cx[v] = nx[v];
      cr[v] = nr[v];
    }
    rs = nrs;
    gs = ngs;
  }
  if (NORM && row0 < A.T) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (has[v]) store_cols(A.part_gain + worker * (nv * 8LL) + (lane + v * G) * 8, dg[v]);
  }
}

// Joins the groups' column sums: blockIdx.x picks 32 columns, 8 warps take the
// groups in turn, then one fixed tree. blockIdx.y = 0 sums dgain; y = 1 + w the
// span that begins in group w's rows and ends in a later group's.
constexpr int kJoinWarps = 16;

__global__ void __launch_bounds__(kJoinWarps * 32)
norm_join_kernel(const float* part_gain, const float* part_gate0, const float* part_gate1, int d,
                 long long workers, long long chunk, long long T, long long span, float* dgain,
                 float* dgate) {
  pdl_enter();
  __shared__ float acc[kJoinWarps][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  const float* first = nullptr;   // a row added to the sum of rows [a, b) of `rest`
  const float* rest;
  float* to;
  long long a, b;
  if (blockIdx.y == 0) {
    if (!dgain) return;
    rest = part_gain;
    a = 0;
    b = workers;
    to = dgain;
  } else {
    const long long w = blockIdx.y - 1;
    const long long row0 = w * chunk, row1 = row0 + chunk;
    if (row1 >= T) return;                                     // nothing goes on past the last row
    const long long s = (row1 - 1) / span;
    const long long begin = s * span, end = (s + 1) * span < T ? (s + 1) * span : T;
    if (begin < row0 || end <= row1) return;
    first = part_gate1 + w * d;
    rest = part_gate0;
    a = w + 1;
    b = (end - 1) / chunk + 1;
    to = dgate + s * d;
  }
  float s = 0.f;
  if (c < d) {
#pragma unroll 4
    for (long long w = a + warp; w < b; w += kJoinWarps) s += __ldcg(rest + w * d + c);
  }
  acc[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < d) {
    float t = first ? __ldcg(first + c) : 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) t += acc[w][lane];
    to[c] = t;
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
  int grid;
  long long chunk, workers;
};

BackwardPlan plan_backward(int T, int d) {
  BackwardPlan p;
  p.rows = plan_rows(d);
  const long long most = static_cast<long long>(num_sms()) * resident(p.rows) * p.rows.groups;
  p.chunk = (T + most - 1) / most;
  if (p.chunk < 1) p.chunk = 1;
  p.workers = (T + p.chunk - 1) / p.chunk;
  p.grid = static_cast<int>((p.workers + p.rows.groups - 1) / p.rows.groups);
  return p;
}

bool norm_shape_ok(int T, int d) { return T >= 0 && d >= 8 && d % 8 == 0; }

template <int V>
int run_backward(const BackwardPlan& p, const BackwardArgs& a, bool norm, int gate,
                 cudaStream_t st) {
  auto go = [&](auto kern) { return launch_pdl(kern, p.grid, p.rows.block(), 0, st, 1, a); };
  if (norm) {
    if (gate == kGateNone) return go(norm_backward_kernel<V, true, kGateNone>);
    if (gate == kGateScalar) return go(norm_backward_kernel<V, true, kGateScalar>);
    return go(norm_backward_kernel<V, true, kGateVector>);
  }
  if (gate == kGateNone) return go(norm_backward_kernel<V, false, kGateNone>);
  if (gate == kGateScalar) return go(norm_backward_kernel<V, false, kGateScalar>);
  return go(norm_backward_kernel<V, false, kGateVector>);
}

int launch_backward(const char* name, BackwardArgs a, int T, int d, bool norm, int gate,
                    float* dgain, void* ws, cudaStream_t st) {
  const BackwardPlan p = plan_backward(T, d);
  float* scratch = reinterpret_cast<float*>(static_cast<char*>(ws) + kWorkspaceHeader);
  a.part_gain = scratch;
  a.part_gate0 = a.part_gain + p.workers * d;
  a.part_gate1 = a.part_gate0 + p.workers * d;
  const bool direct = gate == kGateScalar && a.span == 1;
  a.row_dot = direct ? a.dgate : a.part_gate1 + p.workers * d;
  a.T = T;
  a.chunk = p.chunk;
  a.inv_d = 1.f / static_cast<float>(d);
  a.nv = d / 8;
  a.G = p.rows.G;
  int rc;
  {
    ProfScope prof(name, st);
    rc = p.rows.V == 1 ? run_backward<1>(p, a, norm, gate, st)
                       : run_backward<2>(p, a, norm, gate, st);
  }
  if (rc != MOE_OK) return rc;
  if (norm || gate == kGateVector) {
    ProfScope prof("norm_join", st);
    const dim3 grid((d + 31) / 32, gate == kGateVector ? 1 + static_cast<unsigned>(p.workers) : 1);
    rc = launch_pdl(norm_join_kernel, grid, kJoinWarps * 32, 0, st, 1, a.part_gain, a.part_gate0,
                    a.part_gate1, d, p.workers, p.chunk, static_cast<long long>(T), a.span,
                    norm ? dgain : nullptr, a.dgate);
    if (rc != MOE_OK) return rc;
  }
  if (gate == kGateScalar && !direct) {
    ProfScope prof("norm_join_rows", st);
    const long long rows = (T + a.span - 1) / a.span;
    rc = launch_pdl(norm_join_rows_kernel, static_cast<unsigned>(rows), 256, 0, st, 1, a.row_dot,
                    static_cast<long long>(T), a.span, a.dgate);
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
  if (!norm_shape_ok(T, d) || d > kMaxD) return 0;
  const BackwardPlan p = plan_backward(T, d);
  return kWorkspaceHeader + sizeof(float) * (static_cast<size_t>(p.workers) * d * 3 + T);
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
  const RowPlan p = plan_rows(d);
  const long long blocks = (static_cast<long long>(T) + p.groups - 1) / p.groups;
  const long long cap = static_cast<long long>(num_sms()) * resident(p);
  const unsigned grid = static_cast<unsigned>(std::min(blocks, cap));
  cudaStream_t st = as_stream(stream);
  ProfScope prof("norm_in", st);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, p.block(), 0, st, 1, reinterpret_cast<const uint4*>(x), gain, eps,
                      1.f / static_cast<float>(d), static_cast<long long>(T), d / 8, p.G,
                      reinterpret_cast<uint4*>(xn), rstd);
  };
  if (p.V == 1) return go(norm_in_kernel<1>);
  return go(norm_in_kernel<2>);
}

extern "C" int moe_norm_in_backward(const moe_bf16* dxn, const moe_bf16* x, const float* gain,
                                    const float* rstd, const moe_bf16* dres, int T, int d,
                                    moe_bf16* dx, float* dgain, void* ws, size_t ws_bytes,
                                    void* stream) {
  using namespace moe;
  if (!norm_shape_ok(T, d)) return MOE_ERR_INVALID_ARG;
  if (d > kMaxD) return MOE_ERR_UNSUPPORTED;
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
  const RowPlan p = plan_rows(d);
  const long long blocks = (static_cast<long long>(T) + p.groups - 1) / p.groups;
  const long long cap = static_cast<long long>(num_sms()) * resident(p);
  const unsigned grid = static_cast<unsigned>(std::min(blocks, cap));
  cudaStream_t st = as_stream(stream);
  ProfScope prof("norm_out", st);
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, p.block(), 0, st, 1, reinterpret_cast<const uint4*>(y), topk_w,
                      inv_perm, K, reinterpret_cast<const uint4*>(shared_y),
                      reinterpret_cast<const uint4*>(resid), gain, gate,
                      static_cast<unsigned>(gate ? span : 1), gate_cols, scale, eps,
                      1.f / static_cast<float>(d), static_cast<long long>(T), d / 8, p.G,
                      reinterpret_cast<uint4*>(out), reinterpret_cast<uint4*>(zsum), rstd);
  };
  auto by_k = [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (K == 1) return go(norm_out_kernel<1, V>);
    if (K <= 2) return go(norm_out_kernel<2, V>);
    if (K <= 4) return go(norm_out_kernel<4, V>);
    return go(norm_out_kernel<8, V>);
  };
  if (p.V == 1) return by_k(std::integral_constant<int, 1>());
  return by_k(std::integral_constant<int, 2>());
}

extern "C" int moe_norm_out_backward(const moe_bf16* dout, const moe_bf16* zsum, const float* rstd,
                                     const float* gain, const float* gate, int span, int gate_cols,
                                     float scale, int T, int d, moe_bf16* dz, float* dgain,
                                     float* dgate, void* ws, size_t ws_bytes, void* stream) {
  using namespace moe;
  if (!norm_shape_ok(T, d)) return MOE_ERR_INVALID_ARG;
  if (gate && (span < 1 || (gate_cols != 1 && gate_cols != d))) return MOE_ERR_INVALID_ARG;
  if (d > kMaxD) return MOE_ERR_UNSUPPORTED;
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
