// The residual step between two branches, with the norms around it, for packed documents
// (wan_gated_residual_norm_*):
//   x' = a x + gate_d post(y) w_post,   h = (pre(x') w + b)(1 + scale_d) + shift_d.
//
// Gradient, with G = dx_out + (d h / d x')^T dh: dn = dh (1 + scale_d) w;
// d x' = G = dx_out + r (dn - [mean(dn)] - n mean(dn n)) (the bracket for LAYER only);
// dx = a G; the branch gets dyn = G gate_d w_post and dy through its own norm. Everything
// that is summed over rows follows from three sums per document and column:
//   S0 = sum dh, S1 = sum dh n, S2 = sum G yn:   dshift = S0, dscale = w S1 + b S0,
//   dgate = w_post S2, dw = sum_d (1 + scale_d) S1, db = sum_d (1 + scale_d) S0,
//   dw_post = sum_d gate_d S2.
//
// HBM-bound: 4 + es bytes in, 4 + es out per element (es = 2 or 4), the gradient 8 + 2 es
// in. A block owns one row at a time, 8 columns per thread and unit, and walks a contiguous
// range of rows, so the per-document vectors (folded to three) and, in the gradient, the three
// column sums are at hand until the document changes: in registers in the forward, in
// lane-private shared memory in the gradient. Sums leave as partial rows, one per (block,
// document) that meet, at slot block + document (both only grow along the rows, so slots never
// collide), and are added in order by a second kernel: no atomics. Statistics are fp32, squares
// about a mean (the row's, or, in the gradient, the warp's and then moved). What bounds them
// now are the barriers and the latencies between them: forward 124 us for 604 MB (4.9 TB/s,
// 32,760 rows of 1536; a block's rows consecutive, 134 us with rows dealt out in turn), gradient 552 to 562 us (three cards) for 2.07 GB (3.7 TB/s, 22,501 rows of 5120;
// 1263 us with five barriers a row and the sums in registers).
#include <cuda_bf16.h>

#include "checks.h"
#include "internal.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace wan {
namespace {

constexpr int kMaxBlocks = 148 * 8;

struct ResNormParams {
  const float* x;      // forward: x; gradient: x_out of the forward
  const void* y;
  const float *e, *mod_bias;
  const int32_t* cu;
  int n_docs, rows, D;
  int pre, post, gate, chunk;
  float residual_scale, eps;
  const void *w_pre, *b_pre, *w_post;
  float* x_out;
  void* h_out;
  const void* dh;      // gradient
  const float* dx_out;
  float* dx;
  void* dy;
  float* part;         // [slot][3][D]
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of K values over the block, the same in every thread and run. `buf` alternates
// between two halves, so that one barrier per call is enough.
template <int K>
__device__ __forceinline__ void block_sums(float (&v)[K], float (&buf)[2][32][2], int& half) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) buf[half][threadIdx.x >> 5][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += buf[half][w][k];
    v[k] = s;
  }
  half ^= 1;
}

// Document of `row` (the last one that begins at or before it and is not empty there), by
// bisection; row lies in [cu[0], cu[n_docs]).
__device__ __forceinline__ int doc_of_row(const int32_t* cu, int n_docs, int row) {
  int lo = 0, hi = n_docs;  // cu[lo] <= row < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= row) lo = mid; else hi = mid;
  }
  return lo;
}

// Rows [lo, hi) of the documents and this block's share of them, cut evenly.
struct RowSpan {
  int64_t lo, hi;
};
__device__ __forceinline__ RowSpan block_rows(const ResNormParams& p, int block, int blocks) {
  const int64_t a = min(max(__ldg(p.cu), 0), p.rows);
  const int64_t b = min(max(__ldg(p.cu + p.n_docs), static_cast<int>(a)), p.rows);
  const int64_t n = b - a;
  return {a + n * block / blocks, a + n * (block + 1) / blocks};
}

template <typename T>
__device__ __forceinline__ float at(const void* w, int i, float absent) {
  return w ? to_f32<T>(static_cast<const T*>(w)[i]) : absent;
}
__device__ __forceinline__ float mod_at(const ResNormParams& p, int doc, int which, int col) {
  float v = __ldg(p.e + (static_cast<int64_t>(doc) * 6 + which) * p.D + col);
  if (p.mod_bias) v += __ldg(p.mod_bias + static_cast<int64_t>(which) * p.D + col);
  return v;
}

// v -> (v - mean) r (LAYER) or v r (RMS), in place; returns r.
template <int NU>
__device__ __forceinline__ float normalise(float (&v)[NU][8], const bool (&on)[NU], int kind, float inv_d, float eps,
                                           float (&buf)[2][32][2], int& half) {
  if (kind == WAN_NORM_LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[u][i];  // absent units hold zeros
    block_sums<1>(s, buf, half);
    const float mean = s[0] * inv_d;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = on[u] ? v[u][i] - mean : 0.f;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) q[0] += v[u][i] * v[u][i];
  block_sums<1>(q, buf, half);
  const float r = rsqrtf(q[0] * inv_d + eps);  // within 2 units in the last place; the exact root cost 5 % of the time
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] *= r;
  return r;
}

template <typename T, int NU, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) gated_residual_norm_kernel(const ResNormParams p) {
  __shared__ float buf[2][32][2];
  int half = 0;
  const int tpr = blockDim.x;
  int col[NU];
  bool on[NU];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    col[u] = (u * tpr + threadIdx.x) * 8;
    on[u] = col[u] < p.D;
  }
  const float inv_d = 1.0f / static_cast<float>(p.D);
  const RowSpan span = block_rows(p, blockIdx.x, gridDim.x);
  if (span.lo >= span.hi) return;
  float g[NU][8], sc[NU][8], sh[NU][8];  // gate w_post; w (1 + scale); b (1 + scale) + shift
  int64_t doc_end = -1;
  Raw8<float> rx[NU];
  Raw8<T> ry[NU];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int u = 0; u < NU; ++u)
      if (on[u]) {
        load_raw8(rx[u], p.x + row * p.D + col[u]);
        load_raw8(ry[u], static_cast<const T*>(p.y) + row * p.D + col[u]);
      }
  };
  load(span.lo);
  for (int64_t row = span.lo; row < span.hi; ++row) {
    if (row >= doc_end) {
      const int doc = doc_of_row(p.cu, p.n_docs, static_cast<int>(row));
      doc_end = max(__ldg(p.cu + doc + 1), static_cast<int>(row) + 1);
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = col[u] + i;
          if (!on[u]) continue;
          g[u][i] = at<T>(p.w_post, c, 1.f) * (p.gate >= 0 ? mod_at(p, doc, p.gate, c) : 1.f);
          const float s1 = p.chunk >= 0 ? 1.f + mod_at(p, doc, 3 * p.chunk + 1, c) : 1.f;
          sc[u][i] = at<T>(p.w_pre, c, 1.f) * s1;
          sh[u][i] = at<T>(p.b_pre, c, 0.f) * s1 + (p.chunk >= 0 ? mod_at(p, doc, 3 * p.chunk, c) : 0.f);
        }
    }
    float x[NU][8], y[NU][8];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      if (on[u]) {
        unpack8(rx[u], x[u]);
        unpack8(ry[u], y[u]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = y[u][i] = 0.f;
      }
    }
    if (row + 1 < span.hi) load(row + 1);  // in flight while this row's sums are formed
    if (p.post != WAN_NORM_NONE) normalise<NU>(y, on, p.post, inv_d, p.eps, buf, half);
#pragma unroll
    for (int u = 0; u < NU; ++u)
      if (on[u]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = fmaf(y[u][i], g[u][i], p.residual_scale * x[u][i]);
        store_vec8(p.x_out + row * p.D + col[u], x[u]);
      }
    normalise<NU>(x, on, p.pre, inv_d, p.eps, buf, half);
#pragma unroll
    for (int u = 0; u < NU; ++u)
      if (on[u]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = fmaf(x[u][i], sc[u][i], sh[u][i]);
        store_vec8(static_cast<T*>(p.h_out) + row * p.D + col[u], x[u]);
      }
  }
}

// The gradient's statistics with one barrier for both norms: sums that would need the row's mean
// first are taken about the warp's own mean and moved to the row's. Every warp leaves its
// sums, every lane then takes one warp's; rows alternate between two halves.
struct RowSums {
  float4 x[2][32];   // columns, their sum, squares about the warp's mean (RMS: about 0)
  float2 xg[2][32];  // sums of dn (x - the warp's mean) and of dn
  float4 y[2][32];
  float2 k[2][32];
};

__device__ __forceinline__ void ask_l2(const void* at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at)); }

// The row's mean (0 for RMS), r, and sums of g (v - mean) and g, from the warps' (lane w: warp w).
__device__ __forceinline__ void join_warps(float4 s, float2 g, int kind, float inv_d, float eps, float& mean, float& r,
                                           float& a, float& b) {
  mean = kind == WAN_NORM_LAYER ? warp_sum(s.y) * inv_d : 0.f;
  const float own = kind == WAN_NORM_LAYER && s.x > 0.f ? s.y / s.x : 0.f, off = own - mean;
  const float m2 = warp_sum(fmaf(s.x * off, off, s.z));
  r = rsqrtf(fmaf(m2, inv_d, eps));
  a = warp_sum(fmaf(g.y, off, g.x));
  b = kind == WAN_NORM_LAYER ? warp_sum(g.y) : 0.f;
}

using F2 = unsigned long long;  // two fp32
__device__ __forceinline__ float sum_of(F2 v) {
  const float2 f = f2_unpack(v);
  return f.x + f.y;
}
__device__ __forceinline__ void unpack4(const Raw8<__nv_bfloat16>& r, F2 (&v)[4]) {
  v[0] = f2_pack(bf16_lo(r.u.x), bf16_hi(r.u.x)), v[1] = f2_pack(bf16_lo(r.u.y), bf16_hi(r.u.y));
  v[2] = f2_pack(bf16_lo(r.u.z), bf16_hi(r.u.z)), v[3] = f2_pack(bf16_lo(r.u.w), bf16_hi(r.u.w));
}
__device__ __forceinline__ void unpack4(const Raw8<float>& r, F2 (&v)[4]) {
  v[0] = f2_pack(r.a.x, r.a.y), v[1] = f2_pack(r.a.z, r.a.w), v[2] = f2_pack(r.b.x, r.b.y), v[3] = f2_pack(r.b.z, r.b.w);
}
template <typename T>
__device__ __forceinline__ void store4(T* at, const F2 (&v)[4]) {
  float f[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = f2_unpack(v[k]);
    f[2 * k] = x.x, f[2 * k + 1] = x.y;
  }
  store_vec8(at, f);
}

// A thread's 8 columns of `units` vectors in shared memory, 16 bytes apart by thread: no
// conflicts, no exchange.
__device__ __forceinline__ void sm_get(const float4* sm, int which, F2 (&v)[4]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(sm + (2 * which) * blockDim.x + threadIdx.x);
  const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(sm + (2 * which + 1) * blockDim.x + threadIdx.x);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
__device__ __forceinline__ void sm_put(float4* sm, int which, const F2 (&v)[4]) {
  *reinterpret_cast<ulonglong2*>(sm + (2 * which) * blockDim.x + threadIdx.x) = make_ulonglong2(v[0], v[1]);
  *reinterpret_cast<ulonglong2*>(sm + (2 * which + 1) * blockDim.x + threadIdx.x) = make_ulonglong2(v[2], v[3]);
}
size_t bwd_smem(int threads, int nu) { return static_cast<size_t>(threads) * nu * 5 * 32; }

// The document's vectors (gate w_post, w (1 + scale)) and the three column sums live in shared
// memory: in registers they left room for one block an SM, or spilled more. (Two blocks of 320 threads
// have 96 registers a thread; at widths from 2049 to 5120 that still spills 84 bytes in bf16, 220 in
// fp32.)
template <typename T, int NU, int kMaxThreads, int kMinBlocks>
__global__ void __launch_bounds__(kMaxThreads, kMinBlocks) gated_residual_norm_bwd_kernel(const ResNormParams p) {
  extern __shared__ float4 vec[];  // per unit: g, sc, s0, s1, s2
  __shared__ RowSums sm;
  const int tpr = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int col[NU];
  bool on[NU];
  float mine = 0.f;  // columns of this thread
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    col[u] = (u * tpr + threadIdx.x) * 8;
    on[u] = col[u] < p.D;
    mine += on[u] ? 8.f : 0.f;
  }
  const float warp_cols = warp_sum(mine), inv_cols = warp_cols > 0.f ? 1.0f / warp_cols : 0.f;
  const float inv_d = 1.0f / static_cast<float>(p.D);
  for (int i = threadIdx.x; i < 64; i += tpr) {  // entries of absent warps stay 0
    sm.x[0][i] = sm.y[0][i] = make_float4(0.f, 0.f, 0.f, 0.f);
    sm.xg[0][i] = sm.k[0][i] = make_float2(0.f, 0.f);
  }
  const F2 zero[4] = {};
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int k = 0; k < 5; ++k) sm_put(vec, 5 * u + k, zero);
  __syncthreads();
  const RowSpan span = block_rows(p, blockIdx.x, gridDim.x);
  if (span.lo >= span.hi) return;
  int doc = -1, half = 0;
  int64_t doc_end = -1;
  auto flush = [&]() {
    if (!p.part) return;
    float* out = p.part + (static_cast<int64_t>(blockIdx.x) + doc) * 3 * p.D;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        F2 v[4];
        sm_get(vec, 5 * u + 2 + k, v);
        if (on[u]) store4(out + static_cast<int64_t>(k) * p.D + col[u], v);
        sm_put(vec, 5 * u + 2 + k, zero);
      }
  };
  const float *xp = p.x + span.lo * p.D, *up = p.dx_out + (p.dx_out ? span.lo * p.D : 0);
  const T *hp = static_cast<const T*>(p.dh) + span.lo * p.D, *yp = static_cast<const T*>(p.y) + span.lo * p.D;
  float* dxp = p.dx + span.lo * p.D;
  T* dyp = static_cast<T*>(p.dy) + span.lo * p.D;
  for (int64_t row = span.lo; row < span.hi;
       ++row, half ^= 1, xp += p.D, hp += p.D, yp += p.D, dxp += p.D, dyp += p.D, up += p.dx_out ? p.D : 0) {
    Raw8<float> rx[NU], rg[NU];
    Raw8<T> ry[NU], rh[NU];
    const bool more = row + 1 < span.hi;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      rx[u] = Raw8<float>{}, rg[u] = Raw8<float>{}, ry[u] = Raw8<T>{}, rh[u] = Raw8<T>{};
      if (!on[u]) continue;
      load_raw8(rx[u], xp + col[u]);
      load_raw8(rh[u], hp + col[u]);
      load_raw8(ry[u], yp + col[u]);
      if (more) {  // the next row on its way into L2
        ask_l2(xp + p.D + col[u]);
        ask_l2(hp + p.D + col[u]);
        ask_l2(yp + p.D + col[u]);
        if (p.dx_out) ask_l2(up + p.D + col[u]);
      }
    }
    if (row >= doc_end) {
      if (doc >= 0) flush();
      doc = doc_of_row(p.cu, p.n_docs, static_cast<int>(row));
      doc_end = max(__ldg(p.cu + doc + 1), static_cast<int>(row) + 1);
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        if (!on[u]) continue;
        float g[8], sc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = col[u] + i;
          g[i] = at<T>(p.w_post, c, 1.f) * (p.gate >= 0 ? mod_at(p, doc, p.gate, c) : 1.f);
          sc[i] = at<T>(p.w_pre, c, 1.f) * (p.chunk >= 0 ? 1.f + mod_at(p, doc, 3 * p.chunk + 1, c) : 1.f);
        }
        const F2 g4[4] = {f2_pack(g[0], g[1]), f2_pack(g[2], g[3]), f2_pack(g[4], g[5]), f2_pack(g[6], g[7])};
        const F2 s4[4] = {f2_pack(sc[0], sc[1]), f2_pack(sc[2], sc[3]), f2_pack(sc[4], sc[5]), f2_pack(sc[6], sc[7])};
        sm_put(vec, 5 * u, g4);
        sm_put(vec, 5 * u + 1, s4);
      }
    }
    // This warp's sums: of x about its own mean, with dn = dh sc, and of y. Columns that are
    // not there hold zeros and add their own mean's squares: they are left out.
    float own = 0.f, sum = 0.f, yown = 0.f, ysum = 0.f;
    if (p.pre == WAN_NORM_LAYER || p.post == WAN_NORM_LAYER) {
      F2 a = 0ull, b = 0ull;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        F2 x[4], y[4];
        unpack4(rx[u], x);
        unpack4(ry[u], y);
#pragma unroll
        for (int k = 0; k < 4; ++k) a = f2_add(a, x[k]), b = f2_add(b, y[k]);
      }
      if (p.pre == WAN_NORM_LAYER) sum = warp_sum(sum_of(a)), own = sum * inv_cols;
      if (p.post == WAN_NORM_LAYER) ysum = warp_sum(sum_of(b)), yown = ysum * inv_cols;
    }
    {
      F2 m2 = 0ull, ga = 0ull, gb = 0ull, ym2 = 0ull;
      const F2 own2 = f2_splat(-own), yown2 = f2_splat(-yown);
#pragma unroll
      for (int u = 0; u < NU; ++u)
        if (on[u]) {
          F2 x[4], y[4], h[4], sc[4];
          unpack4(rx[u], x);
          unpack4(rh[u], h);
          sm_get(vec, 5 * u + 1, sc);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const F2 v = f2_add(x[k], own2), dn = f2_mul(h[k], sc[k]);
            m2 = f2_fma(v, v, m2);
            ga = f2_fma(dn, v, ga);
            gb = f2_add(gb, dn);
          }
          if (p.post != WAN_NORM_NONE) {
            unpack4(ry[u], y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const F2 v = f2_add(y[k], yown2);
              ym2 = f2_fma(v, v, ym2);
            }
          }
        }
      const float m = warp_sum(sum_of(m2)), a = warp_sum(sum_of(ga));
      const float c = p.pre == WAN_NORM_LAYER ? warp_sum(sum_of(gb)) : 0.f;
      const float ym = p.post != WAN_NORM_NONE ? warp_sum(sum_of(ym2)) : 0.f;
      if (lane == 0) {
        sm.x[half][warp] = make_float4(warp_cols, sum, m, 0.f);
        sm.xg[half][warp] = make_float2(a, c);
        sm.y[half][warp] = make_float4(warp_cols, ysum, ym, 0.f);
      }
    }
    // Read as late as the barrier still hides it: held from the start it cost the second block.
#pragma unroll
    for (int u = 0; u < NU; ++u)
      if (on[u] && p.dx_out) load_raw8(rg[u], up + col[u]);
    __syncthreads();
    float mean, r, a, c;
    join_warps(sm.x[half][lane], sm.xg[half][lane], p.pre, inv_d, p.eps, mean, r, a, c);
    // dn n sums to a r; G = dx_out + r (dn - [mean dn] - n mean(dn n))
    a *= r * r * inv_d;
    c *= inv_d;
    float ymean = 0.f, ry_ = 1.f;
    if (p.post != WAN_NORM_NONE) {
      float d0, d1;
      join_warps(sm.y[half][lane], make_float2(0.f, 0.f), p.post, inv_d, p.eps, ymean, ry_, d0, d1);
    }
    F2 yn[NU][4], gg[NU][4], k0 = 0ull, k1 = 0ull;
    const F2 mean2 = f2_splat(-mean), r2 = f2_splat(r), a2 = f2_splat(-a), c2 = f2_splat(-c), ymean2 = f2_splat(-ymean),
             ry2 = f2_splat(ry_), scale2 = f2_splat(p.residual_scale);
#pragma unroll
    for (int u = 0; u < NU; ++u)
      if (on[u]) {
        F2 x[4], h[4], sc[4], s0[4], s1[4], s2[4], g[4], dx[4], gv[4];
        unpack4(rx[u], x);
        unpack4(rh[u], h);
        unpack4(ry[u], yn[u]);
        unpack4(rg[u], gv);
        sm_get(vec, 5 * u + 1, sc);
        sm_get(vec, 5 * u + 2, s0);
        sm_get(vec, 5 * u + 3, s1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const F2 v = f2_add(x[k], mean2);
          s0[k] = f2_add(s0[k], h[k]);
          s1[k] = f2_fma(h[k], f2_mul(v, r2), s1[k]);
          gv[k] = f2_fma(r2, f2_fma(v, a2, f2_fma(h[k], sc[k], c2)), gv[k]);
          dx[k] = f2_mul(scale2, gv[k]);
        }
        sm_put(vec, 5 * u + 2, s0);
        sm_put(vec, 5 * u + 3, s1);
        store4(dxp + col[u], dx);
        sm_get(vec, 5 * u + 4, s2);
        sm_get(vec, 5 * u, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          yn[u][k] = f2_mul(f2_add(yn[u][k], ymean2), ry2);
          s2[k] = f2_fma(gv[k], yn[u][k], s2[k]);
          gg[u][k] = f2_mul(gv[k], g[k]);
          k0 = f2_fma(gg[u][k], yn[u][k], k0);
          k1 = f2_add(k1, gg[u][k]);
        }
        sm_put(vec, 5 * u + 4, s2);
      }
    float ka = 0.f, kc = 0.f;
    if (p.post != WAN_NORM_NONE) {
      const float x0 = warp_sum(sum_of(k0)), x1 = p.post == WAN_NORM_LAYER ? warp_sum(sum_of(k1)) : 0.f;
      if (lane == 0) sm.k[half][warp] = make_float2(x0, x1);
      __syncthreads();
      const float2 k = sm.k[half][lane];
      ka = warp_sum(k.x) * inv_d;
      if (p.post == WAN_NORM_LAYER) kc = warp_sum(k.y) * inv_d;
    }
    const F2 ka2 = f2_splat(-ka), kc2 = f2_splat(-kc);
#pragma unroll
    for (int u = 0; u < NU; ++u)
      if (on[u]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) gg[u][k] = f2_mul(ry2, f2_fma(yn[u][k], ka2, f2_add(gg[u][k], kc2)));
        store4(dyp + col[u], gg[u]);
      }
  }
  flush();
}

// Sums over a document's rows: slots block + doc of the blocks whose span meets the
// document, in order (thread row y takes every 32nd). Writes S0..S2 to `total` and, when
// asked, the document's rows of de.
template <typename T>
__global__ void __launch_bounds__(1024) resnorm_doc_sums_kernel(const ResNormParams p, int blocks, float* total, float* de) {
  __shared__ float acc[3][32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  const int64_t a = min(max(__ldg(p.cu), 0), p.rows);
  const int64_t b = min(max(__ldg(p.cu + p.n_docs), static_cast<int>(a)), p.rows);
  const int64_t n = b - a;
  for (int doc = blockIdx.y; doc < p.n_docs; doc += gridDim.y) {
    const DocRange dr = doc_range(p.cu, doc, p.rows);
    float s[3] = {0.f, 0.f, 0.f};
    if (dr.count > 0 && dr.first >= a && n > 0 && c < p.D) {
      // block k holds rows [a + n k / B, a + n (k + 1) / B): none, if there are more blocks
      // than rows and both cuts lie at one place
      const int k0 = static_cast<int>(((dr.first - a + 1) * blocks - 1) / n);
      const int k1 = static_cast<int>(min((dr.first - a + dr.count) * blocks - 1, n * blocks - 1) / n);
      const float* first = p.part + static_cast<int64_t>(doc) * 3 * p.D + c;
#pragma unroll 4
      for (int k = k0 + threadIdx.y; k <= k1; k += 32) {
        const bool rows = n >= blocks || n * k / blocks < n * (k + 1) / blocks;
        const float* row = first + static_cast<int64_t>(k) * 3 * p.D;
#pragma unroll
        for (int q = 0; q < 3; ++q) s[q] += rows ? row[static_cast<int64_t>(q) * p.D] : 0.f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; ++q) acc[q][threadIdx.y][threadIdx.x] = s[q];
    __syncthreads();
    if (threadIdx.y < 3 && c < p.D) {
      float v = 0.f;
#pragma unroll
      for (int y = 0; y < 32; ++y) v += acc[threadIdx.y][y][threadIdx.x];
      acc[threadIdx.y][0][threadIdx.x] = v;
      total[(static_cast<int64_t>(doc) * 3 + threadIdx.y) * p.D + c] = v;
    }
    __syncthreads();
    if (threadIdx.y == 0 && de && c < p.D) {
      float* out = de + static_cast<int64_t>(doc) * 6 * p.D + c;
      const float S0 = acc[0][0][threadIdx.x], S1 = acc[1][0][threadIdx.x], S2 = acc[2][0][threadIdx.x];
      if (p.chunk >= 0) {
        out[static_cast<int64_t>(3 * p.chunk) * p.D] = S0;
        out[static_cast<int64_t>(3 * p.chunk + 1) * p.D] = at<T>(p.w_pre, c, 1.f) * S1 + at<T>(p.b_pre, c, 0.f) * S0;
      }
      if (p.gate >= 0) out[static_cast<int64_t>(p.gate) * p.D] = at<T>(p.w_post, c, 1.f) * S2;
    }
  }
}

// Sums over documents, in order: the gradients of the weights and of mod_bias.
template <typename T>
__global__ void __launch_bounds__(128) resnorm_weight_sums_kernel(const ResNormParams p, const float* total,
                                                                  wan_residual_norm_grads out) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (c >= p.D) return;
  float dw = 0.f, db = 0.f, dwp = 0.f, m0 = 0.f, m1 = 0.f, m2 = 0.f;
  const float w = at<T>(p.w_pre, c, 1.f), b = at<T>(p.b_pre, c, 0.f), wp = at<T>(p.w_post, c, 1.f);
  for (int doc = 0; doc < p.n_docs; ++doc) {
    if (doc_range(p.cu, doc, p.rows).count == 0) continue;  // its modulation may hold anything: 0 * NaN
    const float* t = total + static_cast<int64_t>(doc) * 3 * p.D + c;
    const float S0 = t[0], S1 = t[p.D], S2 = t[2 * static_cast<int64_t>(p.D)];
    const float s1 = p.chunk >= 0 ? 1.f + mod_at(p, doc, 3 * p.chunk + 1, c) : 1.f;
    dw = fmaf(s1, S1, dw);
    db = fmaf(s1, S0, db);
    dwp = fmaf(p.gate >= 0 ? mod_at(p, doc, p.gate, c) : 1.f, S2, dwp);
    m0 += S0;
    m1 += w * S1 + b * S0;
    m2 += wp * S2;
  }
  if (out.dw_pre) out.dw_pre[c] = dw;
  if (out.db_pre) out.db_pre[c] = db;
  if (out.dw_post) out.dw_post[c] = dwp;
  if (out.dmod_bias) {
    if (p.chunk >= 0) {
      out.dmod_bias[static_cast<int64_t>(3 * p.chunk) * p.D + c] = m0;
      out.dmod_bias[static_cast<int64_t>(3 * p.chunk + 1) * p.D + c] = m1;
    }
    if (p.gate >= 0) out.dmod_bias[static_cast<int64_t>(p.gate) * p.D + c] = m2;
  }
}

// Threads of a block: as many units of 8 columns per thread as NU, whole warps.
int block_threads(int D, int nu) { return (D / 8 + nu * 32 - 1) / (nu * 32) * 32; }

// Blocks of one launch: every resident slot of the card, no more than rows.
int blocks_of(int resident, int rows) {
  const int n = resident < kMaxBlocks ? resident : kMaxBlocks;
  return n < rows ? n : (rows > 0 ? rows : 1);
}

template <typename T, int NU, int kMaxThreads>
int launch_fwd(const ResNormParams& p, cudaStream_t s) {
  static ResidentCache resident;
  const int th = block_threads(p.D, NU);
  auto kernel = gated_residual_norm_kernel<T, NU, kMaxThreads>;
  kernel<<<blocks_of(resident.get(reinterpret_cast<const void*>(kernel), th, 0), p.rows), th, 0, s>>>(p);
  return check_launch();
}
template <typename T>
int run_fwd(const ResNormParams& p, cudaStream_t s) {
  if (p.D <= 2048) return launch_fwd<T, 1, 256>(p, s);
  return launch_fwd<T, 2, 512>(p, s);
}

template <typename T, int NU, int kMaxThreads, int kMinBlocks>
int launch_bwd(const ResNormParams& p, cudaStream_t s, int* blocks) {
  const int th = block_threads(p.D, NU);
  auto kernel = gated_residual_norm_bwd_kernel<T, NU, kMaxThreads, kMinBlocks>;
  const size_t smem = bwd_smem(th, NU);
  static ResidentCache resident;
  *blocks = blocks_of(resident.get(reinterpret_cast<const void*>(kernel), th, smem, bwd_smem(kMaxThreads, NU)), p.rows);
  kernel<<<*blocks, th, smem, s>>>(p);
  return check_launch();
}
template <typename T>
int run_bwd(const ResNormParams& p, const wan_residual_norm_grads& g, float* total, cudaStream_t s) {
  const bool weights = g.dmod_bias || g.dw_pre || g.db_pre || g.dw_post;
  int blocks = 0, st = WAN_OK;
  if (p.n_docs > 0)
    st = p.D <= 2048 ? launch_bwd<T, 1, 256, 3>(p, s, &blocks)
                     : p.D <= 5120 ? launch_bwd<T, 2, 320, 2>(p, s, &blocks) : launch_bwd<T, 2, 512, 1>(p, s, &blocks);
  else
    count_launches(-1);  // the call was counted as one
  if (st != WAN_OK || !(weights || g.de)) return st;
  if (p.n_docs > 0) {
    const int docs_y = p.n_docs < 1024 ? p.n_docs : 1024;
    resnorm_doc_sums_kernel<T><<<dim3((p.D + 31) / 32, docs_y), dim3(32, 32), 0, s>>>(p, blocks, total, g.de);
    count_launches(1);
    st = check_launch();
  }
  if (st != WAN_OK || !weights) return st;
  resnorm_weight_sums_kernel<T><<<(p.D + 127) / 128, 128, 0, s>>>(p, total, g);
  count_launches(1);
  return check_launch();
}

int check_op(const wan_dit_config* cfg, const wan_residual_norm* op, const float* e, const float* mod_bias,
             const int32_t* cu, int n_docs, int rows) {
  WAN_TRY(check_cfg(cfg));
  WAN_REQUIRE(op, WAN_ERR_NULL);
  WAN_REQUIRE(op->pre == WAN_NORM_LAYER || op->pre == WAN_NORM_RMS, WAN_ERR_SHAPE);
  WAN_REQUIRE(op->post >= WAN_NORM_NONE && op->post <= WAN_NORM_RMS, WAN_ERR_SHAPE);
  WAN_REQUIRE(op->gate >= -1 && op->gate <= 5 && op->chunk >= -1 && op->chunk <= 1, WAN_ERR_SHAPE);
  // one row of e is either the gate or a shift or scale: its gradient has one place
  WAN_REQUIRE(op->gate < 0 || op->chunk < 0 || (op->gate != 3 * op->chunk && op->gate != 3 * op->chunk + 1),
              WAN_ERR_SHAPE);
  WAN_REQUIRE(op->residual_scale - op->residual_scale == 0.f, WAN_ERR_SHAPE);  // finite
  WAN_REQUIRE(op->post != WAN_NORM_NONE || !op->w_post, WAN_ERR_SHAPE);
  WAN_REQUIRE(cfg->dim <= 8192, WAN_ERR_UNSUPPORTED);
  WAN_REQUIRE(rows >= 0 && n_docs >= 0, WAN_ERR_SHAPE);
  WAN_TRY(check_opt_ptr(op->w_pre));
  WAN_TRY(check_opt_ptr(op->b_pre));
  WAN_TRY(check_opt_ptr(op->w_post));
  WAN_TRY(check_opt_ptr(mod_bias));
  if (op->gate >= 0 || op->chunk >= 0) WAN_TRY(check_array(e, n_docs));
  WAN_TRY(check_ints(cu, n_docs + 1));
  return WAN_OK;
}

ResNormParams make_params(const wan_dit_config* cfg, const wan_residual_norm* op, const float* x, const void* y,
                          const float* e, const float* mod_bias, const int32_t* cu, int n_docs, int rows) {
  ResNormParams p{};
  p.x = x, p.y = y, p.e = e, p.mod_bias = mod_bias, p.cu = cu;
  p.n_docs = n_docs, p.rows = rows, p.D = cfg->dim;
  p.pre = op->pre, p.post = op->post, p.gate = op->gate, p.chunk = op->chunk;
  p.residual_scale = op->residual_scale, p.eps = cfg->eps;
  p.w_pre = op->w_pre, p.b_pre = op->b_pre, p.w_post = op->w_post;
  return p;
}

}  // namespace
}  // namespace wan

using namespace wan;

extern "C" {

int wan_gated_residual_norm_fwd(const wan_dit_config* cfg, const wan_residual_norm* op, const float* x, const void* y,
                                const float* e, const float* mod_bias, const int32_t* cu_rows, int n_docs, int rows,
                                float* x_out, void* h_out, void* stream) {
  WAN_TRY(check_op(cfg, op, e, mod_bias, cu_rows, n_docs, rows));
  WAN_TRY(check_array(x, rows));
  WAN_TRY(check_array(y, rows));
  WAN_TRY(check_array(x_out, rows));
  WAN_TRY(check_array(h_out, rows));
  if (rows == 0 || n_docs == 0) return WAN_OK;
  ResNormParams p = make_params(cfg, op, x, y, e, mod_bias, cu_rows, n_docs, rows);
  p.x_out = x_out, p.h_out = h_out;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  trace_launch_begin(WAN_KIND_NORM, s, static_cast<double>(rows) * cfg->dim * 2.0 * (4 + dtype_size(cfg->dtype)));
  const int st = cfg->dtype == WAN_BF16 ? run_fwd<__nv_bfloat16>(p, s) : run_fwd<float>(p, s);
  trace_launch_end(WAN_KIND_NORM, s);
  return st;
}

size_t wan_gated_residual_norm_workspace_bytes(const wan_dit_config* cfg, int rows, int n_docs) {
  if (check_cfg(cfg) != WAN_OK || rows < 0 || n_docs < 0) return 0;
  const int64_t blocks = rows < kMaxBlocks ? rows : kMaxBlocks;
  // partial rows of every (block, document) slot, then the documents' sums
  return static_cast<size_t>(blocks + 2 * static_cast<int64_t>(n_docs)) * 3 * cfg->dim * 4;
}

int wan_gated_residual_norm_bwd(const wan_dit_config* cfg, const wan_residual_norm* op, const float* x_out,
                                const void* y, const float* e, const float* mod_bias, const int32_t* cu_rows,
                                int n_docs, int rows, const void* dh, const float* dx_out, float* dx, void* dy,
                                const wan_residual_norm_grads* grads, void* workspace, size_t ws_bytes, void* stream) {
  WAN_TRY(check_op(cfg, op, e, mod_bias, cu_rows, n_docs, rows));
  WAN_TRY(check_array(x_out, rows));
  WAN_TRY(check_array(y, rows));
  WAN_TRY(check_array(dh, rows));
  WAN_TRY(check_opt_ptr(dx_out));
  WAN_TRY(check_array(dx, rows));
  WAN_TRY(check_array(dy, rows));
  wan_residual_norm_grads g{};
  if (grads) g = *grads;
  for (const float* q : {g.de, g.dmod_bias, g.dw_pre, g.db_pre, g.dw_post}) WAN_TRY(check_opt_ptr(q));
  const bool sums = g.de || g.dmod_bias || g.dw_pre || g.db_pre || g.dw_post;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((n_docs == 0 || rows == 0) && !sums) return WAN_OK;
  ResNormParams p = make_params(cfg, op, x_out, y, e, mod_bias, cu_rows, n_docs, rows);
  p.dh = dh, p.dx_out = dx_out, p.dx = dx, p.dy = dy;
  float* total = nullptr;
  if (sums) {
    const size_t need = wan_gated_residual_norm_workspace_bytes(cfg, rows, n_docs);
    if (need > 0) WAN_TRY(check_ptr(workspace));  // no rows and no documents: none
    WAN_REQUIRE(ws_bytes >= need, WAN_ERR_WORKSPACE);
    p.part = static_cast<float*>(workspace);
    const int64_t blocks = rows < kMaxBlocks ? rows : kMaxBlocks;
    total = p.part + (blocks + n_docs) * 3 * static_cast<int64_t>(cfg->dim);
  }
  trace_launch_begin(WAN_KIND_NORM, s, static_cast<double>(rows) * cfg->dim * (12 + 3.0 * dtype_size(cfg->dtype)));
  const int st = cfg->dtype == WAN_BF16 ? run_bwd<__nv_bfloat16>(p, g, total, s) : run_bwd<float>(p, g, total, s);
  trace_launch_end(WAN_KIND_NORM, s);
  return st;
}

}  // extern "C"
