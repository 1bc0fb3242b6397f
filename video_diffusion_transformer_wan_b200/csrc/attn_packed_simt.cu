// Attention inside packed documents in fp32 on the CUDA cores, and its gradient: one pass
// over the keys with a running maximum and sum; the gradient recomputes the probabilities
// from the stored log-sums, p = e^(s - lse), ds = p (dp - delta) (1 - tanh^2) with
// delta = sum(do * o), in one kernel per side (dq over the keys, dk and dv over the queries),
// so that nothing is added across blocks.
//
// A block of 128 threads owns 16 rows (queries, or keys) of one document and head and walks
// tiles of 32 rows of the other side, double-buffered by cp.async. 16 threads share two rows:
// in a score product each has 2 x 2 entries, 16 multiply-adds per four 16-byte shared loads;
// in a product with the tile's values 2 rows x 4 (or 2 x 4) dims. Row maxima and sums are
// shuffles over the 16. fp32 models are small: few rows and long latencies bound this, hence
// tiles of 16 rows (346 rows of 2 heads are 48 blocks).
#include <math.h>

#include "internal.h"
#include "packed.cuh"

namespace wan {
namespace {

constexpr int kR = 16;         // rows of a block
constexpr int kC = 32;         // rows of a tile of the other side
constexpr int kThreads = 128;
constexpr int kSp = kC + 4;    // pitch of a tile of probabilities

struct Doc {
  int q0, Lq, k0, Lk, off, prefix;
};
__device__ __forceinline__ Doc load_doc(const PackedAttn& p, int d) {
  const DocRange a = doc_range(p.cu_q, d, p.q_rows), b = doc_range(p.cu_k, d, p.k_rows);
  return {a.first, a.count, b.first, b.count, b.count - a.count, p.prefix ? __ldg(p.prefix + d) : 0};
}

// This block's tile (the first warp finds it); false for a block past the last tile.
__device__ __forceinline__ bool block_tile(const int32_t* cu, int n_docs, int rows, int& doc, int& tile) {
  __shared__ int found[3];
  if (threadIdx.x < 32) {
    int d = 0, t = 0;
    const bool ok = find_doc_tile(cu, n_docs, rows, kR, blockIdx.x, d, t);
    if (threadIdx.x == 0) found[0] = ok, found[1] = d, found[2] = t;
  }
  __syncthreads();
  doc = found[1], tile = found[2];
  return found[0] != 0;
}

// Rows [row0, row0 + n) of a matrix into shared memory (pitch D + 4), rows from `valid` on and
// dims from d on as zeros.
template <int D>
__device__ __forceinline__ void load_async(float* dst, const void* src, int64_t stride, int64_t row0, int n, int valid,
                                           int col0, int d) {
  for (int i = threadIdx.x; i < n * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = i - r * (D / 4);
    const bool there = r < valid && 4 * c < d;
    const float* from = static_cast<const float*>(src) + (there ? (row0 + r) * stride + col0 + 4 * c : 0);
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst + r * (D + 4) + 4 * c));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
  }
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void async_wait_groups() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
// Those of no group too: a block without a tile of the other side commits none, and leaves
// only when its own rows have landed.
__device__ __forceinline__ void async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// s[i][j] = row (2 ty + i) of a . row (tx + 16 j) of b.
template <int D>
__device__ __forceinline__ void dot_2x2(const float* a, const float* b, float (&s)[2][2]) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const float4 *a0 = reinterpret_cast<const float4*>(a + (2 * ty) * (D + 4)), *a1 = reinterpret_cast<const float4*>(a + (2 * ty + 1) * (D + 4));
  const float4 *b0 = reinterpret_cast<const float4*>(b + tx * (D + 4)), *b1 = reinterpret_cast<const float4*>(b + (tx + 16) * (D + 4));
  s[0][0] = s[0][1] = s[1][0] = s[1][1] = 0.f;
#pragma unroll 8
  for (int c = 0; c < D / 4; ++c) {
    const float4 x0 = a0[c], x1 = a1[c], y0 = b0[c], y1 = b1[c];
    s[0][0] = fmaf(x0.w, y0.w, fmaf(x0.z, y0.z, fmaf(x0.y, y0.y, fmaf(x0.x, y0.x, s[0][0]))));
    s[0][1] = fmaf(x0.w, y1.w, fmaf(x0.z, y1.z, fmaf(x0.y, y1.y, fmaf(x0.x, y1.x, s[0][1]))));
    s[1][0] = fmaf(x1.w, y0.w, fmaf(x1.z, y0.z, fmaf(x1.y, y0.y, fmaf(x1.x, y0.x, s[1][0]))));
    s[1][1] = fmaf(x1.w, y1.w, fmaf(x1.z, y1.z, fmaf(x1.y, y1.y, fmaf(x1.x, y1.x, s[1][1]))));
  }
}
// o[i] += row (2 ty + i) of p (32 entries) times b, dims 4 tx + 64 k.
template <int D>
__device__ __forceinline__ void add_product(const float* p, const float* b, float4 (&o)[2][D / 64]) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 2
  for (int j = 0; j < kC; j += 4) {
    const float4 p0 = *reinterpret_cast<const float4*>(p + (2 * ty) * kSp + j), p1 = *reinterpret_cast<const float4*>(p + (2 * ty + 1) * kSp + j);
    const float w0[4] = {p0.x, p0.y, p0.z, p0.w}, w1[4] = {p1.x, p1.y, p1.z, p1.w};
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(b + (j + jj) * (D + 4) + 4 * tx + 64 * k);
        o[0][k].x = fmaf(w0[jj], v.x, o[0][k].x), o[0][k].y = fmaf(w0[jj], v.y, o[0][k].y);
        o[0][k].z = fmaf(w0[jj], v.z, o[0][k].z), o[0][k].w = fmaf(w0[jj], v.w, o[0][k].w);
        o[1][k].x = fmaf(w1[jj], v.x, o[1][k].x), o[1][k].y = fmaf(w1[jj], v.y, o[1][k].y);
        o[1][k].z = fmaf(w1[jj], v.z, o[1][k].z), o[1][k].w = fmaf(w1[jj], v.w, o[1][k].w);
      }
  }
}
template <int D>
__device__ __forceinline__ void store_rows(void* base, int64_t stride, int64_t row0, int valid, int col0, int d,
                                           const float4 (&o)[2][D / 64], const float (&f)[2]) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
      if (2 * ty + i < valid && 4 * tx + 64 * k < d)
        *reinterpret_cast<float4*>(static_cast<float*>(base) + (row0 + 2 * ty + i) * stride + col0 + 4 * tx + 64 * k) =
            make_float4(o[i][k].x * f[i], o[i][k].y * f[i], o[i][k].z * f[i], o[i][k].w * f[i]);
}

__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, 16);
  return v;
}
__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o, 16));
  return v;
}
// Score of query position `pos` (i + off) and key j from q.k; d s / d(q.k) / scale in `turn`.
__device__ __forceinline__ float score(float dot, const PackedAttn& p, float slope, int pos, int j, float& turn) {
  float s = dot * p.scale;
  turn = 1.f;
  if (p.cap > 0.f) {
    const float t = tanhf(s / p.cap);
    s = p.cap * t;
    turn = 1.f - t * t;
  }
  return s - slope * fabsf(static_cast<float>(pos - j));
}

template <int D>
__global__ void __launch_bounds__(kThreads) packed_fwd_kernel(const PackedAttn p) {
  extern __shared__ float4 smem4[];
  float* sm = reinterpret_cast<float*>(smem4);
  constexpr int kTile = kC * (D + 4);
  float *sq = sm, *skv = sq + kR * (D + 4), *sp = skv + 4 * kTile;  // skv: K, V of two stages
  int d, tile;
  if (!block_tile(p.cu_q, p.n_docs, p.q_rows, d, tile)) return;
  const Doc doc = load_doc(p, d);
  const int h = blockIdx.y, hk = h / (p.H / p.Hk);
  const int i0 = tile * kR, rows = min(kR, doc.Lq - i0);
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int most = seen_keys(i0 + rows - 1, doc.off, doc.Lk, doc.prefix, p.causal_block);
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  auto load = [&](int j0, int stage) {
    const int keys = min(kC, doc.Lk - j0);
    load_async<D>(skv + 2 * stage * kTile, p.k, p.k_stride, static_cast<int64_t>(doc.k0) + j0, kC, keys, hk * p.d, p.d);
    load_async<D>(skv + (2 * stage + 1) * kTile, p.v, p.v_stride, static_cast<int64_t>(doc.k0) + j0, kC, keys, hk * p.d, p.d);
    async_commit();
  };
  load_async<D>(sq, p.q, p.q_stride, doc.q0 + i0, kR, rows, h * p.d, p.d);
  if (most > 0) load(0, 0);
  int seen[2];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float4 o[2][D / 64] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    seen[i] = 2 * ty + i < rows ? seen_keys(i0 + 2 * ty + i, doc.off, doc.Lk, doc.prefix, p.causal_block) : 0;
  for (int j0 = 0, st = 0; j0 < most; j0 += kC, st ^= 1) {
    async_wait_groups();
    __syncthreads();  // this tile is there; the other stage has been read
    if (j0 + kC < most) load(j0 + kC, st ^ 1);
    float s[2][2];
    dot_2x2<D>(sq, skv + 2 * st * kTile, s);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float turn, mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int key = j0 + tx + 16 * j;
        s[i][j] = key < seen[i] ? score(s[i][j], p, slope, i0 + 2 * ty + i + doc.off, key, turn) : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      const float m_new = fmaxf(m[i], max16(mx));
      const float base = m_new == -INFINITY ? 0.f : m_new;  // a row that has seen nothing yet
      const float alpha = expf(m[i] - base);
      const float e0 = expf(s[i][0] - base), e1 = expf(s[i][1] - base);
      sp[(2 * ty + i) * kSp + tx] = e0;
      sp[(2 * ty + i) * kSp + tx + 16] = e1;
      l[i] = l[i] * alpha + sum16(e0 + e1);
      m[i] = m_new;
#pragma unroll
      for (int k = 0; k < D / 64; ++k) o[i][k].x *= alpha, o[i][k].y *= alpha, o[i][k].z *= alpha, o[i][k].w *= alpha;
    }
    __syncwarp();  // two rows of sp belong to one half-warp
    add_product<D>(sp, skv + (2 * st + 1) * kTile, o);
  }
  async_wait_all();
  float inv[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    inv[i] = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);  // NaN passes
    if (p.lse && tx == 0 && 2 * ty + i < rows)
      p.lse[static_cast<int64_t>(h) * p.q_rows + doc.q0 + i0 + 2 * ty + i] = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
  }
  store_rows<D>(p.o, p.o_stride, static_cast<int64_t>(doc.q0) + i0, rows, h * p.d, p.d, o, inv);
}

// dq, and delta of the block's rows for the other kernel.
template <int D>
__global__ void __launch_bounds__(kThreads) packed_dq_kernel(const PackedAttn p) {
  extern __shared__ float4 smem4[];
  float* sm = reinterpret_cast<float*>(smem4);
  constexpr int kTile = kC * (D + 4);
  float *sq = sm, *so = sq + kR * (D + 4), *skv = so + kR * (D + 4), *sp = skv + 4 * kTile;
  int d, tile;
  if (!block_tile(p.cu_q, p.n_docs, p.q_rows, d, tile)) return;
  const Doc doc = load_doc(p, d);
  const int h = blockIdx.y, hk = h / (p.H / p.Hk);
  const int i0 = tile * kR, rows = min(kR, doc.Lq - i0);
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int most = seen_keys(i0 + rows - 1, doc.off, doc.Lk, doc.prefix, p.causal_block);
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  auto load = [&](int j0, int stage) {
    const int keys = min(kC, doc.Lk - j0);
    load_async<D>(skv + 2 * stage * kTile, p.k, p.k_stride, static_cast<int64_t>(doc.k0) + j0, kC, keys, hk * p.d, p.d);
    load_async<D>(skv + (2 * stage + 1) * kTile, p.v, p.v_stride, static_cast<int64_t>(doc.k0) + j0, kC, keys, hk * p.d, p.d);
    async_commit();
  };
  load_async<D>(sq, p.q, p.q_stride, doc.q0 + i0, kR, rows, h * p.d, p.d);
  load_async<D>(so, p.d_o, p.do_stride, doc.q0 + i0, kR, rows, h * p.d, p.d);
  if (most > 0) load(0, 0);
  int seen[2];
  float lse[2], delta[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * ty + i;
    float x = 0.f;
    seen[i] = 0, lse[i] = 0.f;
    if (r < rows) {
      const int64_t row = static_cast<int64_t>(doc.q0) + i0 + r;
      seen[i] = seen_keys(i0 + r, doc.off, doc.Lk, doc.prefix, p.causal_block);
      if (seen[i] > 0) lse[i] = p.lse[static_cast<int64_t>(h) * p.q_rows + row];
      for (int c = 4 * tx; c < p.d; c += 64) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p.o) + row * p.o_stride + h * p.d + c);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p.d_o) + row * p.do_stride + h * p.d + c);
        x = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, x))));
      }
    }
    delta[i] = sum16(x);
    if (r < rows && tx == 0) p.delta[static_cast<int64_t>(h) * p.q_rows + doc.q0 + i0 + r] = delta[i];
  }
  float4 g[2][D / 64] = {};
  for (int j0 = 0, st = 0; j0 < most; j0 += kC, st ^= 1) {
    async_wait_groups();
    __syncthreads();
    if (j0 + kC < most) load(j0 + kC, st ^ 1);
    float s[2][2], dp[2][2];
    dot_2x2<D>(sq, skv + 2 * st * kTile, s);
    dot_2x2<D>(so, skv + (2 * st + 1) * kTile, dp);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int key = j0 + tx + 16 * j;
        float ds = 0.f;
        if (key < seen[i]) {
          float turn;
          const float z = score(s[i][j], p, slope, i0 + 2 * ty + i + doc.off, key, turn);
          ds = expf(z - lse[i]) * (dp[i][j] - delta[i]) * turn;
        }
        sp[(2 * ty + i) * kSp + tx + 16 * j] = ds;
      }
    __syncwarp();
    add_product<D>(sp, skv + 2 * st * kTile, g);
  }
  async_wait_all();
  const float f[2] = {p.scale, p.scale};
  store_rows<D>(p.dq, p.dq_stride, static_cast<int64_t>(doc.q0) + i0, rows, h * p.d, p.d, g, f);
}

template <int D>
__global__ void __launch_bounds__(kThreads) packed_dkv_kernel(const PackedAttn p) {
  extern __shared__ float4 smem4[];
  float* sm = reinterpret_cast<float*>(smem4);
  constexpr int kTile = kC * (D + 4);
  float *sk = sm, *sv = sk + kR * (D + 4), *sqo = sv + kR * (D + 4), *sp = sqo + 4 * kTile, *ss = sp + kR * kSp;
  int d, tile;
  if (!block_tile(p.cu_k, p.n_docs, p.k_rows, d, tile)) return;
  const Doc doc = load_doc(p, d);
  const int hk = blockIdx.y, group = p.H / p.Hk;
  const int j0 = tile * kR, keys = min(kR, doc.Lk - j0);
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int first = first_query(j0, doc.off, doc.Lk, doc.prefix, p.causal_block);
  const int per_head = first < doc.Lq ? (doc.Lq - first + kC - 1) / kC : 0, n = per_head * group;
  auto load = [&](int t, int stage) {
    const int h = hk * group + t / per_head, i0 = first + t % per_head * kC, rows = min(kC, doc.Lq - i0);
    load_async<D>(sqo + 2 * stage * kTile, p.q, p.q_stride, static_cast<int64_t>(doc.q0) + i0, kC, rows, h * p.d, p.d);
    load_async<D>(sqo + (2 * stage + 1) * kTile, p.d_o, p.do_stride, static_cast<int64_t>(doc.q0) + i0, kC, rows, h * p.d, p.d);
    async_commit();
  };
  load_async<D>(sk, p.k, p.k_stride, static_cast<int64_t>(doc.k0) + j0, kR, keys, hk * p.d, p.d);
  load_async<D>(sv, p.v, p.v_stride, static_cast<int64_t>(doc.k0) + j0, kR, keys, hk * p.d, p.d);
  if (n > 0) load(0, 0);
  float4 gk[2][D / 64] = {}, gv[2][D / 64] = {};
  for (int t = 0, st = 0; t < n; ++t, st ^= 1) {
    const int h = hk * group + t / per_head, i0 = first + t % per_head * kC;
    const float slope = p.slopes ? p.slopes[h] : 0.f;
    float lse[2], delta[2];
    int seen[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i = i0 + tx + 16 * x;
      seen[x] = 0, lse[x] = delta[x] = 0.f;
      if (i < doc.Lq) {
        const int64_t stat = static_cast<int64_t>(h) * p.q_rows + doc.q0 + i;
        seen[x] = seen_keys(i, doc.off, doc.Lk, doc.prefix, p.causal_block);
        lse[x] = p.lse[stat], delta[x] = p.delta[stat];
      }
    }
    async_wait_groups();
    __syncthreads();
    if (t + 1 < n) load(t + 1, st ^ 1);
    float s[2][2], dp[2][2];
    dot_2x2<D>(sk, sqo + 2 * st * kTile, s);
    dot_2x2<D>(sv, sqo + (2 * st + 1) * kTile, dp);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int key = j0 + 2 * ty + i;
        float pr = 0.f, ds = 0.f;
        if (2 * ty + i < keys && key < seen[x]) {
          float turn;
          const float z = score(s[i][x], p, slope, i0 + tx + 16 * x + doc.off, key, turn);
          pr = expf(z - lse[x]);
          ds = pr * (dp[i][x] - delta[x]) * turn;
        }
        sp[(2 * ty + i) * kSp + tx + 16 * x] = pr;
        ss[(2 * ty + i) * kSp + tx + 16 * x] = ds;
      }
    __syncwarp();
    add_product<D>(sp, sqo + (2 * st + 1) * kTile, gv);
    add_product<D>(ss, sqo + 2 * st * kTile, gk);
  }
  async_wait_all();
  const float one[2] = {1.f, 1.f}, f[2] = {p.scale, p.scale};
  store_rows<D>(p.dk, p.dk_stride, static_cast<int64_t>(doc.k0) + j0, keys, hk * p.d, p.d, gk, f);
  store_rows<D>(p.dv, p.dv_stride, static_cast<int64_t>(doc.k0) + j0, keys, hk * p.d, p.d, gv, one);
}

// delta[h, row] = sum(do * o) of bf16 rows of 128 dims (for the tensor-core gradient): 16 lanes
// a (row, head), four of them at a time.
__global__ void __launch_bounds__(256) packed_delta_kernel(const PackedAttn p) {
  const int lane = threadIdx.x & 15;
  const int64_t all = static_cast<int64_t>(p.q_rows) * p.H, first = (static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4)) * 4;
  uint4 x[4], y[4];
  int64_t row[4];
  int h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t w = first + i < all ? first + i : all - 1;
    row[i] = w / p.H, h[i] = static_cast<int>(w - row[i] * p.H);
    x[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.d_o) + row[i] * p.do_stride + h[i] * 128) + lane);
    y[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.o) + row[i] * p.o_stride + h[i] * 128) + lane);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a[8], b[8], s = 0.f;
    Raw8<__nv_bfloat16> r;
    r.u = x[i];
    unpack8(r, a);
    r.u = y[i];
    unpack8(r, b);
#pragma unroll
    for (int c = 0; c < 8; ++c) s = fmaf(a[c], b[c], s);
    s = sum16(s);
    if (lane == 0 && first + i < all) p.delta[static_cast<int64_t>(h[i]) * p.q_rows + row[i]] = s;
  }
}

// At most this many tiles: every document adds less than one partial tile.
unsigned most_tiles(int rows, int n_docs) { return static_cast<unsigned>(rows / kR) + static_cast<unsigned>(n_docs); }

// Shared memory of a block: `own` tiles of its rows, two stages of two tiles, `squares` of
// probabilities.
template <int D>
constexpr size_t smem_bytes(int own, int squares) {
  return (static_cast<size_t>(own * kR + 4 * kC) * (D + 4) + static_cast<size_t>(squares) * kR * kSp) * sizeof(float);
}
template <typename K>
int launch(K kernel, size_t smem, dim3 grid, const PackedAttn& p, cudaStream_t s) {
  if (smem > 48 * 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  kernel<<<grid, kThreads, smem, s>>>(p);
  return check_launch();
}
template <int D>
int fwd(const PackedAttn& p, cudaStream_t s) {
  return launch(packed_fwd_kernel<D>, smem_bytes<D>(1, 1), dim3(most_tiles(p.q_rows, p.n_docs), p.H), p, s);
}
template <int D>
int bwd(const PackedAttn& p, cudaStream_t s) {
  int st = WAN_OK, launched = 0;
  if (p.q_rows > 0) {
    st = launch(packed_dq_kernel<D>, smem_bytes<D>(2, 1), dim3(most_tiles(p.q_rows, p.n_docs), p.H), p, s);
    ++launched;
  }
  if (st == WAN_OK && p.k_rows > 0) {
    st = launch(packed_dkv_kernel<D>, smem_bytes<D>(2, 2), dim3(most_tiles(p.k_rows, p.n_docs), p.Hk), p, s);
    ++launched;
  }
  count_launches(launched - 1);
  return st;
}
int delta(const PackedAttn& p, cudaStream_t s) {
  if (p.q_rows == 0) {
    count_launches(-1);
    return WAN_OK;
  }
  const int64_t all = static_cast<int64_t>(p.q_rows) * p.H;
  packed_delta_kernel<<<static_cast<unsigned>((all + 63) / 64), 256, 0, s>>>(p);
  return check_launch();
}

}  // namespace

int launch_attn_packed_simt(const PackedAttn& p, cudaStream_t s) {
  trace_launch_begin(WAN_KIND_ATTN, s);
  const int st = p.d <= 64 ? fwd<64>(p, s) : fwd<128>(p, s);
  trace_launch_end(WAN_KIND_ATTN, s);
  return st;
}

int launch_attn_packed_bwd(const PackedAttn& p, int dtype, cudaStream_t s) {
  trace_launch_begin(WAN_KIND_ATTN, s);
  int st = WAN_OK;
  if (dtype == WAN_BF16) {
    st = delta(p, s);
    if (st == WAN_OK) st = launch_attn_packed_tc_bwd(p, s);
  } else {
    st = p.d <= 64 ? bwd<64>(p, s) : bwd<128>(p, s);
  }
  trace_launch_end(WAN_KIND_ATTN, s);
  return st;
}

}  // namespace wan
