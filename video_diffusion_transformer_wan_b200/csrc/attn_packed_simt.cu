// Attention inside packed documents on the CUDA cores, with full fp32 arithmetic, and its
// gradient: one pass over the keys with a running maximum and sum; the gradient recomputes
// the probabilities from the stored log-sums, p = e^(s - lse), ds = p (dp - delta) with
// delta = sum(do * o), in one kernel per side (dq over the keys, dk and dv over the
// queries), so that nothing is added across blocks.
//
// A block takes 32 rows of one document and head; eight lanes hold a row (a quarter of a
// 32-wide tile of scores and an eighth of the head each), so row maxima and sums stay
// inside a warp. Bound by shared-memory reads (two per multiply-add).
#include <math.h>

#include "internal.h"
#include "packed.cuh"

namespace wan {
namespace {

constexpr int kR = 32;         // rows and columns of a tile
constexpr int kThreads = 256;  // eight lanes a row
constexpr int kMaxD = 128;

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

template <typename T>
__device__ __forceinline__ void load_tile(float* dst, const void* src, int64_t stride, int64_t row0, int valid, int col0,
                                          int d) {
  for (int i = threadIdx.x; i < kR * d; i += kThreads) {
    const int r = i / d, c = i - r * d;
    dst[r * (d + 1) + c] = r < valid ? to_f32<T>(static_cast<const T*>(src)[(row0 + r) * stride + col0 + c]) : 0.f;
  }
}

__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, 8);
  return v;
}
__device__ __forceinline__ float max8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o, 8));
  return v;
}
__device__ __forceinline__ float dot_rows(const float* a, const float* b, int d) {
  float s = 0.f;
  for (int c = 0; c < d; ++c) s = fmaf(a[c], b[c], s);
  return s;
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

template <typename T>
__global__ void __launch_bounds__(kThreads) packed_fwd_kernel(const PackedAttn p) {
  extern __shared__ float sm[];
  const int ld = p.d + 1;
  float *sq = sm, *sk = sq + kR * ld, *sv = sk + kR * ld, *sp = sv + kR * ld;  // sp [kR][kR + 1]
  int d, tile;
  if (!block_tile(p.cu_q, p.n_docs, p.q_rows, d, tile)) return;
  const Doc doc = load_doc(p, d);
  const int h = blockIdx.y, hk = h / (p.H / p.Hk);
  const int i0 = tile * kR, rows = min(kR, doc.Lq - i0);
  const int r = threadIdx.x >> 3, c = threadIdx.x & 7, i = i0 + r;
  const int seen = r < rows ? seen_keys(i, doc.off, doc.Lk, doc.prefix, p.causal_block) : 0;
  const int most = seen_keys(i0 + rows - 1, doc.off, doc.Lk, doc.prefix, p.causal_block);
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  load_tile<T>(sq, p.q, p.q_stride, doc.q0 + i0, rows, h * p.d, p.d);
  float m = -INFINITY, l = 0.f, o[kMaxD / 8] = {};
  for (int j0 = 0; j0 < most; j0 += kR) {
    __syncthreads();
    const int keys = min(kR, doc.Lk - j0);
    load_tile<T>(sk, p.k, p.k_stride, static_cast<int64_t>(doc.k0) + j0, keys, hk * p.d, p.d);
    load_tile<T>(sv, p.v, p.v_stride, static_cast<int64_t>(doc.k0) + j0, keys, hk * p.d, p.d);
    __syncthreads();
    float s[4], mx = -INFINITY, turn;
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const int j = c + 8 * jj;
      s[jj] = j0 + j < seen ? score(dot_rows(sq + r * ld, sk + j * ld, p.d), p, slope, i + doc.off, j0 + j, turn) : -INFINITY;
      mx = fmaxf(mx, s[jj]);
    }
    const float m_new = fmaxf(m, max8(mx));
    const float base = m_new == -INFINITY ? 0.f : m_new;  // a row that has seen nothing yet
    const float alpha = expf(m - base);
    float sum = 0.f;
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const float e = expf(s[jj] - base);
      sp[r * (kR + 1) + c + 8 * jj] = e;
      sum += e;
    }
    l = l * alpha + sum8(sum);
    m = m_new;
    __syncwarp();
#pragma unroll
    for (int x = 0; x < kMaxD / 8; ++x)
      if (c + 8 * x < p.d) {
        float a = o[x] * alpha;
        for (int j = 0; j < keys; ++j) a = fmaf(sp[r * (kR + 1) + j], sv[j * ld + c + 8 * x], a);
        o[x] = a;
      }
    __syncwarp();
  }
  if (r >= rows) return;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN passes
  T* out = static_cast<T*>(p.o) + static_cast<int64_t>(doc.q0 + i) * p.o_stride + h * p.d;
#pragma unroll
  for (int x = 0; x < kMaxD / 8; ++x)
    if (c + 8 * x < p.d) out[c + 8 * x] = from_f32<T>(o[x] * inv);
  if (p.lse && c == 0) p.lse[static_cast<int64_t>(h) * p.q_rows + doc.q0 + i] = l == 0.f ? -INFINITY : m + logf(l);
}

// delta[h, row] = sum(do * o), one warp per (row, head).
template <typename T>
__global__ void __launch_bounds__(256) packed_delta_kernel(const PackedAttn p) {
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t row = w / p.H;
  const int h = static_cast<int>(w - row * p.H);
  if (row >= p.q_rows) return;
  const T* a = static_cast<const T*>(p.d_o) + row * p.do_stride + h * p.d;
  const T* b = static_cast<const T*>(p.o) + row * p.o_stride + h * p.d;
  float s = 0.f;
  for (int c = lane; c < p.d; c += 32) s = fmaf(to_f32<T>(a[c]), to_f32<T>(b[c]), s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) p.delta[static_cast<int64_t>(h) * p.q_rows + row] = s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) packed_dq_kernel(const PackedAttn p) {
  extern __shared__ float sm[];
  const int ld = p.d + 1;
  float *sq = sm, *so = sq + kR * ld, *sk = so + kR * ld, *sv = sk + kR * ld, *sp = sv + kR * ld;
  int d, tile;
  if (!block_tile(p.cu_q, p.n_docs, p.q_rows, d, tile)) return;
  const Doc doc = load_doc(p, d);
  const int h = blockIdx.y, hk = h / (p.H / p.Hk);
  const int i0 = tile * kR, rows = min(kR, doc.Lq - i0);
  const int r = threadIdx.x >> 3, c = threadIdx.x & 7, i = i0 + r;
  const int seen = r < rows ? seen_keys(i, doc.off, doc.Lk, doc.prefix, p.causal_block) : 0;
  const int most = seen_keys(i0 + rows - 1, doc.off, doc.Lk, doc.prefix, p.causal_block);
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  load_tile<T>(sq, p.q, p.q_stride, doc.q0 + i0, rows, h * p.d, p.d);
  load_tile<T>(so, p.d_o, p.do_stride, doc.q0 + i0, rows, h * p.d, p.d);
  const int64_t stat = static_cast<int64_t>(h) * p.q_rows + doc.q0 + i;
  const float lse = seen > 0 ? p.lse[stat] : 0.f, delta = seen > 0 ? p.delta[stat] : 0.f;
  float g[kMaxD / 8] = {};
  for (int j0 = 0; j0 < most; j0 += kR) {
    __syncthreads();
    const int keys = min(kR, doc.Lk - j0);
    load_tile<T>(sk, p.k, p.k_stride, static_cast<int64_t>(doc.k0) + j0, keys, hk * p.d, p.d);
    load_tile<T>(sv, p.v, p.v_stride, static_cast<int64_t>(doc.k0) + j0, keys, hk * p.d, p.d);
    __syncthreads();
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const int j = c + 8 * jj;
      float ds = 0.f;
      if (j0 + j < seen) {
        float turn;
        const float s = score(dot_rows(sq + r * ld, sk + j * ld, p.d), p, slope, i + doc.off, j0 + j, turn);
        ds = expf(s - lse) * (dot_rows(so + r * ld, sv + j * ld, p.d) - delta) * turn * p.scale;
      }
      sp[r * (kR + 1) + j] = ds;
    }
    __syncwarp();
#pragma unroll
    for (int x = 0; x < kMaxD / 8; ++x)
      if (c + 8 * x < p.d)
        for (int j = 0; j < keys; ++j) g[x] = fmaf(sp[r * (kR + 1) + j], sk[j * ld + c + 8 * x], g[x]);
    __syncwarp();
  }
  if (r >= rows) return;
  T* out = static_cast<T*>(p.dq) + static_cast<int64_t>(doc.q0 + i) * p.dq_stride + h * p.d;
#pragma unroll
  for (int x = 0; x < kMaxD / 8; ++x)
    if (c + 8 * x < p.d) out[c + 8 * x] = from_f32<T>(g[x]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) packed_dkv_kernel(const PackedAttn p) {
  extern __shared__ float sm[];
  const int ld = p.d + 1;
  float *sk = sm, *sv = sk + kR * ld, *sq = sv + kR * ld, *so = sq + kR * ld, *sp = so + kR * ld, *ss = sp + kR * (kR + 1);
  int d, tile;
  if (!block_tile(p.cu_k, p.n_docs, p.k_rows, d, tile)) return;
  const Doc doc = load_doc(p, d);
  const int hk = blockIdx.y, group = p.H / p.Hk;
  const int j0 = tile * kR, keys = min(kR, doc.Lk - j0);
  const int r = threadIdx.x >> 3, c = threadIdx.x & 7, j = j0 + r;
  load_tile<T>(sk, p.k, p.k_stride, static_cast<int64_t>(doc.k0) + j0, keys, hk * p.d, p.d);
  load_tile<T>(sv, p.v, p.v_stride, static_cast<int64_t>(doc.k0) + j0, keys, hk * p.d, p.d);
  const int first = first_query(j0, doc.off, doc.Lk, doc.prefix, p.causal_block);
  float gk[kMaxD / 8] = {}, gv[kMaxD / 8] = {};
  for (int h = hk * group; h < (hk + 1) * group; ++h) {
    const float slope = p.slopes ? p.slopes[h] : 0.f;
    for (int i0 = first; i0 < doc.Lq; i0 += kR) {
      __syncthreads();
      const int rows = min(kR, doc.Lq - i0);
      load_tile<T>(sq, p.q, p.q_stride, static_cast<int64_t>(doc.q0) + i0, rows, h * p.d, p.d);
      load_tile<T>(so, p.d_o, p.do_stride, static_cast<int64_t>(doc.q0) + i0, rows, h * p.d, p.d);
      __syncthreads();
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const int x = c + 8 * ii, i = i0 + x;
        float pr = 0.f, ds = 0.f;
        if (x < rows && r < keys && j < seen_keys(i, doc.off, doc.Lk, doc.prefix, p.causal_block)) {
          const int64_t stat = static_cast<int64_t>(h) * p.q_rows + doc.q0 + i;
          float turn;
          const float s = score(dot_rows(sk + r * ld, sq + x * ld, p.d), p, slope, i + doc.off, j, turn);
          pr = expf(s - p.lse[stat]);
          ds = pr * (dot_rows(sv + r * ld, so + x * ld, p.d) - p.delta[stat]) * turn * p.scale;
        }
        sp[r * (kR + 1) + x] = pr;
        ss[r * (kR + 1) + x] = ds;
      }
      __syncwarp();
#pragma unroll
      for (int x = 0; x < kMaxD / 8; ++x)
        if (c + 8 * x < p.d)
          for (int y = 0; y < rows; ++y) {
            gv[x] = fmaf(sp[r * (kR + 1) + y], so[y * ld + c + 8 * x], gv[x]);
            gk[x] = fmaf(ss[r * (kR + 1) + y], sq[y * ld + c + 8 * x], gk[x]);
          }
      __syncwarp();
    }
  }
  if (r >= keys) return;
  T* ok = static_cast<T*>(p.dk) + static_cast<int64_t>(doc.k0 + j) * p.dk_stride + hk * p.d;
  T* ov = static_cast<T*>(p.dv) + static_cast<int64_t>(doc.k0 + j) * p.dv_stride + hk * p.d;
#pragma unroll
  for (int x = 0; x < kMaxD / 8; ++x)
    if (c + 8 * x < p.d) {
      ok[c + 8 * x] = from_f32<T>(gk[x]);
      ov[c + 8 * x] = from_f32<T>(gv[x]);
    }
}

size_t tile_bytes(int d, int tiles, int squares) {
  return (static_cast<size_t>(tiles) * kR * (d + 1) + static_cast<size_t>(squares) * kR * (kR + 1)) * sizeof(float);
}

// At most this many tiles: every document adds less than one partial tile.
unsigned most_tiles(int rows, int n_docs) { return static_cast<unsigned>(rows / kR) + static_cast<unsigned>(n_docs); }

template <typename K>
void allow_smem(K kernel, size_t bytes) {
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

template <typename T>
int fwd(const PackedAttn& p, cudaStream_t s) {
  const size_t sm = tile_bytes(p.d, 3, 1);
  allow_smem(packed_fwd_kernel<T>, sm);
  packed_fwd_kernel<T><<<dim3(most_tiles(p.q_rows, p.n_docs), p.H), kThreads, sm, s>>>(p);
  return check_launch();
}
template <typename T>
int delta(const PackedAttn& p, cudaStream_t s) {
  if (p.q_rows == 0) {
    count_launches(-1);
    return WAN_OK;
  }
  const int64_t warps = static_cast<int64_t>(p.q_rows) * p.H;
  packed_delta_kernel<T><<<static_cast<unsigned>((warps + 7) / 8), 256, 0, s>>>(p);
  return check_launch();
}
template <typename T>
int bwd(const PackedAttn& p, cudaStream_t s) {
  int st = WAN_OK;
  if (p.q_rows > 0) {
    const size_t sm = tile_bytes(p.d, 4, 1);
    allow_smem(packed_dq_kernel<T>, sm);
    packed_dq_kernel<T><<<dim3(most_tiles(p.q_rows, p.n_docs), p.H), kThreads, sm, s>>>(p);
    count_launches(1);
    st = check_launch();
  }
  if (st == WAN_OK && p.k_rows > 0) {
    const size_t sm = tile_bytes(p.d, 4, 2);
    allow_smem(packed_dkv_kernel<T>, sm);
    packed_dkv_kernel<T><<<dim3(most_tiles(p.k_rows, p.n_docs), p.Hk), kThreads, sm, s>>>(p);
    count_launches(1);
    st = check_launch();
  }
  return st;
}

}  // namespace

int launch_attn_packed_simt(const PackedAttn& p, cudaStream_t s) {
  trace_launch_begin(WAN_KIND_ATTN, s);
  const int st = fwd<float>(p, s);
  trace_launch_end(WAN_KIND_ATTN, s);
  return st;
}

int launch_attn_packed_bwd(const PackedAttn& p, int dtype, cudaStream_t s) {
  trace_launch_begin(WAN_KIND_ATTN, s);
  int st = dtype == WAN_BF16 ? delta<__nv_bfloat16>(p, s) : delta<float>(p, s);
  if (st == WAN_OK) st = dtype == WAN_BF16 ? launch_attn_packed_tc_bwd(p, s) : bwd<float>(p, s);
  trace_launch_end(WAN_KIND_ATTN, s);
  return st;
}

}  // namespace wan
