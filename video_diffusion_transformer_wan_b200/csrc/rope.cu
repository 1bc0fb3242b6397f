// Rotary positions with the q/k norm, and their gradient (wan_qk_norm_rope_*).
//
// Per head of a row: x -> x r w (r = 1/sqrt(mean(x^2) + eps) over the head or the whole
// width, or no norm), then every pair (a, b) of the rotated part turns by its angle:
// (a c - b s, a s + b c). The gradient turns back, g = R^T dout, and with m = mean(g w x)
// gives dx = r (g w - x r^2 m) and dw = sum over rows of g x r.
//
// HBM-bound: the forward reads and writes every element once, the gradient reads two and
// writes one; what has to be kept down is the instructions per element and what warps wait
// for. A warp of qk_norm_rope_kernel takes a row of q or of k by itself, a lane 8 columns (four
// whole pairs: 8 neighbours, or 4 of each half) of every 256, the same place in every head: its
// cosines serve all heads, sums are shuffles, and no warp waits for another. (Blocks that
// shared a row, a thread for the same columns of every row, spent 4 times the instructions on
// exchanges and waited at barriers: 108 us against 75 us forward, 179 against 154 us gradient, on
// 32,760 and 27,569 rows of 12 + 12 heads.) The cosines of a row are made once per pair, the
// turns reduced in fp64 (positions may be far) and the sine taken in fp32. Up to 6 x 256 columns
// of a side (forward: 20 x 256) stay in registers between the norm's sums and their use; wider
// rows are read twice, the second time from the caches.
// qk_norm_rope_any_kernel serves what this layout does not divide: rows that are not 16-byte
// aligned, heads that do not divide 256 dims or are below 8, halves of odd quads (on the rows
// above it takes 332 us forward and 1553 us for the gradient).
#include <cuda_bf16.h>

#include <math.h>

#include "checks.h"
#include "internal.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace wan {
namespace {

constexpr int kMaxPairs = 64;   // head_dim <= 128
constexpr int kMaxTb = 16;      // rows a block holds at once
constexpr int kDwBlocks = 296;  // blocks of the gradient with a norm: 2 per SM, each leaves one partial sum

struct RopeParams {
  const void *q_in, *k_in, *w_q, *w_k;  // q_in, k_in: the (gradient's) normed inputs
  void *q_out, *k_out;
  const void *gq, *gk;  // gradient: dq_out, dk_out
  int64_t q_stride, k_stride, qo_stride, ko_stride, gq_stride, gk_stride;
  float* part;          // gradient: the blocks' partial rows of the weights' gradients
  const int32_t* pos;
  int rows, H, n, d, tb, norm, layout, pairs, n_axes;  // n = heads of q and k together
  float eps, amplitude;
  double freq[kMaxPairs];  // turns per position: frequency / 2 pi
  uint8_t axis[kMaxPairs];
};

// A lane's pairs u, u + 16, ..., element by element.
struct Lane {
  int u, d, n_pairs;
  bool half;
  __device__ Lane(const RopeParams& p, int lane)
      : u(lane), d(p.d), n_pairs(p.pairs), half(p.layout == WAN_ROPE_HALF) {}
  __device__ __forceinline__ bool on(int k) const { return 2 * (u + 16 * k) < d; }
  __device__ __forceinline__ int pair(int k) const { return u + 16 * k; }
  __device__ __forceinline__ int first(int k) const {
    const int m = u + 16 * k;
    return half && m < n_pairs ? m : 2 * m;
  }
  __device__ __forceinline__ int second(int k) const {
    const int m = u + 16 * k;
    return half && m < n_pairs ? m + n_pairs : 2 * m + 1;
  }
  __device__ __forceinline__ void load(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* x) const {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = on(k) ? static_cast<uint32_t>(__bfloat16_as_ushort(x[first(k)])) |
                         (static_cast<uint32_t>(__bfloat16_as_ushort(x[second(k)])) << 16)
                   : 0u;
    r.u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void load(Raw8<float>& r, const float* x) const {
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[2 * k] = on(k) ? x[first(k)] : 0.f, v[2 * k + 1] = on(k) ? x[second(k)] : 0.f;
    r.a = make_float4(v[0], v[1], v[2], v[3]);
    r.b = make_float4(v[4], v[5], v[6], v[7]);
  }
  template <typename T>
  __device__ __forceinline__ void pairs_of(const Raw8<T>& r, float (&a)[4], float (&b)[4]) const {
    float v[8];
    unpack8(r, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = v[2 * k], b[k] = v[2 * k + 1];
  }
  template <typename T>
  __device__ __forceinline__ void store(T* x, const float (&a)[4], const float (&b)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (on(k)) x[first(k)] = from_f32<T>(a[k]), x[second(k)] = from_f32<T>(b[k]);
  }
};

__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, 16);
  return v;
}

// amplitude (cos, sin) of the angle of position * freq turns.
__device__ __forceinline__ float2 turn(int pos, double freq, float amplitude) {
  const double turns = static_cast<double>(pos) * freq;
  float s, c;
  sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
  return make_float2(c * amplitude, s * amplitude);
}

template <typename T, int NI, bool kBwd>
__global__ void __launch_bounds__(256) qk_norm_rope_any_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kHw = 16;  // half-warps per block
  __shared__ float2 cs[kMaxTb][kMaxPairs + 1];  // the last entry: no turn (1, 0)
  __shared__ float red[kBwd ? 2 : 1][kHw * NI];
  const int hw = threadIdx.x >> 4, u = threadIdx.x & 15;
  const Lane lane(p, u);
  const int items = p.tb * p.n;
  if (threadIdx.x < kMaxTb) cs[threadIdx.x][kMaxPairs] = make_float2(1.f, 0.f);
  float dw[kBwd ? NI : 1][8] = {};

  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.tb; row0 < p.rows; row0 += static_cast<int64_t>(gridDim.x) * p.tb) {
    Raw8<T> rx[NI], rg[kBwd ? NI : 1];
    int head[NI], tok[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int item = i * kHw + hw;
      tok[i] = item / p.n;
      head[i] = item - tok[i] * p.n;
      const int64_t row = row0 + tok[i];
      if (item >= items || row >= p.rows) tok[i] = -1;
      if (tok[i] >= 0) {
        const bool is_q = head[i] < p.H;
        const int h = is_q ? head[i] : head[i] - p.H;
        if (!kBwd || p.norm != WAN_QK_NORM_NONE)
          lane.load(rx[i], static_cast<const T*>(is_q ? p.q_in : p.k_in) + row * (is_q ? p.q_stride : p.k_stride) + h * p.d);
        if constexpr (kBwd)
          lane.load(rg[i], static_cast<const T*>(is_q ? p.gq : p.gk) + row * (is_q ? p.gq_stride : p.gk_stride) + h * p.d);
      }
    }
    // Cosines of this block's rows, while the loads fly.
    for (int w = threadIdx.x; w < p.tb * p.pairs; w += 256) {
      const int t = w / p.pairs, j = w - t * p.pairs;
      if (row0 + t < p.rows) {
        cs[t][j] = turn(p.pos[(row0 + t) * p.n_axes + p.axis[j]], p.freq[j], p.amplitude);
      }
    }
    __syncthreads();
    float inv[NI], mean_gx[kBwd ? NI : 1];
    if (p.norm != WAN_QK_NORM_NONE) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float s = 0.f, m = 0.f;
        if (tok[i] >= 0) {
          float a[4], b[4];
          lane.pairs_of(rx[i], a, b);
#pragma unroll
          for (int k = 0; k < 4; ++k) s += a[k] * a[k] + b[k] * b[k];
          if constexpr (kBwd) {
            const bool is_q = head[i] < p.H;
            const int h = is_q ? head[i] : head[i] - p.H;
            Raw8<T> rw;
            lane.load(rw, static_cast<const T*>(is_q ? p.w_q : p.w_k) + (p.norm == WAN_QK_NORM_WIDTH ? h * p.d : 0));
            float ga[4], gb[4], wa[4], wb[4];
            lane.pairs_of(rg[i], ga, gb);
            lane.pairs_of(rw, wa, wb);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 c = cs[tok[i]][lane.pair(k) < p.pairs ? lane.pair(k) : kMaxPairs];
              m += (ga[k] * c.x + gb[k] * c.y) * wa[k] * a[k] + (gb[k] * c.x - ga[k] * c.y) * wb[k] * b[k];
            }
          }
        }
        s = sum16(s);
        if constexpr (kBwd) m = sum16(m);
        if (p.norm == WAN_QK_NORM_HEAD) {
          inv[i] = 1.0f / sqrtf(s / p.d + p.eps);
          if constexpr (kBwd) mean_gx[i] = m / p.d;
        } else if (u == 0) {
          red[0][i * kHw + hw] = s;
          if constexpr (kBwd) red[1][i * kHw + hw] = m;
        }
      }
      if (p.norm == WAN_QK_NORM_WIDTH) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const bool is_q = head[i] < p.H;
          const int first = tok[i] < 0 ? 0 : tok[i] * p.n + (is_q ? 0 : p.H);
          const int count = tok[i] < 0 ? 0 : (is_q ? p.H : p.n - p.H);
          float s = 0.f, m = 0.f;
          for (int h = u; h < count; h += 16) {
            s += red[0][first + h];
            if constexpr (kBwd) m += red[1][first + h];
          }
          const float width = static_cast<float>(max(count, 1) * p.d);
          inv[i] = 1.0f / sqrtf(sum16(s) / width + p.eps);
          if constexpr (kBwd) mean_gx[i] = sum16(m) / width;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (tok[i] < 0) continue;
      const bool is_q = head[i] < p.H;
      const int h = is_q ? head[i] : head[i] - p.H;
      float a[4], b[4], wa[4], wb[4];
      if (p.norm != WAN_QK_NORM_NONE) {
        Raw8<T> rw;
        lane.load(rw, static_cast<const T*>(is_q ? p.w_q : p.w_k) + (p.norm == WAN_QK_NORM_WIDTH ? h * p.d : 0));
        lane.pairs_of(rw, wa, wb);
      }
      if (!kBwd || p.norm != WAN_QK_NORM_NONE) lane.pairs_of(rx[i], a, b);
      float oa[4], ob[4];
      if constexpr (!kBwd) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 c = cs[tok[i]][lane.pair(k) < p.pairs ? lane.pair(k) : kMaxPairs];
          if (p.norm != WAN_QK_NORM_NONE) a[k] *= inv[i] * wa[k], b[k] *= inv[i] * wb[k];
          oa[k] = a[k] * c.x - b[k] * c.y;
          ob[k] = a[k] * c.y + b[k] * c.x;
        }
      } else {
        float ga[4], gb[4];
        lane.pairs_of(rg[i], ga, gb);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 c = cs[tok[i]][lane.pair(k) < p.pairs ? lane.pair(k) : kMaxPairs];
          oa[k] = ga[k] * c.x + gb[k] * c.y;
          ob[k] = gb[k] * c.x - ga[k] * c.y;
          if (p.norm != WAN_QK_NORM_NONE) {
            const float r = inv[i], f = r * r * mean_gx[i];
            dw[i][2 * k] += oa[k] * a[k] * r;
            dw[i][2 * k + 1] += ob[k] * b[k] * r;
            oa[k] = r * (oa[k] * wa[k] - a[k] * f);
            ob[k] = r * (ob[k] * wb[k] - b[k] * f);
          }
        }
      }
      const int64_t row = row0 + tok[i];
      lane.store(static_cast<T*>(is_q ? p.q_out : p.k_out) + row * (is_q ? p.qo_stride : p.ko_stride) + h * p.d, oa, ob);
    }
    __syncthreads();
  }
  if constexpr (kBwd) {
    if (p.norm != WAN_QK_NORM_NONE) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int item = i * kHw + hw;
        if (item >= items) continue;
        float a[4], b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = dw[i][2 * k], b[k] = dw[i][2 * k + 1];
        lane.store(p.part + (static_cast<int64_t>(blockIdx.x) * items + item) * p.d, a, b);
      }
    }
  }
}

using F2 = unsigned long long;  // two fp32

constexpr int kMaxHeads = 96;  // q and k heads of one row together
constexpr int kWarps = 8;      // per block
// Groups of 256 columns that stay in registers. The gradient, 20,000 rows of 12 + 12 heads of 128:
// held 116 us in bf16 and 181 in fp32 (which spills 80 to 92 bytes), read twice 219 and 299. Beyond 6
// it reads twice, with one block an SM for its sums: 390 us for 20 + 20 heads and 876 for 40 + 40
// (the general kernel 1940 and 3801), 4.2 and 4.7 times the bytes' time, against 2.1 at 12 + 12.
constexpr int kHeld = 6;
// More of them in the forward (read twice: 143, 161 and 268 us for 20, 24 and 40 heads of q and
// of k on 20,000 rows; held: 98, 106 and 153), the last only of two bytes each.
constexpr int kHeldMore = 12, kHeldMost = 20;

// A thread's 8 columns of a head: two quads at da and db; pairs (da + 2k, da + 2k + 1), or,
// split, (da + k, db + k).
template <bool kHalf>
struct Cols {
  int da, db, quad;  // quad: entry of the cosine table (16: the columns only pass)
  bool on, split;
  __device__ Cols(const RopeParams& p, int u) {
    on = 8 * u < p.d;
    const int turning = p.pairs >> 2;
    split = kHalf && u < turning;
    if (kHalf) {
      da = split ? 4 * u : 2 * p.pairs + 8 * (u - turning);
      db = split ? 4 * u + p.pairs : da + 4;
      quad = split ? u : 16;
    } else {
      da = 8 * u, db = da + 4, quad = u;
    }
  }
  __device__ __forceinline__ void load(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* x) const {
    if (kHalf) {
      const uint2 a = __ldcs(reinterpret_cast<const uint2*>(x + da)), b = __ldcs(reinterpret_cast<const uint2*>(x + db));
      r.u = make_uint4(a.x, a.y, b.x, b.y);
    } else {
      load_raw8(r, x + da);
    }
  }
  __device__ __forceinline__ void load(Raw8<float>& r, const float* x) const {
    r.a = __ldcs(reinterpret_cast<const float4*>(x + da));
    r.b = __ldcs(reinterpret_cast<const float4*>(x + db));
  }
  // The first and second parts of the four pairs, two to a register pair (of passing columns:
  // any order, the inverse of `store`).
  template <typename T>
  __device__ __forceinline__ void pairs_of(const Raw8<T>& r, F2 (&a)[2], F2 (&b)[2]) const {
    float v[8];
    unpack8(r, v);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      a[k] = kHalf ? f2_pack(v[2 * k], v[2 * k + 1]) : f2_pack(v[4 * k], v[4 * k + 2]);
      b[k] = kHalf ? f2_pack(v[4 + 2 * k], v[5 + 2 * k]) : f2_pack(v[4 * k + 1], v[4 * k + 3]);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* x, const F2 (&a2)[2], const F2 (&b2)[2]) const {
    float v[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 a = f2_unpack(a2[k]), b = f2_unpack(b2[k]);
      v[kHalf ? 2 * k : 4 * k] = a.x, v[kHalf ? 2 * k + 1 : 4 * k + 2] = a.y;
      v[kHalf ? 4 + 2 * k : 4 * k + 1] = b.x, v[kHalf ? 5 + 2 * k : 4 * k + 3] = b.y;
    }
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(x + da) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(x + db) = make_float4(v[4], v[5], v[6], v[7]);
    } else if (kHalf) {
      *reinterpret_cast<uint2*>(x + da) = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
      *reinterpret_cast<uint2*>(x + db) = make_uint2(pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7]));
    } else {
      store_vec8(x + da, v);
    }
  }
};

// A turn's cosines, sines and negated sines of a thread's four pairs.
struct Turns {
  F2 c[2], s[2], ns[2];
  __device__ __forceinline__ Turns(const float4& co, const float4& si) {
    c[0] = f2_pack(co.x, co.y), c[1] = f2_pack(co.z, co.w), s[0] = f2_pack(si.x, si.y), s[1] = f2_pack(si.z, si.w);
    ns[0] = f2_pack(-si.x, -si.y), ns[1] = f2_pack(-si.z, -si.w);
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float sum_of(F2 v) {
  const float2 f = f2_unpack(v);
  return f.x + f.y;
}

// Four pairs as two float4, `apart` float4 from one another.
__device__ __forceinline__ void put_pairs(float4* at, int apart, const F2 (&a)[2], const F2 (&b)[2]) {
  *reinterpret_cast<ulonglong2*>(at) = make_ulonglong2(a[0], a[1]);
  *reinterpret_cast<ulonglong2*>(at + apart) = make_ulonglong2(b[0], b[1]);
}
__device__ __forceinline__ void get_pairs(const float4* at, int apart, F2 (&a)[2], F2 (&b)[2]) {
  const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(at), y = *reinterpret_cast<const ulonglong2*>(at + apart);
  a[0] = x.x, a[1] = x.y, b[0] = y.x, b[1] = y.y;
}

// One side's rows: q (blocks [0, q_blocks)) or k (the others), a warp each, in turn. CH: groups
// of 256 columns held in registers; 0: any number, read twice. Dynamic shared memory, fp32: the
// weights, then (gradient) each warp's sums of their gradients, both in the order in which
// lanes take them (four first parts of pairs per lane, then, from chunks * 128 on, the
// second parts), so that they move in 16 bytes without conflicts.
template <typename T, int CH, bool kHalf, bool kBwd>
__global__ void __launch_bounds__(kWarps * 32, kBwd && CH > 0 ? 2 : 1) qk_norm_rope_kernel(const __grid_constant__ RopeParams p, int q_blocks) {
  extern __shared__ float4 dyn[];
  __shared__ float4 cosv[kWarps][17], sinv[kWarps][17];  // entry 16: no turn
  const bool is_q = static_cast<int>(blockIdx.x) < q_blocks;
  const int block = is_q ? blockIdx.x : blockIdx.x - q_blocks, blocks = is_q ? q_blocks : gridDim.x - q_blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = (is_q ? p.H : p.n - p.H) * p.d, groups = (W + 255) / 256, chunks = CH > 0 ? CH : groups;
  const Cols<kHalf> cols(p, lane * 8 % p.d / 8);
  const int head0 = lane * 8 / p.d * p.d;  // the lane's head in a group of 256 columns
  const bool normed = p.norm != WAN_QK_NORM_NONE;
  float4* w_sm = dyn;                                            // [2][groups][32]
  float4* dw_sm = dyn + (normed ? groups * 64 * (1 + warp) : 0);  // the same for each warp
  auto on = [&](int c) { return c * 256 + lane * 8 < W; };
  if (normed) {
    const T* w = static_cast<const T*>(is_q ? p.w_q : p.w_k);
    for (int c = warp; c < groups; c += kWarps) {
      F2 a[2] = {}, b[2] = {};
      if (on(c)) {
        Raw8<T> r;
        cols.load(r, w + (p.norm == WAN_QK_NORM_WIDTH ? c * 256 + head0 : 0));
        cols.pairs_of(r, a, b);
      }
      put_pairs(w_sm + c * 32 + lane, groups * 32, a, b);
    }
    if (kBwd)
      for (int i = lane; i < groups * 64; i += 32) dw_sm[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int i = lane; i < 17; i += 32) cosv[warp][i] = make_float4(1.f, 1.f, 1.f, 1.f), sinv[warp][i] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  const int j1 = lane + 32 < p.pairs ? lane + 32 : 0;
  const double freq0 = p.pairs > 0 && lane < p.pairs ? p.freq[lane] : 0.0, freq1 = p.freq[j1];
  const int axis0 = lane < p.pairs ? p.axis[lane] : 0, axis1 = p.axis[j1];
  const T* in = static_cast<const T*>(is_q ? p.q_in : p.k_in);
  const T* grad = static_cast<const T*>(is_q ? p.gq : p.gk);
  T* out = static_cast<T*>(is_q ? p.q_out : p.k_out);
  const int64_t in_stride = is_q ? p.q_stride : p.k_stride, g_stride = is_q ? p.gq_stride : p.gk_stride;
  const int64_t out_stride = is_q ? p.qo_stride : p.ko_stride;
  const float inv_d = 1.0f / p.d, inv_w = 1.0f / W;
  const int lanes = p.d / 8;
  auto head_sum = [&](float v) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };

  // The next positions are read a row ahead. The gradient, whose registers leave only 16 warps
  // an SM, asks rows into L2 two ahead (201 us without, 164 one ahead, 154 two; the forward
  // gains nothing from it).
  const int64_t step = static_cast<int64_t>(blocks) * kWarps;
  auto ask = [&](const T* base, int64_t stride, int64_t row) {
    const char* line = reinterpret_cast<const char*>(base + row * stride);
    for (int i = lane * 128; i < W * static_cast<int>(sizeof(T)); i += 4096)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(line + i));
  };
  int64_t row = static_cast<int64_t>(block) * kWarps + warp;
  int pos0 = 0, pos1 = 0;
  auto read_pos = [&](int64_t at) {
    if (at >= p.rows) return;
    pos0 = __ldg(p.pos + at * p.n_axes + axis0);
    pos1 = __ldg(p.pos + at * p.n_axes + axis1);
  };
  read_pos(row);
  for (; row < p.rows; row += step) {
    const T* xr = in + row * in_stride + head0;
    const T* gr = grad + row * g_stride + head0;
    T* orow = out + row * out_stride + head0;
    Raw8<T> rx[CH > 0 ? CH : 1], rg[CH > 0 && kBwd ? CH : 1];
    if constexpr (CH > 0) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (on(c)) {
          if (!kBwd || normed) cols.load(rx[c], xr + c * 256);
          if constexpr (kBwd) cols.load(rg[c], gr + c * 256);
        } else {
          rx[c] = Raw8<T>{};
          if constexpr (kBwd) rg[c] = Raw8<T>{};
        }
      }
    }
    if (kBwd && row + 2 * step < p.rows) {
      if (normed) ask(in, in_stride, row + 2 * step);
      ask(grad, g_stride, row + 2 * step);
    }
    {
      float2 t = turn(pos0, freq0, p.amplitude);
      if (lane < p.pairs) reinterpret_cast<float*>(cosv[warp])[lane] = t.x, reinterpret_cast<float*>(sinv[warp])[lane] = t.y;
      if (p.pairs > 32) {
        t = turn(pos1, freq1, p.amplitude);
        if (lane + 32 < p.pairs) reinterpret_cast<float*>(cosv[warp])[lane + 32] = t.x, reinterpret_cast<float*>(sinv[warp])[lane + 32] = t.y;
      }
    }
    read_pos(row + step);
    __syncwarp();
    const Turns w(cosv[warp][cols.quad], sinv[warp][cols.quad]);
    __syncwarp();  // read before the next row's are written
    // The columns of group c: input pairs, and, for the gradient, the turned-back gradient.
    auto x_of = [&](int c, F2 (&a)[2], F2 (&b)[2]) {
      Raw8<T> r{};
      if constexpr (CH > 0)
        r = rx[c];
      else if (on(c) && (!kBwd || normed))
        cols.load(r, xr + c * 256);
      cols.pairs_of(r, a, b);
    };
    auto turn_back = [&](const Raw8<T>& r, F2 (&ga)[2], F2 (&gb)[2]) {
      F2 a[2], b[2];
      cols.pairs_of(r, a, b);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ga[k] = f2_fma(a[k], w.c[k], f2_mul(b[k], w.s[k]));
        gb[k] = f2_fma(b[k], w.c[k], f2_mul(a[k], w.ns[k]));
      }
    };
    F2 ha[CH > 0 && kBwd ? CH : 1][2], hb[CH > 0 && kBwd ? CH : 1][2];  // the turned gradient, held
    if constexpr (CH > 0 && kBwd) {
#pragma unroll
      for (int c = 0; c < CH; ++c) turn_back(rg[c], ha[c], hb[c]);
    }
    auto g_of = [&](int c, F2 (&ga)[2], F2 (&gb)[2]) {
      if constexpr (CH > 0 && kBwd) {
#pragma unroll
        for (int k = 0; k < 2; ++k) ga[k] = ha[c][k], gb[k] = hb[c][k];
      } else {
        Raw8<T> r{};
        if (on(c)) cols.load(r, gr + c * 256);
        turn_back(r, ga, gb);
      }
    };
    auto w_of = [&](int c, F2 (&a)[2], F2 (&b)[2]) {
      if (CH > 0 && c >= groups) {
        a[0] = a[1] = b[0] = b[1] = 0ull;
      } else {
        get_pairs(w_sm + c * 32 + lane, groups * 32, a, b);
      }
    };
    // Sums of x^2 and g w x over group c.
    auto sums = [&](int c, float& s, float& m) {
      F2 xa[2], xb[2];
      x_of(c, xa, xb);
      s = sum_of(f2_fma(xa[0], xa[0], f2_fma(xb[0], xb[0], f2_fma(xa[1], xa[1], f2_mul(xb[1], xb[1])))));
      m = 0.f;
      if constexpr (kBwd) {
        F2 ga[2], gb[2], wa[2], wb[2];
        g_of(c, ga, gb);
        w_of(c, wa, wb);
        F2 v = f2_mul(f2_mul(ga[0], wa[0]), xa[0]);
        v = f2_fma(f2_mul(gb[0], wb[0]), xb[0], v);
        v = f2_fma(f2_mul(ga[1], wa[1]), xa[1], v);
        m = sum_of(f2_fma(f2_mul(gb[1], wb[1]), xb[1], v));
      }
    };
    float r = 1.f, mean = 0.f;
    if (p.norm == WAN_QK_NORM_WIDTH) {
      float s = 0.f, m = 0.f;
#pragma unroll
      for (int c = 0; c < chunks; ++c) {
        float sc, mc;
        sums(c, sc, mc);
        s += sc, m += mc;
      }
      r = rsqrtf(fmaf(warp_sum(s), inv_w, p.eps));
      if (kBwd) mean = warp_sum(m) * inv_w;
    }
#pragma unroll
    for (int c = 0; c < chunks; ++c) {
      if (p.norm == WAN_QK_NORM_HEAD) {
        float s, m;
        sums(c, s, m);
        r = rsqrtf(fmaf(head_sum(s), inv_d, p.eps));
        if (kBwd) mean = head_sum(m) * inv_d;
      }
      F2 oa[2], ob[2], xa[2], xb[2], wa[2], wb[2];
      if (!kBwd || normed) x_of(c, xa, xb);
      if (normed) w_of(c, wa, wb);
      if constexpr (!kBwd) {
        if (normed) {
          const F2 r2 = f2_splat(r);
#pragma unroll
          for (int k = 0; k < 2; ++k) xa[k] = f2_mul(xa[k], f2_mul(r2, wa[k])), xb[k] = f2_mul(xb[k], f2_mul(r2, wb[k]));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          oa[k] = f2_fma(xa[k], w.c[k], f2_mul(xb[k], w.ns[k]));
          ob[k] = f2_fma(xa[k], w.s[k], f2_mul(xb[k], w.c[k]));
        }
      } else {
        F2 ga[2], gb[2];
        g_of(c, ga, gb);
        if (normed) {
          // xh = x r:  dx = g r w - xh r^2 mean,  dw += g xh
          const F2 r2 = f2_splat(r), f = f2_splat(-r * r * mean);
          float4* mine = dw_sm + c * 32 + lane;
          F2 da[2], db[2];
          if (CH == 0 || c < groups) get_pairs(mine, groups * 32, da, db);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            xa[k] = f2_mul(xa[k], r2), xb[k] = f2_mul(xb[k], r2);
            da[k] = f2_fma(ga[k], xa[k], da[k]), db[k] = f2_fma(gb[k], xb[k], db[k]);
            oa[k] = f2_fma(xa[k], f, f2_mul(ga[k], f2_mul(r2, wa[k])));
            ob[k] = f2_fma(xb[k], f, f2_mul(gb[k], f2_mul(r2, wb[k])));
          }
          if (CH == 0 || c < groups) put_pairs(mine, groups * 32, da, db);
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) oa[k] = ga[k], ob[k] = gb[k];
        }
      }
      if (on(c)) cols.store(orow + c * 256, oa, ob);
    }
  }
  if constexpr (kBwd) {
    if (!normed) return;
    __syncthreads();
    // The block's sums, warp after warp, back in the columns' order.
    float* part = p.part + (is_q ? static_cast<int64_t>(block) * W : static_cast<int64_t>(q_blocks) * p.H * p.d + static_cast<int64_t>(block) * W);
    for (int c = warp; c < groups; c += kWarps) {
      F2 a[2] = {}, b[2] = {};
      for (int v = 0; v < kWarps; ++v) {
        F2 x[2], y[2];
        get_pairs(dyn + groups * 64 * (1 + v) + c * 32 + lane, groups * 32, x, y);
#pragma unroll
        for (int k = 0; k < 2; ++k) a[k] = f2_add(a[k], x[k]), b[k] = f2_add(b[k], y[k]);
      }
      if (on(c)) cols.store(part + c * 256 + head0, a, b);
    }
  }
}

// dw[col] = sum over partial rows and (per-head norm) heads, in a fixed order: thread row y
// takes every 32nd summand, the 32 partial sums are added in shared memory. blockIdx.y: q or k,
// whose partial rows begin at part + at and lie `pitch` apart.
struct DwSide {
  int64_t at;
  int rows, heads;
  float* out;
};
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* __restrict__ part, DwSide q, DwSide k, int64_t pitch_q,
                                                       int64_t pitch_k, int d, bool per_head) {
  __shared__ float acc[32][33];
  const DwSide side = blockIdx.y == 0 ? q : k;
  const int64_t pitch = blockIdx.y == 0 ? pitch_q : pitch_k;
  const int cols = per_head ? d : side.heads * d;
  if (!side.out || static_cast<int>(blockIdx.x) * 32 >= cols) return;
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (col < cols) {
    const int hs = per_head ? side.heads : 1;
    for (int h = 0; h < hs; ++h) {
      const float* first = part + side.at + h * d + col;
#pragma unroll 4
      for (int i = threadIdx.y; i < side.rows; i += 32) s += first[i * pitch];
    }
  }
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < cols) {
    float v = 0.f;
#pragma unroll
    for (int y = 0; y < 32; ++y) v += acc[y][threadIdx.x];
    side.out[col] = v;
  }
}

// Blocks of one launch; any_kernel: heads per half-warp, rows per block; the other: blocks of q.
struct RopePlan {
  int ni, tb, blocks, q_blocks;
};
// Few rows: one row a block, the most blocks; else the split that leaves the fewest idle
// half-warps, the larger one of equals.
RopePlan plan_any(int rows, int n, bool dw) {
  RopePlan best{(n + 15) / 16, 1, rows, 0};
  if (rows > 2 * 148) {
    float most = 0.f;
    for (int ni = (n + 15) / 16; ni <= 6; ++ni) {
      const int tb = 16 * ni / n < kMaxTb ? 16 * ni / n : kMaxTb;
      const float used = static_cast<float>(tb * n) / (16 * ni);
      if (used >= most) most = used, best.ni = ni, best.tb = tb;
    }
  }
  best.blocks = (rows + best.tb - 1) / best.tb;
  if (dw && best.blocks > kDwBlocks) best.blocks = kDwBlocks;
  return best;
}
template <typename T, int NI, bool kBwd>
int launch_any(const RopeParams& p, const RopePlan& pl, cudaStream_t s) {
  qk_norm_rope_any_kernel<T, NI, kBwd><<<static_cast<unsigned>(pl.blocks), 256, 0, s>>>(p);
  return check_launch();
}
template <typename T, bool kBwd>
int run_any(const RopeParams& p, const RopePlan& pl, cudaStream_t s) {
  switch (pl.ni) {
    case 1: return launch_any<T, 1, kBwd>(p, pl, s);
    case 2: return launch_any<T, 2, kBwd>(p, pl, s);
    case 3: return launch_any<T, 3, kBwd>(p, pl, s);
    case 4: return launch_any<T, 4, kBwd>(p, pl, s);
    case 5: return launch_any<T, 5, kBwd>(p, pl, s);
    case 6: return launch_any<T, 6, kBwd>(p, pl, s);
  }
  return WAN_ERR_UNSUPPORTED;
}

// Dynamic shared memory of one block (see the kernel), and the most that its own leaves of 227 KB.
constexpr size_t kMostSmem = 220 * 1024;
size_t vec_smem(const RopeParams& p, bool bwd) {
  if (p.norm == WAN_QK_NORM_NONE) return 0;
  const size_t widest = static_cast<size_t>(p.H > p.n - p.H ? p.H : p.n - p.H) * p.d;
  return (widest + 255) / 256 * 1024 * (bwd ? 1 + kWarps : 1);
}
// As many blocks as are resident at once, no more than rows need, shared out between q and k
// by their widths. The weights' gradients take one partial row per block, for which the
// workspace has kDwBlocks.
template <typename T, int CH, bool kHalf, bool kBwd>
int launch_vec(const RopeParams& p, RopePlan& pl, bool dw, cudaStream_t s) {
  auto kernel = qk_norm_rope_kernel<T, CH, kHalf, kBwd>;
  const size_t smem = vec_smem(p, kBwd);
  static ResidentCache resident;
  int most = resident.get(reinterpret_cast<const void*>(kernel), kWarps * 32, smem, kMostSmem);
  if (dw && most > kDwBlocks) most = kDwBlocks;
  const int need = (p.rows + kWarps - 1) / kWarps;  // of each side
  pl.q_blocks = static_cast<int>(static_cast<int64_t>(most) * p.H / p.n);
  pl.q_blocks = pl.q_blocks < 1 ? 1 : (pl.q_blocks < need ? pl.q_blocks : need);
  int k_blocks = 0;
  if (p.n > p.H) {
    k_blocks = most - pl.q_blocks;
    k_blocks = k_blocks < 1 ? 1 : (k_blocks < need ? k_blocks : need);
  }
  pl.blocks = pl.q_blocks + k_blocks;
  kernel<<<static_cast<unsigned>(pl.blocks), kWarps * 32, smem, s>>>(p, pl.q_blocks);
  return check_launch();
}
template <typename T, bool kHalf, bool kBwd>
int run_vec(const RopeParams& p, RopePlan& pl, bool dw, cudaStream_t s) {
  const int widest = (p.H > p.n - p.H ? p.H : p.n - p.H) * p.d;
  if (widest <= kHeld * 256) return launch_vec<T, kHeld, kHalf, kBwd>(p, pl, dw, s);
  if constexpr (!kBwd) {
    if (widest <= kHeldMore * 256) return launch_vec<T, kHeldMore, kHalf, kBwd>(p, pl, dw, s);
    if (sizeof(T) == 2 && widest <= kHeldMost * 256) return launch_vec<T, sizeof(T) == 2 ? kHeldMost : 0, kHalf, kBwd>(p, pl, dw, s);
  }
  return launch_vec<T, 0, kHalf, kBwd>(p, pl, dw, s);
}

int check_rope(const wan_rope* r, int head_dim) {
  WAN_REQUIRE(r, WAN_ERR_NULL);
  WAN_REQUIRE(r->layout == WAN_ROPE_INTERLEAVED || r->layout == WAN_ROPE_HALF, WAN_ERR_SHAPE);
  WAN_REQUIRE(r->scaling >= WAN_ROPE_SCALE_NONE && r->scaling <= WAN_ROPE_SCALE_RAMP, WAN_ERR_SHAPE);
  WAN_REQUIRE(r->n_axes >= 1 && r->n_axes <= 3, WAN_ERR_SHAPE);
  WAN_REQUIRE(isfinite(r->theta) && r->theta > 1.0 && isfinite(r->amplitude) && r->amplitude != 0.0, WAN_ERR_SHAPE);
  int total = 0;
  for (int a = 0; a < r->n_axes; ++a) {
    WAN_REQUIRE(r->axis_dim[a] >= 2 && r->axis_dim[a] % 2 == 0 && r->axis_dim[a] <= head_dim, WAN_ERR_SHAPE);
    total += r->axis_dim[a];
    if (r->scaling != WAN_ROPE_SCALE_NONE) WAN_REQUIRE(isfinite(r->factor[a]) && r->factor[a] > 0.0, WAN_ERR_SHAPE);
    if (r->scaling == WAN_ROPE_SCALE_BASE) WAN_REQUIRE(r->axis_dim[a] > 2, WAN_ERR_SHAPE);
    if (r->scaling == WAN_ROPE_SCALE_RAMP)
      WAN_REQUIRE(r->orig_len[a] > 0 && isfinite(r->fast) && isfinite(r->slow) && r->fast > r->slow, WAN_ERR_SHAPE);
  }
  WAN_REQUIRE(total <= head_dim, WAN_ERR_SHAPE);
  return WAN_OK;
}

void fill_frequencies(const wan_rope* r, RopeParams& p) {
  p.pairs = 0;
  for (int a = 0; a < r->n_axes; ++a) {
    const int n = r->axis_dim[a];
    const double theta =
        r->scaling == WAN_ROPE_SCALE_BASE ? r->theta * pow(r->factor[a], n / (n - 2.0)) : r->theta;
    for (int i = 0; i < n / 2; ++i) {
      double f = pow(theta, -2.0 * i / n);
      if (r->scaling == WAN_ROPE_SCALE_LINEAR) f /= r->factor[a];
      if (r->scaling == WAN_ROPE_SCALE_RAMP) {
        const double turns = r->orig_len[a] * f / 6.283185307179586;
        const double keep = fmin(1.0, fmax(0.0, (turns - r->slow) / (r->fast - r->slow)));
        f *= keep + (1.0 - keep) / r->factor[a];
      }
      p.freq[p.pairs] = f / 6.283185307179586;
      p.axis[p.pairs++] = static_cast<uint8_t>(a);
    }
  }
}

// Whether a view's rows are 16-byte aligned (the vector path needs it of every view).
bool rows_aligned(const wan_rows* v, int dtype) { return !v || v->row_stride % (dtype == WAN_BF16 ? 8 : 4) == 0; }

int check_common(const wan_dit_config* cfg, const wan_rope* rope, const int32_t* positions, int rows, int kv_heads,
                 int norm, bool with_k) {
  WAN_TRY(check_cfg(cfg));
  WAN_REQUIRE(cfg->head_dim <= 128 && cfg->head_dim % 2 == 0, WAN_ERR_SHAPE);
  WAN_REQUIRE(rows >= 0 && kv_heads >= 1, WAN_ERR_SHAPE);
  WAN_REQUIRE(norm >= WAN_QK_NORM_NONE && norm <= WAN_QK_NORM_WIDTH, WAN_ERR_SHAPE);
  WAN_TRY(check_rope(rope, cfg->head_dim));
  WAN_TRY(check_ints(positions, rows));
  const int64_t n = static_cast<int64_t>(cfg->heads) + (with_k ? kv_heads : 0);
  WAN_REQUIRE(n <= kMaxHeads, WAN_ERR_UNSUPPORTED);
  return WAN_OK;
}

template <typename T, bool kBwd>
int run_typed(RopeParams& p, bool vec, bool dw, RopePlan& pl, cudaStream_t s) {
  if (!vec) {
    pl = plan_any(p.rows, p.n, dw);
    p.tb = pl.tb;
    return run_any<T, kBwd>(p, pl, s);
  }
  return p.layout == WAN_ROPE_HALF ? run_vec<T, true, kBwd>(p, pl, dw, s) : run_vec<T, false, kBwd>(p, pl, dw, s);
}
template <bool kBwd>
int run_rope(const wan_dit_config* cfg, RopeParams& p, bool vec, bool dw, RopePlan& pl, cudaStream_t s) {
  return cfg->dtype == WAN_BF16 ? run_typed<__nv_bfloat16, kBwd>(p, vec, dw, pl, s) : run_typed<float, kBwd>(p, vec, dw, pl, s);
}

// Every lane has whole groups of 8 dims at one place of every head (the head divides 256 dims,
// split halves are whole quads), and the block's sums fit into shared memory (sides of up to
// 6144 dims, where the gradient takes 1108 us on 20,000 rows and the general kernel 4523; any for
// the forward).
bool wide_fit(const wan_rope* r, const RopeParams& p, bool bwd) {
  if (p.d < 8 || 256 % p.d != 0 || (r->layout == WAN_ROPE_HALF && p.pairs % 4 != 0)) return false;
  return vec_smem(p, bwd) <= kMostSmem;
}

}  // namespace
}  // namespace wan

using namespace wan;

extern "C" {

int wan_qk_norm_rope_fwd(const wan_dit_config* cfg, const wan_rope* rope, const int32_t* positions, int rows,
                         int kv_heads, int norm, const wan_rows* q, const wan_rows* k, const void* w_q,
                         const void* w_k, const wan_rows* q_out, const wan_rows* k_out, void* stream) {
  const bool with_k = k != nullptr;
  WAN_REQUIRE(with_k == (k_out != nullptr), WAN_ERR_NULL);
  WAN_TRY(check_common(cfg, rope, positions, rows, kv_heads, norm, with_k));
  const int64_t wq = static_cast<int64_t>(cfg->heads) * cfg->head_dim;
  const int64_t wk = static_cast<int64_t>(kv_heads) * cfg->head_dim;
  WAN_TRY(check_view(q, rows, wq, cfg->dtype, false));
  WAN_TRY(check_view(q_out, rows, wq, cfg->dtype, false));
  if (with_k) {
    WAN_TRY(check_view(k, rows, wk, cfg->dtype, false));
    WAN_TRY(check_view(k_out, rows, wk, cfg->dtype, false));
  }
  if (norm != WAN_QK_NORM_NONE) {
    WAN_TRY(check_ptr(w_q));
    if (with_k) WAN_TRY(check_ptr(w_k));
  }
  if (rows == 0) return WAN_OK;
  RopeParams p{};
  p.q_in = q->ptr, p.q_stride = q->row_stride;
  p.q_out = q_out->ptr, p.qo_stride = q_out->row_stride;
  if (with_k) p.k_in = k->ptr, p.k_stride = k->row_stride, p.k_out = k_out->ptr, p.ko_stride = k_out->row_stride;
  p.w_q = w_q, p.w_k = w_k;
  p.pos = positions, p.rows = rows, p.H = cfg->heads, p.n = cfg->heads + (with_k ? kv_heads : 0);
  p.d = cfg->head_dim, p.norm = norm, p.layout = rope->layout, p.n_axes = rope->n_axes;
  p.eps = cfg->eps, p.amplitude = static_cast<float>(rope->amplitude);
  fill_frequencies(rope, p);
  const bool vec = wide_fit(rope, p, false) && rows_aligned(q, cfg->dtype) && rows_aligned(k, cfg->dtype) &&
                   rows_aligned(q_out, cfg->dtype) && rows_aligned(k_out, cfg->dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  trace_launch_begin(WAN_KIND_NORM, s, 2.0 * rows * p.n * p.d * dtype_size(cfg->dtype));
  RopePlan pl{};
  const int st = run_rope<false>(cfg, p, vec, false, pl, s);
  trace_launch_end(WAN_KIND_NORM, s);
  return st;
}

size_t wan_qk_norm_rope_workspace_bytes(const wan_dit_config* cfg, int rows, int kv_heads, int norm) {
  if (check_cfg(cfg) != WAN_OK || cfg->head_dim > 128 || rows < 0 || kv_heads < 1 || norm == WAN_QK_NORM_NONE) return 0;
  size_t most = 0;
  for (int n : {cfg->heads, cfg->heads + kv_heads}) {
    if (n > kMaxHeads) continue;
    const RopePlan any = plan_any(rows, n, true);
    const int64_t vec = kDwBlocks + 1, other = static_cast<int64_t>(any.blocks) * any.tb;
    const size_t b = static_cast<size_t>(vec > other ? vec : other) * n * cfg->head_dim * 4;
    most = b > most ? b : most;
  }
  return most;
}

int wan_qk_norm_rope_bwd(const wan_dit_config* cfg, const wan_rope* rope, const int32_t* positions, int rows,
                         int kv_heads, int norm, const wan_rows* dq_out, const wan_rows* dk_out, const wan_rows* q,
                         const wan_rows* k, const void* w_q, const void* w_k, const wan_rows* dq, const wan_rows* dk,
                         float* dw_q, float* dw_k, void* workspace, size_t ws_bytes, void* stream) {
  const bool with_k = dk_out != nullptr;
  WAN_REQUIRE(with_k == (dk != nullptr), WAN_ERR_NULL);
  WAN_TRY(check_common(cfg, rope, positions, rows, kv_heads, norm, with_k));
  const int64_t wq = static_cast<int64_t>(cfg->heads) * cfg->head_dim;
  const int64_t wk = static_cast<int64_t>(kv_heads) * cfg->head_dim;
  WAN_TRY(check_view(dq_out, rows, wq, cfg->dtype, false));
  WAN_TRY(check_view(dq, rows, wq, cfg->dtype, false));
  if (with_k) {
    WAN_TRY(check_view(dk_out, rows, wk, cfg->dtype, false));
    WAN_TRY(check_view(dk, rows, wk, cfg->dtype, false));
  }
  const bool normed = norm != WAN_QK_NORM_NONE;
  if (normed) {
    WAN_TRY(check_view(q, rows, wq, cfg->dtype, false));
    WAN_TRY(check_ptr(w_q));
    if (with_k) {
      WAN_TRY(check_view(k, rows, wk, cfg->dtype, false));
      WAN_TRY(check_ptr(w_k));
    }
    WAN_TRY(check_opt_ptr(dw_q));
    WAN_TRY(check_opt_ptr(dw_k));
    if (rows > 0) {
      WAN_TRY(check_ptr(workspace));
      WAN_REQUIRE(ws_bytes >= wan_qk_norm_rope_workspace_bytes(cfg, rows, kv_heads, norm), WAN_ERR_WORKSPACE);
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    // no rows: the weights' gradients are sums of nothing
    const size_t nq = (norm == WAN_QK_NORM_HEAD ? cfg->head_dim : wq) * 4, nk = (norm == WAN_QK_NORM_HEAD ? cfg->head_dim : wk) * 4;
    if (normed && dw_q && cudaMemsetAsync(dw_q, 0, nq, s) != cudaSuccess) return WAN_ERR_CUDA;
    if (normed && with_k && dw_k && cudaMemsetAsync(dw_k, 0, nk, s) != cudaSuccess) return WAN_ERR_CUDA;
    return WAN_OK;
  }
  RopeParams p{};
  p.gq = dq_out->ptr, p.gq_stride = dq_out->row_stride;
  p.q_out = dq->ptr, p.qo_stride = dq->row_stride;
  if (with_k) p.gk = dk_out->ptr, p.gk_stride = dk_out->row_stride, p.k_out = dk->ptr, p.ko_stride = dk->row_stride;
  if (normed) {
    p.q_in = q->ptr, p.q_stride = q->row_stride;
    if (with_k) p.k_in = k->ptr, p.k_stride = k->row_stride;
  }
  p.w_q = w_q, p.w_k = w_k;
  p.part = static_cast<float*>(workspace);
  p.pos = positions, p.rows = rows, p.H = cfg->heads, p.n = cfg->heads + (with_k ? kv_heads : 0);
  p.d = cfg->head_dim, p.norm = norm, p.layout = rope->layout, p.n_axes = rope->n_axes;
  p.eps = cfg->eps, p.amplitude = static_cast<float>(rope->amplitude);
  fill_frequencies(rope, p);
  const bool vec = wide_fit(rope, p, true) && rows_aligned(dq_out, cfg->dtype) && rows_aligned(dk_out, cfg->dtype) &&
                   rows_aligned(dq, cfg->dtype) && rows_aligned(dk, cfg->dtype) &&
                   (!normed || (rows_aligned(q, cfg->dtype) && rows_aligned(k, cfg->dtype)));
  trace_launch_begin(WAN_KIND_NORM, s, (normed ? 3.0 : 2.0) * rows * p.n * p.d * dtype_size(cfg->dtype));
  RopePlan pl{};
  int st = run_rope<true>(cfg, p, vec, normed, pl, s);
  if (st == WAN_OK && normed && (dw_q || dw_k)) {
    const bool per_head = norm == WAN_QK_NORM_HEAD;
    const int most = per_head ? p.d : (p.H > p.n - p.H ? p.H : p.n - p.H) * p.d;
    const int64_t wide = static_cast<int64_t>(p.n) * p.d, side_q = static_cast<int64_t>(p.H) * p.d;
    const int part_rows = vec ? 0 : pl.blocks * pl.tb;
    const DwSide dq_side{0, vec ? pl.q_blocks : part_rows, p.H, dw_q};
    const DwSide dk_side{vec ? pl.q_blocks * side_q : side_q, vec ? pl.blocks - pl.q_blocks : part_rows, p.n - p.H, dw_k};
    rope_dw_kernel<<<dim3((most + 31) / 32, with_k ? 2 : 1), dim3(32, 32), 0, s>>>(
        p.part, dq_side, dk_side, vec ? side_q : wide, vec ? wide - side_q : wide, p.d, per_head);
    count_launches(1);
    st = check_launch();
  }
  trace_launch_end(WAN_KIND_NORM, s);
  return st;
}

}  // extern "C"
