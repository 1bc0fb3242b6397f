// Rotary positions with the q/k norm, and their gradient (wan_qk_norm_rope_*).
//
// Per head of a row: x -> x r w (r = 1/sqrt(mean(x^2) + eps) over the head or the whole
// width, or no norm), then every pair (a, b) of the rotated part turns by its angle:
// (a c - b s, a s + b c). The gradient turns back, g = R^T dout, and with m = mean(g w x)
// gives dx = r (g w - x r^2 m) and dw = sum over rows of g x r.
//
// HBM-bound: the forward reads and writes every element once, the gradient reads two and
// writes one. A half-warp holds one head of one row, 8 elements (four whole pairs) a lane,
// so a rotation needs no exchange: with interleaved pairs a lane owns 8 consecutive
// elements, with split halves 4 of each half. A block takes `tb` rows and holds NI heads
// per half-warp in registers; all its loads are issued before anything waits, and the
// cosines are made while they fly: one (row, pair) each, shared by all heads of q and k
// through shared memory, the angle reduced in fp64 (positions may be far), the sine in
// fp32. The width norm adds one exchange of the heads' partial sums through shared memory.
#include <cuda_bf16.h>

#include <math.h>

#include "checks.h"
#include "internal.h"
#include "packed.cuh"

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
  float* part;          // gradient: [block][tb * n][head_dim] partial weight gradients
  const int32_t* pos;
  int rows, H, n, d, tb, norm, layout, pairs, n_axes;  // n = heads of q and k together
  float eps, amplitude;
  double freq[kMaxPairs];
  uint8_t axis[kMaxPairs];
};

// A lane's four pairs. V = 4: two quads of elements (16-byte accesses where the quads are
// neighbours); V = 1: single elements, for shapes that quads do not divide.
template <int V>
struct Lane;
template <>
struct Lane<4> {
  int da, db, p0;  // first elements of the quads; first pair (or -1: the quads only pass)
  bool on, split;  // split: pair k is (da + k, db + k); else (da + 2k, da + 2k + 1) over both quads
  __device__ Lane(const RopeParams& p, int u) {
    split = false;
    if (p.layout == WAN_ROPE_HALF) {
      const int turning = p.pairs >> 2;
      split = u < turning;
      da = split ? 4 * u : 2 * p.pairs + 8 * (u - turning);
      db = split ? 4 * u + p.pairs : da + 4;
      p0 = split ? 4 * u : -1;
    } else {
      da = 8 * u, db = da + 4, p0 = 4 * u;
    }
    on = 8 * u < p.d;
  }
  __device__ __forceinline__ int pair(int k) const { return p0 < 0 ? kMaxPairs : p0 + k; }
  __device__ __forceinline__ void load(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* x) const {
    if (!on) {
      r.u = make_uint4(0, 0, 0, 0);
    } else if (split) {
      const uint2 a = __ldcs(reinterpret_cast<const uint2*>(x + da)), b = __ldcs(reinterpret_cast<const uint2*>(x + db));
      r.u = make_uint4(a.x, a.y, b.x, b.y);
    } else {
      load_raw8(r, x + da);
    }
  }
  __device__ __forceinline__ void load(Raw8<float>& r, const float* x) const {
    if (!on) {
      r.a = r.b = make_float4(0, 0, 0, 0);
    } else {
      r.a = __ldcs(reinterpret_cast<const float4*>(x + da));
      r.b = __ldcs(reinterpret_cast<const float4*>(x + db));
    }
  }
  template <typename T>
  __device__ __forceinline__ void pairs_of(const Raw8<T>& r, float (&a)[4], float (&b)[4]) const {
    float v[8];
    unpack8(r, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = split ? v[k] : v[2 * k], b[k] = split ? v[4 + k] : v[2 * k + 1];
  }
  __device__ __forceinline__ void join(const float (&a)[4], const float (&b)[4], float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = split ? a[k] : ((k & 1) ? b[k >> 1] : a[k >> 1]);
      v[4 + k] = split ? b[k] : ((k & 1) ? b[2 + (k >> 1)] : a[2 + (k >> 1)]);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* x, const float (&a)[4], const float (&b)[4]) const {
    if (!on) return;
    float v[8];
    join(a, b, v);
    if (split) {
      *reinterpret_cast<uint2*>(x + da) = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
      *reinterpret_cast<uint2*>(x + db) = make_uint2(pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7]));
    } else {
      store_vec8(x + da, v);
    }
  }
  __device__ __forceinline__ void store(float* x, const float (&a)[4], const float (&b)[4]) const {
    if (!on) return;
    float v[8];
    join(a, b, v);
    *reinterpret_cast<float4*>(x + da) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(x + db) = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <>
struct Lane<1> {
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

template <typename T, int V, int NI, bool kBwd>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kHw = 16;  // half-warps per block
  __shared__ float2 cs[kMaxTb][kMaxPairs + 1];  // the last entry: no turn (1, 0)
  __shared__ float red[kBwd ? 2 : 1][kHw * NI];
  const int hw = threadIdx.x >> 4, u = threadIdx.x & 15;
  const Lane<V> lane(p, u);
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
        const double angle = static_cast<double>(p.pos[(row0 + t) * p.n_axes + p.axis[j]]) * p.freq[j];
        const double turns = rint(angle * 0.15915494309189535);  // 1 / (2 pi)
        float s, c;
        sincosf(static_cast<float>(fma(turns, -6.283185307179586, angle)), &s, &c);
        cs[t][j] = make_float2(c * p.amplitude, s * p.amplitude);
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

// dw[col] = sum over blocks, their rows and (per-head norm) heads of the partial sums, in a
// fixed order: thread row y takes every 32nd summand, the 32 partial sums are added in
// shared memory. blockIdx.y: q or k.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* __restrict__ part, int blocks, int tb, int n, int H,
                                                       int d, bool per_head, float* dw_q, float* dw_k) {
  __shared__ float acc[32][33];
  const bool is_q = blockIdx.y == 0;
  float* out = is_q ? dw_q : dw_k;
  const int h0 = is_q ? 0 : H, heads = is_q ? H : n - H;
  const int cols = per_head ? d : heads * d;
  if (!out || static_cast<int>(blockIdx.x) * 32 >= cols) return;
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (col < cols) {
    const int hs = per_head ? heads : 1;
    const int64_t count = static_cast<int64_t>(blocks) * tb * hs;
    const int first = h0 * d + col;
#pragma unroll 4
    for (int64_t i = threadIdx.y; i < count; i += 32) {
      const int64_t bt = i / hs;
      s += part[bt * n * d + (i - bt * hs) * d + first];
    }
  }
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < cols) {
    float v = 0.f;
#pragma unroll
    for (int y = 0; y < 32; ++y) v += acc[y][threadIdx.x];
    out[col] = v;
  }
}

// Heads per half-warp and rows per block. Few rows: one row a block, the most blocks;
// else the split that leaves the fewest idle half-warps, the larger one of equals.
struct RopePlan {
  int ni, tb, blocks;
};
RopePlan plan_rope(int rows, int n, bool dw) {
  RopePlan best{(n + 15) / 16, 1, rows};
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

template <typename T, int V, int NI, bool kBwd>
int launch_ni(const RopeParams& p, int blocks, cudaStream_t s) {
  qk_norm_rope_kernel<T, V, NI, kBwd><<<static_cast<unsigned>(blocks), 256, 0, s>>>(p);
  return check_launch();
}
template <typename T, int V, bool kBwd>
int launch_v(const RopeParams& p, const RopePlan& pl, cudaStream_t s) {
  switch (pl.ni) {
    case 1: return launch_ni<T, V, 1, kBwd>(p, pl.blocks, s);
    case 2: return launch_ni<T, V, 2, kBwd>(p, pl.blocks, s);
    case 3: return launch_ni<T, V, 3, kBwd>(p, pl.blocks, s);
    case 4: return launch_ni<T, V, 4, kBwd>(p, pl.blocks, s);
    case 5: return launch_ni<T, V, 5, kBwd>(p, pl.blocks, s);
    case 6: return launch_ni<T, V, 6, kBwd>(p, pl.blocks, s);
  }
  return WAN_ERR_UNSUPPORTED;
}

constexpr int kMaxHeads = 96;  // q and k heads of one row together (six per half-warp)

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
      p.freq[p.pairs] = f;
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
  WAN_TRY(check_array(positions, rows));
  const int64_t n = static_cast<int64_t>(cfg->heads) + (with_k ? kv_heads : 0);
  WAN_REQUIRE(n <= kMaxHeads, WAN_ERR_UNSUPPORTED);
  return WAN_OK;
}

template <bool kBwd>
int run_rope(const wan_dit_config* cfg, RopeParams& p, bool vec, bool dw, cudaStream_t s) {
  const RopePlan pl = plan_rope(p.rows, p.n, dw);
  p.tb = pl.tb;
  if (cfg->dtype == WAN_BF16)
    return vec ? launch_v<__nv_bfloat16, 4, kBwd>(p, pl, s) : launch_v<__nv_bfloat16, 1, kBwd>(p, pl, s);
  return vec ? launch_v<float, 4, kBwd>(p, pl, s) : launch_v<float, 1, kBwd>(p, pl, s);
}

// Quads divide the head: whole lanes of 8, and with split halves whole quads of each half.
bool quads_fit(const wan_rope* r, const RopeParams& p) {
  return p.d % 8 == 0 && (r->layout == WAN_ROPE_INTERLEAVED || p.pairs % 4 == 0);
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
  const bool vec = quads_fit(rope, p) && rows_aligned(q, cfg->dtype) && rows_aligned(k, cfg->dtype) &&
                   rows_aligned(q_out, cfg->dtype) && rows_aligned(k_out, cfg->dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  trace_launch_begin(WAN_KIND_NORM, s, 2.0 * rows * p.n * p.d * dtype_size(cfg->dtype));
  const int st = run_rope<false>(cfg, p, vec, false, s);
  trace_launch_end(WAN_KIND_NORM, s);
  return st;
}

size_t wan_qk_norm_rope_workspace_bytes(const wan_dit_config* cfg, int rows, int kv_heads, int norm) {
  if (check_cfg(cfg) != WAN_OK || cfg->head_dim > 128 || rows < 0 || kv_heads < 1 || norm == WAN_QK_NORM_NONE) return 0;
  size_t most = 0;
  for (int n : {cfg->heads, cfg->heads + kv_heads}) {
    if (n > kMaxHeads) continue;
    const RopePlan pl = plan_rope(rows, n, true);
    const size_t b = static_cast<size_t>(pl.blocks) * pl.tb * n * cfg->head_dim * 4;
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
  const bool vec = quads_fit(rope, p) && rows_aligned(dq_out, cfg->dtype) && rows_aligned(dk_out, cfg->dtype) &&
                   rows_aligned(dq, cfg->dtype) && rows_aligned(dk, cfg->dtype) &&
                   (!normed || (rows_aligned(q, cfg->dtype) && rows_aligned(k, cfg->dtype)));
  trace_launch_begin(WAN_KIND_NORM, s, (normed ? 3.0 : 2.0) * rows * p.n * p.d * dtype_size(cfg->dtype));
  int st = run_rope<true>(cfg, p, vec, normed, s);
  if (st == WAN_OK && normed && (dw_q || dw_k)) {
    const RopePlan pl = plan_rope(rows, p.n, true);
    const bool per_head = norm == WAN_QK_NORM_HEAD;
    const int most = per_head ? p.d : (p.H > p.n - p.H ? p.H : p.n - p.H) * p.d;
    rope_dw_kernel<<<dim3((most + 31) / 32, with_k ? 2 : 1), dim3(32, 32), 0, s>>>(p.part, pl.blocks, pl.tb, p.n, p.H,
                                                                                  p.d, per_head, dw_q, dw_k);
    count_launches(1);
    st = check_launch();
  }
  trace_launch_end(WAN_KIND_NORM, s);
  return st;
}

}  // extern "C"
