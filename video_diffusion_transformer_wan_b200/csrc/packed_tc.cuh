// Device helpers shared by the tensor-core kernels of the attention inside packed
// documents: tiles of packed rows, the capped score, and ragged tiles.
#pragma once
#include "internal.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace wan {

constexpr int kPkTile = 128;                 // packed query rows per tile = keys per tile
constexpr int kPkD = 128;                    // head dim
constexpr int kPkSpan = kPkTile * 128;       // 128 rows of one 128-byte swizzled span
constexpr int kPkTileBytes = 2 * kPkSpan;    // a bf16 tile: two 64-column spans
constexpr float kLog2e = 1.4426950408889634f;

// Query heads that share a key head lie next to one another, so a tile of 128 rows takes
// `pack` heads of 128 / pack queries: row m is query m / pack, head m % pack of the tile.
// pack is the largest divisor of heads / kv_heads up to 128; the key head is then read once
// for all of them, which is what bounds a step of single tokens over long keys. (A "head
// group" below is such a set of `pack` heads.)
struct DocRows {
  int q0, Lq, k0, Lk, off, prefix;
};
__device__ __forceinline__ DocRows load_doc(const PackedAttn& p, int d) {
  const DocRange a = doc_range(p.cu_q, d, p.q_rows), b = doc_range(p.cu_k, d, p.k_rows);
  return {a.first, a.count, b.first, b.count, b.count - a.count, p.prefix ? __ldg(p.prefix + d) : 0};
}

// The warp that issues tensor-core instructions runs as a whole, one elected lane issues. A
// value that all its lanes share is taken from lane 0 by a shuffle: the compiler then knows
// that it is uniform and forms addresses and descriptors from it in uniform registers, which
// these instructions read. (From vector registers every operand of every instruction was moved
// across; the forward spent 20 % more time per key tile.)
__device__ __forceinline__ bool elect_lane() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
template <typename T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// Zero rows [row0, kRows) of a bf16 tile (two spans of kRows swizzled rows) in shared memory, by
// one warp: rows behind a document's end may hold anything (NaN too), and 0 * NaN would reach
// the sums. Whole rows are cleared, so the swizzle inside a row does not matter. Ordered
// before tensor-core reads of the tile that follow an arrival of this warp (after the call).
template <int kRows = kPkTile>
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int row0) {
  const int lane = threadIdx.x & 31;
  for (int i = row0 * 8 + lane; i < kRows * 8; i += 32) {
    *reinterpret_cast<uint4*>(tile + i * 16) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(tile + kRows * 128 + i * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// A pair of 2^x on the FMA pipes, x from -125 up (below: 2^-125; NaN stays NaN): Cody-Waite
// range reduction (W. J. Cody and W. Waite, "Software Manual for the Elementary Functions",
// 1980) to f in [-1/2, 1/2], a degree-5 polynomial fitted for least largest relative error
// there, the integer part added to the exponent field. Relative error with these fp32
// coefficients and fp32 steps: 2.2e-7.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ unsigned long long exp2_poly2(unsigned long long y) {
  const float2 v = f2_unpack(y);
  const unsigned long long x = f2_pack(max_nan(v.x, -125.0f), max_nan(v.y, -125.0f));
  const unsigned long long t = f2_add(x, f2_splat(12582912.0f));  // 1.5 2^23: the low bits hold round(x)
  const unsigned long long f = f2_fma(f2_add(t, f2_splat(-12582912.0f)), f2_splat(-1.0f), x);
  unsigned long long q = f2_fma(f2_splat(0.0013276472454890609f), f, f2_splat(0.009675540961325169f));
  q = f2_fma(q, f, f2_splat(0.05550713092088699f));
  q = f2_fma(q, f, f2_splat(0.24022120237350464f));
  q = f2_fma(q, f, f2_splat(0.6931469440460205f));
  q = f2_fma(q, f, f2_splat(1.0000001192092896f));
  const float2 n = f2_unpack(t), e = f2_unpack(q);
  return f2_pack(__int_as_float(__float_as_int(e.x) + (__float_as_int(n.x) << 23)),
                 __int_as_float(__float_as_int(e.y) + (__float_as_int(n.y) << 23)));
}

// tanh on the FMA pipes for |y| <= 1/2: an odd polynomial fitted for least largest error of
// tanh(y)/y on that range. With these fp32 coefficients and fp32 steps: relative error 1.2e-7,
// absolute 4.4e-8.
constexpr float kTanhPolyLimit = 0.5f;
__device__ __forceinline__ unsigned long long tanh_poly2(unsigned long long y) {
  const unsigned long long z = f2_mul(y, y);
  unsigned long long p = f2_fma(f2_splat(0.017151299864053726f), z, f2_splat(-0.05299423262476921f));
  p = f2_fma(p, z, f2_splat(0.13324907422065735f));
  p = f2_fma(p, z, f2_splat(-0.33333075046539307f));
  p = f2_fma(p, z, f2_splat(1.0f));
  return f2_mul(p, y);
}
// Any y, 2^-22 absolute: 1 - 2 / (e^(2|y|) + 1) with y's sign.
__device__ __forceinline__ float tanh_exp(float y) {
  const float e = ex2_approx(2.0f * kLog2e * fabsf(y));
  return copysignf(1.0f - __fdividef(2.0f, e + 1.0f), y);
}
// In place over N scores s: tanh(s * c), by the polynomial where |s c| <= 1/2 and by the
// exponential elsewhere: a score's bits depend on it alone, whatever stands beside it (columns
// that the row does not see may hold anything), and the gradient forms the forward's. A warp whose
// scores all stay under half the cap (ordinary ones do) leaves the exponentials out; with them 9,360
// frame-causal rows of 12 heads take 512 us against 302. (Columns not seen kept out of the vote too:
// 322 us, 4 to 5 % of every call, for the time of those beside large neighbours.) Rows that are not
// `live` do not decide.
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t (&r)[N], float c, bool live) {
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) big = fmax3(big, fabsf(__uint_as_float(r[i])), fabsf(__uint_as_float(r[i + 1])));
  const unsigned long long c2 = f2_splat(c);
  if (__all_sync(0xffffffffu, !live || big * fabsf(c) <= kTanhPolyLimit)) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 t = f2_unpack(tanh_poly2(f2_mul(f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), c2)));
      r[i] = __float_as_uint(t.x), r[i + 1] = __float_as_uint(t.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const unsigned long long y2 = f2_mul(f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), c2);
      const float2 y = f2_unpack(y2), t = f2_unpack(tanh_poly2(y2));
      r[i] = __float_as_uint(fabsf(y.x) <= kTanhPolyLimit ? t.x : tanh_exp(y.x));
      r[i + 1] = __float_as_uint(fabsf(y.y) <= kTanhPolyLimit ? t.y : tanh_exp(y.y));
    }
  }
}

}  // namespace wan
