// Device helpers of the packed-document kernels: document offsets, the order mask's key
// count, and 8-wide loads and stores of fp32 and bf16 rows.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace wan {

// Rows [first, first + count) of document d, clamped into [0, total) and into order, so
// that malformed offsets cannot reach outside the tensor.
struct DocRange {
  int first, count;
};
__device__ __forceinline__ DocRange doc_range(const int32_t* __restrict__ cu, int d, int total) {
  const int a = min(max(__ldg(cu + d), 0), total);
  const int b = min(max(__ldg(cu + d + 1), a), total);
  return {a, b - a};
}

// Tile `idx` of the documents cut into tiles of `tile` rows (documents in order), found by
// one whole warp: 32 documents at a time, a prefix sum of their tile counts by shuffles.
// Returns false (in all lanes) past the last tile.
__device__ __forceinline__ bool find_doc_tile(const int32_t* __restrict__ cu, int n_docs, int total, int tile, int idx,
                                              int& doc, int& tile_in_doc) {
  const int lane = threadIdx.x & 31;
  for (int d0 = 0; d0 < n_docs; d0 += 32) {
    int n = 0;
    if (d0 + lane < n_docs) n = (doc_range(cu, d0 + lane, total).count + tile - 1) / tile;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const int sum = __shfl_sync(0xffffffffu, incl, 31);
    if (idx < sum) {
      const unsigned hit = __ballot_sync(0xffffffffu, idx < incl);
      const int src = __ffs(hit) - 1;
      doc = d0 + src;
      tile_in_doc = idx - __shfl_sync(0xffffffffu, incl - n, src);
      return true;
    }
    idx -= sum;
  }
  return false;
}

// Keys seen by query row i (see wan_documents): `off` = Lk - Lq, `block` = causal_block.
__device__ __forceinline__ int seen_keys(int i, int off, int Lk, int prefix, int block) {
  if (block == 0) return Lk;
  const int pos = i + off;
  int n = 0;
  if (pos >= 0) {
    const int64_t end = (static_cast<int64_t>(pos / block) + 1) * block;
    n = end < Lk ? static_cast<int>(end) : Lk;
  }
  return max(n, min(prefix, Lk));
}

// First query row of a document that sees key j (Lq or more if none does); the key count
// only grows along the rows.
__device__ __forceinline__ int first_query(int j, int off, int Lk, int prefix, int block) {
  if (block == 0 || j < min(prefix, Lk)) return 0;
  return max(0, j / block * block - off);
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Eight (or four) consecutive values as they lie in memory, 16-byte (8-byte) aligned.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
};
template <>
struct Raw8<float> {
  float4 a, b;
};
__device__ __forceinline__ void load_raw8(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* p) {
  r.u = __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void load_raw8(Raw8<float>& r, const float* p) {
  r.a = __ldcs(reinterpret_cast<const float4*>(p));
  r.b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  v[0] = bf16_lo(r.u.x), v[1] = bf16_hi(r.u.x), v[2] = bf16_lo(r.u.y), v[3] = bf16_hi(r.u.y);
  v[4] = bf16_lo(r.u.z), v[5] = bf16_hi(r.u.z), v[6] = bf16_lo(r.u.w), v[7] = bf16_hi(r.u.w);
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
  v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w;
  v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}
__device__ __forceinline__ void store_vec8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store_vec8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

}  // namespace wan
