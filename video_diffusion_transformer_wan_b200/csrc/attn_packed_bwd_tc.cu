// Gradient of the attention inside packed documents on the sm_100a tensor cores (bf16,
// head_dim 128). With s the (capped, distance-biased) score, p = e^(s - lse) recomputed from
// the stored log-sums, delta = sum(do * o) per row and turn = 1 - tanh^2 of a capped score:
//   dp = do v^T,   ds = p (dp - delta) turn,
//   dq = scale ds k,   dk = scale ds^T q,   dv = p^T do.
//
// Two kernels, one per side, so that every sum is formed in one place in a fixed order
// (nothing is added across CTAs): 3 tile products a (query tile, key tile) for dq, 4 for
// dk and dv, against 5 if one kernel did both and added dq through memory. p and ds are
// rounded to bf16, the tensor cores' operand; everything else is fp32.
//
// A CTA owns 128 rows (packed query rows, or keys) and walks the tiles of the other side;
// 384 threads, one CTA per SM: warp 0 loads by TMA, warp 1 issues tcgen05.mma, warp 2 (keys'
// kernel) stages the per-query numbers, warp 3 clears ragged tiles, warps 4-11 do the scores:
// a thread has half of a row's 128 columns (warps 4-7 the first, 8-11 the second).
//   dq:  TMEM holds S twice, dP and dQ. While the score warps work on tile j the tensor core
//        forms S(j+1), and dP(j+1) as soon as dP(j) is read; ds goes back over S(j) in bf16
//        (each half into its own columns) as the A operand of dQ += ds K_j.
//   dkv: the transposed scores, S^T = K Q^T and dP^T = V dO^T, so that p^T and ds^T are A
//        operands too; both go back over S^T. Query tiles have 64 rows, so that TMEM holds
//        S^T and dP^T twice beside dV and dK: while the score warps work on tile i the tensor
//        core forms tile i+1's scores and tile i-1's products, and four tiles are on their
//        way. (With 128 rows, held once, it waited for loads and scores in turn: 697 us
//        against 465 us on 9,371 rows of 12 heads.)
// Rows behind a document's end belong to others: where they are summed over (K rows in dq; Q
// and dO rows in dkv) they are cleared in shared memory, elsewhere masked or not stored.
#include <math.h>

#include <mutex>

#include "internal.h"
#include "packed_tc.cuh"

namespace wan {
namespace {

constexpr int kThreads = 384;
constexpr int kScoreThreads = 256;
constexpr int kDqStages = 5;
constexpr int kDkvStages = 4;                // query tiles of 64 rows on their way
constexpr int kHalfSpan = 64 * 128;          // 64 rows of one 128-byte swizzled span
constexpr int kHalfBytes = 2 * kHalfSpan;    // 64 rows of 128 dims
constexpr size_t kDqSmem = 1024 + static_cast<size_t>(kPkTileBytes) * (2 + kDqStages) + 1280;
// per staged query: float2 (log-sum, delta) or, with distances, float4; and a key count
constexpr int kStatBytes = 64 * (16 + 4);
constexpr int kStatBufs = 4;
constexpr size_t kDkvSmem =
    1024 + 2 * static_cast<size_t>(kPkTileBytes) + 2 * static_cast<size_t>(kHalfBytes) * kDkvStages + kStatBufs * kStatBytes + 512;
static_assert(kDqSmem <= 232448 && kDkvSmem <= 232448, "shared memory of an SM");

struct BwdParams {
  PackedAttn a;
  int pack, per_tile, groups;
  float mult;      // log2 units per (possibly capped) score
  float cap_in;    // scale / cap
  int* err;
};

// This CTA's tile of documents' rows (found by warp 0); false past the last one.
__device__ __forceinline__ bool cta_tile(const int32_t* cu, int n_docs, int rows, int per_tile, int* found, int& doc, int& tile) {
  if (threadIdx.x < 32) {
    int d = 0, t = 0;
    const bool ok = find_doc_tile(cu, n_docs, rows, per_tile, blockIdx.x, d, t);
    if (threadIdx.x == 0) found[0] = ok, found[1] = d, found[2] = t;
  }
  __syncthreads();
  doc = found[1], tile = found[2];
  return found[0] != 0;
}

// D (+)= A B over a 128-deep sum whose A halves lie at a and a + 64 columns in TMEM.
__device__ __forceinline__ void mma_ts_halves(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool first) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    tc_mma_bf16_ts(d, a + (k >> 2) * 64 + (k & 3) * 8, b + ((k * 16 * 128) >> 4), idesc, (!first || k > 0) ? 1u : 0u);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t off = ((k >> 2) * kPkSpan + (k & 3) * 32) >> 4;
    tc_mma_bf16(d, a + off, b + off, idesc, k > 0 ? 1u : 0u);
  }
}

// Slot and phase of load 2 j (K_j) or 2 j + 1 (V_j): three slots of keys, which are held until
// their product with ds, and two of values, which are free after dP. (In one ring of five a
// value tile waited for the slot of a key tile: 40 us more on 9,371 rows of 12 heads.)
struct DqSlot {
  int slot;
  uint32_t phase;
};
__device__ __forceinline__ DqSlot dq_slot(int load) {
  const int j = load >> 1;
  if (load & 1) return {3 + (j & 1), static_cast<uint32_t>((j >> 1) & 1)};
  return {j % 3, static_cast<uint32_t>((j / 3) & 1)};
}

template <bool kPlain>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dq_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapO,
                        const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                        const __grid_constant__ BwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                      // Q, then dO
  uint8_t* sKV = sQ + 2 * kPkTileBytes;    // [kDqStages], see dq_slot
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + kDqStages * kPkTileBytes);
  uint64_t* q_full = bars;
  uint64_t* kv_full = bars + 1;
  uint64_t* kv_empty = kv_full + kDqStages;
  uint64_t* s_full = kv_empty + kDqStages;  // S(j) and dP(j) are there
  uint64_t* y_free = s_full + 1;            // dP(j) has been read
  // [2] ds(j) is in place (j & 1): S(j+1) and dP(j+1) do not wait for ds(j), so a warp may be a tile
  // ahead of another, and on one barrier its arrival would stand for the late one's.
  uint64_t* ds_full = s_full + 2;
  uint64_t* done = s_full + 4;
  uint64_t* ragged = s_full + 5;
  uint64_t* cleared = s_full + 6;
  uint64_t* halves = s_full + 7;            // both halves' parts of delta are there
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(s_full + 8);
  int* found = reinterpret_cast<int*>(s_full + 9);
  float* part = reinterpret_cast<float*>(s_full + 11);  // [2][128]
  static_assert(8 * (1 + 2 * kDqStages + 11) + 2 * kPkTile * 4 <= 1280, "barriers and parts");

  int di, tile;
  if (!cta_tile(p.a.cu_q, p.a.n_docs, p.a.q_rows, p.per_tile, found, di, tile)) return;
  const DocRows doc = load_doc(p.a, di);
  tile = div_up(doc.Lq, p.per_tile) - 1 - tile;  // the tiles that see the most keys first
  const int first = tile * p.per_tile, rows = min(p.per_tile, doc.Lq - first);
  const int n = div_up(seen_keys(first + rows - 1, doc.off, doc.Lk, doc.prefix, p.a.causal_block), kPkTile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < kDqStages; ++s) mbar_init(&kv_full[s], 1), mbar_init(&kv_empty[s], 1);
    mbar_init(s_full, 1);
    mbar_init(y_free, kScoreThreads);
    for (int b = 0; b < 2; ++b) mbar_init(&ds_full[b], kScoreThreads);
    mbar_init(done, 1);
    mbar_init(ragged, 1);
    mbar_init(cleared, 1);
    mbar_init(halves, kScoreThreads);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder, Y = tmem + 256, Z = tmem + 384;  // S(j) at tmem + 128 (j & 1)
  const int end = doc.Lk - (n - 1) * kPkTile;  // keys of the last tile that are the document's

  if (warp == 0) {
    if (lane == 0 && n > 0) {
      const uint32_t bytes = static_cast<uint32_t>(p.per_tile * p.pack) * 256u;
      mbar_arrive_expect_tx(q_full, 2 * bytes);
      for (int c = 0; c < 2; ++c) {
        tma_load_3d(sQ + c * kPkSpan, &mapQ, q_full, 64 * c, blockIdx.y * p.pack, doc.q0 + first);
        tma_load_3d(sQ + kPkTileBytes + c * kPkSpan, &mapO, q_full, 64 * c, blockIdx.y * p.pack, doc.q0 + first);
      }
      const int col = static_cast<int>(blockIdx.y) * p.pack / (p.a.H / p.a.Hk) * kPkD;
      int issued = 0;
      for (; issued < 2 * n; ++issued) {
        const DqSlot at = dq_slot(issued);
        if (!mbar_wait(&kv_empty[at.slot], at.phase ^ 1u, p.err)) break;
        mbar_arrive_expect_tx(&kv_full[at.slot], kPkTileBytes);
        for (int c = 0; c < 2; ++c)
          tma_load_2d(sKV + at.slot * kPkTileBytes + c * kPkSpan, issued & 1 ? &mapV : &mapK, &kv_full[at.slot], col + 64 * c,
                      doc.k0 + (issued >> 1) * kPkTile);
      }
      mbar_wait(q_full, 0, p.err);  // every copy this thread started has landed before it leaves
      for (int load = issued > 6 ? issued - 6 : 0; load < issued; ++load) {
        const DqSlot at = dq_slot(load);
        // the last load of its slot
        if (load + (load & 1 ? 4 : 6) >= issued) mbar_wait(&kv_full[at.slot], at.phase, p.err);
      }
    }
  } else if (warp == 1) {
    const int nu = uniform(n);
    if (nu > 0) {
      const uint32_t id_kk = idesc_bf16_f32(kPkTile, kPkTile, 0, 0), id_mn = idesc_bf16_f32(kPkTile, kPkD, 0, 1);
      const uint32_t tm = uniform(tmem);
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024), o_desc = sdesc_sw128(smem_u32(sQ + kPkTileBytes), 16, 1024);
      const uint64_t kv_desc = sdesc_sw128(smem_u32(sKV), 16, 1024), kt_desc = sdesc_sw128(smem_u32(sKV), kPkSpan, 1024);
      auto stage_off = [](int load) { return static_cast<uint32_t>((dq_slot(load).slot * kPkTileBytes) >> 4); };
      auto wait_pos = [&](int load) {
        const DqSlot at = dq_slot(load);
        return mbar_wait_warp(&kv_full[at.slot], at.phase, p.err);
      };
      // S(j), then dP(j) once dP(j-1) has been read
      auto scores = [&](int j) {
        if (!wait_pos(2 * j)) return false;
        if (j == nu - 1 && uniform(end) < kPkTile) {
          if (lane == 0) mbar_arrive(ragged);
          if (!mbar_wait_warp(cleared, 0, p.err)) return false;
        }
        const uint64_t kd = kv_desc + stage_off(2 * j), vd = kv_desc + stage_off(2 * j + 1);
        if (elect_lane()) mma_ss(tm + 128 * (j & 1), q_desc, kd, id_kk);
        if (!wait_pos(2 * j + 1)) return false;
        if (j > 0 && !mbar_wait_warp(y_free, static_cast<uint32_t>((j - 1) & 1), p.err)) return false;
        tc_fence_after();
        if (elect_lane()) {
          mma_ss(tm + 256, o_desc, vd, id_kk);
          tc_commit(&kv_empty[dq_slot(2 * j + 1).slot]);
          tc_commit(s_full);
        }
        return true;
      };
      bool ok = mbar_wait_warp(q_full, 0, p.err) && scores(0);
      for (int j = 0; ok && j < nu; ++j) {
        if (j + 1 < nu && !scores(j + 1)) break;
        if (!mbar_wait_warp(&ds_full[j & 1], static_cast<uint32_t>((j >> 1) & 1), p.err)) break;
        tc_fence_after();
        const uint64_t kd = kt_desc + stage_off(2 * j);
        if (elect_lane()) {
          mma_ts_halves(tm + 384, tm + 128 * (j & 1), kd, id_mn, j == 0);
          tc_commit(&kv_empty[dq_slot(2 * j).slot]);
        }
      }
      if (elect_lane()) tc_commit(done);
      mbar_wait_warp(done, 0, p.err);
    }
  } else if (warp == 3) {
    if (n > 0 && end < kPkTile && mbar_wait_warp(ragged, 0, p.err)) {
      zero_tile_rows(sKV + dq_slot(2 * (n - 1)).slot * kPkTileBytes, end);
      if (lane == 0) mbar_arrive(cleared);
    }
  } else if (warp >= 4) {
    const int half = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t at = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int query = row / p.pack, i = first + query, head = static_cast<int>(blockIdx.y) * p.pack + row - query * p.pack;
    const bool live = query < rows;
    const int seen = live ? seen_keys(i, doc.off, doc.Lk, doc.prefix, p.a.causal_block) : 0x7fffffff;
    const int64_t stat = static_cast<int64_t>(head) * p.a.q_rows + doc.q0 + i;
    const float nl = live ? -p.a.lse[stat] * kLog2e : 0.f;
    float nd = live ? -p.a.delta[stat] : 0.f;
    const float slope2 = !kPlain && p.a.slopes && live ? __ldg(p.a.slopes + head) * kLog2e : 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!mbar_wait_warp(s_full, static_cast<uint32_t>(j & 1), p.err)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t x = tmem + 128 * (j & 1) + at + 64 * half;
      uint32_t s[64], g[64];
      tmem_ld32(x, *reinterpret_cast<uint32_t(*)[32]>(s));
      tmem_ld32(x + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
      tmem_ld32(Y + at + 64 * half, *reinterpret_cast<uint32_t(*)[32]>(g));
      tmem_ld32(Y + at + 64 * half + 32, *reinterpret_cast<uint32_t(*)[32]>(g + 32));
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(y_free);
      const int key0 = j * kPkTile + 64 * half;
      const unsigned long long nl2 = f2_splat(nl), mult2 = f2_splat(p.mult);
      const float from = static_cast<float>(i + doc.off - key0);
      const int valid = seen - key0;
      auto log2_p = [&](int c) {
        const unsigned long long y = f2_fma(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), mult2, nl2);
        if (kPlain || !p.a.slopes) return f2_unpack(y);
        return f2_unpack(f2_add(y, f2_pack(-slope2 * fabsf(from - static_cast<float>(c)), -slope2 * fabsf(from - static_cast<float>(c + 1)))));
      };
      if (!kPlain && p.a.cap > 0.f) cap_scores(s, p.cap_in, live);
      if (n == 1) {
        // All keys of the row are at hand: delta = sum(p dp) itself, since with few keys the
        // rounding of o to bf16 weighs in do * o (dq and dk of documents of 2 keys were 2.3
        // times as far off as the plain form's). The keys' kernel takes it from here too. Over
        // more key tiles delta is do * o: it would take the scores and dp of all of them twice.
        // (Rows that rest on few of many keys feel it: one query over 131 keys with steep distance
        // slopes 6.5e-3 off, 3.8 times the plain form; 1,145 rows of them 2.6e-3, 1.6 times.)
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 e = log2_p(c);
          if (c < valid) sum = fmaf(ex2_approx(e.x), __uint_as_float(g[c]), sum);
          if (c + 1 < valid) sum = fmaf(ex2_approx(e.y), __uint_as_float(g[c + 1]), sum);
        }
        part[half * kPkTile + row] = sum;
        mbar_arrive(halves);
        if (!mbar_wait_warp(halves, 0, p.err)) {
          ok = false;
          break;
        }
        nd = -(part[row] + part[kPkTile + row]);
        if (live && half == 0) p.a.delta[stat] = -nd;
      }
      const unsigned long long nd2 = f2_splat(nd);
      if (!kPlain && p.a.cap > 0.f) {
#pragma unroll
        for (int c = 0; c < 64; c += 2) {  // g = (dp - delta)(1 - t^2)
          const unsigned long long t = f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
          const unsigned long long d = f2_add(f2_pack(__uint_as_float(g[c]), __uint_as_float(g[c + 1])), nd2);
          const float2 v = f2_unpack(f2_mul(d, f2_fma(f2_mul(t, f2_splat(-1.f)), t, f2_splat(1.f))));
          g[c] = __float_as_uint(v.x), g[c + 1] = __float_as_uint(v.y);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 v = f2_unpack(f2_add(f2_pack(__uint_as_float(g[c]), __uint_as_float(g[c + 1])), nd2));
          g[c] = __float_as_uint(v.x), g[c + 1] = __float_as_uint(v.y);
        }
      }
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float2 e = log2_p(c);
        const float2 d = f2_unpack(f2_mul(f2_pack(ex2_approx(e.x), ex2_approx(e.y)),
                                          f2_pack(__uint_as_float(g[c]), __uint_as_float(g[c + 1]))));
        s[c] = __float_as_uint(d.x), s[c + 1] = __float_as_uint(d.y);
      }
      if (__any_sync(0xffffffffu, valid < 64)) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c >= valid) s[c] = 0u;
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) s[c] = pack_bf16x2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
      tmem_st32(x, *reinterpret_cast<uint32_t(*)[32]>(s));
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&ds_full[j & 1]);
    }
    if (ok && n > 0) ok = mbar_wait_warp(done, 0, p.err);
    if (ok) {
      tc_fence_after();
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.dq) + (static_cast<int64_t>(doc.q0) + i) * p.a.dq_stride + head * kPkD + 64 * half;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32];
        if (n > 0) {
          tmem_ld32(Z + at + 64 * half + 32 * c, r);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int q = 0; q < 32; ++q) r[q] = 0u;
        }
        if (live) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 v;
            v.x = pack_bf16x2(__uint_as_float(r[8 * q]) * p.a.scale, __uint_as_float(r[8 * q + 1]) * p.a.scale);
            v.y = pack_bf16x2(__uint_as_float(r[8 * q + 2]) * p.a.scale, __uint_as_float(r[8 * q + 3]) * p.a.scale);
            v.z = pack_bf16x2(__uint_as_float(r[8 * q + 4]) * p.a.scale, __uint_as_float(r[8 * q + 5]) * p.a.scale);
            v.w = pack_bf16x2(__uint_as_float(r[8 * q + 6]) * p.a.scale, __uint_as_float(r[8 * q + 7]) * p.a.scale);
            reinterpret_cast<uint4*>(out + c * 32)[q] = v;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Query tiles (64 packed rows) of a document that see key tile `key0`, over the head groups of
// one key head: tile i of the walk is query tile first_tile + i % per_group of group
// i / per_group.
struct QueryWalk {
  int first_tile, per_group, n;
};
__device__ __forceinline__ QueryWalk query_walk(const DocRows& d, const BwdParams& p, int key0) {
  const int tiles = div_up(d.Lq, p.per_tile);
  const int f = first_query(key0, d.off, d.Lk, d.prefix, p.a.causal_block) / p.per_tile;
  const int per = f < tiles ? tiles - f : 0;
  return {f, per, per * (p.a.H / p.a.Hk / p.pack)};
}

template <bool kPlain>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dkv_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapO,
                         const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                         const __grid_constant__ BwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = smem;                      // K, then V
  uint8_t* sQ = sKV + 2 * kPkTileBytes;     // [kDkvStages]: Q_i (64 rows), dO_i
  uint8_t* stats = sQ + kDkvStages * 2 * kHalfBytes;  // [kStatBufs] per query: -log-sum, -delta (, slope, position), then keys seen
  uint64_t* bars = reinterpret_cast<uint64_t*>(stats + kStatBufs * kStatBytes);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;
  uint64_t* q_empty = q_full + kDkvStages;
  uint64_t* s_full = q_empty + kDkvStages;  // [2] S^T(i) and dP^T(i) are there (i & 1)
  uint64_t* p_full = s_full + 2;            // [2] p^T and ds^T are in place
  uint64_t* done = s_full + 4;
  uint64_t* ragged = s_full + 5;
  uint64_t* cleared = s_full + 6;
  uint64_t* st_full = s_full + 7;           // [kStatBufs]
  uint64_t* st_empty = st_full + kStatBufs;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(st_empty + kStatBufs);
  int* found = reinterpret_cast<int*>(st_empty + kStatBufs + 1);

  int di, tile;
  if (!cta_tile(p.a.cu_k, p.a.n_docs, p.a.k_rows, kPkTile, found, di, tile)) return;
  const DocRows doc = load_doc(p.a, di);
  const int key0 = tile * kPkTile, keys = min(kPkTile, doc.Lk - key0);
  const QueryWalk w = query_walk(doc, p, key0);
  const int used = p.per_tile * p.pack;     // rows of a tile that are queries
  const int last_rows = (doc.Lq - (div_up(doc.Lq, p.per_tile) - 1) * p.per_tile) * p.pack;  // of a document's last tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < kDkvStages; ++s) mbar_init(&q_full[s], 1), mbar_init(&q_empty[s], 1);
    for (int b = 0; b < 2; ++b) mbar_init(&s_full[b], 1), mbar_init(&p_full[b], kScoreThreads);
    mbar_init(done, 1);
    mbar_init(ragged, 1);
    mbar_init(cleared, 1);
    for (int b = 0; b < kStatBufs; ++b) mbar_init(&st_full[b], 1), mbar_init(&st_empty[b], kScoreThreads);
    fence_mbar_init();
  }
  // Rows that no copy writes take part in the sums over queries.
  if (used < 64 && warp >= 4 && warp < 4 + 2 * kDkvStages) zero_tile_rows<64>(sQ + (warp - 4) * kHalfBytes, used);
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // S^T(i) at 64 (i & 1), dP^T(i) 128 columns on
  const uint32_t tmem = *tmem_holder, dV = tmem + 256, dK = tmem + 384;
  const int hk = blockIdx.y, group0 = hk * (p.a.H / p.a.Hk / p.pack);

  if (warp == 0) {
    if (lane == 0 && w.n > 0) {
      mbar_arrive_expect_tx(kv_full, 2 * kPkTileBytes);
      for (int c = 0; c < 2; ++c) {
        tma_load_2d(sKV + c * kPkSpan, &mapK, kv_full, hk * kPkD + 64 * c, doc.k0 + key0);
        tma_load_2d(sKV + kPkTileBytes + c * kPkSpan, &mapV, kv_full, hk * kPkD + 64 * c, doc.k0 + key0);
      }
      int i = 0;
      for (; i < w.n; ++i) {
        const int stage = i % kDkvStages, g = i / w.per_group;
        if (!mbar_wait(&q_empty[stage], static_cast<uint32_t>((i / kDkvStages) & 1) ^ 1u, p.err)) break;
        mbar_arrive_expect_tx(&q_full[stage], 2 * static_cast<uint32_t>(used) * 256u);
        uint8_t* at = sQ + stage * 2 * kHalfBytes;
        const int y = (group0 + g) * p.pack, z = doc.q0 + (w.first_tile + i - g * w.per_group) * p.per_tile;
        for (int c = 0; c < 2; ++c) {
          tma_load_3d(at + c * kHalfSpan, &mapQ, &q_full[stage], 64 * c, y, z);
          tma_load_3d(at + kHalfBytes + c * kHalfSpan, &mapO, &q_full[stage], 64 * c, y, z);
        }
      }
      mbar_wait(kv_full, 0, p.err);  // every copy this thread started has landed before it leaves
      for (int s = 0; s < kDkvStages; ++s) {
        const int m = i / kDkvStages + (s < i % kDkvStages ? 1 : 0);
        if (m > 0) mbar_wait(&q_full[s], static_cast<uint32_t>((m - 1) & 1), p.err);
      }
    }
  } else if (warp == 1) {
    const int nu = uniform(w.n), per_group = uniform(w.per_group);
    if (nu > 0) {
      const uint32_t id_kk = idesc_bf16_f32(kPkTile, 64, 0, 0), id_mn = idesc_bf16_f32(kPkTile, kPkD, 0, 1);
      const uint32_t tm = uniform(tmem);
      const uint64_t k_desc = sdesc_sw128(smem_u32(sKV), 16, 1024), v_desc = sdesc_sw128(smem_u32(sKV + kPkTileBytes), 16, 1024);
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024), qt_desc = sdesc_sw128(smem_u32(sQ), kHalfSpan, 1024);
      int ragged_seen = 0;
      const bool ragged_end = uniform(last_rows) < used;
      // S^T(i) = K Q_i^T and dP^T(i) = V dO_i^T, once the tile is there and its rows behind the
      // document's end are cleared.
      auto scores = [&](int i) {
        const int stage = i % kDkvStages;
        if (!mbar_wait_warp(&q_full[stage], static_cast<uint32_t>((i / kDkvStages) & 1), p.err)) return false;
        if (ragged_end && (i + 1) % per_group == 0) {
          if (lane == 0) mbar_arrive(ragged);
          if (!mbar_wait_warp(cleared, static_cast<uint32_t>(ragged_seen++ & 1), p.err)) return false;
        }
        const uint64_t qd = q_desc + static_cast<uint32_t>((stage * 2 * kHalfBytes) >> 4);
        const uint64_t od = qd + (kHalfBytes >> 4);
        const uint32_t to = tm + 64 * (i & 1);
        if (elect_lane()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_bf16(to, k_desc + (((k >> 2) * kPkSpan + (k & 3) * 32) >> 4), qd + (((k >> 2) * kHalfSpan + (k & 3) * 32) >> 4),
                        id_kk, k > 0 ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_bf16(to + 128, v_desc + (((k >> 2) * kPkSpan + (k & 3) * 32) >> 4),
                        od + (((k >> 2) * kHalfSpan + (k & 3) * 32) >> 4), id_kk, k > 0 ? 1u : 0u);
          tc_commit(&s_full[i & 1]);
        }
        return true;
      };
      bool ok = mbar_wait_warp(kv_full, 0, p.err) && scores(0);
      if (ok && nu > 1) ok = scores(1);
      for (int i = 0; ok && i < nu; ++i) {
        if (!mbar_wait_warp(&p_full[i & 1], static_cast<uint32_t>((i >> 1) & 1), p.err)) break;
        tc_fence_after();
        const int stage = i % kDkvStages;
        const uint64_t qd = qt_desc + static_cast<uint32_t>((stage * 2 * kHalfBytes) >> 4), od = qd + (kHalfBytes >> 4);
        const uint32_t from = tm + 64 * (i & 1);
        if (elect_lane()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_bf16_ts(tm + 256, from + (k >> 1) * 32 + (k & 1) * 8, od + ((k * 16 * 128) >> 4), id_mn, (i > 0 || k > 0) ? 1u : 0u);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_bf16_ts(tm + 384, from + 16 + (k >> 1) * 32 + (k & 1) * 8, qd + ((k * 16 * 128) >> 4), id_mn,
                           (i > 0 || k > 0) ? 1u : 0u);
          tc_commit(&q_empty[stage]);
        }
        if (i + 2 < nu) ok = scores(i + 2);
      }
      if (elect_lane()) tc_commit(done);
      mbar_wait_warp(done, 0, p.err);
    }
  } else if (warp == 2) {
    // The numbers of each query tile's columns. A column of no query, and a query that sees
    // nothing, get p = 2^(s - infinity) = 0. Four tiles' loads are in flight (with one, this
    // warp held up all others: 786 us against 465).
    float lse[kStatBufs][2], delta[kStatBufs][2];
    int place[2], in_tile[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int m = c * 32 + lane;
      in_tile[c] = m / p.pack;
      place[c] = m - in_tile[c] * p.pack;
      if (in_tile[c] >= p.per_tile) in_tile[c] = 1 << 30;  // no query
    }
    int fetch_tile = 0, fetch_group = 0;  // the next tile to fetch
    auto fetch = [&](float (&l)[2], float (&d)[2]) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int64_t q = static_cast<int64_t>(w.first_tile + fetch_tile) * p.per_tile + in_tile[c];
        l[c] = -INFINITY, d[c] = 0.f;
        if (q < doc.Lq) {
          const int64_t stat = static_cast<int64_t>((group0 + fetch_group) * p.pack + place[c]) * p.a.q_rows + doc.q0 + q;
          l[c] = p.a.lse[stat], d[c] = p.a.delta[stat];
        }
      }
      if (++fetch_tile == w.per_group) fetch_tile = 0, ++fetch_group;
    };
#pragma unroll
    for (int u = 0; u < kStatBufs; ++u)
      if (u < w.n) fetch(lse[u], delta[u]);
    int tile_i = 0, group_i = 0;
    bool ok = true;
    for (int i0 = 0; ok && i0 < w.n; i0 += kStatBufs) {
#pragma unroll
      for (int u = 0; u < kStatBufs; ++u) {
        const int i = i0 + u;
        if (!ok || i >= w.n) continue;
        uint8_t* st = stats + u * kStatBytes;
        if (i0 > 0 && !mbar_wait_warp(&st_empty[u], static_cast<uint32_t>((i0 / kStatBufs - 1) & 1), p.err)) {
          ok = false;
          continue;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int m = c * 32 + lane;
          const int64_t q = static_cast<int64_t>(w.first_tile + tile_i) * p.per_tile + in_tile[c];
          const bool there = q < doc.Lq, sees = lse[u][c] != -INFINITY;
          const float nl = sees ? -lse[u][c] * kLog2e : -INFINITY, nd = sees ? -delta[u][c] : 0.f;
          if (kPlain) {
            reinterpret_cast<float2*>(st)[m] = make_float2(nl, nd);
          } else {
            const float slope2 = p.a.slopes && there ? __ldg(p.a.slopes + (group0 + group_i) * p.pack + place[c]) * kLog2e : 0.f;
            reinterpret_cast<float4*>(st)[m] =
                make_float4(nl, nd, slope2, there ? static_cast<float>(static_cast<int>(q) + doc.off - key0) : 0.f);
          }
          reinterpret_cast<int*>(st + 64 * 16)[m] =
              there ? seen_keys(static_cast<int>(q), doc.off, doc.Lk, doc.prefix, p.a.causal_block) : 0;
        }
        if (++tile_i == w.per_group) tile_i = 0, ++group_i;
        if (i + kStatBufs < w.n) fetch(lse[u], delta[u]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&st_full[u]);
      }
    }
  } else if (warp == 3) {
    if (last_rows < used) {
      int k = 0;
      for (int i = w.per_group - 1; w.per_group > 0 && i < w.n; i += w.per_group, ++k) {
        if (!mbar_wait_warp(ragged, static_cast<uint32_t>(k & 1), p.err)) break;
        zero_tile_rows<64>(sQ + i % kDkvStages * 2 * kHalfBytes, last_rows);
        zero_tile_rows<64>(sQ + i % kDkvStages * 2 * kHalfBytes + kHalfBytes, last_rows);
        if (lane == 0) mbar_arrive(cleared);
      }
    }
  } else {
    const int half = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t at = (static_cast<uint32_t>((warp & 3) * 32) << 16) + 32 * half;
    const bool live = row < keys;
    bool ok = true;
    for (int i = 0; i < w.n; ++i) {
      const int b = i % kStatBufs;
      if (!mbar_wait_warp(&st_full[b], static_cast<uint32_t>((i / kStatBufs) & 1), p.err) ||
          !mbar_wait_warp(&s_full[i & 1], static_cast<uint32_t>((i >> 1) & 1), p.err)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t x = tmem + 64 * (i & 1) + at;
      uint32_t s[32], g[32];
      tmem_ld32(x, s);
      tmem_ld32(x + 128, g);
      tmem_ld_wait();
      const uint8_t* st = stats + b * kStatBytes;
      if (!kPlain && p.a.cap > 0.f) cap_scores(s, p.cap_in, live);
      const unsigned long long mult2 = f2_splat(p.mult);
      const float key = static_cast<float>(row);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float2 nl, nd;
        const unsigned long long t = f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        if constexpr (kPlain) {
          const float4 v = reinterpret_cast<const float4*>(st)[16 * half + (c >> 1)];
          nl = make_float2(v.x, v.z), nd = make_float2(v.y, v.w);
        } else {
          const float4 v0 = reinterpret_cast<const float4*>(st)[32 * half + c], v1 = reinterpret_cast<const float4*>(st)[32 * half + c + 1];
          nl = make_float2(v0.x - v0.z * fabsf(v0.w - key), v1.x - v1.z * fabsf(v1.w - key)), nd = make_float2(v0.y, v1.y);
        }
        const float2 e = f2_unpack(f2_fma(t, mult2, f2_pack(nl.x, nl.y)));
        unsigned long long d = f2_add(f2_pack(__uint_as_float(g[c]), __uint_as_float(g[c + 1])), f2_pack(nd.x, nd.y));
        if (!kPlain && p.a.cap > 0.f) d = f2_mul(d, f2_fma(f2_mul(t, f2_splat(-1.f)), t, f2_splat(1.f)));
        const float e0 = ex2_approx(e.x), e1 = ex2_approx(e.y);
        const float2 v = f2_unpack(f2_mul(f2_pack(e0, e1), d));
        s[c] = __float_as_uint(e0), s[c + 1] = __float_as_uint(e1);
        g[c] = __float_as_uint(v.x), g[c + 1] = __float_as_uint(v.y);
      }
      if (p.a.causal_block > 0) {
        // queries see ever more keys: the tile's first column decides whether any is masked
        const int* seen = reinterpret_cast<const int*>(st + 64 * 16);
        if (seen[0] < key0 + keys) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (key0 + row >= seen[32 * half + c]) s[c] = 0u, g[c] = 0u;
        }
      }
      mbar_arrive(&st_empty[b]);
      uint32_t out[32];  // p^T, then ds^T, over this half of S^T
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        out[c] = pack_bf16x2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
        out[16 + c] = pack_bf16x2(__uint_as_float(g[2 * c]), __uint_as_float(g[2 * c + 1]));
      }
      tmem_st32(x, out);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[i & 1]);
    }
    if (ok && w.n > 0) ok = mbar_wait_warp(done, 0, p.err);
    if (ok) {
      tc_fence_after();
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const int64_t key_row = static_cast<int64_t>(doc.k0) + key0 + row;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {  // two quarters of dV, two of dK
        uint32_t r[32];
        const int col = 64 * half + 32 * (c & 1);
        if (w.n > 0) {
          tmem_ld32((c < 2 ? dV : dK) + lanes + col, r);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int q = 0; q < 32; ++q) r[q] = 0u;
        }
        if (live) {
          const float f = c < 2 ? 1.0f : p.a.scale;
          __nv_bfloat16* out = c < 2 ? static_cast<__nv_bfloat16*>(p.a.dv) + key_row * p.a.dv_stride
                                     : static_cast<__nv_bfloat16*>(p.a.dk) + key_row * p.a.dk_stride;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 v;
            v.x = pack_bf16x2(__uint_as_float(r[8 * q]) * f, __uint_as_float(r[8 * q + 1]) * f);
            v.y = pack_bf16x2(__uint_as_float(r[8 * q + 2]) * f, __uint_as_float(r[8 * q + 3]) * f);
            v.z = pack_bf16x2(__uint_as_float(r[8 * q + 4]) * f, __uint_as_float(r[8 * q + 5]) * f);
            v.w = pack_bf16x2(__uint_as_float(r[8 * q + 6]) * f, __uint_as_float(r[8 * q + 7]) * f);
            reinterpret_cast<uint4*>(out + hk * kPkD + col)[q] = v;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

int launch_attn_packed_tc_bwd(const PackedAttn& a, cudaStream_t s) {
  BwdParams p{};
  p.a = a;
  p.pack = packed_heads_per_tile(a.H, a.Hk);
  p.per_tile = kPkTile / p.pack;
  p.groups = a.H / p.pack;
  p.mult = (a.cap > 0.f ? a.cap : a.scale) * kLog2e;
  p.cap_in = a.cap > 0.f ? a.scale / a.cap : 0.f;
  p.err = device_error_flag();
  int dev = 0;
  cudaGetDevice(&dev);
  static std::once_flag once[64];
  std::call_once(once[dev & 63], [] {
    for (auto kernel : {packed_dq_tc_kernel<true>, packed_dq_tc_kernel<false>})
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kDqSmem));
    for (auto kernel : {packed_dkv_tc_kernel<true>, packed_dkv_tc_kernel<false>})
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kDkvSmem));
  });
  BwdParams p2 = p;  // the keys' kernel: query tiles of 64 rows
  p2.pack = packed_heads_per_tile(a.H, a.Hk, 64);
  p2.per_tile = 64 / p2.pack;
  p2.groups = a.H / p2.pack;
  CUtensorMap mq, mo, mk, mv, mq2, mo2;
  // without queries (or keys) none is loaded: any valid map will do
  const bool qs = a.q_rows > 0, ks = a.k_rows > 0;
  if (!make_packed_kv_map(&mk, ks ? a.k : a.q, ks ? a.k_stride : a.q_stride, ks ? a.k_rows : 1, a.Hk) ||
      !make_packed_kv_map(&mv, ks ? a.v : a.q, ks ? a.v_stride : a.q_stride, ks ? a.k_rows : 1, a.Hk))
    return WAN_ERR_CUDA;
  if (!qs) {
    mq = mo = mq2 = mo2 = mk;
  } else if (!make_packed_q_map(&mq, a.q, a.q_stride, a.q_rows, a.H, p.pack) ||
             !make_packed_q_map(&mo, a.d_o, a.do_stride, a.q_rows, a.H, p.pack) ||
             !make_packed_q_map(&mq2, a.q, a.q_stride, a.q_rows, a.H, p2.pack, 64) ||
             !make_packed_q_map(&mo2, a.d_o, a.do_stride, a.q_rows, a.H, p2.pack, 64)) {
    return WAN_ERR_CUDA;
  }
  const bool plain = a.cap == 0.f && !a.slopes;
  // every document adds less than one partial tile
  if (qs) {
    const dim3 grid(static_cast<unsigned>(a.q_rows / p.per_tile + a.n_docs), static_cast<unsigned>(p.groups));
    (plain ? packed_dq_tc_kernel<true> : packed_dq_tc_kernel<false>)<<<grid, kThreads, kDqSmem, s>>>(mq, mo, mk, mv, p);
    count_launches(1);
    const int st = check_launch();
    if (st != WAN_OK) return st;
  }
  if (ks) {
    const dim3 grid(static_cast<unsigned>(a.k_rows / kPkTile + a.n_docs), static_cast<unsigned>(a.Hk));
    (plain ? packed_dkv_tc_kernel<true> : packed_dkv_tc_kernel<false>)<<<grid, kThreads, kDkvSmem, s>>>(mq2, mo2, mk, mv, p2);
    count_launches(1);
    return check_launch();
  }
  return WAN_OK;
}

}  // namespace wan
