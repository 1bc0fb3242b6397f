// Attention inside packed documents on the sm_100a tensor cores (bf16, head_dim 128):
// o = softmax(s) v over each query's seen keys, one pass over the keys with a running
// maximum and sum, and the log-sum for the gradient.
//
// A unit of work is two 128-row query tiles of one document and head group (see
// packed_tc.cuh) against the document's keys. A CTA's warps share it as follows (384
// threads, one CTA per SM, looping over its work):
//   warp 0   : TMA loads: both Q tiles, then K_0, K_1, V_0, K_2, V_1, ... through a
//              5-stage ring of 32 KB tiles;
//   warp 1   : tcgen05.mma, issued by one lane: for key tile j and query tile t,
//              O_t += P_t(j-1) V_{j-1} with P from tensor memory, then S_t = Q_t K_j^T;
//   warp 3   : finds this CTA's share of the work, later clears ragged V tiles; warp 2 notes
//              where the share ends;
//   warps 4-7, 8-11: softmax of tile 0 and tile 1, a thread per row: the row's 128 scores
//              come from TMEM at once; cap, distance and mask passes run over them only
//              where the call, or the tile, has any; P goes back over S in bf16 (the
//              operand's rounding; sums stay fp32), and the product over its first 96 keys
//              starts while the last 32 are still formed (1.78 M clocks without, 1.67 M
//              with 64 + 64, 1.62 M so, 14,080 rows of 12 heads). The base of the
//              exponentials moves only when the row maximum grew by more than 2^8.
// While one tile's softmax runs, the tensor core works on the other's products. What bounds it
// is that chain: about 3,300 clocks per key tile for 2,048 of tensor work and as many of
// exponentials. 4 clips of 23,400 rows, 12 heads: 1.36 to 1.38 ms, 1080 TFLOP/s under the power cap; 8
// single tokens over 117 k keys, 12/4 heads: 71 us, 3.4 TB/s.
//
// Whole waves of equal units (a document's, as many as there are CTAs) come first. What they
// leave is cut by key tiles: of T key tiles (and unit costs), CTA c of C takes
// [T c / C, T (c+1) / C), so that any mix of document lengths, orders of keys and few queries
// over many keys load the SMs alike. A unit cut between CTAs leaves unnormalised outputs with
// their base and sum in the workspace, merged in CTA order by a second kernel (nothing depends
// on timing). Units of up to 8 key tiles, and all units when there is no workspace, stay whole
// in the CTA in which they begin.
//
// Keys behind a document's end are masked by position, and their V rows, which belong to
// other documents or to none, are cleared in shared memory before the product.
#include <math.h>

#include <mutex>

#include "internal.h"
#include "packed_tc.cuh"

namespace wan {
namespace {

constexpr int kRegsLow = 88;    // warps 0-3
constexpr int kRegsHigh = 208;  // softmax warps: a whole score row in registers
static_assert(128 * kRegsLow + 256 * kRegsHigh <= 384 * 168, "register split above the launch");
constexpr int kThreads = 384;
constexpr int kStages = 5;
constexpr int kMaxCtas = 148;
// A unit of more key tiles may be cut: a cut costs its parts' way through memory (ragged texts
// 86 us with 2 against 73; single tokens over long keys 69 with 2, 71 with 8, 82 with 16).
constexpr int kMinSplit = 8;
constexpr int kMinShare = 4;         // key tiles a CTA takes at least (12: ragged texts 82 us)
constexpr int kUnitCost = 2;         // see unit_weight
constexpr float kRescaleLog2 = 8.0f;
constexpr int kPolyEvery = 8;        // one pair of exponentials in this many runs on the FMA pipes
constexpr size_t kSmem = 1024 + static_cast<size_t>(kPkTileBytes) * (2 + kStages) + 2048;
static_assert(kSmem <= 232448, "shared memory of an SM");

// Where a CTA's share ends inside a unit that begins in it: what the merge needs.
struct Cut {
  int crosses, first_slot, last_cta, row0, rows, group;
};

template <bool kV>
struct BoolConstant {
  static constexpr bool value = kV;
};

struct FwdParams {
  PackedAttn a;
  int pack, per_tile, groups;   // heads per tile, queries per tile, head groups
  int ctas, may_split, slot_rows;
  float mult;                   // log2 units per (possibly capped) score
  float cap_in;                 // scale / cap (cap > 0)
  int prescale;                 // slopes, or a negative scale: scores are scaled before the maximum
  float* part_o;                // [2 ctas][slot_rows][128]
  float2* part_ml;              // [2 ctas][slot_rows]: base (log2 units), sum
  Cut* cuts;                    // [ctas]
  int* err;
};

// ------------------------------------------------------------------ the share of a CTA
__device__ __forceinline__ int tiles_seen(const DocRows& d, const FwdParams& p, int first, int count) {
  const int last = min(first + count, d.Lq) - 1;  // rows see ever more keys
  return div_up(seen_keys(last, d.off, d.Lk, d.prefix, p.a.causal_block), kPkTile);
}
// Key tiles of unit `u` (pair of query tiles) of a document; a unit that sees none counts
// as one, it still writes its rows.
__device__ __forceinline__ int unit_tiles(const DocRows& d, const FwdParams& p, int u) {
  return max(1, tiles_seen(d, p, u * 2 * p.per_tile, 2 * p.per_tile));
}

// A unit's weight in the shares: loading Q, the first scores and the output cost about as much
// as two key tiles (texts of 1 to 4 tiles: without it some CTAs took three times the work).
__device__ __forceinline__ int unit_weight(const DocRows& d, const FwdParams& p, int u) { return unit_tiles(d, p, u) + kUnitCost; }

template <typename T>
__device__ __forceinline__ T warp_incl_scan(T v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// Units of a document, in the order (head group, pair of query tiles), and how many of them
// are taken in waves: every CTA one unit at a time, so that all CTAs read the same keys at the
// same time (measured 15 % faster on 14,080-row documents than consecutive units per CTA).
// Only documents whose units are all alike have waves.
__device__ __forceinline__ int doc_pairs(const DocRows& d, const FwdParams& p) { return div_up(d.Lq, 2 * p.per_tile); }
__device__ __forceinline__ int doc_waves(const DocRows& d, const FwdParams& p) {
  return p.a.causal_block == 0 ? doc_pairs(d, p) * p.groups / p.ctas : 0;
}

constexpr int kWaveDocs = 32;  // documents with waves (the first ones; more are shared out by key tiles)
struct Share {
  int64_t s, e;   // this CTA's part of what the waves leave, in key tiles and unit costs
  int64_t total;  // all of it
  int64_t at;     // first key tile of the unit below
  int ctas;       // CTAs that share it
  int doc, unit;
  int n_wave, wave_doc[kWaveDocs];
  __device__ bool in_waves(int d) const { return n_wave < kWaveDocs || d <= wave_doc[kWaveDocs - 1]; }
};

// Key tiles that the waves leave of the lane's document d0 + lane (whole warp; past the last
// document: 0). `n_wave`: documents with waves before d0, updated; listed in `list` if given.
__device__ int64_t doc_left(const FwdParams& p, int d0, int& n_wave, int* list) {
  const int lane = threadIdx.x & 31, d = d0 + lane;
  int64_t w = 0;
  int waves = 0;
  bool walk = false;
  DocRows doc{};
  if (d < p.a.n_docs) {
    doc = load_doc(p.a, d);
    const int pairs = doc_pairs(doc, p);
    waves = doc_waves(doc, p);
    if (pairs > 8 && p.a.causal_block > 0) {
      walk = true;
    } else if (pairs > 0) {
      int64_t one = 0;
      if (p.a.causal_block == 0)
        one = static_cast<int64_t>(pairs) * unit_weight(doc, p, 0);
      else
        for (int u = 0; u < pairs; ++u) one += unit_weight(doc, p, u);
      w = one * p.groups;
    }
  }
  const unsigned has = __ballot_sync(0xffffffffu, waves > 0);
  const int rank = n_wave + __popc(has & ((1u << lane) - 1u));
  if (waves > 0 && rank < kWaveDocs) {
    w -= static_cast<int64_t>(waves) * p.ctas * unit_weight(doc, p, 0);
    if (list) list[rank] = d;
  }
  n_wave = min(n_wave + __popc(has), kWaveDocs);
  for (unsigned todo = __ballot_sync(0xffffffffu, walk); todo; todo &= todo - 1) {
    const int src = __ffs(todo) - 1;
    const DocRows x = load_doc(p.a, d0 + src);
    const int n = doc_pairs(x, p);
    int64_t s = 0;
    for (int u = lane; u < n; u += 32) s += unit_weight(x, p, u);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == src) w = s * p.groups;
  }
  return w;
}

// By one warp; `out` in shared memory.
__device__ void find_share(const FwdParams& p, Share& out) {
  const int lane = threadIdx.x & 31;
  int n_wave = 0;
  int64_t total = 0;
  for (int d0 = 0; d0 < p.a.n_docs; d0 += 32)
    total += __shfl_sync(0xffffffffu, warp_incl_scan(doc_left(p, d0, n_wave, out.wave_doc)), 31);
  const int64_t most = total / kMinShare;
  const int ctas = most < 1 ? 1 : (most < p.ctas ? static_cast<int>(most) : p.ctas);
  const int c = blockIdx.x;
  const int64_t s = c < ctas ? total * c / ctas : total, e = c < ctas ? total * (c + 1) / ctas : total;
  if (lane == 0) out.n_wave = n_wave, out.total = total, out.ctas = ctas, out.s = s, out.e = e;
  __syncwarp();
  if (s >= e) return;
  int64_t left = s, at = 0;
  int doc_i = 0, unit = 0;
  n_wave = 0;
  for (int d0 = 0;; d0 += 32) {
    const int64_t w = doc_left(p, d0, n_wave, nullptr), incl = warp_incl_scan(w), sum = __shfl_sync(0xffffffffu, incl, 31);
    if (left >= sum) {
      left -= sum, at += sum;
      continue;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, left < incl)) - 1;
    const int64_t before = __shfl_sync(0xffffffffu, incl - w, src);
    doc_i = d0 + src;
    left -= before, at += before;
    break;
  }
  const DocRows doc = load_doc(p.a, doc_i);
  const int pairs = doc_pairs(doc, p);
  if (p.a.causal_block == 0) {
    const int n = unit_weight(doc, p, 0), k = static_cast<int>(left / n);
    unit = k + (out.in_waves(doc_i) ? doc_waves(doc, p) * p.ctas : 0);
    at += static_cast<int64_t>(k) * n;
  } else {
    int64_t one = 0;
    for (int u0 = 0; u0 < pairs; u0 += 32)
      one += __shfl_sync(0xffffffffu, warp_incl_scan(static_cast<int64_t>(u0 + lane < pairs ? unit_weight(doc, p, u0 + lane) : 0)), 31);
    const int group = static_cast<int>(left / one);
    left -= one * group, at += one * group;
    for (int u0 = 0;; u0 += 32) {
      const int64_t w = u0 + lane < pairs ? unit_weight(doc, p, u0 + lane) : 0, incl = warp_incl_scan(w);
      const int64_t sum = __shfl_sync(0xffffffffu, incl, 31);
      if (left >= sum) {
        left -= sum, at += sum;
        continue;
      }
      const int src = __ffs(__ballot_sync(0xffffffffu, left < incl)) - 1;
      unit = group * pairs + u0 + src;
      at += __shfl_sync(0xffffffffu, incl - w, src);
      break;
    }
  }
  if (lane == 0) out.at = at, out.doc = doc_i, out.unit = unit;
}

// One piece of a CTA's work: key tiles [k0, k0 + nmax) of a unit.
struct Piece {
  int group, first;     // head group, first query row of the unit
  int k0, n[2], nmax;   // key tiles of each query tile from key tile k0 on
  bool whole, begins;   // the unit is not cut; the piece holds its beginning
  int slot;             // partial results of a cut unit
  int unit_end;         // the unit's end, relative to the share
};

// Walks the pieces of a CTA in order: its unit of every wave, then its share of the rest. The
// walk lives in shared memory, one per warp, so that it holds no registers of the softmax loop
// (where every one counts). Positions are relative to the share's first key tile.
struct Walk {
  int wave_doc, wave;  // next wave
  int at, end, weight;  // unit's first key tile, the share's end, the unit's weight (0: none yet)
  int doc, unit;
  DocRows d;           // document of the piece
  Piece x;
};
__device__ __forceinline__ void walk_begin(Walk& w, const Share& s) {
  w.wave_doc = w.wave = 0;
  w.end = static_cast<int>(s.e - s.s), w.weight = 0;
  w.at = w.end > 0 ? static_cast<int>(s.at - s.s) : 0;
  w.doc = s.doc, w.unit = s.unit - 1;
}
// Piece [a, b) of the key tiles of unit `unit` of document d, which has n.
__device__ __forceinline__ void make_piece(Piece& x, const DocRows& d, const FwdParams& p, int unit, int a, int b, int n) {
  const int pairs = doc_pairs(d, p), group = unit / pairs;
  x.group = group, x.first = (unit - group * pairs) * 2 * p.per_tile;
  x.k0 = a;
  int most = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int f = x.first + t * p.per_tile;
    const int nt = f < d.Lq ? max(0, min(tiles_seen(d, p, f, p.per_tile), b) - a) : 0;
    x.n[t] = nt;
    most = max(most, nt);
  }
  x.nmax = most;
  x.whole = a == 0 && b == n;
  x.begins = a == 0;
}
// By one thread: the next piece, or false.
__device__ __forceinline__ bool walk_step(Walk& w, const FwdParams& p, const Share& s) {
  for (; w.wave_doc < s.n_wave; ++w.wave_doc, w.wave = 0) {
    const DocRows d = load_doc(p.a, s.wave_doc[w.wave_doc]);
    if (w.wave < doc_waves(d, p)) {
      const int n = unit_tiles(d, p, 0);
      make_piece(w.x, d, p, w.wave++ * p.ctas + static_cast<int>(blockIdx.x), 0, n, n);
      w.d = d;
      return true;
    }
  }
  int at = w.at, weight = w.weight, unit = w.unit;
  if (at + weight >= w.end) return false;
  DocRows d = load_doc(p.a, w.doc);
  while (at + weight < w.end) {
    at += weight;
    ++unit;
    while (unit >= doc_pairs(d, p) * p.groups) {
      d = load_doc(p.a, ++w.doc);
      unit = s.in_waves(w.doc) ? doc_waves(d, p) * p.ctas : 0;
    }
    const int n = unit_tiles(d, p, unit % doc_pairs(d, p));
    weight = n + kUnitCost;  // the cost lies behind the key tiles
    const bool may_cut = p.may_split && n > kMinSplit;
    int a = 0, b = n;
    bool mine = at >= 0;
    if (may_cut) {
      a = max(0, -at);
      b = min(n, w.end - at);
      mine = a < b;
    }
    if (!mine) continue;
    make_piece(w.x, d, p, unit, a, b, n);
    w.x.slot = 2 * static_cast<int>(blockIdx.x) + (at <= 0 ? 0 : 1);  // the share's first piece, or its last
    w.x.unit_end = at + n;
    w.at = at, w.weight = weight, w.unit = unit, w.d = d;
    return true;
  }
  w.at = at, w.weight = weight;
  return false;
}
// The same for a whole warp. The barriers order the other lanes' reads of the piece before with
// lane 0's writes, and those with the reads that follow: a shuffle alone orders no memory.
__device__ __forceinline__ bool walk_next(Walk& w, const FwdParams& p, const Share& s) {
  __syncwarp();
  bool more = false;
  if ((threadIdx.x & 31) == 0) more = walk_step(w, p, s);
  __syncwarp();
  return __shfl_sync(0xffffffffu, more, 0);
}

// Ring position of K_j / V_j in the load order K_0, K_1, V_0, K_2, V_1, ..., V_{n-1}.
__device__ __forceinline__ int pos_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int pos_v(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

// kPlain: scores are neither capped nor scaled before their maximum. The passes for those
// cost registers even where a call skips them (each instance spills a little: 4 bytes the plain
// one, 12 the other).
template <bool kPlain>
__global__ void __launch_bounds__(kThreads, 1)
    packed_fwd_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                         const __grid_constant__ CUtensorMap mapV, const __grid_constant__ FwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                        // [2][tile]
  uint8_t* sKV = sQ + 2 * kPkTileBytes;      // [kStages][tile]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + kStages * kPkTileBytes);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* kv_full = bars + 2;
  uint64_t* kv_empty = kv_full + kStages;
  uint64_t* s_full = kv_empty + kStages;     // [2]
  uint64_t* p_full = s_full + 2;             // [2]
  uint64_t* p_half = p_full + 2;             // [2]: its first 96 columns
  uint64_t* o_final = p_half + 2;            // [2]
  uint64_t* ragged = o_final + 2;            // a ragged V tile has landed; its end is cleared
  uint64_t* cleared = ragged + 1;
  uint64_t* drain = ragged + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  Share* share = reinterpret_cast<Share*>(drain + 2);

  static_assert(24 * 8 + sizeof(Share) + 12 * sizeof(Walk) <= 2048, "barriers and walks");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 128);
      mbar_init(&p_half[t], 128);
      mbar_init(&o_final[t], 1);
    }
    mbar_init(ragged, 1);
    mbar_init(cleared, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&mapQ);
    tma_prefetch_desc(&mapK);
    tma_prefetch_desc(&mapV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == 3) find_share(p, *share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  Walk& walk = reinterpret_cast<Walk*>(share + 1)[warp];
  const Piece& x = walk.x;
  const DocRows& doc = walk.d;
  if (lane == 0) walk_begin(walk, *share);

  if (warp < 4) {
    setmaxnreg_dec<kRegsLow>();
    if (warp == 0) {
      if (lane == 0) {
        int issued = 0, q_loads = 0;
        bool ok = true;
        const uint32_t q_bytes = static_cast<uint32_t>(p.per_tile * p.pack) * 256u;
        while (ok && walk_step(walk, p, *share)) {
          if (x.nmax == 0) continue;
          if (q_loads > 0 && !mbar_wait(q_empty, static_cast<uint32_t>((q_loads - 1) & 1), p.err)) break;
          mbar_arrive_expect_tx(q_full, q_bytes * ((x.n[0] > 0) + (x.n[1] > 0)));
          for (int t = 0; t < 2; ++t)
            if (x.n[t] > 0)
              for (int c = 0; c < 2; ++c)
                tma_load_3d(sQ + t * kPkTileBytes + c * kPkSpan, &mapQ, q_full, 64 * c, x.group * p.pack,
                            doc.q0 + x.first + t * p.per_tile);
          ++q_loads;
          const int nmax = x.nmax, key_row = doc.k0 + x.k0 * kPkTile;
          const int col = x.group * p.pack / (p.a.H / p.a.Hk) * kPkD;
          const int n_loads = 2 * nmax;
          for (int ld = 0; ld < n_loads; ++ld) {
            const int stage = issued % kStages;
            if (!mbar_wait(&kv_empty[stage], static_cast<uint32_t>((issued / kStages) & 1) ^ 1u, p.err)) {
              ok = false;
              break;
            }
            const bool is_v = ld == n_loads - 1 || (ld > 0 && !(ld & 1));
            const int j = is_v ? (ld == n_loads - 1 ? nmax - 1 : (ld >> 1) - 1) : (ld + 1) >> 1;
            mbar_arrive_expect_tx(&kv_full[stage], kPkTileBytes);
            for (int c = 0; c < 2; ++c)
              tma_load_2d(sKV + stage * kPkTileBytes + c * kPkSpan, is_v ? &mapV : &mapK, &kv_full[stage], col + 64 * c,
                          key_row + j * kPkTile);
            ++issued;
          }
        }
        // Wait for every copy this thread started (the last fill of each buffer and stage).
        if (q_loads > 0) mbar_wait(q_full, static_cast<uint32_t>((q_loads - 1) & 1), p.err);
        for (int s = 0; s < kStages; ++s) {
          const int n_s = issued / kStages + (s < issued % kStages ? 1 : 0);
          if (n_s > 0) mbar_wait(&kv_full[s], static_cast<uint32_t>((n_s - 1) & 1), p.err);
        }
      }
    } else if (warp == 1) {
      const uint32_t idesc_qk = idesc_bf16_f32(kPkTile, kPkTile, 0, 0), idesc_pv = idesc_bf16_f32(kPkTile, kPkD, 0, 1);
      const uint32_t tm = uniform(tmem_base);
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(sKV), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(sKV), kPkSpan, 1024);
      auto wait_pos = [&](int pos) {
        return mbar_wait_warp(&kv_full[pos % kStages], static_cast<uint32_t>((pos / kStages) & 1), p.err);
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_lane()) tc_commit(bar);
      };
      auto qk = [&](int t, int stage) {
        const uint64_t qd = q_desc + static_cast<uint32_t>((t * kPkTileBytes) >> 4);
        const uint64_t kd = k_desc + static_cast<uint32_t>((stage * kPkTileBytes) >> 4);
        if (elect_lane()) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t off = ((k >> 2) * kPkSpan + (k & 3) * 32) >> 4;
            tc_mma_bf16(tm + t * kPkTile, qd + off, kd + off, idesc_qk, k > 0 ? 1u : 0u);
          }
          tc_commit(&s_full[t]);
        }
      };
      int base = 0, units = 0, ragged_seen = 0;
      uint32_t seen0 = 0, seen1 = 0;  // key tiles whose P was waited for
      // O_t += P_t V. The first product of a piece overwrites O_t: the softmax threads read
      // the piece before out of it before they arrived on p_full for this one.
      auto next_pv = [&](int t, uint32_t& seen, bool first, int stage) {
        const uint64_t vd = v_desc + static_cast<uint32_t>((stage * kPkTileBytes) >> 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!mbar_wait_warp(h == 0 ? &p_half[t] : &p_full[t], seen & 1u, p.err)) return false;
          tc_fence_after();
          if (elect_lane()) {
#pragma unroll
            for (int k = 6 * h; k < 6 + 2 * h; ++k)
              tc_mma_bf16_ts(tm + 256 + t * kPkTile, tm + t * kPkTile + k * 8, vd + ((k * 16 * 128) >> 4), idesc_pv,
                             (!first || k > 0) ? 1u : 0u);
          }
        }
        ++seen;
        return true;
      };
      bool ok = true;
      while (ok && walk_next(walk, p, *share)) {
        const int nmax = uniform(x.nmax), n0 = uniform(x.n[0]), n1 = uniform(x.n[1]);
        if (nmax == 0) continue;
        if (!mbar_wait_warp(q_full, static_cast<uint32_t>(units & 1), p.err)) break;
        ++units;
        for (int j = 0; j < nmax; ++j) {
          const int pk = base + pos_k(j), pvp = base + pos_v(j - 1, nmax);
          const int ks = pk % kStages, vs = pvp % kStages;
          ok = wait_pos(pk) && (j == 0 || wait_pos(pvp));
          if (!ok) break;
          if (j > 0 && j <= n0) {
            ok = next_pv(0, seen0, j == 1, vs);
            if (!ok) break;
            if (j == n0) commit(&o_final[0]);  // tile 0 ends before tile 1
          }
          if (j < n0) qk(0, ks);
          if (j > 0 && j <= n1) {
            ok = next_pv(1, seen1, j == 1, vs);
            if (!ok) break;
            if (j == n1) commit(&o_final[1]);
          }
          if (j < n1) qk(1, ks);
          commit(&kv_empty[ks]);
          if (j > 0) commit(&kv_empty[vs]);
        }
        if (!ok) break;
        commit(q_empty);
        const int pvp = base + pos_v(nmax - 1, nmax), vs = pvp % kStages;
        if (!wait_pos(pvp)) break;
        if (uniform(doc.Lk - (x.k0 + nmax - 1) * kPkTile) < kPkTile) {
          if (lane == 0) mbar_arrive(ragged);
          if (!mbar_wait_warp(cleared, static_cast<uint32_t>(ragged_seen & 1), p.err)) break;
          ++ragged_seen;
        }
        if (n0 == nmax) {
          ok = next_pv(0, seen0, nmax == 1, vs);
          if (!ok) break;
          commit(&o_final[0]);
        }
        if (n1 == nmax) {
          ok = next_pv(1, seen1, nmax == 1, vs);
          if (!ok) break;
          commit(&o_final[1]);
        }
        commit(&kv_empty[vs]);
        base += 2 * nmax;
      }
      commit(drain);
      mbar_wait_warp(drain, 0, p.err);
    } else if (warp == 3) {
      int base = 0, ragged_seen = 0;
      while (walk_next(walk, p, *share)) {
        if (x.nmax == 0) continue;
        const int end = doc.Lk - (x.k0 + x.nmax - 1) * kPkTile;  // keys of the last tile that are the document's
        if (end < kPkTile) {
          if (!mbar_wait_warp(ragged, static_cast<uint32_t>(ragged_seen & 1), p.err)) break;
          ++ragged_seen;
          zero_tile_rows(sKV + (base + pos_v(x.nmax - 1, x.nmax)) % kStages * kPkTileBytes, end);
          if (lane == 0) mbar_arrive(cleared);
        }
        base += 2 * x.nmax;
      }
    } else if (warp == 2 && p.may_split) {
      Cut cut{};
      while (walk_next(walk, p, *share)) {
        if (x.whole || !x.begins) continue;
        cut.crosses = 1;
        cut.first_slot = x.slot;
        // CTA of the unit's last key tile
        cut.last_cta = static_cast<int>(((share->s + x.unit_end) * share->ctas - 1) / share->total);
        cut.row0 = doc.q0 + x.first;
        cut.rows = min(2 * p.per_tile, doc.Lq - x.first);
        cut.group = x.group;
      }
      if (lane == 0) p.cuts[blockIdx.x] = cut;
    }
  } else {
    setmaxnreg_inc<kRegsHigh>();
    const int t = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_row = tmem_base + lane_off + t * kPkTile;
    const uint32_t o_row = tmem_base + lane_off + 256 + t * kPkTile;
    const int query = row / p.pack, head_in = row - query * p.pack;
    uint32_t s_seen = 0, o_seen = 0;
    bool ok = true;
    while (ok && walk_next(walk, p, *share)) {
      const int i = x.first + t * p.per_tile + query;
      const bool live = query < p.per_tile && i < doc.Lq;
      const int head = x.group * p.pack + head_in;
      // Rows of no query are not masked: what they hold goes nowhere.
      const int seen = live ? seen_keys(i, doc.off, doc.Lk, doc.prefix, p.a.causal_block) : 0x7fffffff;
      const float slope2 = p.a.slopes && live ? __ldg(p.a.slopes + head) * kLog2e : 0.f;
      const float mult = !kPlain && p.prescale ? 1.0f : p.mult;
      float m_run = -INFINITY, l_run = 0.f;
      const int n = x.n[t];
      int valid = seen - x.k0 * kPkTile;                                      // keys of the tile that the row sees
      float from = static_cast<float>(i + doc.off - x.k0 * kPkTile);          // distance from the tile's first key
      for (int j = 0; j < n; ++j, valid -= kPkTile, from -= kPkTile) {
        if (!mbar_wait_warp(&s_full[t], s_seen & 1u, p.err)) {
          ok = false;
          break;
        }
        ++s_seen;
        tc_fence_after();
        uint32_t r[kPkTile];
        tmem_ld32(s_row, *reinterpret_cast<uint32_t(*)[32]>(r));
        tmem_ld32(s_row + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
        tmem_ld32(s_row + 64, *reinterpret_cast<uint32_t(*)[32]>(r + 64));
        tmem_ld32(s_row + 96, *reinterpret_cast<uint32_t(*)[32]>(r + 96));
        tmem_ld_wait();
        if (!kPlain && p.a.cap > 0.f) cap_scores(r, p.cap_in, live);
        if (!kPlain && p.prescale) {
          const unsigned long long m2 = f2_splat(p.mult);
          if (__all_sync(0xffffffffu, !live || from >= kPkTile - 1 || from <= 0.f)) {
            // every key lies on one side of the row's own place: the distance is linear
            const float w = from > 0.f ? slope2 : -slope2, b = -w * from;
#pragma unroll
            for (int c = 0; c < kPkTile; c += 2) {
              const float2 v = f2_unpack(f2_fma(f2_pack(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), m2,
                                                f2_pack(fmaf(w, static_cast<float>(c), b), fmaf(w, static_cast<float>(c + 1), b))));
              r[c] = __float_as_uint(v.x), r[c + 1] = __float_as_uint(v.y);
            }
          } else {
#pragma unroll
            for (int c = 0; c < kPkTile; ++c)
              r[c] = __float_as_uint(fmaf(__uint_as_float(r[c]), p.mult, -slope2 * fabsf(from - static_cast<float>(c))));
          }
        }
        const bool cut = __any_sync(0xffffffffu, valid < kPkTile);
        if (cut) {
#pragma unroll
          for (int c = 0; c < kPkTile; ++c)
            if (c >= valid) r[c] = __float_as_uint(-INFINITY);
        }
        float mx8[8];
#pragma unroll
        for (int a = 0; a < 8; ++a) mx8[a] = __uint_as_float(r[a]);
#pragma unroll
        for (int c = 8; c < kPkTile; c += 2)
          mx8[(c >> 1) & 7] = fmax3(mx8[(c >> 1) & 7], __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
        const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                               fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        const bool grow = live && (mx - m_run) * mult > kRescaleLog2;
        float alpha = 1.0f;
        bool rescale = false;
        if (j == 0) {
          m_run = mx;
        } else if (__any_sync(0xffffffffu, grow)) {
          const float m_new = fmaxf(m_run, mx);
          alpha = m_new == -INFINITY ? 1.0f : ex2_approx((m_run - m_new) * mult);
          m_run = m_new;
          rescale = true;
        }
        const float nb = m_run == -INFINITY ? 0.f : -m_run * mult;  // a row that has seen nothing yet
        const unsigned long long mult2 = f2_pack(mult, mult), nb2 = f2_pack(nb, nb);
        unsigned long long rs4[4] = {0ull, 0ull, 0ull, 0ull};
        // Masked entries are exactly 0 (the polynomial stops at 2^-125), so it is left out there.
        auto exps = [&](int c0, auto poly) {
#pragma unroll
          for (int c = c0; c < (c0 ? 64 : 48); ++c) {
            const unsigned long long y2 = f2_fma(f2_pack(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1])), mult2, nb2);
            float2 e;
            if (poly.value && c % kPolyEvery == kPolyEvery - 1) {
              e = f2_unpack(exp2_poly2(y2));
            } else {
              const float2 y = f2_unpack(y2);
              e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            }
            rs4[c & 3] = f2_add(rs4[c & 3], f2_pack(e.x, e.y));
            r[c] = pack_bf16x2(e.x, e.y);
          }
        };
        if (cut)
          exps(0, BoolConstant<false>{});
        else
          exps(0, BoolConstant<true>{});
        tmem_st32(s_row, *reinterpret_cast<uint32_t(*)[32]>(r));
        tmem_st16(s_row + 32, *reinterpret_cast<uint32_t(*)[16]>(r + 32));
        if (rescale) {
          // S_t(j) ready implies that PV_t(j-1) completed, and PV_t(j) waits for this
          // thread's arrival below: O_t is current and idle here.
#pragma unroll 1
          for (int c = 0; c < kPkD / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_row + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
            tmem_st32(o_row + c * 32, o);
          }
          l_run *= alpha;
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_half[t]);  // the product over the first 96 keys may begin
        if (cut)
          exps(48, BoolConstant<false>{});
        else
          exps(48, BoolConstant<true>{});
        tmem_st16(s_row + 48, *reinterpret_cast<uint32_t(*)[16]>(r + 48));
        {
          const float2 s01 = f2_unpack(f2_add(rs4[0], rs4[1])), s23 = f2_unpack(f2_add(rs4[2], rs4[3]));
          l_run += (s01.x + s01.y) + (s23.x + s23.y);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      if (n > 0) {
        if (!mbar_wait_warp(&o_final[t], o_seen & 1u, p.err)) break;
        ++o_seen;
        tc_fence_after();
      }
      const int64_t grow_row = static_cast<int64_t>(doc.q0) + i;
      const float base2 = m_run * mult;  // log2 units
      if (!x.whole) {
        const int64_t slot = static_cast<int64_t>(x.slot) * p.slot_rows + t * kPkTile + row;
        float4* po = reinterpret_cast<float4*>(p.part_o + slot * kPkD);
        if (n > 0) {
#pragma unroll 1
          for (int c = 0; c < kPkD / 32; ++c) {
            uint32_t r0[32];
            tmem_ld32(o_row + c * 32, r0);
            tmem_ld_wait();
            if (live) {
#pragma unroll
              for (int g = 0; g < 8; ++g)
                po[c * 8 + g] = make_float4(__uint_as_float(r0[4 * g]), __uint_as_float(r0[4 * g + 1]),
                                            __uint_as_float(r0[4 * g + 2]), __uint_as_float(r0[4 * g + 3]));
            }
          }
        }
        if (live) p.part_ml[slot] = make_float2(base2, l_run);
      } else {
        const float inv = l_run == 0.f ? 0.f : 1.0f / l_run;
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.a.o) + grow_row * p.a.o_stride + head * kPkD;
#pragma unroll 1
        for (int c = 0; c < kPkD / 32; ++c) {
          uint32_t r0[32];
          if (n > 0) {
            tmem_ld32(o_row + c * 32, r0);
            tmem_ld_wait();
          }
          if (live) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint4 v;  // a row without a seen key: 0, whatever O holds
              v.x = l_run == 0.f ? 0u : pack_bf16x2(__uint_as_float(r0[8 * g]) * inv, __uint_as_float(r0[8 * g + 1]) * inv);
              v.y = l_run == 0.f ? 0u : pack_bf16x2(__uint_as_float(r0[8 * g + 2]) * inv, __uint_as_float(r0[8 * g + 3]) * inv);
              v.z = l_run == 0.f ? 0u : pack_bf16x2(__uint_as_float(r0[8 * g + 4]) * inv, __uint_as_float(r0[8 * g + 5]) * inv);
              v.w = l_run == 0.f ? 0u : pack_bf16x2(__uint_as_float(r0[8 * g + 6]) * inv, __uint_as_float(r0[8 * g + 7]) * inv);
              reinterpret_cast<uint4*>(orow + c * 32)[g] = v;
            }
          }
        }
        if (live && p.a.lse)
          p.a.lse[static_cast<int64_t>(head) * p.a.q_rows + grow_row] =
              l_run == 0.f ? -INFINITY : (base2 + log2f(l_run)) * 0.6931471805599453f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Merge the parts of the unit that begins in CTA blockIdx.x and ends in a later one: with
// base b = max b_c and w_c = 2^(b_c - b), o = sum w_c o_c / sum w_c l_c, in CTA order. A
// warp takes a row, a lane 4 of its 128 columns; the lanes first fetch the parts' bases and
// sums side by side (32 at a time).
__global__ void __launch_bounds__(256) packed_merge_kernel(const __grid_constant__ FwdParams p) {
  const Cut cut = p.cuts[blockIdx.x];
  if (!cut.crosses) return;
  const int lane = threadIdx.x & 31, step = gridDim.y * 8;
  const int c0 = blockIdx.x, parts = cut.last_cta - c0 + 1;
  for (int m = blockIdx.y * 8 + (threadIdx.x >> 5); m < cut.rows * p.pack; m += step) {
    const int query = m / p.pack, head = cut.group * p.pack + m - query * p.pack;
    const int t = query >= p.per_tile ? 1 : 0;
    const int in_slot = t * kPkTile + m - t * p.per_tile * p.pack;
    auto slot_of = [&](int i) { return static_cast<int64_t>(i == 0 ? cut.first_slot : 2 * (c0 + i)) * p.slot_rows + in_slot; };
    float base = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += 32) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (i0 + lane < parts) ml = p.part_ml[slot_of(i0 + lane)];
      if (ml.y == 0.f) ml.x = -INFINITY;  // a part that saw nothing
      float top = ml.x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      top = fmaxf(top, base);
      const float back = base == -INFINITY ? 0.f : exp2f(base - top), w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
      base = top;
      l *= back;
      o.x *= back, o.y *= back, o.z *= back, o.w *= back;
      const int n = min(32, parts - i0);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i), li = __shfl_sync(0xffffffffu, ml.y, i);
        if (li == 0.f) continue;  // its output was not written
        const float4 v = reinterpret_cast<const float4*>(p.part_o + slot_of(i0 + i) * kPkD)[lane];
        l = fmaf(wi, li, l);
        o.x = fmaf(wi, v.x, o.x), o.y = fmaf(wi, v.y, o.y), o.z = fmaf(wi, v.z, o.z), o.w = fmaf(wi, v.w, o.w);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const int64_t row = static_cast<int64_t>(cut.row0) + query;
    __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.a.o) + row * p.a.o_stride + head * kPkD;
    reinterpret_cast<uint2*>(orow)[lane] = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (lane == 0 && p.a.lse)
      p.a.lse[static_cast<int64_t>(head) * p.a.q_rows + row] = l == 0.f ? -INFINITY : (base + log2f(l)) * 0.6931471805599453f;
  }
}

struct SplitLayout {
  int slot_rows;
  size_t o_bytes, ml_bytes, total;
};
SplitLayout split_layout(const PackedAttn& a) {
  const int pack = packed_heads_per_tile(a.H, a.Hk), per_tile = kPkTile / pack;
  SplitLayout l{};
  l.slot_rows = a.q_rows <= per_tile ? a.q_rows * pack : 2 * kPkTile;
  l.o_bytes = static_cast<size_t>(2 * kMaxCtas) * l.slot_rows * kPkD * 4;
  l.ml_bytes = (static_cast<size_t>(2 * kMaxCtas) * l.slot_rows * 8 + 15) / 16 * 16;
  l.total = l.o_bytes + l.ml_bytes + kMaxCtas * sizeof(Cut);
  return l;
}

}  // namespace

int packed_heads_per_tile(int H, int Hk, int rows) {
  const int group = H / Hk;
  for (int n = group < rows ? group : rows; n > 1; --n)
    if (group % n == 0) return n;
  return 1;
}

bool make_packed_q_map(CUtensorMap* map, const void* ptr, int64_t stride, int n_rows, int H, int pack, int tile_rows) {
  const uint64_t dims[3] = {kPkD, static_cast<uint64_t>(H), static_cast<uint64_t>(n_rows)};
  const uint64_t strides[2] = {kPkD * 2, static_cast<uint64_t>(stride) * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(pack), static_cast<uint32_t>(tile_rows / pack)};
  return make_tmap_bf16(map, ptr, 3, dims, strides, box);
}

bool make_packed_kv_map(CUtensorMap* map, const void* ptr, int64_t stride, int n_rows, int Hk, int tile_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(Hk) * kPkD, static_cast<uint64_t>(n_rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(stride) * 2};
  const uint32_t box[2] = {64, static_cast<uint32_t>(tile_rows)};
  return make_tmap_bf16(map, ptr, 2, dims, strides, box);
}

size_t attn_packed_tc_workspace(const PackedAttn& a) { return split_layout(a).total; }

int launch_attn_packed_tc(const PackedAttn& a, void* ws, size_t ws_bytes, cudaStream_t s) {
  FwdParams p{};
  p.a = a;
  p.pack = packed_heads_per_tile(a.H, a.Hk);
  p.per_tile = kPkTile / p.pack;
  p.groups = a.H / p.pack;
  p.mult = (a.cap > 0.f ? a.cap : a.scale) * kLog2e;
  p.cap_in = a.cap > 0.f ? a.scale / a.cap : 0.f;
  p.prescale = a.slopes || p.mult < 0.f;
  p.err = device_error_flag();
  int dev = 0;
  cudaGetDevice(&dev);
  p.ctas = device_sms() < kMaxCtas ? device_sms() : kMaxCtas;
  const SplitLayout l = split_layout(a);
  p.slot_rows = l.slot_rows;
  if (ws && ws_bytes < l.total) return WAN_ERR_WORKSPACE;
  if (ws && a.k_rows > kMinSplit * kPkTile) {  // no unit of fewer keys is cut
    uint8_t* w = static_cast<uint8_t*>(ws);
    p.part_o = reinterpret_cast<float*>(w);
    p.part_ml = reinterpret_cast<float2*>(w + l.o_bytes);
    p.cuts = reinterpret_cast<Cut*>(w + l.o_bytes + l.ml_bytes);
    p.may_split = 1;
  }
  CUtensorMap mq, mk, mv;
  // without keys no key is loaded: any valid map will do
  const bool keys = a.k_rows > 0;
  if (!make_packed_q_map(&mq, a.q, a.q_stride, a.q_rows, a.H, p.pack) ||
      !make_packed_kv_map(&mk, keys ? a.k : a.q, keys ? a.k_stride : a.q_stride, keys ? a.k_rows : 1, a.Hk) ||
      !make_packed_kv_map(&mv, keys ? a.v : a.q, keys ? a.v_stride : a.q_stride, keys ? a.k_rows : 1, a.Hk))
    return WAN_ERR_CUDA;
  static std::once_flag once[64];
  std::call_once(once[dev & 63], [] {
    for (auto kernel : {packed_fwd_tc_kernel<true>, packed_fwd_tc_kernel<false>})
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  });
  trace_launch_begin(WAN_KIND_ATTN, s);
  (a.cap > 0.f || p.prescale ? packed_fwd_tc_kernel<false> : packed_fwd_tc_kernel<true>)<<<p.ctas, kThreads, kSmem, s>>>(mq, mk, mv, p);
  int st = check_launch();
  if (st == WAN_OK && p.may_split) {
    packed_merge_kernel<<<dim3(p.ctas, l.slot_rows < 128 ? (l.slot_rows + 7) / 8 : 16), 256, 0, s>>>(p);
    count_launches(1);
    st = check_launch();
  }
  trace_launch_end(WAN_KIND_ATTN, s);
  return st;
}

}  // namespace wan
