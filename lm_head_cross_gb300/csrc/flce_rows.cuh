// What the epilogues that walk a row of logits share: the candidates of its largest
// values, and the arithmetic of its softmax in log2 units.
#pragma once

#include <stdint.h>

#include "flce_device.cuh"

namespace flce {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Below every finite logit's distance from the maximum, in log2 units: 2^it is 0, and 0
// times it is 0, where a logit of minus infinity (a column past V, an infinite weight)
// would make 0 * infinity.
constexpr float kNoLogit = -1e30f;

// max(a, b) that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// A log probability and an entropy are kept on their side of 0, which rounding can cross by
// 1e-7 (a NaN stays one).
__device__ __forceinline__ float at_most_zero(float v) { return v > 0.f ? 0.f : v; }
__device__ __forceinline__ float at_least_zero(float v) { return v < 0.f ? 0.f : v; }

// ----------------------------------------------------------------------------- top-k candidates
// Each epilogue thread (one row) appends (logit, id) candidates that beat its
// row's threshold to a buffer in the warp's shared-memory staging area (entry e
// of lane l at topk_slot(e, l)).  Whenever a lane holds more than
// kTopkCand - 8, the whole warp ranks that lane's entries (one per lane) and
// keeps the best k; the threshold becomes the smallest kept.

constexpr int kTopkCand = 32;

struct TopkBuf {
  float* val;    // [kTopkCand][32]
  int* idx;      // [kTopkCand][32]
  int count;
  float thr;
  unsigned* shared_thr;  // the row's threshold shared by all its vocabulary ranges (global memory), or null
};

// Word of entry e of lane l's buffer.  Rows of 32 words, the lane index XORed
// with the entry: a warp appending at equal counts, and a warp reading one
// lane's whole buffer (entry e by lane e), both touch 32 different banks.
__device__ __forceinline__ int topk_slot(int e, int l) { return e * 32 + (l ^ e); }

// The same word where lanes append at their own pace and hardly ever read each other's buffer
// (the score passes): lane l's entries stay in bank l.
__device__ __forceinline__ int best_slot(int e, int l) { return e * 32 + l; }
template <bool OWN_BANK>
__device__ __forceinline__ int buffer_slot(int e, int l) {
  return OWN_BANK ? best_slot(e, l) : topk_slot(e, l);
}

// Order-preserving map of a float to an unsigned (0 stands below every float).
__device__ __forceinline__ unsigned topk_key(float f) {
  const unsigned b = __float_as_uint(f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float topk_unkey(unsigned u) {
  if (u == 0u) return -INFINITY;
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}

// (value, id) as one number that grows with the value and, among equal ones, as the id falls; 0: none.
__device__ __forceinline__ uint64_t candidate_key(float v, int id) {
  return (static_cast<uint64_t>(topk_key(v + 0.f)) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}

// The nth (from 0) of the ids that are not among `count` candidates: the alternatives that
// follow where a row has fewer logits above minus infinity than are asked for.  Those are all
// candidates, the other ids are equal, and the lowest goes first.  (Each round moves the answer
// past the candidates that are not above it: at most count + 1.)
__device__ __forceinline__ int nth_other_id(const uint64_t* cand, int count, int nth) {
  int id = nth;
  while (true) {
    int past = 0;
    for (int q = 0; q < count; ++q) past += 0xffffffffu - static_cast<uint32_t>(cand[q]) <= static_cast<uint32_t>(id);
    if (nth + past == id) return id;
    id = nth + past;
  }
}
// Its key: minus infinity, which topk_unkey makes of 0.
__device__ __forceinline__ uint64_t other_key(int id) { return 0xffffffffu - static_cast<uint32_t>(id); }

__device__ __forceinline__ bool topk_better(float av, int ai, float bv, int bi) {
  return av > bv || (av == bv && static_cast<unsigned>(ai) < static_cast<unsigned>(bi));
}

// How many of 32 values reach `at`, in four independent chains.
__device__ __forceinline__ int count_reaching(const float (&v)[32], float at) {
  int n[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 32; ++e) n[e & 3] += v[e] >= at ? 1 : 0;
  return (n[0] + n[1]) + (n[2] + n[3]);
}

// Compact the buffers of every lane in `mask` (whole-warp call), keeping each
// row's best `keep` (= k, at most kTopkMax).  Lane e holds entry e of the
// buffer; its rank (how many entries beat it) comes from 32 independent shuffle
// rounds, and the best `keep` go to slots 0..keep-1 in rank order.  Entries are
// distinct (value, id) pairs, so the ranks of the filled slots are distinct.
template <bool OWN_BANK = false>
__device__ __forceinline__ void topk_compact_lanes(TopkBuf& b, int lane, unsigned mask, int keep) {
  while (mask) {
    const int L = __ffs(mask) - 1;
    mask &= mask - 1;
    const int cnt = __shfl_sync(0xffffffffu, b.count, L);
    const bool filled = lane < cnt;
    const float v = filled ? b.val[buffer_slot<OWN_BANK>(lane, L)] : -INFINITY;
    const int i = filled ? b.idx[buffer_slot<OWN_BANK>(lane, L)] : -1;
    int rank = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float ov = __shfl_sync(0xffffffffu, v, j);
      const int oi = __shfl_sync(0xffffffffu, i, j);
      rank += topk_better(ov, oi, v, i) ? 1 : 0;
    }
    __syncwarp();  // every entry is in registers before the slots are rewritten
    if (filled && rank < keep) {
      b.val[buffer_slot<OWN_BANK>(rank, L)] = v;
      b.idx[buffer_slot<OWN_BANK>(rank, L)] = i;
    }
    const unsigned at_k = __ballot_sync(0xffffffffu, filled && rank == keep - 1);
    const float kth = __shfl_sync(0xffffffffu, v, at_k ? __ffs(at_k) - 1 : 0);
    __syncwarp();
    if (lane == L) {
      b.count = min(cnt, keep);
      if (cnt >= keep && at_k) {
        b.thr = kth;
        // `keep` values of this row are >= kth, so any value below it, in any range, is out
        if (b.shared_thr) atomicMax(b.shared_thr, topk_key(kth));
      }
    }
  }
}

// A floor under a row's best k values, from `valid` columns of a tile in TMEM (at most 64
// GROUP of them), before anything is kept: with the columns in groups of GROUP neighbours (64
// groups cover the window), k groups whose maxima reach a value hold k values that do.
// Bisection between the least and the greatest maximum finds nearly the greatest such value,
// in the same instructions for every row; the columns that pass it are few (kept and ranked
// whole instead, they took 20 instructions a column and row).  Whole-warp call; minus
// infinity where fewer than k groups hold a column.
template <int GROUP>
__device__ __forceinline__ float first_floor(uint32_t tbase, int valid, int k) {
  constexpr int kPer = 32 / GROUP;  // groups of a 32-column chunk
  float g[2][32];
  float lo[4] = {INFINITY, INFINITY, INFINITY, INFINITY}, hi[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 2 * GROUP; ++c) {
    const int left = valid - c * 32;
    if (left > 0) {  // the same for the whole warp
      uint32_t v[32];
      __syncwarp();
      tmem_ld_32x32(tbase + c * 32, v);
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        float m = __uint_as_float(v[q * GROUP]);
#pragma unroll
        for (int j = q * GROUP + 1; j < (q + 1) * GROUP; ++j)
          if (j < left) m = fmaxf(m, __uint_as_float(v[j]));
        const bool in = q * GROUP < left;
        g[(c * kPer + q) / 32][(c * kPer + q) % 32] = in ? m : -INFINITY;
        lo[q & 3] = fminf(lo[q & 3], in ? m : INFINITY);
        hi[q & 3] = fmaxf(hi[q & 3], in ? m : -INFINITY);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kPer; ++q) g[(c * kPer + q) / 32][(c * kPer + q) % 32] = -INFINITY;
    }
  }
  if ((valid + GROUP - 1) / GROUP < k) return -INFINITY;
  float least = fminf(fminf(lo[0], lo[1]), fminf(lo[2], lo[3]));
  float most = fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3]));
#pragma unroll 1
  for (int i = 0; i < 7; ++i) {
    const float mid = 0.5f * least + 0.5f * most;
    if (count_reaching(g[0], mid) + count_reaching(g[1], mid) >= k) least = mid;
    else most = mid;
  }
  return least;
}

// Drops what cannot be among a row's best k from every lane's buffer at once (whole-warp
// call): bisection between the least and the greatest entry of a lane that holds more than
// k finds a value that k entries reach and few others do; those stay, in their order, and
// the value is returned as the row's new floor (the old one for other lanes).  About 900
// instructions for the warp, where ranking takes 220 for each lane; out of line, as is the
// ranking behind it, so that the code that every chunk runs through stays short.
struct Trimmed {
  int count;
  float thr;
};
static __device__ __noinline__ Trimmed topk_trim(float* val, int* idx, int count, int lane, int k, float floor_thr) {
  float v[kTopkCand];
  float lo4[4], hi4[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo4[i] = INFINITY;
    hi4[i] = -INFINITY;
  }
#pragma unroll
  for (int e = 0; e < kTopkCand; ++e) {
    v[e] = e < count ? val[best_slot(e, lane)] : -INFINITY;
    if (e < count) lo4[e & 3] = fminf(lo4[e & 3], v[e]);
    hi4[e & 3] = fmaxf(hi4[e & 3], v[e]);
  }
  float lo = fminf(fminf(lo4[0], lo4[1]), fminf(lo4[2], lo4[3]));
  float hi = fmaxf(fmaxf(hi4[0], hi4[1]), fmaxf(hi4[2], hi4[3]));
  if (count <= k) lo = -INFINITY;  // everything stays
#pragma unroll 1
  for (int i = 0; i < 7; ++i) {
    const float mid = 0.5f * lo + 0.5f * hi;
    const bool up = count_reaching(v, mid) >= k && count > k;
    lo = up ? mid : lo;
    hi = up ? hi : mid;
  }
  int id[kTopkCand];  // read whole before anything is rewritten
#pragma unroll
  for (int e = 0; e < kTopkCand; ++e) id[e] = idx[best_slot(e, lane)];
  int at = 0;
#pragma unroll
  for (int e = 0; e < kTopkCand; ++e) {
    const bool keep = e < count && v[e] >= lo;
    if (keep) {
      val[best_slot(at, lane)] = v[e];
      idx[best_slot(at, lane)] = id[e];
    }
    at += keep ? 1 : 0;
  }
  __syncwarp();
  return Trimmed{at, fmaxf(floor_thr, lo)};
}

// topk_compact_lanes for the lanes that hold more than `most`: their new count and threshold.
static __device__ __noinline__ Trimmed topk_cut(float* val, int* idx, int count, float thr, int lane, int k, int most) {
  TopkBuf b;
  b.val = val;
  b.idx = idx;
  b.count = count;
  b.thr = thr;
  b.shared_thr = nullptr;
  topk_compact_lanes<true>(b, lane, __ballot_sync(0xffffffffu, count > most), k);
  return Trimmed{b.count, b.thr};
}

// ----------------------------------------------------------------------------- a row's walk over its logits

// Softmax statistics of the logits seen so far, in log2 units: the maximum m, l = sum 2^(t - m)
// and es = sum 2^(t - m) (t - m).  entropy = ln l - ln 2 (es / l): two terms of like sign, where
// lse - sum p z would cancel.
struct RowSum {
  float m, l, es;
};

// Maxima of 32 logits' blocks of 8, and of all.
__device__ __forceinline__ float block_maxima(const uint32_t (&v)[32], float (&gmax)[4]) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const auto x = [&](int j) { return __uint_as_float(v[8 * g + j]); };
    gmax[g] = fmaxf(fmaxf(fmaxf(fmaxf(x(0), x(1)), x(2)), fmaxf(fmaxf(x(3), x(4)), x(5))), fmaxf(x(6), x(7)));
  }
  return fmaxf(fmaxf(gmax[0], gmax[1]), fmaxf(gmax[2], gmax[3]));
}

// 32 logits, the largest of them cmax (in their own units), zs log2 units each.  3 instructions
// a logit (two at a time but for 2^u), where logits of minus infinity would make 0 * infinity:
// the NaN that it leaves is the sign to take them one by one.
__device__ __forceinline__ void add_chunk(RowSum& r, const uint32_t (&v)[32], float cmax, float zs) {
  const float new_m = fmaxf(r.m, cmax * zs);
  const float2 scale = both(zs), back = both(-new_m);
  float2 s2[2] = {}, e2[2] = {};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 u = fma2(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), scale, back);
    const float2 w = make_float2(fast_exp2(u.x), fast_exp2(u.y));
    s2[j & 1] = add2(s2[j & 1], w);
    e2[j & 1] = fma2(w, u, e2[j & 1]);
  }
  const float2 st = add2(s2[0], s2[1]), et = add2(e2[0], e2[1]);
  float s = st.x + st.y, e = et.x + et.y;
  if (!(e == e)) {
    const float from = new_m == -INFINITY ? 0.f : new_m;  // nothing but minus infinity so far: adds 0
    s = e = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float u = max_nan(fmaf(__uint_as_float(v[j]), zs, -from), kNoLogit);
      const float w = fast_exp2(u);
      s += w;
      e = fmaf(w, u, e);
    }
  }
  const float d = fmaxf(r.m - new_m, kNoLogit);  // (minus infinity twice: the sums are 0 or NaN)
  const float f = fast_exp2(d);
  r.es = f * fmaf(r.l, d, r.es) + e;
  r.l = r.l * f + s;
  r.m = new_m;
}

// The float below f: x > it exactly where x >= f.
__device__ __forceinline__ float float_below(float f) {
  if (f == -INFINITY) return f;
  return topk_unkey(topk_key(f == 0.f ? -0.f : f) - 1u);
}

// A lane's candidates for its row's best k.
struct RowBest {
  float* val;  // [kTopkCand][32], the warp's
  int* idx;
  int at;       // count * 32 + lane: where the next one goes
  float thr;    // the range's own k-th best, once it is known: ids grow, so an equal later value is out
  float floor;  // nothing below it is among the row's best
  float bar;    // what a candidate passes: both in one
};
__device__ __forceinline__ void set_bar(RowBest& b) { b.bar = b.floor > b.thr ? float_below(b.floor) : b.thr; }

// Trims every lane to about k, and ranks the lanes that stay above `most`.
__device__ __forceinline__ void trim_best(RowBest& b, int lane, int k, int most) {
  Trimmed t = topk_trim(b.val, b.idx, b.at >> 5, lane, k, b.floor);
  b.floor = t.thr;
  t = topk_cut(b.val, b.idx, t.count, b.thr, lane, k, most);  // (many equal values)
  b.at = best_slot(t.count, lane);
  b.thr = t.thr;
  set_bar(b);
}

// Appends what passes the bar of 32 logits that start at id col0 (whole-warp call): 5
// instructions a logit in the blocks of 8 where any lane's passes.  A buffer that holds at
// most kTopkCand - 8 does not overflow.  Returns whether the lane's floor rose.
__device__ __forceinline__ bool append_chunk(RowBest& b, const uint32_t (&v)[32], const float (&gmax)[4], float cmax,
                                             int col0, int lane, int k) {
  const float floor0 = b.floor;
  if (!__any_sync(0xffffffffu, cmax > b.bar)) return false;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (!__any_sync(0xffffffffu, gmax[g] > b.bar)) continue;
#pragma unroll
    for (int j = 8 * g; j < 8 * g + 8; ++j) {
      const float x = __uint_as_float(v[j]);
      const bool keep = x > b.bar;
      if (keep) {  // predicated stores, no branch
        b.val[b.at] = x;
        b.idx[b.at] = col0 + j;
      }
      b.at += keep ? 32 : 0;
    }
    if (__any_sync(0xffffffffu, b.at >= 32 * (kTopkCand - 7))) trim_best(b, lane, k, kTopkCand - 8);
  }
  return b.floor > floor0;
}

}  // namespace flce
