// Work split of the shared-prefix decode, used by its attention kernels and
// by the merge.
//
// Every attention unit is a tile of query rows against a run of keys:
//   prefix units (n, h, tile): the queries of up to R rows of the sequences of
//     group n (row = sequence * G + head of the group) against prefix n;
//   own units (b, h): the G query heads of one sequence against its own cache.
// A unit's keys are cut into chunks of kPdChunk.  All chunks of all units lie
// end to end (prefixes first; within a prefix by head, then row tile) and CTA
// c of P = min(CTAs, W) takes chunks [W c / P, W (c + 1) / P): every SM streams the same
// number of keys whatever the lengths.  A CTA that holds any of unit i's
// chunks writes one partial (normalised rows and their log2-sum-exp) to slot
// c + i: the pairs (c, i) met along the line grow by one in c or in i at a
// time, so slots are distinct and number at most P + units.
#pragma once

#include "internal.h"

namespace csa {

constexpr int kPdChunk = 64;      // keys per chunk
constexpr int kPdMaxPrefixes = 64;

// Sanitised lengths: out of range is flagged and clamped.
__device__ __forceinline__ int pd_clamp(int v, int64_t hi, const DevErr& e) {
  if (v < 0 || v > hi) {
    dev_flag(e, DEV_BAD_INDEX);
    v = v < 0 ? 0 : static_cast<int>(hi);
  }
  return v;
}

struct PdShape {
  int B, Hkv, G, N, R, P;
  int64_t Tp, T;
  const int32_t* prefix_len;   // [N] or null: Tp
  const int32_t* group_start;  // [N + 1] or null: one group of all sequences
  const int32_t* len;          // [B] or null: T
  DevErr err;
};

__device__ __forceinline__ int pd_prefix_len(const PdShape& s, int n) {
  return s.prefix_len ? pd_clamp(__ldg(s.prefix_len + n), s.Tp, s.err) : static_cast<int>(s.Tp);
}
__device__ __forceinline__ int pd_own_len(const PdShape& s, int b) {
  if (s.T == 0) return 0;
  return s.len ? pd_clamp(__ldg(s.len + b), s.T, s.err) : static_cast<int>(s.T);
}
__device__ __forceinline__ int pd_chunks(int keys) { return (keys + kPdChunk - 1) / kPdChunk; }
__device__ __forceinline__ int pd_tiles(const PdShape& s, int seqs) {
  return (seqs * s.G + s.R - 1) / s.R;
}

// gs[0 .. N]: the groups' bounds, clamped to [0, B] and made non-decreasing
// (a bound below an earlier one is flagged).  One warp.
__device__ __forceinline__ void pd_groups(const PdShape& s, int* gs) {
  const int lane = threadIdx.x & 31;
  if (s.N == 0) return;
  if (s.group_start == nullptr) {
    if (lane < 2) gs[lane] = lane ? s.B : 0;
    return;
  }
  int carry = 0;
  for (int i0 = 0; i0 <= s.N; i0 += 32) {
    const int i = i0 + lane;
    int v = i <= s.N ? pd_clamp(__ldg(s.group_start + i), s.B, s.err) : 0;
    const int raw = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, t);
    }
    v = max(v, carry);
    if (i <= s.N) {
      if (v != raw) dev_flag(s.err, DEV_BAD_INDEX);
      gs[i] = v;
    }
    carry = __shfl_sync(0xffffffffu, v, 31);
  }
}

// A CTA's place on the line.  `item` < N: prefix item; else sequence item - N.
struct PdStart {
  int total;       // W
  int x0, x1;      // this CTA's chunks
  int item, off;   // the item holding x0 and x0's offset in it
  int units;       // prefix units in all
  int unit0;       // prefix units before `item` (prefix items only)
};

// Block-wide: fills *st (shared).  `gs` is shared, filled by pd_groups.
// starts (global, optional): for every item its first chunk, then W;
// ubase (global, optional): for every prefix its first unit, then the count.
__device__ __forceinline__ void pd_locate(const PdShape& s, const int* gs, int cta, PdStart* st,
                                          int* scan_sh, int32_t* starts, int32_t* ubase) {
  const int items = s.N + s.B, nt = blockDim.x, tid = threadIdx.x;
  auto weight = [&](int i) -> int {
    if (i < s.N) return pd_tiles(s, gs[i + 1] - gs[i]) * s.Hkv * pd_chunks(pd_prefix_len(s, i));
    return i < items ? s.Hkv * pd_chunks(pd_own_len(s, i - s.N)) : 0;
  };
  int run = 0;
  for (int i0 = 0; i0 < items; i0 += nt) {
    const int i = i0 + tid;
    int tot;
    const int ex = block_exclusive_scan(weight(i), scan_sh, &tot);
    if (starts && i < items) starts[i] = run + ex;
    run += tot;
  }
  if (tid == 0) {
    st->total = run;
    // at least one chunk per CTA that takes part: each writes the slots it owns
    const int P = max(1, min(s.P, run));
    st->x0 = cta < P ? static_cast<int>(static_cast<int64_t>(run) * cta / P) : run;
    st->x1 = cta < P ? static_cast<int>(static_cast<int64_t>(run) * (cta + 1) / P) : run;
    if (starts) starts[items] = run;
    int u = 0;
    for (int n = 0; n < s.N; ++n) {
      if (ubase) ubase[n] = u;
      u += pd_tiles(s, gs[n + 1] - gs[n]) * s.Hkv;
    }
    if (ubase) ubase[s.N] = u;
    st->units = u;
  }
  __syncthreads();
  const int x0 = st->x0;
  run = 0;
  for (int i0 = 0; i0 < items; i0 += nt) {
    const int i = i0 + tid, w = weight(i);
    int tot;
    const int ex = run + block_exclusive_scan(w, scan_sh, &tot);
    if (x0 >= ex && x0 < ex + w) {  // at most one item
      st->item = i;
      st->off = x0 - ex;
      int u = 0;
      for (int n = 0; n < min(i, s.N); ++n) u += pd_tiles(s, gs[n + 1] - gs[n]) * s.Hkv;
      st->unit0 = u;
    }
    run += tot;
  }
  __syncthreads();
}

// One CTA's share of one unit.
struct PdSeg {
  bool own;
  int n, b;        // prefix index, or sequence
  int h, tile;
  int unit;        // index among the prefix units, or b * Hkv + h
  int rows;        // query rows of the tile
  int row0;        // prefix: first row (sequence * G + head) of the tile
  int keys;        // keys of the unit
  int j0, j1;      // its chunks taken here
};

// Walks a CTA's segments; every role of a CTA walks the same list.
struct PdWalk {
  const PdShape& s;
  const int* gs;
  int left;        // chunks still to take
  int item, off;   // current item, chunk offset in it
  int unit0;
  __device__ PdWalk(const PdShape& sh, const int* g, const PdStart& st)
      : s(sh), gs(g), left(st.x1 - st.x0), item(st.item), off(st.off), unit0(st.unit0) {}
  __device__ __forceinline__ bool next(PdSeg& q) {
    while (left > 0) {
      if (item < s.N) {
        const int seqs = gs[item + 1] - gs[item], tiles = pd_tiles(s, seqs);
        const int keys = pd_prefix_len(s, item), c = pd_chunks(keys);
        const int ui = c > 0 ? off / c : 0;
        if (ui >= tiles * s.Hkv || c == 0) {
          unit0 += tiles * s.Hkv;
          ++item;
          off = 0;
          continue;
        }
        q.own = false;
        q.n = item;
        q.b = 0;
        q.h = ui / tiles;
        q.tile = ui - q.h * tiles;
        q.unit = unit0 + ui;
        q.row0 = gs[item] * s.G + q.tile * s.R;
        q.rows = min(s.R, seqs * s.G - q.tile * s.R);
        q.keys = keys;
        q.j0 = off - ui * c;
        q.j1 = min(c, q.j0 + left);
      } else {
        const int b = item - s.N;
        if (b >= s.B) return false;
        const int keys = pd_own_len(s, b), c = pd_chunks(keys);
        const int ui = c > 0 ? off / c : 0;
        if (ui >= s.Hkv || c == 0) {
          ++item;
          off = 0;
          continue;
        }
        q.own = true;
        q.n = 0;
        q.b = b;
        q.h = ui;
        q.tile = 0;
        q.unit = b * s.Hkv + ui;
        q.row0 = b * s.G;
        q.rows = s.G;
        q.keys = keys;
        q.j0 = off - ui * c;
        q.j1 = min(c, q.j0 + left);
      }
      left -= q.j1 - q.j0;
      off += q.j1 - q.j0;
      return true;
    }
    return false;
  }
};

// The CTA of `ctas` that holds chunk x of W.
__device__ __forceinline__ int pd_cta_of(int x, int W, int ctas) {
  const int P = min(ctas, W);
  return static_cast<int>(((static_cast<int64_t>(x) + 1) * P - 1) / W);
}

}  // namespace csa
