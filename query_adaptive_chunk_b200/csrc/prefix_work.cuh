// Work split of the shared-prefix decode, used by its attention kernels and
// by the merge.
//
// Every attention unit is a tile of query rows against a run of keys:
//   prefix units (n, h, tile): the queries of up to R rows of the sequences of
//     group n (row = sequence * G + head of the group) against prefix n;
//   own units (b, h): the G query heads of one sequence against its own cache.
// A unit's keys are cut into chunks of kPdChunk.  All chunks of all units lie
// end to end (prefixes first; within a prefix by head, then row tile; own units by
// sequence, then head) and CTA c of P = min(CTAs, W) takes chunks [W c / P,
// W (c + 1) / P): every SM streams the same number of keys whatever the
// lengths.  A CTA that holds any of unit i's chunks writes one partial
// (normalised rows and their log2-sum-exp) to slot c + i: the pairs (c, i) met
// along the line grow by one in c or in i at a time, so slots are distinct
// and number at most P + units.
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
// Keys of item i: prefix i, or the own cache of sequence i - N.
__device__ __forceinline__ int pd_item_keys(const PdShape& s, int i) {
  return i < s.N ? pd_prefix_len(s, i) : pd_own_len(s, i - s.N);
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

// A CTA's place on the line.
struct PdStart {
  int left;             // its chunks
  int item, h, tile, j; // where they start: item, head, row tile, chunk of the unit
  int unit0;            // prefix units before `item` (prefix items only)
};

// What the merge needs to find a unit's partials, written by one CTA.
struct PdPlan {
  int32_t* starts;  // [N + B + 1] first chunk of each item, then W
  int32_t* ubase;   // [N + 1] first unit of each prefix
  int32_t* gsan;    // [N + 1] the sanitised group bounds
  int32_t* group;   // [B] each sequence's prefix, or -1
};

// Block-wide: fills *st (shared).  `gs` (shared) is filled by pd_groups in the
// calling code before a barrier; key0 = pd_item_keys of item threadIdx.x,
// loaded before that barrier (any value for threads past the items).
__device__ __forceinline__ void pd_locate(const PdShape& s, const int* gs, int key0, PdStart* st,
                                          int* scan_sh, const PdPlan* plan) {
  const int items = s.N + s.B, nt = blockDim.x, tid = threadIdx.x;
  auto units = [&](int i) -> int {
    return i < s.N ? pd_tiles(s, gs[i + 1] - gs[i]) * s.Hkv : s.Hkv;
  };
  auto place = [&](int i, int u, int c, int off, int take) {  // one thread: CTA starts in item i
    st->left = take;
    st->item = i;
    const int ui = off / c, tiles = i < s.N ? u / s.Hkv : 1;
    st->h = ui / tiles;
    st->tile = ui - st->h * tiles;
    st->j = off - ui * c;
    int before = 0;
    for (int n = 0; n < min(i, s.N); ++n) before += units(n);
    st->unit0 = before;
  };
  auto share = [&](int W, int* x0, int* x1) {
    // at least one chunk for each CTA that takes part: each writes the slots it owns
    const int P = max(1, min(s.P, W)), c = static_cast<int>(blockIdx.x);
    *x0 = c < P ? static_cast<int>(static_cast<int64_t>(W) * c / P) : W;
    *x1 = c < P ? static_cast<int>(static_cast<int64_t>(W) * (c + 1) / P) : W;
  };
  if (tid == 0) st->left = 0;
  int W, x0, x1;
  if (items <= nt) {
    const int u = tid < items ? units(tid) : 0, c = tid < items ? pd_chunks(key0) : 0;
    const int ex = block_exclusive_scan(u * c, scan_sh, &W);
    share(W, &x0, &x1);
    if (x0 >= ex && x0 < ex + u * c) place(tid, u, c, x0 - ex, x1 - x0);  // at most one item
    if (plan && tid < items) plan->starts[tid] = ex;
  } else {
    W = 0;
    for (int i0 = 0; i0 < items; i0 += nt) {
      const int i = i0 + tid;
      int tot;
      const int ex = block_exclusive_scan(i < items ? units(i) * pd_chunks(pd_item_keys(s, i)) : 0,
                                          scan_sh, &tot);
      if (plan && i < items) plan->starts[i] = W + ex;
      W += tot;
    }
    share(W, &x0, &x1);
    int run = 0;
    for (int i0 = 0; i0 < items; i0 += nt) {
      const int i = i0 + tid;
      const int u = i < items ? units(i) : 0, c = i < items ? pd_chunks(pd_item_keys(s, i)) : 0;
      int tot;
      const int ex = run + block_exclusive_scan(u * c, scan_sh, &tot);
      if (x0 >= ex && x0 < ex + u * c) place(i, u, c, x0 - ex, x1 - x0);
      run += tot;
    }
  }
  if (plan) {
    if (tid == 0) {
      plan->starts[items] = W;
      int u = 0;
      for (int n = 0; n < s.N; ++n) {
        plan->ubase[n] = u;
        u += units(n);
      }
      plan->ubase[s.N] = u;
    }
    if (s.N > 0 && tid <= s.N) plan->gsan[tid] = gs[tid];
    for (int b = tid; b < s.B; b += nt) {
      int g = -1;
      for (int n = 0; n < s.N; ++n)
        if (gs[n] <= b && b < gs[n + 1]) g = n;
      plan->group[b] = g;
    }
  }
  __syncthreads();
}

// One CTA's share of one unit.
struct PdSeg {
  bool own;
  int n, b;        // prefix index, or sequence
  int h;
  int unit;        // index among the prefix units, or b * Hkv + h
  int rows;        // query rows of the tile
  int row0;        // first row (sequence * G + head) of the tile
  int keys;        // keys of the unit
  int j0, j1;      // its chunks taken here
};

// Walks a CTA's segments; every role of a CTA walks the same list.
struct PdWalk {
  const PdShape& s;
  const int* gs;
  int left, item, h, tile, j, unit0;
  int keys = 0, tiles = 0;  // of `item`, once loaded
  bool loaded = false;
  __device__ __forceinline__ PdWalk(const PdShape& sh, const int* g, const PdStart& st)
      : s(sh), gs(g), left(st.left), item(st.item), h(st.h), tile(st.tile), j(st.j),
        unit0(st.unit0) {}
  __device__ __forceinline__ bool next(PdSeg& q) {
    if (left <= 0) return false;
    while (!loaded) {
      if (item >= s.N + s.B) return false;
      keys = pd_item_keys(s, item);
      tiles = item < s.N ? pd_tiles(s, gs[item + 1] - gs[item]) : 1;
      loaded = keys > 0 && tiles > 0;
      if (!loaded) {
        unit0 += tiles * s.Hkv;  // only read for prefixes
        ++item;
      }
    }
    const int c = pd_chunks(keys);
    q.own = item >= s.N;
    q.n = q.own ? 0 : item;
    q.b = q.own ? item - s.N : 0;
    q.h = h;
    q.keys = keys;
    q.unit = q.own ? q.b * s.Hkv + h : unit0 + h * tiles + tile;
    q.row0 = (q.own ? q.b : gs[item]) * s.G + tile * s.R;
    q.rows = q.own ? s.G : min(s.R, (gs[item + 1] - gs[item]) * s.G - tile * s.R);
    q.j0 = j;
    q.j1 = min(c, j + left);
    left -= q.j1 - j;
    j = q.j1;
    if (j == c) {
      j = 0;
      if (++tile == tiles) {
        tile = 0;
        if (++h == s.Hkv) {
          h = 0;
          unit0 += tiles * s.Hkv;
          ++item;
          loaded = false;
        }
      }
    }
    return true;
  }
};

// The CTA of `ctas` that holds chunk x of W.
__device__ __forceinline__ int pd_cta_of(int x, int W, int ctas) {
  const int P = min(ctas, W);
  return static_cast<int>(((static_cast<int64_t>(x) + 1) * P - 1) / W);
}

}  // namespace csa
