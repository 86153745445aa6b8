// Work split of the shared-prefix decode, used by its attention kernels and
// by the merge.
//
// Every attention unit is a tile of query rows against a run of keys:
//   prefix units (n, h, tile): the queries of up to R rows of the sequences of
//     group n (row = sequence * G + head of the group) against prefix n;
//   own units (b, h): the G query heads of one sequence against its own cache.
// Units go to a kernel's line by their kind and by their group's rows.  A
// unit's keys are cut into chunks.  All chunks of a line's units lie end to
// end (prefixes first; within a prefix by head, then row tile; own units by
// sequence, then head) and worker c (a CTA, or a warp) of P = min(workers, W)
// takes chunks [W c / P, W (c + 1) / P): every SM streams the same number of
// keys whatever the lengths.  A worker that holds any of unit i's chunks writes
// one partial (normalised rows and their log2-sum-exp) to slot c + i: the
// pairs (c, i) met along the line grow by one in c or in i at a time, so slots
// are distinct and number at most P + units.
#pragma once

#include "internal.h"

namespace csa {

constexpr int kPdMaxPrefixes = 64;

// Sanitised lengths: out of range is flagged and clamped.
__device__ __forceinline__ int pd_clamp(int v, int64_t hi, const DevErr& e) {
  if (v < 0 || v > hi) {
    dev_flag(e, DEV_BAD_INDEX);
    v = v < 0 ? 0 : static_cast<int>(hi);
  }
  return v;
}

// A line of units.
struct PdShape {
  int B, Hkv, G, N;
  int R;                       // query rows per tile
  int P;                       // workers
  int chunk_log2;              // keys per chunk
  int min_rows, max_rows;      // prefix units of groups of so many rows
  int own;                     // own units too
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
__device__ __forceinline__ int pd_chunks(const PdShape& s, int keys) {
  return (keys + (1 << s.chunk_log2) - 1) >> s.chunk_log2;
}
// Row tiles of a group of `seqs` sequences (0: the group is not on this line).
__device__ __forceinline__ int pd_tiles(const PdShape& s, int seqs) {
  const int rows = seqs * s.G;
  return rows < s.min_rows || rows > s.max_rows ? 0 : (rows + s.R - 1) / s.R;
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

// A worker's place on the line.
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

// Block-wide: fills st[0 .. NW - 1] (shared), the places of the block's NW
// workers.  `gs` (shared) is filled by pd_groups in the calling code before a
// barrier; key0 = pd_item_keys of item threadIdx.x, loaded before that barrier
// (any value for threads past the items).
template <int NW>
__device__ __forceinline__ void pd_locate(const PdShape& s, const int* gs, int key0, PdStart* st,
                                          int* scan_sh, const PdPlan* plan) {
  const int items = s.N + s.B, nt = blockDim.x, tid = threadIdx.x;
  auto units = [&](int i) -> int {
    return i < s.N ? pd_tiles(s, gs[i + 1] - gs[i]) * s.Hkv : s.own ? s.Hkv : 0;
  };
  // chunks [ex, ex + u c) are item i's: the workers that start among them
  auto place = [&](int W, int i, int u, int c, int ex) {
    if (u * c == 0) return;
    // at least one chunk for each worker that takes part: each writes the slots it owns
    const int P = min(s.P, W), w0 = static_cast<int>(blockIdx.x) * NW;
#pragma unroll 1
    for (int k = 0; k < NW; ++k) {
      if (w0 + k >= P) break;
      const int x0 = static_cast<int>(static_cast<int64_t>(W) * (w0 + k) / P);
      if (x0 < ex || x0 >= ex + u * c) continue;
      const int off = x0 - ex, ui = off / c, tiles = i < s.N ? u / s.Hkv : 1;
      int before = 0;
      for (int n = 0; n < min(i, s.N); ++n) before += units(n);
      st[k].left = static_cast<int>(static_cast<int64_t>(W) * (w0 + k + 1) / P) - x0;
      st[k].item = i;
      st[k].h = ui / tiles;
      st[k].tile = ui - st[k].h * tiles;
      st[k].j = off - ui * c;
      st[k].unit0 = before;
    }
  };
  if (tid < NW) st[tid].left = 0;
  int W;
  if (items <= nt) {
    const int u = tid < items ? units(tid) : 0, c = tid < items ? pd_chunks(s, key0) : 0;
    const int ex = block_exclusive_scan(u * c, scan_sh, &W);
    place(W, tid, u, c, ex);
    if (plan && tid < items) plan->starts[tid] = ex;
  } else {
    W = 0;
    for (int i0 = 0; i0 < items; i0 += nt) {
      const int i = i0 + tid;
      int tot;
      const int ex = block_exclusive_scan(
          i < items ? units(i) * pd_chunks(s, pd_item_keys(s, i)) : 0, scan_sh, &tot);
      if (plan && i < items) plan->starts[i] = W + ex;
      W += tot;
    }
    int run = 0;
    for (int i0 = 0; i0 < items; i0 += nt) {
      const int i = i0 + tid;
      const int u = i < items ? units(i) : 0, c = i < items ? pd_chunks(s, pd_item_keys(s, i)) : 0;
      int tot;
      const int ex = run + block_exclusive_scan(u * c, scan_sh, &tot);
      place(W, i, u, c, ex);
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

// One worker's share of one unit.
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

// Walks a worker's segments; every role of a CTA walks the same list.
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
      tiles = item < s.N ? pd_tiles(s, gs[item + 1] - gs[item]) : s.own;
      loaded = keys > 0 && tiles > 0;
      if (!loaded) {
        unit0 += tiles * s.Hkv;  // only read for prefixes
        ++item;
      }
    }
    const int c = pd_chunks(s, keys);
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

// The worker of `workers` that holds chunk x of W.
__device__ __forceinline__ int pd_worker_of(int x, int W, int workers) {
  const int P = min(workers, W);
  return static_cast<int>(((static_cast<int64_t>(x) + 1) * P - 1) / W);
}

}  // namespace csa
