// Work split of the shared-prefix decode, used by its attention kernels and
// by the merge.
//
// Every attention unit is a tile of query rows against a run of keys:
//   prefix units (n, h, tile): the queries of up to R rows of the sequences of
//     group n (row = sequence * G + head of the group) against prefix n;
//   own units (b, h): the G query heads of one sequence against its own cache.
// Units go to one of two lines by their kind and by their group's rows.  The
// lines run side by side in one launch, each on the share of the CTAs (one per
// SM) that its keys are of all (as two launches, the second's CTAs wait for SMs
// at both ends: 42 against 32 us for 32 sequences over 8K tokens).  A unit's
// keys are cut into chunks.  A unit is `lead` places, for what it costs besides
// its keys, and its chunks; all units of a line lie end to end (prefixes first;
// within a prefix by head, then row tile; own units by sequence, then head)
// and worker c (a CTA, or a warp) of P takes places [W c / P, W (c + 1) / P): every
// worker has the same to do whatever the lengths.  A worker that holds any of
// unit i's chunks writes one partial (normalised rows and their log2-sum-exp)
// to slot c + i: the pairs (c, i) met along the line grow by one in c or in i at
// a time, so slots are distinct and number at most P + units.
#pragma once

#include "internal.h"
#include "prefix_split.h"

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
  float inv_R;
  int ctas;                    // CTAs that the lines share (0: no such line)
  int workers;                 // workers per CTA, at most 8
  int spread;                  // worker k of CTA c is number c + k * CTAs (0: c * workers + k)
  int chunk_log2;              // keys per chunk
  int lead;                    // places before a unit's chunks
  int min_rows, max_rows;      // prefix units of groups of so many rows
  int own;                     // own units too
  float cost;                  // of a chunk, relative to the other line's
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
// Item i: prefix i, or the own cache of sequence i - N.  Its keys as they
// stand in memory (pd_raw_keys), and sanitised.
__device__ __forceinline__ int pd_raw_keys(const PdShape& s, int i) {
  if (i < s.N) return s.prefix_len ? __ldg(s.prefix_len + i) : static_cast<int>(s.Tp);
  if (s.T == 0) return 0;
  return s.len ? __ldg(s.len + i - s.N) : static_cast<int>(s.T);
}
__device__ __forceinline__ int pd_item_keys(const PdShape& s, int i) {
  return i < s.N ? pd_prefix_len(s, i) : pd_own_len(s, i - s.N);
}
__device__ __forceinline__ int pd_chunks(const PdShape& s, int keys) {
  return (keys + (1 << s.chunk_log2) - 1) >> s.chunk_log2;
}
// Places of a unit of so many keys.
__device__ __forceinline__ int pd_places(const PdShape& s, int keys) {
  return keys > 0 ? s.lead + pd_chunks(s, keys) : 0;
}
// Row tiles of a group of `seqs` sequences (0: the group is not on this line).
__device__ __forceinline__ int pd_tiles(const PdShape& s, int seqs) {
  const int rows = seqs * s.G;
  // ceil(rows / R): rows < 2^20, so that the product is within 1 / 2R of it
  return rows < s.min_rows || rows > s.max_rows
             ? 0
             : static_cast<int>((static_cast<float>(rows + s.R) - 0.5f) * s.inv_R);
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

// A worker's stretch of the line: `left` places from place `off` of item `item`
// (of `keys` keys) on; unit0 prefix units lie before it (prefix items only).
struct PdStart {
  int left, item, off, unit0, keys;
};

// Shared memory of pd_locate: its result, and the scan's.
struct PdShared {
  PdStart st[8];       // the CTA's workers' stretches
  uint64_t scan[16];   // one entry per warp
  int na;              // CTAs on line a
};

// What the merge needs to find a unit's partials, written by one CTA.
struct PdPlan {
  int32_t* starts;  // [N + B + 2] first place of each item, then W, then P
  int32_t* ubase;   // [N] first unit of each prefix
  int32_t* gsan;    // [N + 1] the sanitised group bounds (line b's plan)
  int32_t* group;   // [B] each sequence's prefix, or -1 (line b's plan)
};

// Exclusive prefix sum over the block's first `warps` warps of two counts packed
// in 64 bits; `sh` holds one entry per warp.  Every thread of the block calls it.
__device__ __forceinline__ uint64_t pd_scan(uint64_t v, uint64_t* sh, int warps, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
  if (warp < warps) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh[warp] = x;
  }
  __syncthreads();
  uint64_t before = 0, all = 0;
#pragma unroll 4
  for (int w = 0; w < warps; ++w) {
    const uint64_t y = sh[w];
    before += w < warp ? y : 0;
    all += y;
  }
  *total = all;
  return before + x - v;
}

// W places over P < 2^11 workers, P <= W < 2^31.
struct PdCut {
  int P, q, r;  // W = q P + r
  float inv_P, per_place;
  __device__ __forceinline__ PdCut(int W, int workers) : P(workers), q(W / workers) {
    r = W - q * P;
    inv_P = __frcp_rn(static_cast<float>(P));
    per_place = static_cast<float>(P) / static_cast<float>(W);
  }
  // Places before worker c <= P: floor(W c / P).  r c < 2^22 is exact, and (r c +
  // 1/2) / P lies 1 / 2P = 2^-12 or more from the integers, its error (two
  // roundings of 2^-24 of less than 2^11) below that.
  __device__ __forceinline__ int before(int c) const {
    return q * c + static_cast<int>((static_cast<float>(r * c) + 0.5f) * inv_P);
  }
  // The worker that holds place x: (x + 1/2) P / W is within one of it.
  __device__ __forceinline__ int worker_of(int x) const {
    const int c = min(P - 1, static_cast<int>((static_cast<float>(x) + 0.5f) * per_place));
    return before(c) > x ? c - 1 : before(c + 1) <= x ? c + 1 : c;
  }
};

// What a CTA works on.
struct PdPlace {
  int line;   // 0: a, 1: b
  int block;  // its number on that line
};

// Block-wide: the CTA's line, and ps->st, the places of its workers there.
// `gs` (shared) is filled by pd_groups before a barrier; key0 = pd_raw_keys of
// item threadIdx.x, loaded before that barrier (any value for threads past the
// items).  One CTA passes plans to write.  Only the warps that hold an
// item take part.
__device__ __forceinline__ PdPlace pd_locate(const PdShape& a, const PdShape& b, const int* gs,
                                             int key0, PdShared* ps, const PdPlan* plan_a,
                                             const PdPlan* plan_b) {
  const int items = b.N + b.B, nt = blockDim.x, tid = threadIdx.x, lane = tid & 31;
  const bool two = a.ctas > 0;
  const bool one = items <= nt;  // one item per thread
  const int warps = one ? (items + 31) >> 5 : nt >> 5;
  auto units = [&](const PdShape& s, int i) -> int {
    return i < s.N ? pd_tiles(s, gs[i + 1] - gs[i]) * s.Hkv : s.own ? s.Hkv : 0;
  };
  auto keys_of = [&](int i, int raw) { return pd_clamp(raw, i < b.N ? b.Tp : b.T, b.err); };
  // places of item i: line a in the high half, line b in the low one
  auto weigh = [&](int i, int keys) -> uint64_t {
    if (i >= items) return 0;
    const uint32_t nb = units(b, i) * pd_places(b, keys);
    const uint32_t na = two && i < b.N ? units(a, i) * pd_places(a, keys) : 0;
    return static_cast<uint64_t>(na) << 32 | nb;
  };
  auto raw_of = [&](int i) { return i < items ? pd_raw_keys(b, i) : 0; };
  if (tid < 8) ps->st[tid].left = 0;
  uint64_t total = 0, v = 0, ex = 0;
  int keys = 0;
  if (one) {
    if (tid < items) keys = keys_of(tid, key0);
    v = weigh(tid, keys);
    ex = pd_scan(v, ps->scan, warps, &total);
  } else {
    for (int i0 = 0; i0 < items; i0 += nt) {
      const int i = i0 + tid;
      uint64_t tot;
      pd_scan(weigh(i, i < items ? keys_of(i, raw_of(i)) : 0), ps->scan, warps, &tot);
      total += tot;
      __syncthreads();  // the scan's memory is used again
    }
  }
  int na = 0;
  if (tid >> 5 < warps) {
    const int Wa = static_cast<int>(total >> 32), Wb = static_cast<int>(total & 0xffffffffu);
    // line a's CTAs: its share of the keys, at least one for each line with work
    if (Wa > 0)
      na = pd_line_a_ctas(Wa * a.cost, Wb * b.cost, b.ctas, b.N == 1 ? units(a, 0) : 0,
                          a.lead * a.cost);
    if (tid == 0) ps->na = na;
    // each worker that takes part has a place
    const int Pa = max(1, min(na, Wa)), Pb = max(1, min((b.ctas - na) * b.workers, Wb));
    const bool on_a = static_cast<int>(blockIdx.x) < na;
    const PdShape& me = on_a ? a : b;
    const int block = static_cast<int>(blockIdx.x) - (on_a ? 0 : na);
    const int W = on_a ? Wa : Wb, P = on_a ? Pa : Pb, nw = me.workers;
    // lane k: worker k's bounds
    const int wk = min(lane, nw);
    const int c_lane = me.spread ? wk * b.ctas + block : block * nw + wk;
    const PdCut cut(max(1, W), P);
    const int x_lane = cut.before(min(P, c_lane)), xe_lane = cut.before(min(P, c_lane + 1));
    // this warp's 32 items, from item i0 on: lane k looks worker k's first place up
    // among them (the last item that starts at or before it)
    auto place = [&](int i0, int n_keys, uint64_t at, uint64_t mine) {
      const int e = static_cast<int>(on_a ? at >> 32 : at & 0xffffffffu);
      const int n = static_cast<int>(on_a ? mine >> 32 : mine & 0xffffffffu);
      int k = 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (__shfl_sync(0xffffffffu, e, k + o) <= x_lane) k += o;
      const int ek = __shfl_sync(0xffffffffu, e, k), nk = __shfl_sync(0xffffffffu, n, k);
      const int keys_k = __shfl_sync(0xffffffffu, n_keys, k);
      if (lane < nw && xe_lane > x_lane && x_lane >= ek && x_lane < ek + nk) {
        const int i = i0 + k;
        int before = 0;
        if (i < me.N)
          for (int m = 0; m < i; ++m) before += units(me, m);
        ps->st[lane] = PdStart{xe_lane - x_lane, i, x_lane - ek, before, keys_k};
      }
    };
    auto write = [&](int i, uint64_t at) {
      if (i >= items) return;
      if (plan_a) plan_a->starts[i] = static_cast<int>(at >> 32);
      if (plan_b) plan_b->starts[i] = static_cast<int>(at & 0xffffffffu);
    };
    if (one) {
      place(tid & ~31, keys, ex, v);
      write(tid, ex);
    } else {
      uint64_t run = 0;
      for (int i0 = 0; i0 < items; i0 += nt) {
        const int i = i0 + tid;
        uint64_t tot;
        const int n_keys = i < items ? keys_of(i, raw_of(i)) : 0;
        const uint64_t w = weigh(i, n_keys);
        const uint64_t at = run + pd_scan(w, ps->scan, warps, &tot);
        place(i & ~31, n_keys, at, w);
        write(i, at);
        run += tot;
        __syncthreads();
      }
    }
    auto finish = [&](const PdShape& s, const PdPlan* plan, int Wl, int Pl) {
      if (plan == nullptr || tid != 0) return;
      plan->starts[items] = Wl;
      plan->starts[items + 1] = Pl;
      int u = 0;
      for (int n = 0; n < s.N; ++n) {
        plan->ubase[n] = u;
        u += units(s, n);
      }
    };
    finish(a, plan_a, Wa, Pa);
    finish(b, plan_b, Wb, Pb);
  }
  if (plan_b) {
    if (b.N > 0 && tid <= b.N) plan_b->gsan[tid] = gs[tid];
    for (int q = tid; q < b.B; q += nt) {
      int g = -1;
      for (int n = 0; n < b.N; ++n)
        if (gs[n] <= q && q < gs[n + 1]) g = n;
      plan_b->group[q] = g;
    }
  }
  __syncthreads();
  na = ps->na;
  const bool on_a = static_cast<int>(blockIdx.x) < na;
  return PdPlace{on_a ? 0 : 1, static_cast<int>(blockIdx.x) - (on_a ? 0 : na)};
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
  int left, item, h = 0, tile = 0, j = 0, unit0;  // j: place in the unit
  int off;                  // places of `item` before the start
  int keys, tiles;          // of `item`, once loaded
  bool loaded;
  __device__ __forceinline__ PdWalk(const PdShape& sh, const int* g, const PdStart& st)
      : s(sh), gs(g), left(st.left), item(st.item), unit0(st.unit0), off(st.off), keys(st.keys) {
    loaded = left > 0;  // the first item has places
    if (loaded) tiles = tiles_of(item);
  }
  __device__ __forceinline__ int tiles_of(int i) const {
    return i < s.N ? pd_tiles(s, gs[i + 1] - gs[i]) : s.own;
  }
  __device__ __forceinline__ bool next(PdSeg& q) {
    while (left > 0) {
      if (!loaded) {
        if (item >= s.N + s.B) return false;
        keys = pd_item_keys(s, item);
        tiles = tiles_of(item);
        loaded = keys > 0 && tiles > 0;
        if (!loaded) {
          unit0 += tiles * s.Hkv;  // only read for prefixes
          ++item;
          continue;
        }
      }
      const int c = pd_places(s, keys);
      if (off > 0) {  // the first segment of all
        const int ui = off / c;
        h = ui / tiles;
        tile = ui - h * tiles;
        j = off - ui * c;
        off = 0;
        if (h >= s.Hkv) return false;  // the lengths have changed since: nothing past the heads
      }
      q.own = item >= s.N;
      q.n = q.own ? 0 : item;
      q.b = q.own ? item - s.N : 0;
      q.h = h;
      q.keys = keys;
      q.unit = q.own ? q.b * s.Hkv + h : unit0 + h * tiles + tile;
      q.row0 = (q.own ? q.b : gs[item]) * s.G + tile * s.R;
      q.rows = q.own ? s.G : min(s.R, (gs[item + 1] - gs[item]) * s.G - tile * s.R);
      const int to = min(c, j + left);
      q.j0 = max(0, j - s.lead);
      q.j1 = max(0, to - s.lead);
      left -= to - j;
      j = to;
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
      if (q.j1 > q.j0) return true;  // (a stretch that ends in a unit's lead has none of it)
    }
    return false;
  }
};

}  // namespace csa
