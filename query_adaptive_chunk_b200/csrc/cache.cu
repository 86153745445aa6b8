// A bounded KV cache kept by accumulated attention weight: one token in at a
// time over the lightest (insert), or many rows into a smaller cache, the
// heaviest kept (compress).
//
// A slot of unit u = (b, h) is protected when its token's position is below
// n_sink or among the last n_local (>= next - n_local).  The others rank by
// weight; NaN counts as -inf, equal weights go by the lower slot.  The rank
// is taken on order-preserving 32-bit keys, so it is exact.
#include <algorithm>
#include <climits>

#include "internal.h"

namespace csa {
namespace {

constexpr uint32_t kKeyProtected = 0xffffffffu;

__device__ __forceinline__ uint32_t weight_key(float w) {
  return w != w ? 0x007fffffu /* -inf's key */ : float_key(w);
}

// `local`: the first of the last n_local positions.
__device__ __forceinline__ bool is_protected(int pos, int n_sink, int local) {
  return pos < n_sink || pos >= local;
}

// One row of `bytes` from src to dst by `n` threads (this one is `t`):
// 16-byte words when every row starts on one, else two bytes at a time (the
// narrowest element).
__device__ __forceinline__ void copy_row(void* dst, const void* src, int bytes, bool wide, int t,
                                         int n) {
  if (wide) {
    for (int i = t; i < bytes / 16; i += n)
      static_cast<uint4*>(dst)[i] = static_cast<const uint4*>(src)[i];
  } else {
    for (int i = t; i < bytes / 2; i += n)
      static_cast<uint16_t*>(dst)[i] = static_cast<const uint16_t*>(src)[i];
  }
}

// ---------------------------------------------------------------- insert
//
// Reads the unit's weights and positions once (8 bytes a slot), so it is
// bound by latency at the usual sizes: one CTA per unit, the minimum of
// (key << 32 | slot) over its threads, eight slots in flight per thread, then
// the first warps write the new row.  The sequence's length and next position are shared
// by its heads: each CTA reads them before it arrives at the sequence's
// counter, and the last one to arrive advances them and clears the counter.
// 4 sequences of 4 heads and 257 slots: 3.6 us; 64 of 8 heads and 4096 slots
// (17 MB, 2.7 us at the copy rate): 7.3 us.
constexpr int kInsThreads = 512;

__global__ void __launch_bounds__(kInsThreads) cache_insert_kernel(
    const CacheArgs c, const char* __restrict__ k, const char* __restrict__ v, int64_t kb,
    int64_t kh, int64_t vb, int64_t vh, int wide, DevErr err) {
  __shared__ int sh_len, sh_next;
  __shared__ unsigned long long sh_best[kInsThreads / 32];
  constexpr int U = 8;  // slots in flight per thread
  const int u = blockIdx.x, b = u / c.Hkv, h = u - b * c.Hkv, tid = threadIdx.x;
  const float* w = c.weights + static_cast<int64_t>(u) * c.T;
  const int32_t* pos = c.positions + static_cast<int64_t>(u) * c.T;
  float x[U];
  int p[U];
  auto load = [&](int j0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * kInsThreads;
      x[i] = j < c.budget ? w[j] : 0.f;
      p[i] = j < c.budget ? pos[j] : 0;
    }
  };
  int arrived = -1;
  if (tid == 0) {
    const int n = *static_cast<volatile int32_t*>(c.len + b);
    const int at = *static_cast<volatile int32_t*>(c.next_pos + b);
    sh_len = n;
    sh_next = at;
    __threadfence();
    if (at >= 0 && at < INT_MAX && n >= 0 && n <= c.budget) arrived = atomicAdd(c.counters + b, 1);
  }
  load(tid);  // most often the cache is full: its slots' loads go out beside the length's
  // and so do the new row's: K by the first 64 threads, V by the next, 16 bytes each
  const int es = c.bf16 ? 2 : 4, bytes = c.D * es;
  const bool is_v = tid >= 64, ahead = wide && bytes <= 1024;
  const char* from = is_v ? v + (b * vb + h * vh) * es : k + (b * kb + h * kh) * es;
  const int off = (tid & 63) * 16;
  uint4 row = make_uint4(0u, 0u, 0u, 0u);
  if (ahead && tid < 128 && off < bytes) row = *reinterpret_cast<const uint4*>(from + off);
  __syncthreads();
  const int len = sh_len, next = sh_next;
  if (next < 0) return;  // an inactive sequence: left alone
  if (len < 0 || len > c.budget || next == INT_MAX) {  // (no position would follow)
    if (tid == 0) dev_flag(err, DEV_BAD_INDEX);
    return;
  }
  int slot = len;
  if (len == c.budget) {
    unsigned long long best = ~0ull;
    for (int j0 = tid; j0 < len; j0 += U * kInsThreads) {
      if (j0 != tid) load(j0);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int j = j0 + i * kInsThreads;
        if (j < len && !is_protected(p[i], c.n_sink, next - c.n_local)) {
          const unsigned long long e =
              (static_cast<unsigned long long>(weight_key(x[i])) << 32) | static_cast<unsigned>(j);
          best = e < best ? e : best;
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long e = __shfl_xor_sync(0xffffffffu, best, o);
      best = e < best ? e : best;
    }
    if ((tid & 31) == 0) sh_best[tid >> 5] = best;
    __syncthreads();
    best = sh_best[tid & (kInsThreads / 32 - 1)];
#pragma unroll
    for (int o = kInsThreads / 64; o > 0; o >>= 1) {
      const unsigned long long e = __shfl_xor_sync(0xffffffffu, best, o);
      best = e < best ? e : best;
    }
    slot = best == ~0ull ? -1 : static_cast<int>(best & 0xffffffffu);
  }
  if (slot >= 0) {
    if (tid < 128) {
      char* to = is_v ? static_cast<char*>(c.V) + (b * c.vst[0] + h * c.vst[1] + slot * c.vst[2]) * es
                      : static_cast<char*>(c.K) + (b * c.kst[0] + h * c.kst[1] + slot * c.kst[2]) * es;
      if (!ahead)
        copy_row(to, from, bytes, wide, tid & 63, 64);
      else if (off < bytes)
        *reinterpret_cast<uint4*>(to + off) = row;
    } else if (tid == 128)
      c.weights[static_cast<int64_t>(u) * c.T + slot] = 0.f;
    else if (tid == 160)
      c.positions[static_cast<int64_t>(u) * c.T + slot] = next;
  } else if (tid == 0) {
    dev_flag(err, DEV_BAD_INDEX);  // every slot protected: positions are not distinct
  }
  if (arrived == c.Hkv - 1) {  // thread 0 of the sequence's last head to have read these
    __threadfence();
    c.counters[b] = 0;
    c.len[b] = len < c.budget ? len + 1 : len;
    c.next_pos[b] = next + 1;
  }
}

// ---------------------------------------------------------------- compress
//
// Selection: one cluster of CS <= 8 CTAs per unit, CTA r holding the keys of rows
// [n r / CS, n (r + 1) / CS) in shared memory (re-read from memory when they
// do not fit).  An MSB-first radix select over the keys' bytes finds the
// budget-th largest key tau, the CTAs' histograms of each pass added through
// distributed shared memory; keys equal to tau are taken lowest row first.
// Each CTA writes its kept rows, ascending, into the destination's positions
// (as row numbers; the copy turns them into positions).  Each warp takes a run of
// consecutive keys, four a lane (histograms by atomics on one copy per warp; a
// match of equal buckets first took four times as long).  A warp's keys above tau
// are counted in its histograms.  The weights are read once, sixteen a thread in
// flight; bound by the passes' latency (four, one cluster barrier each, 2 us a
// pass of few keys) and, with 16K keys a CTA, by the instructions over them.  8
// units of 128K rows: 19 of the call's 31 us, 64 units of 8K rows: 12 of 21.
// CTAs of more keys than this have 1024 threads where each has an SM, the others
// 512 (8 units of 128K rows, 64 CTAs of 16K keys: 31 against 34 us; 128 units of
// 20K, a CTA each: 29 against 31; 32 units of 70K as 256 CTAs: 52 against 30, the
// second half waits for the first).
constexpr int kCmpMany = 8192;
constexpr int kCmpKeys = 45056;  // keys held per CTA (176 KB)

struct CompressParams {
  const float* weights;        // [U, S]
  const int32_t* positions;    // [U, S] or null: the row number
  const int32_t* len;          // [B] or null: S
  const int32_t* next_pos;     // [B] or null: the length
  int64_t S;
  int Hkv, budget, n_sink, n_local;
  int64_t T;
  int32_t* rows;               // destination positions [U, T]
  int held;                    // keys are held in shared memory
  DevErr err;
};

__device__ __forceinline__ int source_len(const int32_t* len, int b, int64_t S, const DevErr& e) {
  if (len == nullptr) return static_cast<int>(S);
  int n = len[b];
  if (n < 0 || n > S) {
    dev_flag(e, DEV_BAD_INDEX);
    n = n < 0 ? 0 : static_cast<int>(S);
  }
  return n;
}

// Four consecutive keys from j on (j a multiple of four); 0, which no key is, for
// those at or past n.
struct Keys4 {
  uint32_t k[4];
};

template <int CS, int kCmpThreads>
__global__ void __launch_bounds__(kCmpThreads) compress_select_kernel(const CompressParams p) {
  if (CS > 1) cluster_arrive_relaxed();
  pdl_next();  // the copy
  constexpr int kWarps = kCmpThreads / 32;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ unsigned int hw[kWarps][256];  // a histogram per warp: no contention between them
  __shared__ unsigned int hc[2][256];       // this CTA's, for the pass's parity
  __shared__ unsigned int gc[256];          // the cluster's
  __shared__ unsigned int part[2][CS];      // keys above tau and at tau of each CTA
  __shared__ unsigned int warp_part[2][kWarps];
  __shared__ unsigned int pick_sh[2];
  __shared__ int warp_last[kWarps], last[CS];  // largest positions (inactive sequences)
  const int rank = CS > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int u = blockIdx.x / CS, b = u / p.Hkv, tid = threadIdx.x, lane = tid & 31;
  const int warp = tid >> 5;
  const int len = source_len(p.len, b, p.S, p.err);
  const int next = p.next_pos ? p.next_pos[b] : len;
  const int lo = static_cast<int>(static_cast<int64_t>(len) * rank / CS);
  const int n = static_cast<int>(static_cast<int64_t>(len) * (rank + 1) / CS) - lo;
  const float* wrow = p.weights + static_cast<int64_t>(u) * p.S + lo;
  const int32_t* prow = p.positions ? p.positions + static_cast<int64_t>(u) * p.S + lo : nullptr;
  const bool select = len > p.budget;
  int32_t* out = p.rows + static_cast<int64_t>(u) * p.T;
  if (CS > 1) cluster_wait();  // every CTA of the cluster is running
  if (!select) {  // uniform over the cluster: all rows stay
    for (int j = tid; j < n; j += kCmpThreads) out[lo + j] = lo + j;
    return;
  }
  // An inactive sequence does not say where it stands: right behind its last row's
  // position (the same branch for the whole cluster).
  int64_t behind = next;
  if (next < 0) {
    if (prow == nullptr) {
      behind = len;
    } else {
      int most = INT_MIN;
      for (int j = tid; j < n; j += kCmpThreads) most = max(most, prow[j]);
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) warp_last[warp] = most;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) most = max(most, warp_last[w]);
      if (CS > 1) {
        if (tid < CS)
          st_cluster_u32(cluster_map(smem_u32(&last[rank]), tid), static_cast<uint32_t>(most));
        cluster_arrive();
        cluster_wait();
        for (int r = 0; r < CS; ++r) most = max(most, last[r]);
      }
      behind = static_cast<int64_t>(most) + 1;
    }
  }
  const int local = static_cast<int>(
      min(static_cast<int64_t>(INT_MAX), max(static_cast<int64_t>(INT_MIN), behind - p.n_local)));
  auto make_key = [&](float w, int pos) -> uint32_t {
    return is_protected(pos, p.n_sink, local) ? kKeyProtected : weight_key(w);
  };
  const bool held = p.held != 0;
  if (held) {
    constexpr int U = 16;  // loads in flight
    for (int j0 = tid; j0 < n; j0 += U * kCmpThreads) {
      float w[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int j = j0 + i * kCmpThreads;
        w[i] = j < n ? wrow[j] : 0.f;
      }
      if (prow == nullptr) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int j = j0 + i * kCmpThreads;
          if (j < n) keys[j] = make_key(w[i], lo + j);
        }
      } else {
        int pos[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int j = j0 + i * kCmpThreads;
          pos[i] = j < n ? prow[j] : 0;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int j = j0 + i * kCmpThreads;
          if (j < n) keys[j] = make_key(w[i], pos[i]);
        }
      }
    }
  }
  __syncthreads();
  auto keys_at = [&](int j) -> Keys4 {
    Keys4 k;
    if (held) {
      const uint4 x = *reinterpret_cast<const uint4*>(keys + j);  // (the buffer is whole fours)
      k.k[0] = x.x;
      k.k[1] = x.y;
      k.k[2] = x.z;
      k.k[3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        k.k[i] = j + i < n ? make_key(wrow[j + i], prow ? prow[j + i] : lo + j + i) : 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j + i >= n) k.k[i] = 0u;
    return k;
  };
  // this warp's run of the CTA's rows, a multiple of 128 rows from its start
  const int run = (n + kWarps * 128 - 1) / (kWarps * 128) * 128;
  const int s0 = min(n, warp * run), s1 = min(n, s0 + run);
  // keys > tau are taken, and the first `need` keys equal to tau
  uint32_t prefix = 0u, mask = 0u;
  unsigned int need = static_cast<unsigned int>(p.budget);
  unsigned int c_gt = 0u, c_eq = 0u;  // this warp's keys above tau and at tau
  for (int shift = 24; shift >= 0; shift -= 8) {
    unsigned int* mine = hc[(shift >> 3) & 1];
    for (int d = lane; d < 256; d += 32) hw[warp][d] = 0u;
    __syncwarp();
    for (int j = s0 + 4 * lane; j < s1; j += 128) {
      const Keys4 k = keys_at(j);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k.k[i] != 0u && (k.k[i] & mask) == prefix) atomicAdd(&hw[warp][(k.k[i] >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid < 256) {
      unsigned int sum = 0u;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += hw[w][tid];
      mine[tid] = sum;
      if (CS == 1) gc[tid] = sum;
    }
    if (CS > 1) {
      // every CTA's histogram of this pass is complete.  The buffer is written
      // again two passes on, behind the next pass's barrier: by then all have
      // read it.
      cluster_arrive();
      cluster_wait();
      if (tid < 256) {
        unsigned int cr[CS], cnt = 0u;
#pragma unroll
        for (int r = 0; r < CS; ++r) cr[r] = ld_cluster_u32(cluster_map(smem_u32(mine + tid), r));
#pragma unroll
        for (int r = 0; r < CS; ++r) cnt += cr[r];
        gc[tid] = cnt;
      }
    }
    __syncthreads();
    if (tid < 32) {  // the bucket where the count from the top reaches `need`
      unsigned int pc[8], lc = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pc[i] = gc[255 - 8 * lane - i];
        lc += pc[i];
      }
      unsigned int sc = lc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned int t = __shfl_up_sync(0xffffffffu, sc, o);
        if (lane >= o) sc += t;
      }
      unsigned int above = sc - lc;  // count in the buckets above this lane's eight
      int sel = -1;
      unsigned int above_sel = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (sel < 0) {
          if (above + pc[i] >= need) {
            sel = 255 - 8 * lane - i;
            above_sel = above;
          } else {
            above += pc[i];
          }
        }
      }
      // `need` never exceeds the count of keys under the prefix: a bucket is hit
      const unsigned int hit = __ballot_sync(0xffffffffu, sel >= 0);
      if (lane == (hit ? __ffs(hit) - 1 : 0)) {
        pick_sh[0] = sel < 0 ? 0u : static_cast<unsigned int>(sel);
        pick_sh[1] = above_sel;
      }
    }
    __syncthreads();
    prefix |= pick_sh[0] << shift;
    mask |= 255u << shift;
    need -= pick_sh[1];
    // this warp's keys above the bucket, and in it, from its own histogram
    const unsigned int sel = pick_sh[0];
    unsigned int over = 0u;
#pragma unroll
    for (int d = lane; d < 256; d += 32) over += static_cast<unsigned int>(d) > sel ? hw[warp][d] : 0u;
    c_gt += __reduce_add_sync(0xffffffffu, over);
    c_eq = hw[warp][sel];
    __syncwarp();  // read before it is cleared for the next pass
  }
  const uint32_t tau = prefix;
  if (lane == 0) {
    warp_part[0][warp] = c_gt;
    warp_part[1][warp] = c_eq;
  }
  __syncthreads();
  unsigned int gt = 0, eq = 0;  // before this warp
  for (int w = 0; w < warp; ++w) {
    gt += warp_part[0][w];
    eq += warp_part[1][w];
  }
  if (CS > 1) {
    if (tid < CS) {
      unsigned int a0 = 0, a1 = 0;
      for (int w = 0; w < kWarps; ++w) {
        a0 += warp_part[0][w];
        a1 += warp_part[1][w];
      }
      st_cluster_u32(cluster_map(smem_u32(&part[0][rank]), tid), a0);
      st_cluster_u32(cluster_map(smem_u32(&part[1][rank]), tid), a1);
    }
    cluster_arrive();
    cluster_wait();  // the last access to another CTA's shared memory is before this barrier
    for (int r = 0; r < rank; ++r) {
      gt += part[0][r];
      eq += part[1][r];
    }
  }
  // Row j goes behind the keys above tau and the kept ties before it: those of
  // the lanes below, which have four rows each, by a vote for each of the four.
  const unsigned int lower = (1u << lane) - 1u;
  for (int j0 = s0; j0 < s1; j0 += 128) {
    const int j = j0 + 4 * lane;
    Keys4 k{};
    if (j < s1) k = keys_at(j);
    unsigned int g = gt, all = 0u, ties = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned int v = __ballot_sync(0xffffffffu, k.k[i] > tau);
      g += __popc(v & lower);
      all += __popc(v);
      ties |= k.k[i] == tau && k.k[i] != 0u ? 1u << i : 0u;
    }
    if (!__any_sync(0xffffffffu, ties != 0u)) {
      unsigned int to = g + min(eq, need);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k.k[i] > tau) {
          if (to < static_cast<unsigned int>(p.budget)) out[to] = lo + j + i;
          ++to;
        }
    } else {
      unsigned int q = eq;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned int v = __ballot_sync(0xffffffffu, ties >> i & 1u);
        q += __popc(v & lower);
        eq += __popc(v);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool above = k.k[i] > tau, tie = ties >> i & 1u;
        const unsigned int to = g + min(q, need);
        if ((above || (tie && q < need)) && to < static_cast<unsigned int>(p.budget)) out[to] = lo + j + i;
        g += above;
        q += tie;
      }
    }
    gt += all;
  }
}

// ---------------------------------------------------------------- copy
// Copy: destination slot i of unit u gets source row rows[u, i] (K, V, the
// weight), and rows[u, i] becomes the row's position.  Bound by HBM: a warp
// takes kCopyRows rows, half of its lanes the K rows and half the V rows,
// every load of the warp in flight before its first store.  8 units of 8K rows
// of D = 128 in bf16 (67 MB read and written): 12 of the call's 31 us, 88% of the
// copy rate.
constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 4;

struct CopyParams {
  CacheArgs dst;
  const char *K, *V;
  int64_t kst[3], vst[3];
  const float* weights;
  const int32_t* positions;
  const int32_t* len;
  const int32_t* next_pos;
  int64_t S;
  int wide;
  DevErr err;
};

__global__ void __launch_bounds__(kCopyThreads) compress_copy_kernel(const CopyParams p) {
  pdl_wait();  // the row numbers are written
  const CacheArgs& d = p.dst;
  const int u = blockIdx.y, b = u / d.Hkv, h = u - b * d.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = source_len(p.len, b, p.S, p.err);
  const int kept = min(len, d.budget);
  const int i0 = (blockIdx.x * (kCopyThreads / 32) + warp) * kCopyRows;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) {
    const int next = p.next_pos ? p.next_pos[b] : len;
    d.len[b] = kept;
    if (d.next_pos) d.next_pos[b] = next;
  }
  if (i0 >= kept) return;
  int32_t* rows = d.positions + static_cast<int64_t>(u) * d.T;
  const int es = d.bf16 ? 2 : 4, bytes = d.D * es;
  const int nr = min(kCopyRows, kept - i0);
  int mine = lane < nr ? rows[i0 + lane] : 0;
  if (lane < nr) {
    if (mine < 0 || mine >= len) {  // cannot happen; never read past the source
      dev_flag(p.err, DEV_BAD_INDEX);
      mine = 0;
    }
    const int64_t src = static_cast<int64_t>(u) * p.S + mine;
    d.weights[static_cast<int64_t>(u) * d.T + i0 + lane] = p.weights[src];
    rows[i0 + lane] = p.positions ? p.positions[src] : mine;
  }
  const bool is_v = lane >= 16;
  const int t = lane & 15;
  const char* sp = is_v ? p.V + (b * p.vst[0] + h * p.vst[1]) * es
                        : p.K + (b * p.kst[0] + h * p.kst[1]) * es;
  char* dp = is_v ? static_cast<char*>(d.V) + (b * d.vst[0] + h * d.vst[1]) * es
                  : static_cast<char*>(d.K) + (b * d.kst[0] + h * d.kst[1]) * es;
  const int64_t ss = (is_v ? p.vst[2] : p.kst[2]) * es, ds = (is_v ? d.vst[2] : d.kst[2]) * es;
  int row[kCopyRows];
#pragma unroll
  for (int r = 0; r < kCopyRows; ++r) row[r] = __shfl_sync(0xffffffffu, mine, r);
  if (p.wide) {
    for (int o = t * 16; o < bytes; o += 256) {
      uint4 x[kCopyRows];
#pragma unroll
      for (int r = 0; r < kCopyRows; ++r)
        if (r < nr) x[r] = __ldcs(reinterpret_cast<const uint4*>(sp + row[r] * ss + o));
#pragma unroll
      for (int r = 0; r < kCopyRows; ++r)
        if (r < nr) *reinterpret_cast<uint4*>(dp + (i0 + r) * ds + o) = x[r];
    }
  } else {
    for (int r = 0; r < nr; ++r) copy_row(dp + (i0 + r) * ds, sp + row[r] * ss, bytes, false, t, 16);
  }
}

template <int CS, int kCmpThreads>
cudaError_t launch_select_threads(const Launch& l, const CompressParams& p, int U, size_t smem) {
  const void* fn = reinterpret_cast<const void*>(compress_select_kernel<CS, kCmpThreads>);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(U) * CS);
  cfg.blockDim = dim3(kCmpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, compress_select_kernel<CS, kCmpThreads>, p);
}

template <int CS>
cudaError_t launch_compress_select(const Launch& l, const CompressParams& p, int U, size_t smem) {
  if ((p.S + CS - 1) / CS > kCmpMany && U * CS <= l.num_sms)
    return launch_select_threads<CS, 1024>(l, p, U, smem);
  return launch_select_threads<CS, 512>(l, p, U, smem);
}

// Rows of `st`-strided tensors at `ptr` all start on a 16-byte boundary.
bool rows_wide(const void* ptr, const int64_t* st, int n, int es, int D) {
  bool ok = reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && (D * es) % 16 == 0;
  for (int i = 0; i < n; ++i) ok = ok && (st[i] * es) % 16 == 0;
  return ok;
}

}  // namespace

cudaError_t launch_cache_insert(const Launch& l, const CacheArgs& c, const void* k,
                                const int64_t* kst, const void* v, const int64_t* vst) {
  const int es = c.bf16 ? 2 : 4;
  const bool wide = rows_wide(c.K, c.kst, 3, es, c.D) && rows_wide(c.V, c.vst, 3, es, c.D) &&
                    rows_wide(k, kst, 2, es, c.D) && rows_wide(v, vst, 2, es, c.D);
  cache_insert_kernel<<<c.B * c.Hkv, kInsThreads, 0, l.stream>>>(
      c, static_cast<const char*>(k), static_cast<const char*>(v), kst[0], kst[1], vst[0], vst[1],
      wide ? 1 : 0, l.err);
  return cudaGetLastError();
}

cudaError_t launch_cache_compress(const Launch& l, const CacheArgs& dst, const CacheSource& s) {
  const int U = dst.B * dst.Hkv, es = dst.bf16 ? 2 : 4;
  if (s.S > 0) {
    CompressParams p{s.weights, s.positions,  s.len,       s.next_pos, s.S,           dst.Hkv,
                     dst.budget, dst.n_sink, dst.n_local, dst.T,      dst.positions, 0,
                     l.err};
    // CTAs per unit: 2048 rows or more each, while each has an SM (two per SM: 32
    // units of 16K rows 19.0 against 16.8 us, 64 of 8K 21.8 against 20.9)
    int CS = 1;
    while (CS < 8 && s.S > 2048ll * CS && 2 * U * CS <= l.num_sms) CS *= 2;
    while (CS < 8 && (s.S + CS - 1) / CS > kCmpKeys) CS *= 2;
    const int64_t per = (s.S + CS - 1) / CS;
    p.held = per <= kCmpKeys ? 1 : 0;
    const size_t smem = p.held ? static_cast<size_t>(per + 3) / 4 * 16 : 0;  // fours of keys
    const cudaError_t e = CS == 1   ? launch_compress_select<1>(l, p, U, smem)
                          : CS == 2 ? launch_compress_select<2>(l, p, U, smem)
                          : CS == 4 ? launch_compress_select<4>(l, p, U, smem)
                                    : launch_compress_select<8>(l, p, U, smem);
    if (e != cudaSuccess) return e;
  }
  CopyParams p{};
  p.dst = dst;
  p.K = static_cast<const char*>(s.K);
  p.V = static_cast<const char*>(s.V);
  for (int i = 0; i < 3; ++i) {
    p.kst[i] = s.kst[i];
    p.vst[i] = s.vst[i];
  }
  p.weights = s.weights;
  p.positions = s.positions;
  p.len = s.len;
  p.next_pos = s.next_pos;
  p.S = s.S;
  p.wide = rows_wide(dst.K, dst.kst, 3, es, dst.D) && rows_wide(dst.V, dst.vst, 3, es, dst.D) &&
           rows_wide(s.K, s.kst, 3, es, dst.D) && rows_wide(s.V, s.vst, 3, es, dst.D);
  p.err = l.err;
  const int64_t most = std::min<int64_t>(dst.budget, s.S);
  const int per_block = kCopyThreads / 32 * kCopyRows;
  const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, (most + per_block - 1) / per_block)),
                  static_cast<unsigned>(U));
  return launch_behind(compress_copy_kernel, grid, dim3(kCopyThreads), 0, l.stream, p);
}

}  // namespace csa
