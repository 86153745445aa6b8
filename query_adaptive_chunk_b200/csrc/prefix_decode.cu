// One decode token per sequence over a prefix that several sequences share
// and over each sequence's own cache, the weights its own tokens received
// added to their running sums.
//
//   s_j = scale q.k_j over the keys of the sequence's prefix and of its cache,
//   lse = log sum_j exp(s_j),  out = sum_j exp(s_j - lse) v_j,
//   weights[b, h, j] <- decay weights[b, h, j] + sum_g exp(s_gj - lse_g).
//
// A prefix is read once for all the sequences of its group: their query rows
// are stacked into tiles against its keys (see prefix_work.cuh for the split
// over the SMs).  The attention kernels write partial rows; the merge below
// joins them and turns the own keys' logits, kept by the attention kernel (4
// bytes per head and key against 4 D for K and V), into weights.
#include <algorithm>
#include <cmath>

#include "prefix_decode.cuh"

namespace csa {
namespace {

// ------------------------------------------------------------------ fp32
//
// Plain fp32 products on the FMA pipe: a tile of up to 32 query rows against
// chunks of 32 keys held in shared memory.  Bound: with few rows HBM (a chunk
// is 256 D bytes), with 32 the FMA pipe (2 * 32 * 32 * D products a chunk).
// For the logits each warp takes a quarter of D for the whole tile, a thread up
// to eight rows by four keys (12 loads from shared memory to 128 products; four
// by two with all of D in each warp: 6 to 32, bound by those loads), and the
// quarters meet in shared memory, on the keys that have been read.  Rows and
// keys are dealt out in turn, so that a tile of few rows still has every warp
// at work.  Four workers of four warps to a CTA, one CTA per SM: the loads of
// one hide under the products of the others, and a short batch still fills
// the SMs.  8 sequences of 16 heads over 4K tokens and 511 own keys each: 32 us
// with the merge, about 23 here: 2 to the split, 4 for the first chunks (25 MB,
// all workers' at once), then one or two chunks a worker, 3 to 6 us each.
constexpr int kF32Rows = 32;
constexpr int kF32Threads = 128;
constexpr int kF32Workers = 4;  // per CTA, one CTA per SM
constexpr int kF32ChunkLog2 = 5, kF32Chunk = 1 << kF32ChunkLog2;
constexpr int kF32Lead = 1;  // a unit's queries and partials, in chunks' time

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// 16 bytes into shared memory, zeros if !in (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}

// A barrier of one worker's threads.
__device__ __forceinline__ void f32_meet(int worker) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + worker), "n"(kF32Threads) : "memory");
}

// Floats of shared memory of a worker: queries, values, weights, keys (the
// logits' quarters later).
__host__ __device__ constexpr int f32_floats(int D) {
  return kF32Rows * (D + 4) + kF32Chunk * D + kF32Rows * kF32Chunk +
         (D > 4 * kF32Rows - 4 ? kF32Chunk * (D + 4) : 4 * kF32Rows * kF32Chunk);
}

// Place of (row, key) in a tile of weights, 32 floats a row: rows of equal
// number mod 4 are turned alike, so that neither a thread's four keys nor
// a row's eight in sequence meet on a bank.
__device__ __forceinline__ int f32_place(int row, int key) {
  return row * kF32Chunk + ((key + 8 * (row & 3)) & (kF32Chunk - 1));
}

// This warp's quarter of D of the logits of rows 0 .. 4 RI - 1, into red once
// every warp has read the keys it lies on.
template <int D, int RI>
__device__ __forceinline__ void f32_logits(const float* sq, const float* sk, float* red, int worker,
                                           int warp, int lane) {
  constexpr int KS = D + 4;
  const int rg = lane >> 3, kg = lane & 7;
  const float* qa = sq + rg * KS + warp * (D / 4);
  const float* ka = sk + kg * KS + warp * (D / 4);
  float s[RI][4] = {};
#pragma unroll 2
  for (int d = 0; d < D / 4; d += 4) {
    float4 k[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) k[c] = ld4(ka + 8 * c * KS + d);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const float4 a = ld4(qa + 4 * i * KS + d);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        s[i][c] = fmaf(a.w, k[c].w, fmaf(a.z, k[c].z, fmaf(a.y, k[c].y, fmaf(a.x, k[c].x, s[i][c]))));
    }
  }
  f32_meet(worker);
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      red[warp * kF32Rows * kF32Chunk + f32_place(rg + 4 * i, kg + 8 * c)] = s[i][c];
}

// o += weights * v for rows ty + 8 i, i < RO, columns 64 e + 4 tx ...
template <int D, int RO>
__device__ __forceinline__ void f32_values(const float* ss, const float* al, const float* sv, int tx,
                                           int ty, float (&o)[kF32Rows / 8][D / 16]) {
#pragma unroll
  for (int r = 0; r < RO; ++r) {
    const float f = al[ty + 8 * r];
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[r][d] *= f;
  }
#pragma unroll 2
  for (int t = 0; t < kF32Chunk; t += 4) {
    float4 pw[RO];
#pragma unroll
    for (int r = 0; r < RO; ++r) pw[r] = ld4(ss + f32_place(ty + 8 * r, t));
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int d = 0; d < D / 64; ++d) {
        const float4 v = ld4(sv + (t + k) * D + d * 64 + tx * 4);
#pragma unroll
        for (int r = 0; r < RO; ++r) {
          const float w = k == 0 ? pw[r].x : k == 1 ? pw[r].y : k == 2 ? pw[r].z : pw[r].w;
          o[r][4 * d] += w * v.x;
          o[r][4 * d + 1] += w * v.y;
          o[r][4 * d + 2] += w * v.z;
          o[r][4 * d + 3] += w * v.w;
        }
      }
  }
}

template <int D>
__global__ void __launch_bounds__(kF32Workers* kF32Threads) attend_f32_kernel(const PdParams p) {
  constexpr int KS = D + 4;
  constexpr int D4 = D / 4;
  static_assert(kF32Threads == 4 * kF32Rows);
  extern __shared__ __align__(16) float sm[];
  const int worker = threadIdx.x / kF32Threads;
  float* sq = sm + worker * f32_floats(D);  // [32][KS]
  float* sv = sq + kF32Rows * KS;           // [32][D]
  float* ss = sv + kF32Chunk * D;           // [32][32], the weights
  float* sk = ss + kF32Rows * kF32Chunk;    // [32][KS]; then [4][32][32]: the logits' quarters
  float* red = sk;
  __shared__ int gs[kPdMaxPrefixes + 1];
  __shared__ PdShared ps;
  __shared__ float factors[kF32Workers][kF32Rows];  // of each row's output, a chunk's
  float* al = factors[worker];
  const int tid = threadIdx.x % kF32Threads, warp = tid >> 5, lane = tid & 31;
  const int tx = tid & 15, ty = tid >> 4;
  const int row = tid >> 2, key8 = (tid & 3) * 8;  // of the softmax
  const PdShape& shape = p.b.s;
  pdl_next();  // the merge
  const int item = static_cast<int>(threadIdx.x);
  const int key0 = item < shape.N + shape.B ? pd_raw_keys(shape, item) : 0;
  if (item < 32) pd_groups(shape, gs);
  __syncthreads();
  pd_locate(p.a.s, shape, gs, key0, &ps, nullptr, blockIdx.x == 0 ? &p.b.plan : nullptr);
  // from here on each worker by itself, with a barrier of its own
  auto meet = [worker] { f32_meet(worker); };
  PdWalk walk(shape, gs, ps.st[worker]);
  const int64_t number = static_cast<int64_t>(worker) * gridDim.x + blockIdx.x;
  PdSeg g;
  while (walk.next(g)) {
    const int64_t* kst = g.own ? p.ks : p.kps;
    const int64_t* vst = g.own ? p.vs : p.vps;
    const int64_t k0 = g.own ? g.b : g.n;
    const float* Kg = static_cast<const float*>(g.own ? p.K : p.Kp) + k0 * kst[0] + g.h * kst[1];
    const float* Vg = static_cast<const float*>(g.own ? p.V : p.Vp) + k0 * vst[0] + g.h * vst[1];
    const float* q = static_cast<const float*>(p.q);
    // a chunk's rows; those past the keys are zero: whatever the cache holds
    // there, 0 * v stays 0
    auto load = [&](float* to, int ld, const float* from, int64_t stride, int j) {
      const int t0 = j * kF32Chunk, nk = min(kF32Chunk, g.keys - t0);
#pragma unroll 4
      for (int i = tid; i < kF32Chunk * D4; i += kF32Threads) {
        const int t = i / D4, d = (i % D4) * 4;
        copy16(smem_u32(to + t * ld + d), t < nk ? from + (t0 + t) * stride + d : q, t < nk);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    {
      constexpr int kStep = kF32Threads / D4;  // rows from one pass to the next
      const int r0 = tid / D4, d = tid % D4 * 4;
      int b = (g.row0 + r0) / shape.G, hd = g.row0 + r0 - b * shape.G;
      for (int r = r0; r < kF32Rows; r += kStep) {
        const bool in = r < g.rows;
        const int64_t row = static_cast<int64_t>(b) * p.Hq + g.h * shape.G + hd;
        copy16(smem_u32(sq + r * KS + d), in ? q + row * D + d : q, in);
        for (hd += kStep; hd >= shape.G; hd -= shape.G) ++b;
      }
    }
    load(sk, KS, Kg, kst[2], g.j0);
    load(sv, D, Vg, vst[2], g.j0);
    float m = -INFINITY, l = 0.f;
    float o[kF32Rows / 8][D / 16];
#pragma unroll
    for (int r = 0; r < kF32Rows / 8; ++r)
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[r][d] = 0.f;
    for (int j = g.j0; j < g.j1; ++j) {
      const int t0 = j * kF32Chunk, nk = min(kF32Chunk, g.keys - t0);
      asm volatile("cp.async.wait_group 1;" ::: "memory");  // the keys
      meet();
      if (g.rows <= 4)
        f32_logits<D, 1>(sq, sk, red, worker, warp, lane);
      else if (g.rows <= 8)
        f32_logits<D, 2>(sq, sk, red, worker, warp, lane);
      else if (g.rows <= 16)
        f32_logits<D, 4>(sq, sk, red, worker, warp, lane);
      else
        f32_logits<D, 8>(sq, sk, red, worker, warp, lane);
      meet();
      if (warp * 8 < g.rows) {
        // four threads a row, eight keys each; odd rows take their second four
        // first (no bank twice)
        float s[8];
        const int at = f32_place(row, key8), odd = (row & 1) * 4;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (row < g.rows)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float4 y = ld4(red + w * kF32Rows * kF32Chunk + at + (e ^ odd));
              x.x += y.x;
              x.y += y.y;
              x.z += y.z;
              x.w += y.w;
            }
          const int k = key8 + (e ^ odd);
          s[e] = k < nk ? x.x * p.scale_log2 : -INFINITY;
          s[e + 1] = k + 1 < nk ? x.y * p.scale_log2 : -INFINITY;
          s[e + 2] = k + 2 < nk ? x.z * p.scale_log2 : -INFINITY;
          s[e + 3] = k + 3 < nk ? x.w * p.scale_log2 : -INFINITY;
          if (g.own && p.logits && row < g.rows)
            *reinterpret_cast<float4*>(
                p.logits + (static_cast<int64_t>(g.unit) * shape.G + row) * p.Tl + t0 + k) =
                make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
        }
        float mx = s[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) mx = fmaxf(mx, s[e]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - base);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[e] = exp2f(s[e] - base);
          sum += s[e];
        }
#pragma unroll
        for (int e = 0; e < 8; e += 4)
          *reinterpret_cast<float4*>(ss + at + (e ^ odd)) =
              make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        l = l * f + sum;
        m = mn;
        if ((tid & 3) == 0) al[row] = f;
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");  // the values
      meet();
      // the next keys under the products, the next values behind them
      const bool more = j + 1 < g.j1;
      if (more) load(sk, KS, Kg, kst[2], j + 1);
      if (g.rows <= 8) {
        if (ty < g.rows) f32_values<D, 1>(ss, al, sv, tx, ty, o);
      } else if (g.rows <= 16) {
        f32_values<D, 2>(ss, al, sv, tx, ty, o);
      } else {
        f32_values<D, 4>(ss, al, sv, tx, ty, o);
      }
      meet();  // the chunk, and after the last one the queries, have been read
      if (more) load(sv, D, Vg, vst[2], j + 1);
    }
    const int64_t slot = number + g.unit;
    const int rows = g.own ? shape.G : p.b.slot_rows;
    float* po = (g.own ? p.oo : p.b.po) + slot * rows * D;
    float* pl = (g.own ? p.olse : p.b.plse) + slot * rows;
    if (row < g.rows && (tid & 3) == 0) {
      al[row] = l == 0.f ? 0.f : 1.f / l;  // a NaN stays one
      pl[row] = l == 0.f ? -INFINITY : m + log2f(l);
    }
    meet();
#pragma unroll
    for (int r = 0; r < kF32Rows / 8; ++r) {
      const int orow = ty + 8 * r;
      if (orow < g.rows) {
        const float inv = al[orow];
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
          *reinterpret_cast<float4*>(po + static_cast<int64_t>(orow) * D + d * 64 + tx * 4) =
              make_float4(o[r][4 * d] * inv, o[r][4 * d + 1] * inv, o[r][4 * d + 2] * inv,
                          o[r][4 * d + 3] * inv);
      }
    }
  }
}

// ------------------------------------------------------------------ merge
//
// A CTA joins a share of the partials of one (sequence, KV head) into the
// output and adds the weights of a share of its own keys.  Reads the
// partials once (they sit in L2) and 4 bytes per head and own key.  Bound by
// latency at the usual sizes, so each step's loads go out together: where the
// partials lie, their lse, then their rows and the logits.  The shares (of the
// output's columns and of the own keys) are as many as keep every SM busy with
// a few CTAs each.  5 to 8 us after the attention kernel's end for 4 to 32
// sequences.
constexpr int kMergeThreads = 256;
constexpr int kMergeMinKeys = 1024;  // own keys per share at least
constexpr int kMaxG = 16;
constexpr int kMergeKept = 128;  // partials of a head whose weights are kept in shared memory
constexpr int kMergeAhead = 4;   // heads whose logits are fetched ahead

// Partials of one query head: `np` of its prefix unit, then `no` of its own
// unit.  Prefix partial i lies at row (i >> psh) * pstep + (i & psh) * phalf
// from the unit's first: psh = 1 where a CTA's share is in two halves.
struct MergeSrc {
  const float *pl, *po, *ol, *oo;
  int np, no;
  int psh, pstep, phalf;
  int ostep;
  __device__ __forceinline__ int64_t prow(int i) const {
    return static_cast<int64_t>(i >> psh) * pstep + (i & psh) * phalf;
  }
  __device__ __forceinline__ int64_t orow(int i) const { return static_cast<int64_t>(i) * ostep; }
  __device__ __forceinline__ float lse(int i) const {
    return i < np ? pl[prow(i)] : ol[orow(i - np)];
  }
};

template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) merge_kernel(const PdParams p, int share) {
  const PdShape& s = p.b.s;
  const int u = blockIdx.y, b = u / s.Hkv, h = u - b * s.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // An inactive sequence has no keys here.  (The attention kernel takes no notice:
  // looking there costs every call 0.5 us of its start, and 2% of a long one.)
  const int next = p.next_pos ? __ldg(p.next_pos + b) : 0, own = pd_own_len(s, b);
  const int len = next >= 0 ? own : -1;
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * share;
  // this share's output: `tasks` groups of four columns from task0 on
  constexpr int D4 = D / 4;
  const int per = (s.G * D4 + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int task0 = static_cast<int>(blockIdx.x) * per;
  const int tasks = min(per, s.G * D4 - task0);
  if (tasks <= 0 && (p.acc == nullptr || k0 >= len)) return;
  __shared__ float lse2[kMaxG];
  __shared__ MergeSrc src[kMaxG];
  __shared__ float4 red[kMergeThreads];
  __shared__ float part_w[kMaxG][kMergeKept];  // exp(lse - L) of the partials, -1: not written
  __shared__ float4 ahead[kMergeAhead][kMergeThreads];
  // the first four keys' sums and logits of this thread come while the partials
  // are looked up
  float* acc = p.acc ? p.acc + static_cast<int64_t>(u) * s.T : nullptr;
  const float* lg = p.logits + static_cast<int64_t>(u) * s.G * p.Tl;
  const int64_t k1 = min(k0 + share, static_cast<int64_t>(len)), j_first = k0 + 4 * tid;
  // (the lengths, next_pos and the sums are earlier kernels': the attention kernel is an
  // ordinary launch that waited for them, and writes none of them)
  float old_first[4] = {0.f, 0.f, 0.f, 0.f};
  if (acc != nullptr && p.decay != 0.f)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j_first + i < k1) old_first[i] = acc[j_first + i];
  pdl_wait();  // the attention kernel's partials
  if (acc != nullptr && j_first < k1)
    for (int g = 0; g < min(s.G, kMergeAhead); ++g)
      copy16(smem_u32(&ahead[g][tid]), lg + g * p.Tl + j_first, true);
  asm volatile("cp.async.commit_group;" ::: "memory");
  for (int g = warp; g < s.G; g += kMergeThreads / 32) {
    MergeSrc m{};
    // one round of loads: both lines' plans, and with one prefix its entries
    // whether the sequence has it or not
    const int items = s.N + s.B;
    const int32_t* sb = p.b.plan.starts;
    const int W = sb[items], P = sb[items + 1];
    const int x_own = sb[s.N + b];
    const int n = s.N == 0 ? -1 : s.N == 1 ? 0 : p.b.plan.group[b];
    if (n >= 0) {
      const bool two = p.a.s.ctas > 0;
      const int32_t* sa = two ? p.a.plan.starts : sb;
      const int g0 = p.b.plan.gsan[n], g1 = p.b.plan.gsan[n + 1], seqs = g1 - g0;
      const int xa = sa[n], Wa = sa[items], Pa = sa[items + 1];
      const int ua = (two ? p.a.plan.ubase : p.b.plan.ubase)[n];
      const int xb = sb[n], unb = p.b.plan.ubase[n];
      const int keys = pd_prefix_len(s, n);
      const bool on_a = two && seqs * s.G >= p.a.s.min_rows;
      const PdLine& ln = on_a ? p.a : p.b;
      const int x_pre = on_a ? xa : xb, ub = on_a ? ua : unb;
      const int Wl = on_a ? Wa : W, Pl = on_a ? Pa : P;
      const int c = len >= 0 && g0 <= b && b < g1 ? pd_chunks(ln.s, keys) : 0;
      if (c > 0) {
        const int tiles = pd_tiles(ln.s, seqs), R = ln.s.R;
        int r = (b - g0) * s.G + g;
        const int tile = r / R;
        r -= tile * R;
        const int rows = min(R, seqs * s.G - tile * R);
        const int ui = h * tiles + tile, x = x_pre + ui * (c + ln.s.lead) + ln.s.lead;
        const PdCut cut(Wl, Pl);
        const int c0 = cut.worker_of(x), c1 = cut.worker_of(x + c - 1);
        if (ln.halves == 2) {
          const int rh = R / 2;
          m.psh = rows <= rh ? 1 : 0;
          if (r >= rh) r += ln.slot_rows / 2 - rh;
        }
        const int64_t row = (static_cast<int64_t>(c0) + ub + ui) * ln.slot_rows + r;
        m.np = (c1 - c0 + 1) << m.psh;
        m.pl = ln.plse + row;
        m.po = ln.po + row * D;
        m.pstep = ln.slot_rows;
        m.phalf = ln.slot_rows / 2;
      }
    }
    const int c = pd_chunks(s, len);
    if (c > 0) {
      const int x = x_own + h * (c + s.lead) + s.lead;
      const PdCut cut(W, P);
      const int c0 = cut.worker_of(x), c1 = cut.worker_of(x + c - 1);
      m.no = c1 - c0 + 1;
      const int64_t row = (static_cast<int64_t>(c0) + u) * s.G + g;
      m.ostep = s.G;
      m.ol = p.olse + row;
      m.oo = p.oo + row * D;
    }
    const int ns = m.np + m.no;
    // the first 128 partials' stay in registers
    float lv[4];
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lv[k] = lane + 32 * k < ns ? m.lse(lane + 32 * k) : -INFINITY;
      mx = fmaxf(mx, lv[k]);
    }
    for (int i = lane + 128; i < ns; i += 32) mx = fmaxf(mx, m.lse(i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) sum += exp2f(lv[k] - base);
    for (int i = lane + 128; i < ns; i += 32) sum += exp2f(m.lse(i) - base);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float L = sum == 0.f ? -INFINITY : base + log2f(sum);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      part_w[g][lane + 32 * k] = lv[k] == -INFINITY ? -1.f : exp2f(lv[k] - L);
    if (lane == 0) {
      lse2[g] = L;
      src[g] = m;
    }
  }
  __syncthreads();
  if (tasks > 0) {
    constexpr int kFly = 4;
    // few tasks: several threads each, over the partials
    const int parts = max(1, kMergeThreads / tasks);
    for (int t0 = 0; t0 < tasks; t0 += kMergeThreads) {
      const int task = parts > 1 ? tid % tasks : t0 + tid, part = parts > 1 ? tid / tasks : 0;
      const int g = (task0 + task) / D4, d = (task0 + task) % D4 * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (task < tasks && part < parts) {
        const MergeSrc m = src[g];
        const float L = lse2[g];
        const int ns = L == -INFINITY ? 0 : m.np + m.no;
        for (int i = part; i < ns; i += kFly * parts) {  // kFly rows in flight
          float w[kFly];
          float4 v[kFly];
#pragma unroll
          for (int k = 0; k < kFly; ++k) {
            const int j = min(i + k * parts, ns - 1);
            v[k] = ld4(j < m.np ? m.po + m.prow(j) * D + d : m.oo + m.orow(j - m.np) * D + d);
            if (j < kMergeKept) {
              w[k] = part_w[g][j];
            } else {
              const float x = m.lse(j);
              w[k] = x == -INFINITY ? -1.f : exp2f(x - L);
            }
          }
#pragma unroll
          for (int k = 0; k < kFly; ++k) {
            // a row whose lse is -inf was not written (a NaN is one that was)
            if (i + k * parts < ns && !(w[k] < 0.f)) {
              o.x += w[k] * v[k].x;
              o.y += w[k] * v[k].y;
              o.z += w[k] * v[k].z;
              o.w += w[k] * v[k].w;
            }
          }
        }
      }
      if (parts > 1) {
        red[tid] = o;
        __syncthreads();
        // tree over the parts
        int n = parts;
        while (n > 1) {
          const int half = (n + 1) / 2;
          if (part < n - half && task < tasks) {
            const float4 v = red[tid + half * tasks];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
            red[tid] = o;
          }
          __syncthreads();
          n = half;
        }
      }
      if (task < tasks && part == 0) {
        const int64_t at = (static_cast<int64_t>(b) * p.Hq + h * s.G + g) * D + d;
        if (p.out_bf16) {
          uint2 x;
          x.x = pack_bf16x2(o.x, o.y);
          x.y = pack_bf16x2(o.z, o.w);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) = x;
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = o;
        }
      }
    }
  }
  if (blockIdx.x == 0 && p.lse_out && tid < s.G)
    p.lse_out[static_cast<int64_t>(b) * p.Hq + h * s.G + tid] = lse2[tid] * kPdLn2;
  if (acc != nullptr) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // each thread reads its own only
    // four keys a thread, four heads' logits in flight: their rows start on 16
    // bytes, the sums' need not
    for (int64_t j = j_first; j < k1; j += 4 * kMergeThreads) {
      const bool first = j == j_first;
      float w[4] = {0.f, 0.f, 0.f, 0.f}, old[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        old[i] = first ? old_first[i] : p.decay != 0.f && j + i < k1 ? acc[j + i] : 0.f;
      for (int g0 = 0; g0 < s.G; g0 += 4) {
        float4 x[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if (g0 + g < s.G)
            x[g] = first && g0 + g < kMergeAhead ? ahead[(g0 + g) % kMergeAhead][tid]
                                                 : ld4(lg + (g0 + g) * p.Tl + j);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float L = g0 + g < s.G ? lse2[g0 + g] : -INFINITY;
          if (L != -INFINITY) {
            w[0] += fast_exp2(x[g].x - L);
            w[1] += fast_exp2(x[g].y - L);
            w[2] += fast_exp2(x[g].z - L);
            w[3] += fast_exp2(x[g].w - L);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + i < k1) acc[j + i] = p.decay != 0.f ? p.decay * old[i] + w[i] : w[i];
    }
  }
}

int64_t round256(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Hands out the workspace's areas; with base = null only counts.
struct Carver {
  char* base;
  int64_t at = 0;
  template <typename T>
  T* take(int64_t n) {
    T* p = base ? reinterpret_cast<T*>(base + at) : nullptr;
    at += round256(n * static_cast<int64_t>(sizeof(T)));
    return p;
  }
};

void carve_line(Carver* c, PdLine* ln, int D, int64_t units) {
  const PdShape& s = ln->s;
  ln->plan.starts = c->take<int32_t>(s.N + s.B + 2);
  ln->plan.ubase = c->take<int32_t>(s.N);
  ln->plan.gsan = c->take<int32_t>(s.N + 1);
  ln->plan.group = c->take<int32_t>(s.B);
  ln->slots = units > 0 ? s.ctas * s.workers + units : 0;
  ln->plse = c->take<float>(ln->slots * ln->slot_rows);
  ln->po = c->take<float>(ln->slots * ln->slot_rows * D);
}

// The lines' shapes and the workspace (bytes returned).
int64_t pd_layout(PdParams* p, char* ws, bool bf16, int B, int Hkv, int G, int D, int N, int64_t Tp,
                  int64_t T, bool weights, int num_sms) {
  const int64_t rows = static_cast<int64_t>(B) * G, U = static_cast<int64_t>(B) * Hkv;
  PdShape s{};
  s.B = B;
  s.Hkv = Hkv;
  s.G = G;
  s.N = N;
  s.Tp = Tp;
  s.T = T;
  Carver c{ws};
  p->a.s = p->b.s = s;
  // fp32: one line of 32-row tiles.  bf16: one CTA per SM for
  // the groups of many rows, and the warps for everything else.
  PdShape& a = p->a.s;
  PdShape& b = p->b.s;
  b.own = 1;
  b.min_rows = 1;
  if (bf16) {
    a.R = pd_tc_rows(G);
    a.ctas = N > 0 && Tp > 0 && rows > pd_few_rows(G) ? num_sms : 0;
    a.workers = 1;
    // a chunk's time in 16-key steps of the warps: its bytes, and a quarter more for
    // the longer way to its first and from its last chunk, or twice its bytes where
    // both halves' rows are at work (groups taken as of equal size)
    a.cost = 4.f * (N > 0 && rows / N > a.R / 2 ? 2.f : 1.25f);
    b.cost = 1.f;
    a.chunk_log2 = kPdTcChunkLog2;
    a.lead = kPdTcLead;
    a.min_rows = pd_few_rows(G) + 1;
    a.max_rows = 1 << 30;
    p->a.halves = 2;
    p->a.slot_rows = kPdTcSlotRows;
    b.R = pd_few_rows(G);
    b.ctas = num_sms;
    b.workers = kPdWarps;
    b.chunk_log2 = kPdWarpChunkLog2;
    b.lead = kPdWarpLead;
    b.max_rows = b.R;
    p->b.slot_rows = b.R;
  } else {
    b.R = kF32Rows;
    b.ctas = num_sms;
    b.workers = kF32Workers;
    // the line's front (prefixes, many rows) is the dearer part: some on every SM
    b.spread = 1;
    b.chunk_log2 = kF32ChunkLog2;
    b.lead = kF32Lead;
    b.max_rows = 1 << 30;
    p->b.slot_rows = kF32Rows;
  }
  p->b.halves = 1;
  a.inv_R = bf16 ? 1.f / a.R : 0.f;
  b.inv_R = 1.f / b.R;
  // tiles of all groups: at most rows / R + N
  if (a.ctas > 0) carve_line(&c, &p->a, D, Hkv * (rows / a.R + N));
  carve_line(&c, &p->b, D, N > 0 && Tp > 0 ? Hkv * (bf16 ? N : rows / b.R + N) : 0);
  const int64_t oslots = T > 0 ? b.ctas * b.workers + U : 0;
  p->olse = c.take<float>(oslots * G);
  p->oo = c.take<float>(oslots * G * D);
  p->Tl = (T + 63) / 64 * 64;
  p->logits = c.take<float>(weights ? U * G * p->Tl : 0);
  if (!weights) p->logits = nullptr;
  return c.at;
}

template <int D>
cudaError_t launch_attend_f32(const Launch& l, const PdParams& p) {
  const int smem = kF32Workers * f32_floats(D) * 4;
  cudaError_t e = cudaFuncSetAttribute(attend_f32_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // an ordinary launch: the merge behind it reads what earlier kernels wrote
  attend_f32_kernel<D><<<p.b.s.ctas, kF32Workers * kF32Threads, smem, l.stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_pd_merge(const Launch& l, const PdParams& p) {
  const PdShape& s = p.b.s;
  const int64_t U = static_cast<int64_t>(s.B) * s.Hkv;
  // about four CTAs per SM: of at least kMergeMinKeys keys where there are
  // weights, or of eight groups of columns where many partials may meet
  const int64_t by_keys = p.acc ? (s.T + kMergeMinKeys - 1) / kMergeMinKeys : 1;
  const int64_t by_cols = static_cast<int64_t>(s.G) * D / 32;
  const int64_t blocks = std::max<int64_t>(
      1, std::min<int64_t>(std::max(by_keys, by_cols), 4ll * l.num_sms / U));
  int64_t share = (s.T + blocks - 1) / blocks;
  share = std::max<int64_t>(4, (share + 3) / 4 * 4);
  return launch_behind(merge_kernel<D>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(U)),
                       dim3(kMergeThreads), 0, l.stream, p, static_cast<int>(share));
}

}  // namespace

int64_t prefix_decode_workspace_bytes(bool bf16, int B, int Hkv, int G, int D, int N, int64_t Tp,
                                      int64_t T, bool weights, int num_sms) {
  PdParams p{};
  return pd_layout(&p, nullptr, bf16, B, Hkv, G, D, N, Tp, T, weights, num_sms);
}

cudaError_t launch_prefix_decode(const Launch& l, const PrefixDecodeArgs& a, std::string* why) {
  PdParams p{};
  const bool weights = a.weights != nullptr && a.T > 0;
  pd_layout(&p, static_cast<char*>(a.workspace), a.bf16, a.B, a.Hkv, a.Hq / a.Hkv, a.D, a.N, a.Tp,
            a.T, weights, l.num_sms);
  for (PdShape* s : {&p.a.s, &p.b.s}) {
    s->prefix_len = a.prefix_len;
    s->group_start = a.group_start;
    s->len = a.len;
    s->err = l.err;
  }
  p.q = a.q;
  p.Kp = a.Kp;
  p.Vp = a.Vp;
  p.K = a.K;
  p.V = a.V;
  for (int i = 0; i < 3; ++i) {
    p.kps[i] = a.kps[i];
    p.vps[i] = a.vps[i];
    p.ks[i] = a.ks[i];
    p.vs[i] = a.vs[i];
  }
  p.Hq = a.Hq;
  p.scale_log2 = a.scale * kPdLog2e;
  p.out = a.out;
  p.out_bf16 = a.out_bf16 ? 1 : 0;
  p.lse_out = a.lse_out;
  p.acc = weights ? a.weights : nullptr;
  p.decay = a.decay;
  p.next_pos = a.next_pos;
  cudaError_t e = cudaSuccess;
  if (a.bf16) {
    e = launch_attend_bf16(l, p, a.D, why);
  } else {
    e = a.D == 128 ? launch_attend_f32<128>(l, p) : launch_attend_f32<64>(l, p);
  }
  if (e != cudaSuccess) return e;
  return a.D == 128 ? launch_pd_merge<128>(l, p) : launch_pd_merge<64>(l, p);
}

}  // namespace csa
