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
// Plain fp32 products on the FMA pipe: a tile of 32 query rows against chunks
// of 32 keys held in shared memory, a thread four rows by two keys of the logits
// and four rows by D/16 columns of the output.  Bound: with few rows HBM (a
// chunk is 256 D bytes), with 32 the FMA pipe (2 * 32 * 32 * D products a
// chunk).  Small chunks and CTAs, four per SM: the loads of one hide under
// the products of the others, and a short batch still fills the SMs (one
// chunk of 64 keys on 256 threads, two CTAs per SM: 35 us for 8 sequences over
// 4K tokens).
constexpr int kF32Rows = 32;
constexpr int kF32Threads = 128;
constexpr int kF32Ctas = 4;  // per SM
constexpr int kF32ChunkLog2 = 5, kF32Chunk = 1 << kF32ChunkLog2;
constexpr int kF32Lead = 1;  // a unit's queries and partials, in chunks' time

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// 16 bytes into shared memory, zeros if !in (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const float* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kF32Threads) attend_f32_kernel(const PdParams p) {
  constexpr int KS = D + 4, SS = kF32Chunk + 4;
  constexpr int D4 = D / 4;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;                           // [32][KS]
  float* sk = sq + kF32Rows * KS;           // [32][KS]
  float* sv = sk + kF32Chunk * KS;          // [32][D]
  float* ss = sv + kF32Chunk * D;           // [32][SS]
  __shared__ int gs[kPdMaxPrefixes + 1];
  __shared__ PdStart st[8];
  __shared__ uint64_t scan_sh[kF32Threads / 32];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const PdShape& shape = p.b.s;
  pdl_next();  // the merge
  const int key0 = tid < shape.N + shape.B ? pd_raw_keys(shape, tid) : 0;
  if (tid < 32) pd_groups(shape, gs);
  __syncthreads();
  pd_locate(p.a.s, shape, gs, key0, st, scan_sh, nullptr, blockIdx.x == 0 ? &p.b.plan : nullptr);
  PdWalk walk(shape, gs, st[0]);
  PdSeg g;
  while (walk.next(g)) {
    const int64_t* kst = g.own ? p.ks : p.kps;
    const int64_t* vst = g.own ? p.vs : p.vps;
    const int64_t k0 = g.own ? g.b : g.n;
    const float* Kg = static_cast<const float*>(g.own ? p.K : p.Kp) + k0 * kst[0] + g.h * kst[1];
    const float* Vg = static_cast<const float*>(g.own ? p.V : p.Vp) + k0 * vst[0] + g.h * vst[1];
    const float* q = static_cast<const float*>(p.q);
    for (int i = tid; i < kF32Rows * D4; i += kF32Threads) {
      const int r = i / D4, d = (i % D4) * 4;
      const int row = g.row0 + r, b = row / shape.G, hd = g.h * shape.G + row % shape.G;
      const bool in = r < g.rows;
      copy16(smem_u32(sq + r * KS + d), in ? q + (static_cast<int64_t>(b) * p.Hq + hd) * D + d : q, in);
    }
    // warps whose rows are past the unit's only help with the loads
    const bool active = (ty & ~1) * 4 < g.rows;
    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[r][d] = 0.f;
    }
    for (int j = g.j0; j < g.j1; ++j) {
      const int t0 = j * kF32Chunk, nk = min(kF32Chunk, g.keys - t0);
      // rows past the keys are zero: whatever the cache holds there, 0 * v stays 0
#pragma unroll 4
      for (int i = tid; i < kF32Chunk * D4; i += kF32Threads) {
        const int t = i / D4, d = (i % D4) * 4;
        copy16(smem_u32(sk + t * KS + d), t < nk ? Kg + (t0 + t) * kst[2] + d : q, t < nk);
        copy16(smem_u32(sv + t * D + d), t < nk ? Vg + (t0 + t) * vst[2] + d : q, t < nk);
      }
      asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      if (active) {
        float s[4][2] = {};
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          float4 a[4], k[2];
#pragma unroll
          for (int r = 0; r < 4; ++r) a[r] = ld4(sq + (ty * 4 + r) * KS + d);
#pragma unroll
          for (int c = 0; c < 2; ++c) k[c] = ld4(sk + (tx + 16 * c) * KS + d);
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              s[r][c] += a[r].x * k[c].x + a[r].y * k[c].y + a[r].z * k[c].z + a[r].w * k[c].w;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = ty * 4 + r;
#pragma unroll
          for (int c = 0; c < 2; ++c)
            s[r][c] = tx + 16 * c < nk ? s[r][c] * p.scale_log2 : -INFINITY;
          if (g.own && p.logits && row < g.rows) {
            float* lg = p.logits + (static_cast<int64_t>(g.unit) * shape.G + row) * p.Tl + t0;
            lg[tx] = s[r][0];
            lg[tx + 16] = s[r][1];
          }
          float mx = fmaxf(s[r][0], s[r][1]);
#pragma unroll
          for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
          const float al = exp2f(m[r] - base);
          const float e0 = exp2f(s[r][0] - base), e1 = exp2f(s[r][1] - base);
          ss[row * SS + tx] = e0;
          ss[row * SS + tx + 16] = e1;
          float sum = e0 + e1;
#pragma unroll
          for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
          l[r] = l[r] * al + sum;
          m[r] = mn;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) o[r][d] *= al;
        }
        __syncwarp();  // a row's weights are written and read by the same half-warp
#pragma unroll 2
        for (int t = 0; t < kF32Chunk; t += 4) {
          float4 pw[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) pw[r] = ld4(ss + (ty * 4 + r) * SS + t);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int d = 0; d < D / 64; ++d) {
              const float4 v = ld4(sv + (t + k) * D + d * 64 + tx * 4);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float w = k == 0 ? pw[r].x : k == 1 ? pw[r].y : k == 2 ? pw[r].z : pw[r].w;
                o[r][4 * d] += w * v.x;
                o[r][4 * d + 1] += w * v.y;
                o[r][4 * d + 2] += w * v.z;
                o[r][4 * d + 3] += w * v.w;
              }
            }
        }
      }
      __syncthreads();  // the chunk, and after the last one the queries, have been read
    }
    if (!active) continue;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) + g.unit;
    const int rows = g.own ? shape.G : p.b.slot_rows;
    float* po = (g.own ? p.oo : p.b.po) + slot * rows * D;
    float* pl = (g.own ? p.olse : p.b.plse) + slot * rows;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = ty * 4 + r;
      if (row < g.rows) {
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];  // a NaN stays one
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
          *reinterpret_cast<float4*>(po + static_cast<int64_t>(row) * D + d * 64 + tx * 4) =
              make_float4(o[r][4 * d] * inv, o[r][4 * d + 1] * inv, o[r][4 * d + 2] * inv,
                          o[r][4 * d + 3] * inv);
        if (tx == 0) pl[row] = l[r] == 0.f ? -INFINITY : m[r] + log2f(l[r]);
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
// a few CTAs each.
constexpr int kMergeThreads = 256;
constexpr int kMergeMinKeys = 1024;  // own keys per share at least
constexpr int kMaxG = 16;

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
  const int len = pd_own_len(s, b);
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
  pdl_wait();  // the attention kernel's partials
  for (int g = warp; g < s.G; g += kMergeThreads / 32) {
    MergeSrc m{};
    const int W = p.b.plan.starts[s.N + s.B], P = p.b.plan.starts[s.N + s.B + 1];
    const int x_own = p.b.plan.starts[s.N + b];
    const int n = s.N > 0 ? p.b.plan.group[b] : -1;
    if (n >= 0) {
      const int g0 = p.b.plan.gsan[n], seqs = p.b.plan.gsan[n + 1] - g0;
      const PdLine& ln = p.a.s.ctas > 0 && seqs * s.G >= p.a.s.min_rows ? p.a : p.b;
      const int x_pre = ln.plan.starts[n], ub = ln.plan.ubase[n];
      const int Wl = ln.plan.starts[s.N + s.B], Pl = ln.plan.starts[s.N + s.B + 1];
      const int c = pd_chunks(ln.s, pd_prefix_len(s, n));
      if (c > 0) {
        const int tiles = pd_tiles(ln.s, seqs), R = ln.s.R;
        int r = (b - g0) * s.G + g;
        const int tile = r / R;
        r -= tile * R;
        const int rows = min(R, seqs * s.G - tile * R);
        const int ui = h * tiles + tile, x = x_pre + ui * (c + ln.s.lead) + ln.s.lead;
        const int c0 = pd_worker_of(x, Wl, Pl), c1 = pd_worker_of(x + c - 1, Wl, Pl);
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
      const int c0 = pd_worker_of(x, W, P), c1 = pd_worker_of(x + c - 1, W, P);
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
    if (lane == 0) {
      lse2[g] = L;
      src[g] = m;
    }
  }
  __syncthreads();
  if (tasks > 0) {
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
        for (int i = part; i < ns; i += 4 * parts) {  // four rows in flight
          float w[4];
          float4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = min(i + k * parts, ns - 1);
            w[k] = m.lse(j);
            v[k] = ld4(j < m.np ? m.po + m.prow(j) * D + d : m.oo + m.orow(j - m.np) * D + d);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // a row whose lse is -inf was not written
            if (i + k * parts < ns && w[k] != -INFINITY) {
              const float e = exp2f(w[k] - L);
              o.x += e * v[k].x;
              o.y += e * v[k].y;
              o.z += e * v[k].z;
              o.w += e * v[k].w;
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
  if (p.acc != nullptr) {
    float* acc = p.acc + static_cast<int64_t>(u) * s.T;
    const float* lg = p.logits + static_cast<int64_t>(u) * s.G * p.Tl;
    const int64_t k1 = min(k0 + share, static_cast<int64_t>(len));
    // four keys a thread, four heads' logits in flight: their rows start on 16
    // bytes, the sums' need not
    for (int64_t j = k0 + 4 * tid; j < k1; j += 4 * kMergeThreads) {
      float w[4] = {0.f, 0.f, 0.f, 0.f}, old[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) old[i] = p.decay != 0.f && j + i < k1 ? acc[j + i] : 0.f;
      for (int g0 = 0; g0 < s.G; g0 += 4) {
        float4 x[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if (g0 + g < s.G) x[g] = ld4(lg + (g0 + g) * p.Tl + j);
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
    b.ctas = kF32Ctas * num_sms;
    b.workers = 1;
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
  const int smem = ((kF32Rows + kF32Chunk) * (D + 4) + kF32Chunk * D + kF32Rows * (kF32Chunk + 4)) * 4;
  cudaError_t e = cudaFuncSetAttribute(attend_f32_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attend_f32_kernel<D><<<p.b.s.ctas, kF32Threads, smem, l.stream>>>(p);
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
