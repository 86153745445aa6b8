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
// of 64 keys held in shared memory.
constexpr int kF32Rows = 32;
constexpr int kF32Threads = 256;

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int D>
__global__ void __launch_bounds__(kF32Threads) attend_f32_kernel(const PdParams p) {
  constexpr int KS = D + 4, SS = kPdChunk + 4;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;                           // [32][KS]
  float* sk = sq + kF32Rows * KS;           // [64][KS]
  float* sv = sk + kPdChunk * KS;           // [64][D]
  float* ss = sv + kPdChunk * D;            // [32][SS]
  __shared__ int gs[kPdMaxPrefixes + 1];
  __shared__ PdStart st;
  __shared__ int scan_sh[33];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  if (tid < 32) pd_groups(p.s, gs);
  __syncthreads();
  const bool plan = blockIdx.x == 0;
  pd_locate(p.s, gs, blockIdx.x, &st, scan_sh, plan ? p.starts : nullptr, plan ? p.ubase : nullptr);
  if (plan && tid <= p.s.N) p.gsan[tid] = gs[tid];
  PdWalk walk(p.s, gs, st);
  PdSeg g;
  while (walk.next(g)) {
    for (int i = tid; i < kF32Rows * (D / 4); i += kF32Threads) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < g.rows) {
        const int row = g.row0 + r, b = row / p.s.G, hd = g.h * p.s.G + row % p.s.G;
        x = ld4(static_cast<const float*>(p.q) + (static_cast<int64_t>(b) * p.Hq + hd) * D + d);
      }
      *reinterpret_cast<float4*>(sq + r * KS + d) = x;
    }
    const int64_t* kst = g.own ? p.ks : p.kps;
    const int64_t* vst = g.own ? p.vs : p.vps;
    const int64_t k0 = g.own ? g.b : g.n;
    const float* Kg = static_cast<const float*>(g.own ? p.K : p.Kp) + k0 * kst[0] + g.h * kst[1];
    const float* Vg = static_cast<const float*>(g.own ? p.V : p.Vp) + k0 * vst[0] + g.h * vst[1];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[2][D / 16];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[r][d] = 0.f;
    for (int j = g.j0; j < g.j1; ++j) {
      const int t0 = j * kPdChunk, nk = min(kPdChunk, g.keys - t0);
      __syncthreads();  // the previous chunk's values have been read
      for (int i = tid; i < kPdChunk * (D / 4); i += kF32Threads) {
        const int t = i / (D / 4), d = (i % (D / 4)) * 4;
        // rows past the keys are zero: whatever the cache holds there, 0 * v stays 0
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (t < nk) {
          x = ld4(Kg + (t0 + t) * kst[2] + d);
          y = ld4(Vg + (t0 + t) * vst[2] + d);
        }
        *reinterpret_cast<float4*>(sk + t * KS + d) = x;
        *reinterpret_cast<float4*>(sv + t * D + d) = y;
      }
      __syncthreads();
      float s[2][4] = {};
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[2], k[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) a[r] = ld4(sq + (ty * 2 + r) * KS + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) k[c] = ld4(sk + (tx + 16 * c) * KS + d);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            s[r][c] += a[r].x * k[c].x + a[r].y * k[c].y + a[r].z * k[c].z + a[r].w * k[c].w;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = ty * 2 + r;
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[r][c] = tx + 16 * c < nk ? s[r][c] * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, s[r][c]);
        }
        if (g.own && p.logits && row < g.rows) {
          float* lg = p.logits + (static_cast<int64_t>(g.unit) * p.s.G + row) * p.Tl + t0;
#pragma unroll
          for (int c = 0; c < 4; ++c) lg[tx + 16 * c] = s[r][c];
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float mn = fmaxf(m[r], mx), base = mn == -INFINITY ? 0.f : mn;
        const float al = exp2f(m[r] - base);
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float e = exp2f(s[r][c] - base);
          sum += e;
          ss[row * SS + tx + 16 * c] = e;
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        l[r] = l[r] * al + sum;
        m[r] = mn;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[r][d] *= al;
      }
      __syncwarp();  // a row's weights are written and read by the same half-warp
#pragma unroll 4
      for (int t = 0; t < kPdChunk; ++t) {
        float pw[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) pw[r] = ss[(ty * 2 + r) * SS + t];
#pragma unroll
        for (int d = 0; d < D / 64; ++d) {
          const float4 v = ld4(sv + t * D + d * 64 + tx * 4);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            o[r][4 * d] += pw[r] * v.x;
            o[r][4 * d + 1] += pw[r] * v.y;
            o[r][4 * d + 2] += pw[r] * v.z;
            o[r][4 * d + 3] += pw[r] * v.w;
          }
        }
      }
    }
    const int64_t slot = static_cast<int64_t>(blockIdx.x) + g.unit;
    const int rows = g.own ? p.s.G : p.s.R;
    float* po = (g.own ? p.oo : p.po) + slot * rows * D;
    float* pl = (g.own ? p.olse : p.plse) + slot * rows;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = ty * 2 + r;
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
    __syncthreads();  // the queries have been read
  }
}

// ------------------------------------------------------------------ merge
//
// A CTA joins the partials of one (sequence, KV head) and, block by block of
// kMergeKeys own keys, adds the keys' weights; the first block's CTA writes
// the output.  Reads the partials once (they sit in L2) and 4 bytes per head
// and own key; bound by latency at the usual sizes.
constexpr int kMergeThreads = 256;
constexpr int kMergeKeys = 1024;
constexpr int kMaxG = 16;

// Partials of one query head: `np` of its prefix unit, then `no` of its own
// unit.  Partial i lies at row (i >> sh) * step + (i & sh) * half from the
// unit's first: sh = 1 where a CTA's share is in two halves.
struct MergeSrc {
  const float *pl, *po, *ol, *oo;
  int np, no;
  int psh, pstep, phalf;
  int osh, ostep, ohalf;
  __device__ __forceinline__ int64_t prow(int i) const {
    return static_cast<int64_t>(i >> psh) * pstep + (i & psh) * phalf;
  }
  __device__ __forceinline__ int64_t orow(int i) const {
    return static_cast<int64_t>(i >> osh) * ostep + (i & osh) * ohalf;
  }
};

template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const PdParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention kernel's partials
  __shared__ float lse2[kMaxG];
  __shared__ MergeSrc src[kMaxG];
  __shared__ float4 red[kMergeThreads];
  const PdShape& s = p.s;
  const int u = blockIdx.y, b = u / s.Hkv, h = u - b * s.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = p.starts[s.N + s.B];
  const int len = pd_own_len(s, b);
  for (int g = warp; g < s.G; g += kMergeThreads / 32) {
    MergeSrc m{};
    // the sequence's group
    int n = -1;
    for (int i0 = 0; i0 < s.N; i0 += 32) {
      const int i = i0 + lane;
      const unsigned hit =
          __ballot_sync(0xffffffffu, i < s.N && p.gsan[i] <= b && b < p.gsan[i + 1]);
      if (hit) n = i0 + __ffs(hit) - 1;
    }
    if (n >= 0) {
      const int seqs = p.gsan[n + 1] - p.gsan[n], tiles = pd_tiles(s, seqs);
      const int c = pd_chunks(pd_prefix_len(s, n));
      if (c > 0) {
        const int row = (b - p.gsan[n]) * s.G + g, tile = row / s.R, r = row - tile * s.R;
        const int ui = h * tiles + tile, x = p.starts[n] + ui * c;
        const int c0 = pd_cta_of(x, W, s.P), c1 = pd_cta_of(x + c - 1, W, s.P);
        const int64_t slot = static_cast<int64_t>(c0) + p.ubase[n] + ui;
        const bool split = p.halves == 2 && min(s.R, seqs * s.G - tile * s.R) <= s.R / 2;
        m.psh = split ? 1 : 0;
        m.np = (c1 - c0 + 1) << m.psh;
        m.pl = p.plse + slot * s.R + r;
        m.po = p.po + (slot * s.R + r) * D;
        m.pstep = s.R;
        m.phalf = s.R / 2;
      }
    }
    const int c = pd_chunks(len);
    if (c > 0) {
      const int x = p.starts[s.N + b] + h * c;
      const int c0 = pd_cta_of(x, W, s.P), c1 = pd_cta_of(x + c - 1, W, s.P);
      const int64_t slot = static_cast<int64_t>(c0) + u;
      m.osh = p.halves - 1;
      m.no = (c1 - c0 + 1) << m.osh;
      m.ostep = p.halves * s.G;
      m.ohalf = s.G;
      m.ol = p.olse + slot * m.ostep + g;
      m.oo = p.oo + (slot * m.ostep + g) * D;
    }
    const int ns = m.np + m.no;
    auto lse_at = [&](int i) -> float {
      return i < m.np ? m.pl[m.prow(i)] : m.ol[m.orow(i - m.np)];
    };
    float mx = -INFINITY;
    for (int i = lane; i < ns; i += 32) mx = fmaxf(mx, lse_at(i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    for (int i = lane; i < ns; i += 32) sum += exp2f(lse_at(i) - base);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      lse2[g] = sum == 0.f ? -INFINITY : base + log2f(sum);
      src[g] = m;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    constexpr int D4 = D / 4;
    const int tasks = s.G * D4;
    const int parts = max(1, kMergeThreads / tasks);
    for (int t0 = 0; t0 < tasks; t0 += kMergeThreads) {
      const int task = parts > 1 ? tid % tasks : t0 + tid, part = parts > 1 ? tid / tasks : 0;
      const int g = task / D4, d = (task % D4) * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (task < tasks && part < parts) {
        const MergeSrc& m = src[g];
        const float L = lse2[g];
        const int ns = L == -INFINITY ? 0 : m.np + m.no;
        for (int i = part; i < ns; i += parts) {
          const bool pre = i < m.np;
          const int64_t k = pre ? m.prow(i) : m.orow(i - m.np);
          const float ls = pre ? m.pl[k] : m.ol[k];
          if (ls == -INFINITY) continue;  // this slot's row was not written
          const float w = exp2f(ls - L);
          const float4 v = ld4((pre ? m.po : m.oo) + k * D + d);
          o.x += w * v.x;
          o.y += w * v.y;
          o.z += w * v.z;
          o.w += w * v.w;
        }
      }
      if (parts > 1) {
        red[tid] = o;
        __syncthreads();
        if (part == 0) {
          for (int k = 1; k < parts; ++k) {
            const float4 v = red[tid + k * tasks];
            o.x += v.x;
            o.y += v.y;
            o.z += v.z;
            o.w += v.w;
          }
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
    if (p.lse_out && tid < s.G)
      p.lse_out[static_cast<int64_t>(b) * p.Hq + h * s.G + tid] = lse2[tid] * kPdLn2;
  }
  if (p.acc != nullptr) {
    const int64_t k0 = static_cast<int64_t>(blockIdx.x) * kMergeKeys;
    float* acc = p.acc + static_cast<int64_t>(u) * s.T;
    const float* lg = p.logits + static_cast<int64_t>(u) * s.G * p.Tl;
    for (int64_t j = k0 + tid; j < min(k0 + kMergeKeys, static_cast<int64_t>(len));
         j += kMergeThreads) {
      float w = 0.f;
      for (int g = 0; g < s.G; ++g)
        if (lse2[g] != -INFINITY) w += exp2f(lg[g * p.Tl + j] - lse2[g]);
      acc[j] = p.decay == 0.f ? w : p.decay * acc[j] + w;
    }
  }
}

struct PdLayout {
  int64_t starts, ubase, gsan, plse, po, olse, oo, logits, total;
  int64_t Tl;
};

// CTAs that share the chunks: one per SM for bf16 (it takes the SM's whole
// shared memory), two for fp32.
int pd_parts(bool bf16, int num_sms) { return bf16 ? num_sms : 2 * num_sms; }
int pd_rows(bool bf16) { return bf16 ? pd_tc_rows() : kF32Rows; }
int pd_halves(bool bf16) { return bf16 ? 2 : 1; }

PdLayout pd_layout(bool bf16, int B, int Hkv, int G, int D, int N, int64_t T, bool weights, int P) {
  const int64_t R = pd_rows(bf16), U = static_cast<int64_t>(B) * Hkv;
  const int64_t pslots = N > 0 ? P + Hkv * (static_cast<int64_t>(B) * G / R + N) : 0;
  const int64_t oslots = T > 0 ? P + U : 0;
  PdLayout w{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t r = at;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  w.Tl = (T + kPdChunk - 1) / kPdChunk * kPdChunk;
  w.starts = take(4ll * (N + B + 1));
  w.ubase = take(4ll * (N + 1));
  w.gsan = take(4ll * (N + 1));
  w.plse = take(4 * pslots * R);
  w.po = take(4 * pslots * R * D);
  w.olse = take(4 * oslots * pd_halves(bf16) * G);
  w.oo = take(4 * oslots * pd_halves(bf16) * G * D);
  w.logits = take(weights ? 4 * U * G * w.Tl : 0);
  w.total = at;
  return w;
}

template <int D>
cudaError_t launch_attend_f32(const Launch& l, const PdParams& p) {
  const int smem = ((kF32Rows + kPdChunk) * (D + 4) + kPdChunk * D + kF32Rows * (kPdChunk + 4)) * 4;
  cudaError_t e = cudaFuncSetAttribute(attend_f32_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attend_f32_kernel<D><<<p.s.P, kF32Threads, smem, l.stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_pd_merge(const Launch& l, const PdParams& p) {
  cudaLaunchConfig_t cfg = {};
  const int64_t blocks =
      p.acc ? std::max<int64_t>(1, (p.s.T + kMergeKeys - 1) / kMergeKeys) : 1;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(p.s.B * p.s.Hkv));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = l.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel<D>, p);
}

}  // namespace

int64_t prefix_decode_workspace_bytes(bool bf16, int B, int Hkv, int G, int D, int N, int64_t T,
                                      bool weights, int num_sms) {
  return pd_layout(bf16, B, Hkv, G, D, N, T, weights, pd_parts(bf16, num_sms)).total;
}

cudaError_t launch_prefix_decode(const Launch& l, const PrefixDecodeArgs& a, std::string* why) {
  const int G = a.Hq / a.Hkv, P = pd_parts(a.bf16, l.num_sms);
  const PdLayout w = pd_layout(a.bf16, a.B, a.Hkv, G, a.D, a.N, a.T, a.weights != nullptr, P);
  char* ws = static_cast<char*>(a.workspace);
  PdParams p{};
  p.s = PdShape{a.B,  a.Hkv, G,            a.N,           pd_rows(a.bf16), P,
                a.Tp, a.T,   a.prefix_len, a.group_start, a.len,           l.err};
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
  p.halves = pd_halves(a.bf16);
  p.scale_log2 = a.scale * kPdLog2e;
  p.starts = reinterpret_cast<int32_t*>(ws + w.starts);
  p.ubase = reinterpret_cast<int32_t*>(ws + w.ubase);
  p.gsan = reinterpret_cast<int32_t*>(ws + w.gsan);
  p.plse = reinterpret_cast<float*>(ws + w.plse);
  p.po = reinterpret_cast<float*>(ws + w.po);
  p.olse = reinterpret_cast<float*>(ws + w.olse);
  p.oo = reinterpret_cast<float*>(ws + w.oo);
  p.logits = a.weights ? reinterpret_cast<float*>(ws + w.logits) : nullptr;
  p.Tl = w.Tl;
  p.out = a.out;
  p.out_bf16 = a.out_bf16 ? 1 : 0;
  p.lse_out = a.lse_out;
  p.acc = a.T > 0 ? a.weights : nullptr;
  p.decay = a.decay;
  cudaError_t e;
  if (a.bf16)
    e = launch_attend_tc(l, p, a.D, why);
  else
    e = a.D == 128 ? launch_attend_f32<128>(l, p) : launch_attend_f32<64>(l, p);
  if (e != cudaSuccess) return e;
  return a.D == 128 ? launch_pd_merge<128>(l, p) : launch_pd_merge<64>(l, p);
}

}  // namespace csa
