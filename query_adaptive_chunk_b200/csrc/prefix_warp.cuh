// Own caches, and prefixes of at most 8 (16 for G > 8) query rows, of the
// shared-prefix decode (bf16).
//
// Every warp works by itself: it takes its share of the line (prefix_work.cuh)
// in steps of 16 keys, with a ring of stages of its own filled by cp.async, so
// no warp waits for another and a short unit costs its warp alone.  Per step,
// with NT tiles of 8 query rows (mma.sync: the rows are the narrow side, N = 8):
//   S^T = K Q^T        16 keys x 8 rows, K from shared memory (ldmatrix)
//   P^T = exp2(S^T sl - m sl)   in registers; a row's m moves only when a logit
//                      passes it by more than 2^8 (one vote per step), the row's
//                      sum stays spread over the lanes until the unit's end
//   O^T += V^T P^T     D x 8, V transposed by ldmatrix, P^T's accumulator
//                      fragment turned into an operand by movmatrix; P is
//                      rounded to bf16 (V's type)
// The logits of own keys go to memory (4 bytes a row and key) for the merge.
//
// Bound by HBM: a step is 64 D bytes of K and V against about 60
// instructions; with all stages of a ring but one on their way while a warp waits
// (128 KB per SM at D = 128, 160 KB at D = 64) the loads run ahead of the products (32
// sequences over 8K tokens, 67 MB here beside 34 MB of line a, on one set of
// inputs and so partly from L2: 5.5 TB/s of both from the first row's arrival to the
// last).  Rows past a unit's keys are filled with zeros by the copy itself,
// so what the cache holds there never enters a product.
#pragma once

#include "prefix_decode.cuh"

namespace csa {
namespace {

constexpr int kStep = 1 << kPdWarpChunkLog2;  // 16 keys
constexpr float kWRescaleLog2 = 8.0f;

template <int D>
struct WCfg {
  static constexpr int kHalf = kStep * D * 2;            // K (or V) bytes of a step
  static constexpr int kStages = 3 * 128 / D;
  static constexpr int kWarpBytes = kStages * 2 * kHalf;  // 24 KB
  static constexpr int kSmem = kPdWarps * kWarpBytes;
  static constexpr int kCh = D / 8;                       // 16-byte chunks of a row
};

__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Chunk c of row r: 16-byte chunks permuted within a row by the row's low bits, so
// that eight rows' chunks of one column lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t cell(int r, int c) {
  return static_cast<uint32_t>(r * D * 2 + ((c ^ (r & 7)) << 4));
}

// One of the kPdWarps warps of CTA `block` of line b; `smem` is the warps' rings.
template <int D, int NT>
__device__ __forceinline__ void attend_warp(const PdParams& p, uint8_t* smem, const int* gs,
                                            const PdStart* st, int block) {
  using C = WCfg<D>;
  const PdShape& shape = p.b.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;
  const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_normal();
  // ---- loads: a walk of its own, kStages - 1 steps ahead
  PdWalk lw(shape, gs, st[warp]);
  PdSeg lg;
  int lj = 0, lj1 = 0;  // next step of the segment being loaded
  const char *kp = nullptr, *vp = nullptr;
  int64_t krow = 0, vrow = 0;
  uint64_t policy = once;
  // lanes: chunk lc of rows lr, lr + kRows, ..
  constexpr int kRows = 32 / C::kCh;
  const int lc = lane % C::kCh, lr = lane / C::kCh;
  auto load_step = [&](int stage) {
    if (lj == lj1) {
      if (lw.next(lg)) {
        lj = lg.j0;
        lj1 = lg.j1;
        const int64_t* ks = lg.own ? p.ks : p.kps;
        const int64_t* vs = lg.own ? p.vs : p.vps;
        const int64_t i0 = lg.own ? lg.b : lg.n;
        krow = ks[2] * 2;
        vrow = vs[2] * 2;
        kp = static_cast<const char*>(lg.own ? p.K : p.Kp) + (i0 * ks[0] + lg.h * ks[1]) * 2 +
             lj * (kStep * krow) + lr * krow + lc * 16;
        vp = static_cast<const char*>(lg.own ? p.V : p.Vp) + (i0 * vs[0] + lg.h * vs[1]) * 2 +
             lj * (kStep * vrow) + lr * vrow + lc * 16;
        policy = lg.own ? once : keep;
      }
    }
    if (lj < lj1) {
      const int nk = lg.keys - lj * kStep;
      const uint32_t kd = ring + stage * 2 * C::kHalf, vd = kd + C::kHalf;
#pragma unroll
      for (int i = 0; i < kStep / kRows; ++i) {
        const int r = lr + i * kRows;
        const int n = r < nk ? 16 : 0;  // rows past the keys: zeros, nothing read
        const uint32_t at = cell<D>(r, lc);
        asm volatile(
            "cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(kd + at),
            "l"(n ? kp + i * (kRows * krow) : static_cast<const char*>(p.q)), "r"(n), "l"(policy)
            : "memory");
      }
#pragma unroll
      for (int i = 0; i < kStep / kRows; ++i) {
        const int r = lr + i * kRows;
        const int n = r < nk ? 16 : 0;
        const uint32_t at = cell<D>(r, lc);
        asm volatile(
            "cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(vd + at),
            "l"(n ? vp + i * (kRows * vrow) : static_cast<const char*>(p.q)), "r"(n), "l"(policy)
            : "memory");
      }
      ++lj;
      kp += kStep * krow;
      vp += kStep * vrow;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < C::kStages - 1; ++i) load_step(i);

  // ---- products
  PdWalk walk(shape, gs, st[warp]);
  PdSeg g;
  const float sl = p.scale_log2;
  int stage = 0;
  const int qr = lane >> 2, qc = (lane & 3) * 2;  // fragment row, first of its two columns
  while (walk.next(g)) {
    // Q fragments: rows (heads) 8 t + qr of the unit, B operand of S^T
    uint32_t qf[NT][D / 16][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + qr;
      const int row = g.row0 + r, b = row / shape.G, hd = g.h * shape.G + (row - b * shape.G);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(
          static_cast<const __nv_bfloat16*>(p.q) + (static_cast<int64_t>(b) * p.Hq + hd) * D + qc);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[t][k][0] = r < g.rows ? __ldg(q + 8 * k) : 0u;
        qf[t][k][1] = r < g.rows ? __ldg(q + 8 * k + 4) : 0u;
      }
    }
    float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[t][d][0] = o[t][d][1] = o[t][d][2] = o[t][d][3] = 0.f;
    }
    float* lg_row = g.own && p.logits
                        ? p.logits + static_cast<int64_t>(g.unit) * shape.G * p.Tl + g.j0 * kStep + qr
                        : nullptr;
    for (int j = g.j0; j < g.j1; ++j) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
      __syncwarp();  // this step's rows are in; the previous step's reads are done
      {
        int ns = stage + C::kStages - 1;
        if (ns >= C::kStages) ns -= C::kStages;
        load_step(ns);
      }
      const uint32_t kb = ring + stage * 2 * C::kHalf, vb = kb + C::kHalf;
      if (++stage == C::kStages) stage = 0;
      float s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4(kb + cell<D>(lane & 15, 2 * k + (lane >> 4)), a0, a1, a2, a3);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma_bf16_16816(s[t], a0, a1, a2, a3, qf[t][k][0], qf[t][k][1]);
      }
      // s[t][0..3]: keys qr, qr, qr + 8, qr + 8; rows 8 t + qc, + 1, + 0, + 1
      if (lg_row) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (8 * t + qc + c < g.rows) {
              float* x = lg_row + (8 * t + qc + c) * p.Tl;
              x[0] = s[t][c] * sl;
              x[8] = s[t][c + 2] * sl;
            }
        lg_row += kStep;
      }
      const int nk = g.keys - j * kStep;
      if (nk < kStep) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (qr >= nk) s[t][0] = s[t][1] = -INFINITY;
          if (qr + 8 >= nk) s[t][2] = s[t][3] = -INFINITY;
        }
      }
      // (a NaN passes no comparison and reaches the sums)
      bool over = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float lim = m[t][c] + kWRescaleLog2 / sl;
          over = over || s[t][c] > lim || s[t][c + 2] > lim;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float al[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(fmaxf(s[t][c], s[t][c + 2]), m[t][c]);
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            al[c] = mx == -INFINITY ? 1.f : fast_exp2((m[t][c] - mx) * sl);
            m[t][c] = mx;
            l[t][c] *= al[c];
          }
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            o[t][d][0] *= al[0];
            o[t][d][1] *= al[1];
            o[t][d][2] *= al[0];
            o[t][d][3] *= al[1];
          }
        }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float n0 = m[t][0] == -INFINITY ? 0.f : -m[t][0] * sl;
        const float n1 = m[t][1] == -INFINITY ? 0.f : -m[t][1] * sl;
        const float e0 = fast_exp2(fmaf(s[t][0], sl, n0)), e1 = fast_exp2(fmaf(s[t][1], sl, n1));
        const float e2 = fast_exp2(fmaf(s[t][2], sl, n0)), e3 = fast_exp2(fmaf(s[t][3], sl, n1));
        l[t][0] += e0 + e2;
        l[t][1] += e1 + e3;
        pf[t][0] = movmatrix_trans(pack_bf16x2(e0, e1));
        pf[t][1] = movmatrix_trans(pack_bf16x2(e2, e3));
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        // V^T's tile of 16 columns: 8 x 8 blocks (keys 0-7, d 0-7), (0-7, 8-15), (8-15, 0-7), ..
        uint32_t a0, a1, a2, a3;
        ldsm_x4_trans(vb + cell<D>((lane & 7) + ((lane >> 4) << 3), 2 * d + ((lane >> 3) & 1)), a0,
                      a1, a2, a3);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_bf16_16816(o[t][d], a0, a1, a2, a3, pf[t][0], pf[t][1]);
      }
    }
    // ---- the unit's share is done: its partial rows
    const int64_t slot = static_cast<int64_t>(block) * kPdWarps + warp + g.unit;
    const int64_t row0 = slot * (g.own ? shape.G : shape.R);
    float* po = (g.own ? p.oo : p.b.po) + row0 * D;
    float* pl = (g.own ? p.olse : p.b.plse) + row0;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[t][c];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        const int r = 8 * t + qc + c;
        if (r < g.rows) {
          const float inv = sum == 0.f ? 0.f : 1.0f / sum;
          if (qr == 0)
            pl[r] = sum == 0.f ? -INFINITY : (m[t][c] == -INFINITY ? 0.f : m[t][c] * sl) + log2f(sum);
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            po[r * D + 16 * d + qr] = o[t][d][c] * inv;
            po[r * D + 16 * d + 8 + qr] = o[t][d][c + 2] * inv;
          }
        }
      }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace
}  // namespace csa
