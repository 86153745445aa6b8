// bf16 attention of the shared-prefix decode on the 5th-generation tensor
// cores (tcgen05, accumulators in tensor memory).
//
// Work unit: up to R <= 256 query rows against a run of keys (prefix_work.cuh),
// in chunks of 64 keys.  Per chunk and 128-row half:
//   S = Q K^T     tcgen05.mma M=128 N=64 K=D, operands in shared memory
//   P = softmax   a warpgroup reads S with tcgen05.ld, keeps each row's running
//                 maximum and sum in registers (fp32) and writes P to tensor
//                 memory as bf16 (the A operand of the second product has V's
//                 type; a rounding of 2^-8 of each weight at most)
//   O += P V      tcgen05.mma M=128 N=D K=64, V from shared memory
// Units of more than R / 2 rows (many sequences on one prefix) give each half
// its own rows and both the same chunk.  Units of fewer (few sequences, or one
// sequence's own cache with G rows) give the halves the even and the odd
// chunks, so two softmax chains share the CTA's chunks; each half writes its
// own partial rows.  A unit of at most 32 rows has them twice, at rows 0 and 32
// of the query tile: half 1 reads the copy, so that the two chains run on
// different warps of the tile's rows and so on different schedulers.  Rows
// past a unit's are garbage that no other row sees; their warps only keep the
// barriers' counts.
//
// Bound: a CTA's chunk is 256 D bytes of K and V.  At the copy rate an SM gets about
// 23 bytes a clock, 1430 clocks a chunk at D = 128, against 512 clocks of
// products per half and 512 of exponentials: memory-bound up to 256 rows per
// key, which is why a unit takes that many.  With both halves' exponentials on
// the special-function unit alone a chunk took 2300 clocks (it serves one warp
// of each half, in step); half of them go to the FMA pipe.
// The keys past a unit's end are masked in S, and their V rows zeroed in
// shared memory, so that neither value reaches a result (0 * NaN is NaN).
//
// Warps: 0 TMA (K and V, a ring of 128 KB), 1 and 2 the halves' MMA issuers
// (1 owns the tensor memory), 3 the queries (TMA; two 128-row slots, so
// that the next small unit's rows arrive early), 4-7 and 8-11 softmax and
// epilogue of half 0 and 1.  Every wait is bounded.
#include <algorithm>

#include "prefix_decode.cuh"
#include "tcgen05.cuh"

namespace csa {
namespace {

constexpr int kTcThreads = 384;
constexpr float kTcRescaleLog2 = 8.0f;

template <int D>
struct TcCfg {
  static constexpr int kQSlot = 128 * D * 2;
  static constexpr int kKV = kPdChunk * D * 2;  // bytes of K (or V) per chunk
  static constexpr int kStage = 2 * kKV;
  static constexpr int kNS = 131072 / kStage;   // 4 stages of 32 KB, or 8 of 16 KB
  static constexpr int kQOff = 0;
  static constexpr int kKVOff = 2 * kQSlot;
  static constexpr int kOOff = kKVOff + kNS * kStage;  // 4 KB of output rows per softmax warp
  static constexpr int kBarOff = kOOff + 8 * 4096;
  static constexpr int kSmem = 1024 + kBarOff + 512;
  static constexpr uint32_t kIdescQK = idesc_bf16(128, kPdChunk, 0);
  static constexpr uint32_t kIdescPV = idesc_bf16(128, D, 1);
};

// TMEM columns, as the prefill's: S of half h at 64 h, P buffer u of half h at
// 128 + 64 u + 32 h, O of half h at 256 + 128 h
constexpr uint32_t kColP = 128, kColO = 256;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_hint(uint32_t dst, const CUtensorMap* map, int c0,
                                                 int c1, int c2, int c3, uint32_t bar,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar),
      "l"(policy)
      : "memory");
}

// Index multipliers (0 for a broadcast dimension, whose map has one entry).
struct TcMaps {
  int kph, kpn, vph, vpn, kh, kb, vh, vb;
  int few;  // rows of a small query box: whole sequences, at most 32
};

// The share of one half: its chunks i0, i0 + step, .. of the segment's.
struct HalfSeg {
  bool both;   // more than R / 2 rows: both halves take every chunk
  bool small;  // the rows lie twice in the query tile, at 0 and 32
  int i0, step, n;
  int rows;    // this half's valid rows
  int first;   // the tile row of the first of them
};
__device__ __forceinline__ HalfSeg half_seg(const PdSeg& g, int hf, int rh, int few) {
  HalfSeg s;
  const int n = g.j1 - g.j0;
  s.both = g.rows > rh;
  s.small = g.rows <= few;
  s.i0 = s.both ? 0 : hf;
  s.step = s.both ? 1 : 2;
  s.n = s.both ? n : (n + 1 - hf) / 2;
  s.rows = s.both ? (hf ? g.rows - rh : rh) : g.rows;
  s.first = s.small ? 32 * hf : 0;
  return s;
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tmKp,
                     const __grid_constant__ CUtensorMap tmVp,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmQs,
                     const __grid_constant__ CUtensorMap tmO, const TcMaps mp, const PdParams p) {
  using C = TcCfg<D>;
  constexpr int NS = C::kNS;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ int gs[kPdMaxPrefixes + 1];
  __shared__ PdStart st;
  __shared__ int scan_sh[33];
  const uint32_t sb = smem_u32(smem);
  const uint32_t sQ = sb + C::kQOff, sKV = sb + C::kKVOff, bar = sb + C::kBarOff;
  const uint32_t q_full = bar, q_empty = bar + 16;  // [2 slots] each
  const uint32_t kv_full = bar + 32, kv_empty = kv_full + 8 * NS;
  const uint32_t s_full = kv_empty + 8 * NS;  // [2 halves]
  const uint32_t s_free = s_full + 16;        // [2]
  const uint32_t p_full = s_free + 16;        // [2 halves][2 P buffers]
  const uint32_t pv_done = p_full + 32;       // [2][2]
  const uint32_t drain = pv_done + 32;        // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + (drain + 16 - bar));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 32) {
    for (int h = 0; h < 2; ++h) {
      mbar_init(q_full + 8 * h, 1);
      mbar_init(q_empty + 8 * h, 2);
      mbar_init(s_full + 8 * h, 1);
      mbar_init(s_free + 8 * h, 4);
      for (int u = 0; u < 2; ++u) {
        mbar_init(p_full + 8 * (2 * h + u), 4);
        mbar_init(pv_done + 8 * (2 * h + u), 1);
      }
      mbar_init(drain + 8 * h, 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(kv_full + 8 * s, 1);
      mbar_init(kv_empty + 8 * s, 2);
    }
    fence_barrier_init();
  }
  const int items = p.s.N + p.s.B;
  const int key0 = static_cast<int>(threadIdx.x) < items ? pd_item_keys(p.s, threadIdx.x) : 0;
  if (warp == 0) pd_groups(p.s, gs);
  if (warp == 1) tmem_alloc<512>(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pd_locate(p.s, gs, key0, &st, scan_sh, blockIdx.x == 0 ? &p.plan : nullptr);
  const int rh = p.s.R / 2;

  PdWalk walk(p.s, gs, st);
  PdSeg g;
  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      const uint64_t once = l2_policy_evict_first();  // own caches are read once per step
      uint32_t it = 0;
      bool ok = true;
      while (ok && walk.next(g)) {
        const CUtensorMap* mk = g.own ? &tmK : &tmKp;
        const CUtensorMap* mv = g.own ? &tmV : &tmVp;
        const int kh = g.h * (g.own ? mp.kh : mp.kph), vh = g.h * (g.own ? mp.vh : mp.vph);
        const int kb = g.own ? g.b * mp.kb : g.n * mp.kpn, vb = g.own ? g.b * mp.vb : g.n * mp.vpn;
        for (int j = g.j0; j < g.j1; ++j, ++it) {
          const uint32_t s = it % NS;
          if (!mbar_wait(kv_empty + 8 * s, ((it / NS) & 1u) ^ 1u, p.s.err)) {
            ok = false;
            break;
          }
          const uint32_t fb = kv_full + 8 * s, dst = sKV + s * C::kStage;
          mbar_arrive_expect_tx(fb, C::kStage);
          const int t0 = j * kPdChunk;
#pragma unroll
          for (int d = 0; d < D / 64; ++d) {
            if (g.own) {
              tma_load_4d_hint(dst + d * 8192, mk, d * 64, t0, kh, kb, fb, once);
              tma_load_4d_hint(dst + C::kKV + d * 8192, mv, d * 64, t0, vh, vb, fb, once);
            } else {
              tma_load_4d(dst + d * 8192, mk, d * 64, t0, kh, kb, fb);
              tma_load_4d(dst + C::kKV + d * 8192, mv, d * 64, t0, vh, vb, fb);
            }
          }
        }
      }
      // let every copy in flight land before the CTA retires
      for (uint32_t i = it > NS ? it - NS : 0u; i < it; ++i)
        mbar_wait(kv_full + 8 * (i % NS), (i / NS) & 1u, p.s.err);
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    // ---------------------------------------------------------------- MMA issuers
    const int hf = warp - 1;
    if (lane == 0) {
      uint32_t it = 0, s_cnt = 0, seg = 0, qn[2] = {0, 0};
      bool ok = true;
      auto qk = [&](uint32_t stage, uint32_t qa) -> bool {
        // S is overwritten only after the softmax has loaded the previous one
        if (s_cnt > 0 && !mbar_wait(s_free + 8 * hf, (s_cnt - 1) & 1u, p.s.err)) return false;
        tc_fence_after();
        const uint32_t d = tmem + hf * 64, kb = sKV + stage * C::kStage;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss(d, smem_desc(qa + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                  smem_desc(kb + (kk >> 2) * 8192 + (kk & 3) * 32, 16, 1024), C::kIdescQK,
                  kk > 0 ? 1u : 0u);
        umma_commit(s_full + 8 * hf);
        ++s_cnt;
        return true;
      };
      while (ok && walk.next(g)) {
        const HalfSeg hs = half_seg(g, hf, rh, mp.few);
        const int n = g.j1 - g.j0;
        const uint32_t slot = hs.both ? hf : (seg & 1u);
        const uint32_t qa = sQ + slot * C::kQSlot;
        // a slot is released by two arrivals: both halves', or this half's twice
        auto release_q = [&]() {
          umma_commit(q_empty + 8 * slot);
          if (hs.both) umma_commit(q_empty + 8 * slot);
        };
        auto stage_of = [&](int i) { return (it + hs.i0 + i * hs.step) % NS; };
        auto kv_wait = [&](int i) -> bool {
          const uint32_t x = it + hs.i0 + i * hs.step;
          return mbar_wait(kv_full + 8 * (x % NS), (x / NS) & 1u, p.s.err);
        };
        if (!mbar_wait(q_full + 8 * slot, qn[slot] & 1u, p.s.err)) break;
        if (hs.n == 0) {
          release_q();
        } else {
          if (!kv_wait(0) || !qk(stage_of(0), qa)) break;
          if (hs.n == 1) release_q();
        }
        for (int i = 0; i < hs.n; ++i) {
          if (i + 1 < hs.n) {
            if (!kv_wait(i + 1) || !qk(stage_of(i + 1), qa)) {
              ok = false;
              break;
            }
            if (i + 2 == hs.n) release_q();
          }
          // chunk i is this half's k-th: S so far minus the one ahead
          const uint32_t k = s_cnt - 1 - (i + 1 < hs.n ? 1u : 0u);
          if (!mbar_wait(p_full + 8 * (2 * hf + (k & 1u)), (k >> 1) & 1u, p.s.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + kColO + hf * 128;
          const uint32_t pa = tmem + kColP + (k & 1u) * 64 + hf * 32;
          const uint32_t vb = sKV + stage_of(i) * C::kStage + C::kKV;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ts(d, pa + kk * 8, smem_desc(vb + kk * 2048, 8192, 1024), C::kIdescPV,
                    (i > 0 || kk > 0) ? 1u : 0u);
          umma_commit(pv_done + 8 * (2 * hf + (k & 1u)));
          // the stage is free once both halves have read it, or its one reader
          umma_commit(kv_empty + 8 * stage_of(i));
          if (!hs.both) umma_commit(kv_empty + 8 * stage_of(i));
        }
        it += n;
        ++qn[slot];
        if (hs.both) ++qn[slot ^ 1u];  // the other half's slot was filled too
        ++seg;
      }
      // every MMA this thread issued has finished before TMEM is released
      umma_commit(drain + 8 * hf);
      mbar_wait(drain + 8 * hf, 0u, p.s.err);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------------------------------------------------------- queries
    if (lane == 0) {
      uint32_t seg = 0, qn[2] = {0, 0};
      bool ok = true;
      while (ok && walk.next(g)) {
        const HalfSeg hs = half_seg(g, 0, rh, mp.few);
        const int b0 = g.row0 / p.s.G;  // tiles start at whole sequences
        for (int k = 0; k < (hs.both ? 2 : 1); ++k) {
          const uint32_t slot = hs.both ? k : (seg & 1u);
          if (!mbar_wait(q_empty + 8 * slot, (qn[slot] & 1u) ^ 1u, p.s.err)) {
            ok = false;
            break;
          }
          ++qn[slot];
          const uint32_t fb = q_full + 8 * slot, dst = sQ + slot * C::kQSlot;
          mbar_arrive_expect_tx(fb, (hs.small ? 2 * mp.few : rh) * D * 2);
#pragma unroll
          for (int d = 0; d < D / 64; ++d) {
            if (hs.small) {
              tma_load_3d(dst + d * 16384, &tmQs, d * 64, g.h * p.s.G, b0, fb);
              tma_load_3d(dst + d * 16384 + 4096, &tmQs, d * 64, g.h * p.s.G, b0, fb);
            } else {
              tma_load_3d(dst + d * 16384, &tmQ, d * 64, g.h * p.s.G, b0 + k * (rh / p.s.G), fb);
            }
          }
        }
        ++seg;
      }
      // the last rows have landed: their readers waited for them, or gave up
      for (int k = 0; k < 2; ++k)
        if (qn[k] > 0) mbar_wait(q_full + 8 * k, (qn[k] - 1) & 1u, p.s.err);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax + epilogue
    const int hf = (warp - 4) >> 2;
    const int wr = warp & 3;        // rows 32 wr .. of the half == TMEM lanes
    const int r = wr * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wr * 32) << 16;
    const uint32_t tS = tmem + lane_base + hf * 64;
    const uint32_t tP = tmem + lane_base + kColP + hf * 32;  // + 64 per buffer
    const uint32_t tO = tmem + lane_base + kColO + hf * 128;
    const float sl = p.scale_log2;
    const uint32_t stage = sb + C::kOOff + (warp - 4) * 4096;
    uint32_t it = 0, s_cnt = 0;
    bool ok = true;
    // PV k of this half: the (k / 2)-th completion of pv_done[hf][k & 1].  S of
    // chunk k + 2 is committed behind PV k, so a full S tells that the PV two
    // chunks back is done (its P buffer is free), and a wait for the last PV
    // finds its barrier at most one completion behind.
    auto wait_pv = [&](uint32_t k) -> bool {
      if (!warp_wait(pv_done + 8 * (2 * hf + (k & 1u)), (k >> 1) & 1u, p.s.err)) return false;
      tc_fence_after();
      return true;
    };
    while (ok && walk.next(g)) {
      const HalfSeg hs = half_seg(g, hf, rh, mp.few);
      const int rr = r - hs.first;  // this thread's row of the half
      const bool active = wr * 32 >= hs.first && wr * 32 < hs.first + hs.rows;  // warp-uniform
      const bool valid = rr >= 0 && rr < hs.rows;
      float m = -INFINITY, l = 0.f;  // running maximum of the raw scores, sum of 2^((s - m) sl)
      for (int i = 0; i < hs.n; ++i) {
        const int j = g.j0 + hs.i0 + i * hs.step;
        const uint32_t kc = s_cnt;
        const uint32_t sph = s_cnt & 1u;
        ++s_cnt;
        if (!warp_wait(s_full + 8 * hf, sph, p.s.err)) {
          ok = false;
          break;
        }
        const int nk = g.keys - j * kPdChunk;  // valid keys, if below the chunk's
        const bool ragged = nk < kPdChunk;
        if (ragged) {
          // zero the V rows past the keys, for this half's product
          const uint32_t x = it + hs.i0 + i * hs.step;
          if (!warp_wait(kv_full + 8 * (x % NS), (x / NS) & 1u, p.s.err)) {
            ok = false;
            break;
          }
          const uint32_t vb = sKV + (x % NS) * C::kStage + C::kKV;
          for (int c = r; c < (kPdChunk - nk) * (D / 8); c += 128) {
            const int row = nk + c / (D / 8), ch = c % (D / 8);
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             vb + (ch >> 3) * 8192 + row * 128 + (ch & 7) * 16),
                         "r"(0)
                         : "memory");
          }
          fence_proxy_async_smem();
        }
        if (!active) {
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(s_free + 8 * hf);
            mbar_arrive(p_full + 8 * (2 * hf + (kc & 1u)));
          }
          continue;
        }
        tc_fence_after();
        uint32_t sr[2][32];
        tmem_ld32(tS, sr[0]);
        tmem_ld32(tS + 32, sr[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free + 8 * hf);  // S is in registers
        float x[kPdChunk];
#pragma unroll
        for (int k = 0; k < kPdChunk; ++k) x[k] = __uint_as_float(sr[k >> 5][k & 31]);
        if (g.own && p.logits != nullptr && valid) {
          float4* lg = reinterpret_cast<float4*>(
              p.logits + (static_cast<int64_t>(g.unit) * p.s.G + rr) * p.Tl + j * kPdChunk);
#pragma unroll
          for (int k = 0; k < kPdChunk / 4; ++k)
            lg[k] = make_float4(x[4 * k] * sl, x[4 * k + 1] * sl, x[4 * k + 2] * sl, x[4 * k + 3] * sl);
        }
        if (ragged) {
#pragma unroll
          for (int k = 0; k < kPdChunk; ++k) x[k] = k < nk ? x[k] : -INFINITY;
        }
        float mq[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          float v = fmax3_nan(x[16 * a], x[16 * a + 1], x[16 * a + 2]);
#pragma unroll
          for (int k = 3; k < 15; k += 2) v = fmax3_nan(v, x[16 * a + k], x[16 * a + k + 1]);
          mq[a] = fmax3_nan(v, x[16 * a + 15], m);
        }
        const float mnew = fmax3_nan(fmax3_nan(mq[0], mq[1], mq[2]), mq[3], m);
        if (!(mnew < INFINITY)) l = NAN;  // a NaN or +inf logit makes the row NaN
        // Lazy rescale: a row moves its maximum only when it grew by more than
        // 2^8; the warp rescales together (the others by 1).  The unit's first
        // chunk has nothing in O yet.
        const bool grow = valid && m != -INFINITY && (mnew - m) * sl > kTcRescaleLog2;
        float alpha = 1.f;
        if (grow) {
          alpha = fast_exp2((m - mnew) * sl);
          l *= alpha;
          m = mnew;
        }
        if (m == -INFINITY) m = mnew;
        if (__any_sync(0xffffffffu, grow)) {
          if (!wait_pv(kc - 1)) {
            ok = false;
            break;
          }
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t ov[32];
            tmem_ld32(tO + cc, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(tO + cc, ov);
          }
          tmem_wait_st();
        }
        const float nm = m == -INFINITY ? 0.f : -m * sl;
        const float2 sl2 = make_float2(sl, sl), nm2 = make_float2(nm, nm);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f)};
        uint32_t pk[32];
        if (!ragged) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float2 xe = __ffma2_rn(make_float2(x[2 * e], x[2 * e + 1]), sl2, nm2);
            const float2 pe = e % 2 ? exp2_fma2_quintic(xe)
                                    : make_float2(fast_exp2(xe.x), fast_exp2(xe.y));
            acc[e & 3] = __fadd2_rn(acc[e & 3], pe);
            pk[e] = pack_bf16x2(pe.x, pe.y);
          }
        } else {  // masked keys must give exactly 0: special-function unit only
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float2 xe = __ffma2_rn(make_float2(x[2 * e], x[2 * e + 1]), sl2, nm2);
            const float2 pe = make_float2(fast_exp2(xe.x), fast_exp2(xe.y));
            acc[e & 3] = __fadd2_rn(acc[e & 3], pe);
            pk[e] = pack_bf16x2(pe.x, pe.y);
          }
        }
        l += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y) + (acc[2].x + acc[2].y) +
             (acc[3].x + acc[3].y);
        tmem_st32(tP + static_cast<uint32_t>(kc & 1) * 64, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * (2 * hf + (kc & 1u)));
      }
      if (!ok) break;
      it += g.j1 - g.j0;
      if (!active) continue;
      // epilogue: this half's partial rows
      const int64_t slot = static_cast<int64_t>(blockIdx.x) + g.unit;
      const int64_t row0 = g.own ? (slot * 2 + hf) * p.s.G : slot * kPdTcSlotRows + hf * 128;
      if (valid)
        (g.own ? p.olse : p.plse)[row0 + rr] =
            hs.n == 0 || l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m * sl) + log2f(l);
      if (hs.n == 0) continue;
      if (!wait_pv(s_cnt - 1)) {
        ok = false;
        break;
      }
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      if (g.own || hs.small) {
        // a few rows: each from its thread
        float* po = (g.own ? p.oo : p.po) + (row0 + rr) * D;
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t ov[32];
          tmem_ld32(tO + cc, ov);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(po + cc + e) =
                  make_float4(__uint_as_float(ov[e]) * inv, __uint_as_float(ov[e + 1]) * inv,
                              __uint_as_float(ov[e + 2]) * inv, __uint_as_float(ov[e + 3]) * inv);
          }
        }
      } else {
        // 32 rows x 32 columns at a time through shared memory (row stores
        // from the threads would touch 32 lines each).  Rows past the unit's
        // land in the slot's unused rows.
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t ov[32];
          tmem_ld32(tO + cc, ov);
          tmem_wait_ld();
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();  // the previous store has read the staged rows
#pragma unroll
          for (int e = 0; e < 8; ++e)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                             stage + lane * 128 + ((e ^ (lane & 7)) << 4)),
                         "f"(__uint_as_float(ov[4 * e]) * inv),
                         "f"(__uint_as_float(ov[4 * e + 1]) * inv),
                         "f"(__uint_as_float(ov[4 * e + 2]) * inv),
                         "f"(__uint_as_float(ov[4 * e + 3]) * inv)
                         : "memory");
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmO, stage, cc, static_cast<int>(row0) + wr * 32);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      }
      // the next unit's first PV overwrites O: it is issued after this
      // warpgroup's next p_full arrivals, which follow these loads
      tc_fence_before();
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<512>(tmem);
}

// A tensor map of [n0, n1, rows, D]; a dimension of one entry, or of stride 0
// (the same rows for all), becomes one entry with multiplier 0.
bool kv_map(CUtensorMap* map, const void* base, int64_t n0, int64_t n1, int64_t rows, int D,
            const int64_t* st, int* m1, int* m0, std::string* why) {
  *m1 = n1 > 1 && st[1] != 0;
  *m0 = n0 > 1 && st[0] != 0;
  const uint64_t rs = rows > 1 ? st[2] : D;
  return make_tmap_bf16_4d(map, base, D, rows, *m1 ? n1 : 1, *m0 ? n0 : 1, rs, *m1 ? st[1] : D,
                           *m0 ? st[0] : D, kPdChunk, 64, why);
}

template <int D>
cudaError_t launch_tc(const Launch& l, const PdParams& p, std::string* why) {
  CUtensorMap kp, vp, k, v, q, qs, o;
  TcMaps m{};
  const bool pre = p.s.N > 0 && p.s.Tp > 0, own = p.s.T > 0;
  if (pre && (!kv_map(&kp, p.Kp, p.s.N, p.s.Hkv, p.s.Tp, D, p.kps, &m.kph, &m.kpn, why) ||
              !kv_map(&vp, p.Vp, p.s.N, p.s.Hkv, p.s.Tp, D, p.vps, &m.vph, &m.vpn, why)))
    return cudaErrorInvalidValue;
  if (own && (!kv_map(&k, p.K, p.s.B, p.s.Hkv, p.s.T, D, p.ks, &m.kh, &m.kb, why) ||
              !kv_map(&v, p.V, p.s.B, p.s.Hkv, p.s.T, D, p.vs, &m.vh, &m.vb, why)))
    return cudaErrorInvalidValue;
  // a side without keys is never loaded: any map will do for it
  if (!pre && own) kp = k, vp = v;
  if (!own && pre) k = kp, v = vp;
  if (!own && !pre) kp = vp = k = v = CUtensorMap{};
  const int G = p.s.G;
  m.few = 32 / G * G;
  const uint64_t D_ = D, Hq = p.Hq;
  if (!make_tmap_3d(&q, p.q, false, D, Hq, p.s.B, D_, Hq * D_, 64, G, 128 / G, why) ||
      !make_tmap_3d(&qs, p.q, false, D, Hq, p.s.B, D_, Hq * D_, 64, G, 32 / G, why))
    return cudaErrorInvalidValue;
  o = q;  // without prefixes there are no staged stores
  if (pre && !make_tmap_3d(&o, p.po, true, D, static_cast<uint64_t>(p.slots) * kPdTcSlotRows, 0, D_,
                           0, 32, 32, 0, why))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attend_tc_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       TcCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  attend_tc_kernel<D><<<p.s.P, kTcThreads, TcCfg<D>::kSmem, l.stream>>>(kp, vp, k, v, q, qs, o, m, p);
  return cudaGetLastError();
}

}  // namespace

// A tile's halves hold whole sequences, at most 128 rows.
int pd_tc_rows(int G) { return 2 * (128 / G * G); }

cudaError_t launch_attend_tc(const Launch& l, const PdParams& p, int D, std::string* why) {
  return D == 128 ? launch_tc<128>(l, p, why) : launch_tc<64>(l, p, why);
}

}  // namespace csa
