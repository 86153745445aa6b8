// Prefix attention of the shared-prefix decode (bf16, groups of more query rows
// than line b takes) on the 5th-generation tensor cores (tcgen05,
// accumulators in tensor memory).
//
// Work unit: up to R <= 256 query rows against a run of keys (prefix_work.cuh),
// in chunks of 64 keys.  Per chunk and 128-row half:
//   S = Q K^T     tcgen05.mma M=128 N=64 K=D, operands in shared memory
//   P = softmax   a warpgroup reads S with tcgen05.ld, keeps each row's running
//                 maximum and sum in registers (fp32) and writes P to tensor
//                 memory as bf16 (the A operand of the second product has V's
//                 type; a rounding of 2^-8 of each weight at most)
//   O += P V      tcgen05.mma M=128 N=D K=64, V from shared memory
// Units of more than R / 2 rows give each half its own rows and both the same
// chunk.  Units of fewer give the halves the even and the odd chunks, so two
// softmax chains share the CTA's chunks; each half writes its own partial
// rows.  A unit of at most 32 rows has them twice, at rows 0 and 32 of the query
// tile: half 1 reads the copy, so that the two chains run on different warps
// of the tile's rows and so on different schedulers.  Rows past a unit's are
// garbage that no other row sees; their warps only keep the barriers' counts.
//
// Bound: a CTA's chunk is 256 D bytes of K and V.  At the copy rate an SM gets about
// 23 bytes a clock, 1430 clocks a chunk at D = 128, against 640 clocks of
// products (QK^T at N = 64 is bound by its shared-memory operands) and 512 of
// exponentials per half: up to 128 rows memory is the bound (128K tokens, 8 KV
// heads, 128 rows: this kernel 95 us, 87% of the copy rate, 1310 clocks a chunk).  With
// 256 rows a chunk takes about 2000 clocks (146 us): the tensor pipe passes between the four groups of
// products per chunk (QK^T and PV of each half), each short.  Measured there
// and not kept: half or a quarter of the exponentials on the FMA pipe (8% and 6%
// slower), four softmax warps per scheduler instead of two, a column half each
// (9%), P written over S with QK^T two chunks ahead (9%).
// The keys past a unit's end are masked in S, and their V rows zeroed in
// shared memory, so that neither value reaches a result (0 * NaN is NaN).
//
// Warps: 0 TMA (K and V, rings of 144 KB in all), 1 and 2 the halves' MMA issuers
// (1 owns the tensor memory), 3 the queries (TMA; two 128-row slots, so
// that the next small unit's rows arrive early), 4-7 and 8-11 softmax and
// epilogue of half 0 and 1.  Every wait is bounded.
#pragma once

#include "prefix_decode.cuh"
#include "tcgen05.cuh"

namespace csa {
namespace {

constexpr int kTcThreads = 384;
constexpr float kTcRescaleLog2 = 8.0f;
constexpr int kChunk = 1 << kPdTcChunkLog2;

template <int D>
struct TcCfg {
  static constexpr int kQSlot = 128 * D * 2;
  static constexpr int kKV = kChunk * D * 2;  // bytes of K (or V) per chunk
  // K and V have rings of their own: a K chunk is free after its QK^T, a V
  // chunk only after the softmax and PV behind it, and each half looks one
  // QK^T ahead (with one ring of 4 stages all were held and none loading)
  static constexpr int kNK = 4 * 128 / D, kNV = 5 * 128 / D;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = 2 * kQSlot;
  static constexpr int kVOff = kKOff + kNK * kKV;
  static constexpr int kOOff = kVOff + kNV * kKV;  // 2 KB of output rows per softmax warp
  static constexpr int kBarOff = kOOff + 8 * 2048;
  static constexpr int kSmem = 1024 + kBarOff + 512;
  static constexpr uint32_t kIdescQK = idesc_bf16(128, kChunk, 0);
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
// Index multipliers (0 for a broadcast dimension, whose map has one entry).
struct TcMaps {
  int kh, kn, vh, vn;
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

// Addresses of the barriers (shared) and the places of the tensor memory's
// address.
template <int D>
struct TcBars {
  static constexpr int NK = TcCfg<D>::kNK, NV = TcCfg<D>::kNV;
  uint32_t q_full, q_empty;    // [2 slots] each
  uint32_t k_full, k_empty, v_full, v_empty;
  uint32_t s_full, s_free;     // [2 halves]
  uint32_t p_full, pv_done;    // [2 halves][2 P buffers]
  uint32_t drain;              // [2]
  uint32_t turn;               // [2 halves][4 warps]
  uint32_t end;
  __device__ __forceinline__ explicit TcBars(uint32_t bar) {
    q_full = bar;
    q_empty = bar + 16;
    k_full = bar + 32;
    k_empty = k_full + 8 * NK;
    v_full = k_empty + 8 * NK;
    v_empty = v_full + 8 * NV;
    s_full = v_empty + 8 * NV;
    s_free = s_full + 16;
    p_full = s_free + 16;
    pv_done = p_full + 32;
    drain = pv_done + 32;
    turn = drain + 16;
    end = turn + 64;
  }
  __device__ __forceinline__ void init() const {  // one thread
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
      for (int w = 0; w < 4; ++w) mbar_init(turn + 8 * (4 * h + w), 1);
    }
    for (int s = 0; s < NK; ++s) {
      mbar_init(k_full + 8 * s, 1);
      mbar_init(k_empty + 8 * s, 2);
    }
    for (int s = 0; s < NV; ++s) {
      mbar_init(v_full + 8 * s, 1);
      mbar_init(v_empty + 8 * s, 2);
    }
    fence_barrier_init();
  }
};

// A CTA of line a: worker `block`.  The barriers are set up and the tensor
// memory is allocated by warp 1, which frees it after this.
template <int D>
__device__ __forceinline__ void attend_tc(const CUtensorMap& tmK, const CUtensorMap& tmV,
                                          const CUtensorMap& tmQ, const CUtensorMap& tmQs,
                                          const CUtensorMap& tmO, const TcMaps& mp,
                                          const PdParams& p, uint8_t* smem, const TcBars<D>& bars,
                                          uint32_t tmem, const int* gs, const PdStart& st,
                                          int block) {
  using C = TcCfg<D>;
  constexpr int NK = C::kNK, NV = C::kNV;
  const uint32_t sb = smem_u32(smem);
  const uint32_t sQ = sb + C::kQOff, sK = sb + C::kKOff, sV = sb + C::kVOff;
  const uint32_t q_full = bars.q_full, q_empty = bars.q_empty;
  const uint32_t k_full = bars.k_full, k_empty = bars.k_empty;
  const uint32_t v_full = bars.v_full, v_empty = bars.v_empty;
  const uint32_t s_full = bars.s_full, s_free = bars.s_free;
  const uint32_t p_full = bars.p_full, pv_done = bars.pv_done;
  const uint32_t drain = bars.drain, turn = bars.turn;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PdShape& shape = p.a.s;
  const int rh = shape.R / 2;

  PdWalk walk(shape, gs, st);
  PdSeg g;
  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      uint32_t it = 0, kn = 0, vn = 0;  // chunks; K and V loads issued
      bool ok = true;
      while (ok && walk.next(g)) {
        const int kh = g.h * mp.kh, vh = g.h * mp.vh, kn_ = g.n * mp.kn, vn_ = g.n * mp.vn;
        for (int j = g.j0; j < g.j1; ++j, ++it) {
          const uint32_t ks = it % NK, vs = it % NV;
          const int t0 = j * kChunk;
          if (!mbar_wait(k_empty + 8 * ks, ((it / NK) & 1u) ^ 1u, shape.err)) {
            ok = false;
            break;
          }
          const uint32_t kf = k_full + 8 * ks, kd = sK + ks * C::kKV;
          mbar_arrive_expect_tx(kf, C::kKV);
#pragma unroll
          for (int d = 0; d < D / 64; ++d)
            tma_load_4d(kd + d * 8192, &tmK, d * 64, t0, kh, kn_, kf);
          ++kn;
          if (!mbar_wait(v_empty + 8 * vs, ((it / NV) & 1u) ^ 1u, shape.err)) {
            ok = false;
            break;
          }
          const uint32_t vf = v_full + 8 * vs, vd = sV + vs * C::kKV;
          mbar_arrive_expect_tx(vf, C::kKV);
#pragma unroll
          for (int d = 0; d < D / 64; ++d)
            tma_load_4d(vd + d * 8192, &tmV, d * 64, t0, vh, vn_, vf);
          ++vn;
        }
      }
      // let every copy in flight land before the CTA retires
      for (uint32_t i = kn > NK ? kn - NK : 0u; i < kn; ++i)
        mbar_wait(k_full + 8 * (i % NK), (i / NK) & 1u, shape.err);
      for (uint32_t i = vn > NV ? vn - NV : 0u; i < vn; ++i)
        mbar_wait(v_full + 8 * (i % NV), (i / NV) & 1u, shape.err);
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2) {
    // ---------------------------------------------------------------- MMA issuers
    // The whole warp walks, waits and forms the descriptors, so that they live
    // in uniform registers; one elected lane issues.  (From one lane's own
    // registers each MMA took about 100 clocks to issue, 1250 a chunk.)
    const int hf = __shfl_sync(0xffffffffu, warp, 0) - 1;
    uint32_t it = 0, s_cnt = 0, seg = 0, qn[2] = {0, 0};
    bool ok = true;
    // S = Q K^T of the CTA's chunk x
    auto qk = [&](uint32_t x, uint32_t qa, bool both) -> bool {
      if (!warp_wait(k_full + 8 * (x % NK), (x / NK) & 1u, shape.err)) return false;
      // S is overwritten only after the softmax has loaded the previous one
      if (s_cnt > 0 && !warp_wait(s_free + 8 * hf, (s_cnt - 1) & 1u, shape.err)) return false;
      tc_fence_after();
      const uint32_t d = tmem + hf * 64;
      const uint64_t qd = smem_desc(qa, 16, 1024), kd = smem_desc(sK + (x % NK) * C::kKV, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss(d, qd + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                  kd + (((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), C::kIdescQK, kk > 0 ? 1u : 0u);
        umma_commit(s_full + 8 * hf);
        // the stage is free once both halves have read it, or its one reader
        umma_commit(k_empty + 8 * (x % NK));
        if (!both) umma_commit(k_empty + 8 * (x % NK));
      }
      __syncwarp();
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
        if (elect_one()) {
          umma_commit(q_empty + 8 * slot);
          if (hs.both) umma_commit(q_empty + 8 * slot);
        }
        __syncwarp();
      };
      auto chunk = [&](int i) -> uint32_t { return it + hs.i0 + i * hs.step; };
      if (!warp_wait(q_full + 8 * slot, qn[slot] & 1u, shape.err)) break;
      if (hs.n == 0) {
        release_q();
      } else {
        if (!qk(chunk(0), qa, hs.both)) break;
        if (hs.n == 1) release_q();
      }
      for (int i = 0; i < hs.n; ++i) {
        if (i + 1 < hs.n) {
          if (!qk(chunk(i + 1), qa, hs.both)) {
            ok = false;
            break;
          }
          if (i + 2 == hs.n) release_q();
        }
        // chunk i is this half's k-th: S so far minus the one ahead
        const uint32_t k = s_cnt - 1 - (i + 1 < hs.n ? 1u : 0u);
        const uint32_t x = chunk(i), vst = x % NV;
        if (!warp_wait(v_full + 8 * vst, (x / NV) & 1u, shape.err) ||
            !warp_wait(p_full + 8 * (2 * hf + (k & 1u)), (k >> 1) & 1u, shape.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + kColO + hf * 128;
        const uint32_t pa = tmem + kColP + (k & 1u) * 64 + hf * 32;
        const uint64_t vd = smem_desc(sV + vst * C::kKV, 8192, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ts(d, pa + kk * 8, vd + ((kk * 2048) >> 4), C::kIdescPV, (i > 0 || kk > 0) ? 1u : 0u);
          umma_commit(pv_done + 8 * (2 * hf + (k & 1u)));
          umma_commit(v_empty + 8 * vst);
          if (!hs.both) umma_commit(v_empty + 8 * vst);
        }
        __syncwarp();
      }
      it += n;
      ++qn[slot];
      if (hs.both) ++qn[slot ^ 1u];  // the other half's slot was filled too
      ++seg;
    }
    // every MMA this warp issued has finished before TMEM is released
    if (elect_one()) umma_commit(drain + 8 * hf);
    __syncwarp();
    warp_wait(drain + 8 * hf, 0u, shape.err);
  } else if (warp == 3) {
    // ---------------------------------------------------------------- queries
    if (lane == 0) {
      uint32_t seg = 0, qn[2] = {0, 0};
      bool ok = true;
      while (ok && walk.next(g)) {
        const HalfSeg hs = half_seg(g, 0, rh, mp.few);
        const int b0 = g.row0 / shape.G;  // tiles start at whole sequences
        for (int k = 0; k < (hs.both ? 2 : 1); ++k) {
          const uint32_t slot = hs.both ? k : (seg & 1u);
          if (!mbar_wait(q_empty + 8 * slot, (qn[slot] & 1u) ^ 1u, shape.err)) {
            ok = false;
            break;
          }
          ++qn[slot];
          const uint32_t fb = q_full + 8 * slot, dst = sQ + slot * C::kQSlot;
          mbar_arrive_expect_tx(fb, (hs.small ? 2 * mp.few : rh) * D * 2);
#pragma unroll
          for (int d = 0; d < D / 64; ++d) {
            if (hs.small) {
              tma_load_3d(dst + d * 16384, &tmQs, d * 64, g.h * shape.G, b0, fb);
              tma_load_3d(dst + d * 16384 + 4096, &tmQs, d * 64, g.h * shape.G, b0, fb);
            } else {
              tma_load_3d(dst + d * 16384, &tmQ, d * 64, g.h * shape.G, b0 + k * (rh / shape.G), fb);
            }
          }
        }
        ++seg;
      }
      // the last rows have landed: their readers waited for them, or gave up
      for (int k = 0; k < 2; ++k)
        if (qn[k] > 0) mbar_wait(q_full + 8 * k, (qn[k] - 1) & 1u, shape.err);
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
    const uint32_t stage = sb + C::kOOff + (warp - 4) * 2048;
    uint32_t it = 0, s_cnt = 0, turns = 0;
    bool ok = true;
    // In a unit of both halves the two warps of a scheduler take turns at the
    // exponentials (half 0 first): in step they share the special-function unit
    // there and leave it idle elsewhere (158 against 151 us, measured
    // in turn).
    auto turn_wait = [&]() -> bool {
      const uint32_t n = turns++;
      return warp_wait(turn + 8 * (4 * hf + wr), hf ? n & 1u : (n & 1u) ^ 1u, shape.err);
    };
    auto turn_pass = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(turn + 8 * (4 * (hf ^ 1) + wr));
    };
    // PV k of this half: the (k / 2)-th completion of pv_done[hf][k & 1].  S of
    // chunk k + 2 is committed behind PV k, so a full S tells that the PV two
    // chunks back is done (its P buffer is free), and a wait for the last PV
    // finds its barrier at most one completion behind.
    auto wait_pv = [&](uint32_t k) -> bool {
      if (!warp_wait(pv_done + 8 * (2 * hf + (k & 1u)), (k >> 1) & 1u, shape.err)) return false;
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
        if (!warp_wait(s_full + 8 * hf, sph, shape.err)) {
          ok = false;
          break;
        }
        const int nk = g.keys - j * kChunk;  // valid keys, if below the chunk's
        const bool ragged = nk < kChunk;
        if (ragged) {
          // zero the V rows past the keys, for this half's product
          const uint32_t x = it + hs.i0 + i * hs.step;
          if (!warp_wait(v_full + 8 * (x % NV), (x / NV) & 1u, shape.err)) {
            ok = false;
            break;
          }
          const uint32_t vb = sV + (x % NV) * C::kKV;
          for (int c = r; c < (kChunk - nk) * (D / 8); c += 128) {
            const int row = nk + c / (D / 8), ch = c % (D / 8);
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             vb + (ch >> 3) * 8192 + row * 128 + (ch & 7) * 16),
                         "r"(0)
                         : "memory");
          }
          fence_proxy_async_smem();
        }
        if (!active) {
          if (hs.both) {
            if (!turn_wait()) {
              ok = false;
              break;
            }
            turn_pass();
          }
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
        float x[kChunk];
#pragma unroll
        for (int k = 0; k < kChunk; ++k) x[k] = __uint_as_float(sr[k >> 5][k & 31]);
        if (ragged) {
#pragma unroll
          for (int k = 0; k < kChunk; ++k) x[k] = k < nk ? x[k] : -INFINITY;
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
        if (hs.both && !turn_wait()) {
          ok = false;
          break;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 xe = __ffma2_rn(make_float2(x[2 * e], x[2 * e + 1]), sl2, nm2);
          const float2 pe = make_float2(fast_exp2(xe.x), fast_exp2(xe.y));
          acc[e & 3] = __fadd2_rn(acc[e & 3], pe);
          pk[e] = pack_bf16x2(pe.x, pe.y);
        }
        if (hs.both) turn_pass();
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
      const int64_t slot = static_cast<int64_t>(block) + g.unit;
      const int64_t row0 = slot * kPdTcSlotRows + hf * 128;
      if (valid)
        p.a.plse[row0 + rr] =
            hs.n == 0 || l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m * sl) + log2f(l);
      if (hs.n == 0) continue;
      if (!wait_pv(s_cnt - 1)) {
        ok = false;
        break;
      }
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      if (hs.small) {
        // a few rows: each from its thread
        float* po = p.a.po + (row0 + rr) * D;
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
        // 32 rows x 16 columns at a time through shared memory (row stores
        // from the threads would touch 32 lines each).  Rows past the unit's
        // land in the slot's unused rows.
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t ov[32];
          tmem_ld32(tO + cc, ov);
          tmem_wait_ld();
#pragma unroll
          for (int c2 = 0; c2 < 32; c2 += 16) {
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();  // the previous store has read the staged rows
            // 64-byte swizzle: 16-byte chunk e of row r at e ^ (r / 2 % 4)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                               stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)),
                           "f"(__uint_as_float(ov[c2 + 4 * e]) * inv),
                           "f"(__uint_as_float(ov[c2 + 4 * e + 1]) * inv),
                           "f"(__uint_as_float(ov[c2 + 4 * e + 2]) * inv),
                           "f"(__uint_as_float(ov[c2 + 4 * e + 3]) * inv)
                           : "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmO, stage, cc + c2, static_cast<int>(row0) + wr * 32);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
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
}

}  // namespace
}  // namespace csa
