// The bf16 attention kernel of the shared-prefix decode: CTAs of line a (groups
// of many query rows, on the tensor memory) and of line b (the rest, warp by
// warp) in one launch, one CTA per SM.
#include <algorithm>

#include "prefix_tc.cuh"
#include "prefix_warp.cuh"

namespace csa {
namespace {

// NT: tiles of 8 query rows in a unit of line b.
template <int D, int NT>
__global__ void __launch_bounds__(kTcThreads, 1)
    attend_bf16_kernel(const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmQs,
                       const __grid_constant__ CUtensorMap tmO, const TcMaps mp,
                       const PdParams p) {
  pdl_next();  // the merge
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ int gs[kPdMaxPrefixes + 1];
  __shared__ PdShared ps;
  __shared__ uint32_t tmem_slot;
  const int tid = threadIdx.x, warp = tid >> 5;
  const bool two = p.a.s.ctas > 0;
  const int key0 = tid < p.b.s.N + p.b.s.B ? pd_raw_keys(p.b.s, tid) : 0;
  const TcBars<D> bars(smem_u32(smem) + TcCfg<D>::kBarOff);
  // what line a needs is set up by every CTA while the lengths are on their way
  if (warp == 0) pd_groups(p.b.s, gs);
  if (two && tid == 64) bars.init();
  if (two && tid == 96) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (two && warp == 1) tmem_alloc<512>(&tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool first = blockIdx.x == 0;
  const PdPlace at = pd_locate(p.a.s, p.b.s, gs, key0, &ps,
                               first && two ? &p.a.plan : nullptr, first ? &p.b.plan : nullptr);
  if (at.line == 0)
    attend_tc<D>(tmK, tmV, tmQ, tmQs, tmO, mp, p, smem, bars, tmem_slot, gs, ps.st[0], at.block);
  if (two && warp == 1) tmem_dealloc<512>(tmem_slot);
  if (at.line == 1 && warp < kPdWarps) attend_warp<D, NT>(p, smem, gs, ps.st, at.block);
}

// A tensor map of [n0, n1, rows, D]; a dimension of one entry, or of stride 0
// (the same rows for all), becomes one entry with multiplier 0.
bool kv_map(CUtensorMap* map, const void* base, int64_t n0, int64_t n1, int64_t rows, int D,
            const int64_t* st, int* m1, int* m0, std::string* why) {
  *m1 = n1 > 1 && st[1] != 0;
  *m0 = n0 > 1 && st[0] != 0;
  const uint64_t rs = rows > 1 ? st[2] : D;
  return make_tmap_bf16_4d(map, base, D, rows, *m1 ? n1 : 1, *m0 ? n0 : 1, rs, *m1 ? st[1] : D,
                           *m0 ? st[0] : D, kChunk, 64, why);
}

template <int D>
constexpr int smem_bytes() {
  return TcCfg<D>::kSmem > WCfg<D>::kSmem + 1024 ? TcCfg<D>::kSmem : WCfg<D>::kSmem + 1024;
}

template <int D, int NT>
cudaError_t launch(const Launch& l, const PdParams& p, std::string* why) {
  const PdShape& s = p.b.s;
  CUtensorMap k{}, v{}, q{}, qs{}, o{};
  TcMaps m{};
  m.few = 32 / s.G * s.G;
  const uint64_t Hq = p.Hq;
  if (p.a.s.ctas > 0 &&
      (!kv_map(&k, p.Kp, s.N, s.Hkv, s.Tp, D, p.kps, &m.kh, &m.kn, why) ||
       !kv_map(&v, p.Vp, s.N, s.Hkv, s.Tp, D, p.vps, &m.vh, &m.vn, why) ||
       !make_tmap_3d(&q, p.q, false, D, Hq, s.B, D, Hq * D, 64, s.G, 128 / s.G, 128, why) ||
       !make_tmap_3d(&qs, p.q, false, D, Hq, s.B, D, Hq * D, 64, s.G, 32 / s.G, 128, why) ||
       !make_tmap_3d(&o, p.a.po, true, D, static_cast<uint64_t>(p.a.slots) * kPdTcSlotRows, 0, D, 0,
                     16, 32, 0, 64, why)))
    return cudaErrorInvalidValue;
  constexpr int smem = smem_bytes<D>();
  cudaError_t e = cudaFuncSetAttribute(attend_bf16_kernel<D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // an ordinary launch: the merge behind it reads what earlier kernels wrote
  attend_bf16_kernel<D, NT><<<s.ctas, kTcThreads, smem, l.stream>>>(k, v, q, qs, o, m, p);
  return cudaGetLastError();
}

}  // namespace

// A tile's halves hold whole sequences, at most 128 rows.
int pd_tc_rows(int G) { return 2 * (128 / G * G); }

cudaError_t launch_attend_bf16(const Launch& l, const PdParams& p, int D, std::string* why) {
  const bool wide = p.b.s.R > 8;
  if (D == 128) return wide ? launch<128, 2>(l, p, why) : launch<128, 1>(l, p, why);
  return wide ? launch<64, 2>(l, p, why) : launch<64, 1>(l, p, why);
}

}  // namespace csa
