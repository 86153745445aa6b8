// Arguments of the shared-prefix decode's kernels.
#pragma once

#include "prefix_work.cuh"

namespace csa {

constexpr float kPdLog2e = 1.4426950408889634f;
constexpr float kPdLn2 = 0.6931471805599453f;

struct PdParams {
  PdShape s;
  const void *q, *Kp, *Vp, *K, *V;
  int64_t kps[3], vps[3], ks[3], vs[3];  // strides in elements: prefix / sequence, head, token
  int Hq;
  float scale_log2;
  // workspace.  A prefix unit's slot holds `slot_rows` rows, an own unit's
  // `halves` * G.  With halves = 2 row r of a tile lies at (r / (R/2)) *
  // slot_rows/2 + r % (R/2), and a unit of at most R / 2 rows (an own one always)
  // is split once more inside its CTA: even chunks' rows in the slot's first
  // half, odd chunks' in its second.
  int halves, slot_rows;
  int64_t slots;  // prefix slots
  PdPlan plan;
  float *plse, *po, *olse, *oo, *logits;
  int64_t Tl;  // logits' row length
  // outputs
  void* out;
  int out_bf16;
  float* lse_out;
  float* acc;
  float decay;
};

// prefix_decode_tc.cu: the bf16 attention kernel.
int pd_tc_rows(int G);           // query rows per tile
constexpr int kPdTcSlotRows = 256;
cudaError_t launch_attend_tc(const Launch& l, const PdParams& p, int D, std::string* why);

}  // namespace csa
