// Arguments of the shared-prefix decode's kernels.
#pragma once

#include "prefix_work.cuh"

namespace csa {

constexpr float kPdLog2e = 1.4426950408889634f;
constexpr float kPdLn2 = 0.6931471805599453f;

// bf16: groups of more rows than line b's tile are line a (prefix_tc.cuh), the
// others and the own units line b (prefix_warp.cuh), whose tile is the G rows of
// an own unit rounded up to eights.  fp32 has line b alone.
inline int pd_few_rows(int G) { return G <= 8 ? 8 : 16; }

// A line of units and where its partials go.  A prefix unit's slot
// holds `slot_rows` rows, an own unit's G.  With halves = 2 row r of a tile
// lies at (r / (R/2)) * slot_rows/2 + r % (R/2), and a unit of at most R / 2
// rows is split once more inside its CTA: even chunks' rows in the slot's first
// half, odd chunks' in its second.
struct PdLine {
  PdShape s;
  PdPlan plan;
  int halves, slot_rows;
  int64_t slots;  // prefix slots
  float *plse, *po;
};

struct PdParams {
  PdLine a;  // bf16: the groups of many rows; a.s.ctas = 0: no such line
  PdLine b;  // the rest
  const void *q, *Kp, *Vp, *K, *V;
  int64_t kps[3], vps[3], ks[3], vs[3];  // strides in elements: prefix / sequence, head, token
  int Hq;
  float scale_log2;
  float *olse, *oo, *logits;  // own units' partials (line b) and logits
  int64_t Tl;                 // logits' row length
  // outputs
  void* out;
  int out_bf16;
  float* lse_out;
  float* acc;
  float decay;
  const int32_t* next_pos;  // [B] or null; negative: the sequence is inactive
};

// prefix_decode_bf16.cu
int pd_tc_rows(int G);  // query rows per tile of line a
constexpr int kPdTcSlotRows = 256;
constexpr int kPdTcChunkLog2 = 6;
constexpr int kPdWarps = 8;  // warps of a CTA on line b
constexpr int kPdWarpChunkLog2 = 4;
// What a unit costs besides its keys, in chunks' time: its queries, the first
// chunk's way and its partials.  (Without, the warps that got many units of a
// few keys were the last by 8 of 30 us.)
constexpr int kPdTcLead = 2, kPdWarpLead = 2;
cudaError_t launch_attend_bf16(const Launch& l, const PdParams& p, int D, std::string* why);

}  // namespace csa
