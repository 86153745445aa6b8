// Internal launcher interface between the C ABI (api.cu) and the kernel files.
// Launchers assume validated arguments and return the launch's cudaError_t.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "common.cuh"

namespace csa {

// Sets the thread-local message returned by csa_last_error_string().
void set_last_error(const std::string& why);

struct Launch {
  cudaStream_t stream;
  DevErr err;
  int num_sms;
  // the launch follows a kernel that writes the query it reads (a host-query
  // copy): a launcher that supports it starts behind that kernel with
  // programmatic dependent launch and waits for it before reading the query
  bool after_query_copy = false;
};

// A launch that may start while the kernel before it on the stream drains
// (programmatic dependent launch): before pdl_wait() the kernel must read nothing
// that the one before it writes, and write nothing that it reads.  What still
// earlier kernels wrote may be read ahead of the wait only where the kernel
// before it is an ordinary launch, which waited for them.  pdl_next() lets the
// next one in.
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// summaries.cu
cudaError_t launch_chunk_summaries(const Launch& l, const void* K, bool bf16, int U, int64_t T,
                                   int D, int L, const float* proj, int R, float* summ);
cudaError_t launch_meta_summaries(const Launch& l, const float* summ, int U, int C, int Ds, int Gm,
                                  float* meta);
cudaError_t launch_tile_mean(const Launch& l, const void* Q, bool bf16, int B, int S, int Hq, int D,
                             int tile_m, float* qbar);

// score.cu
cudaError_t launch_score(const Launch& l, const void* q, bool bf16, const float* proj, int R,
                         const float* summ, int B, int Nq, int Hq, int Hkv, int D, int C,
                         const uint8_t* head_full, int causal_tile_m, int causal_L,
                         float* scores);

// select.cu
// causal_tiles > 0: unit u is query tile u % causal_tiles of a causal
// prefill and sees the chunks c < ((t + 1) * causal_tile_m - 1) / causal_L + 1
// (n_valid is then ignored).  inv (optional, [U, C]): when the long-row
// cluster kernel runs, it also writes every position's slot in its unit's
// list (or -1) and sets *inv_done; otherwise *inv_done is false.
// The long-row top-k (one cluster of 8 CTAs per unit) runs for these sizes
// (rows of C >= 8192 keys, nothing forced).
bool topk_cluster_fits(int U, int C, int num_sms);
cudaError_t launch_select_topk(const Launch& l, const float* scores, int U, int C,
                               const int32_t* n_valid, int k_free, int n_sink, int n_local,
                               int32_t* idx, int32_t* count, int kmax,
                               const int32_t* k_dev = nullptr, int causal_tiles = 0,
                               int causal_tile_m = 0, int causal_L = 0, int32_t* inv = nullptr,
                               bool* inv_done = nullptr);
cudaError_t launch_select_topp(const Launch& l, const float* scores, int U, int C,
                               float logit_scale, float p, int budget, int n_sink, int n_local,
                               int32_t* idx, int32_t* count, int kmax, int32_t* n_p_out);
cudaError_t launch_select_hier(const Launch& l, const void* q, bool bf16, const float* meta,
                               const float* summ, int B, int Hq, int Hkv, int D, int C, int Gm,
                               int top_meta, int k_free, int n_sink, int n_local, int32_t* idx,
                               int32_t* count, int kmax);

cudaError_t launch_score_select_topk(const Launch& l, const void* q, bool bf16, const float* proj,
                                     int R, const float* summ, int B, int Hq, int Hkv, int D, int C,
                                     const uint8_t* head_full, int k_free, int n_sink, int n_local,
                                     int32_t* idx, int32_t* count, int kmax,
                                     bool per_head_union = false);
cudaError_t launch_score_select_topp(const Launch& l, const void* q, bool bf16, const float* proj,
                                     int R, const float* summ, int B, int Hq, int Hkv, int D, int C,
                                     const uint8_t* head_full, float logit_scale, float p,
                                     int budget, int n_sink, int n_local, int32_t* idx,
                                     int32_t* count, int kmax, int32_t* n_p_out);

// token_sparse.cu
size_t token_importance_scratch_bytes(int B, int S, int Hkv, int G, int n_obs);
cudaError_t launch_token_importance(const Launch& l, const void* Q, const void* K, int B, int S,
                                    int Hq, int Hkv, int D, int n_obs, float scale, float* imp,
                                    float* scratch, std::string* why);
// The coverage budget runs one cluster of 8 CTAs per sequence for these
// sizes (else one CTA per sequence, S <= 32768).
bool token_budget_cluster_fits(int B, int num_sms);
cudaError_t launch_token_budget(const Launch& l, const float* imp, int B, int S, int Hkv,
                                float tau, int tile, int32_t* k_seq, int32_t* k_unit);
cudaError_t launch_tsa_gather(const Launch& l, const void* Q, const void* K, const void* V,
                              const int32_t* idx, const int32_t* count, int kmax, int B, int S,
                              int Sc, int Hq, int Hkv, int D, void* Qc, void* Kc, void* Vc);
// inv [B*Hkv, S] (scratch): built here from idx/count unless inv_ready (the
// selection wrote it)
cudaError_t launch_tsa_scatter(const Launch& l, const void* Oc, const int32_t* idx,
                               const int32_t* count, int kmax, int B, int S, int Sc, int Hq,
                               int Hkv, int D, int32_t* inv, void* O, bool inv_ready = false);

// rope.cu
cudaError_t launch_rope(const Launch& l, const void* x, void* y, bool bf16, int64_t rows, int D,
                        int64_t period, int64_t pos0, float theta);

// rotary.cu
enum RotScaling : int { ROT_NONE = 0, ROT_LINEAR = 1, ROT_NTK = 2, ROT_TURNS = 3, ROT_RAMP = 4 };
struct RotaryArgs {
  struct Tensor {  // H = 0: none
    const void* x = nullptr;
    void* y = nullptr;
    int H = 0;
    int64_t xst[3] = {0, 0, 0};  // batch, token, head strides in elements
    int64_t yst[3] = {0, 0, 0};
  } t[2];
  bool bf16 = true, half = true, transpose = false;
  int64_t B = 0, S = 0;
  int D = 0, rot = 0;
  const uint64_t* table = nullptr;
  float amplitude = 1.f;
  const int32_t* positions = nullptr;
  int64_t pos_stride_b = 0, pos0 = 0;
};
// rot/2 entries: the fraction of a turn per position, in units of 2^-64;
// from `freqs` (radians per position) when given, else from the formula.
cudaError_t launch_rotary_table(const Launch& l, int rot, double theta, int scaling, double factor,
                                double orig_len, double low, double high, const double* freqs,
                                uint64_t* table);
// Interleaved pairs need every pair aligned to its two elements.
bool rotary_supported(const RotaryArgs& a);
cudaError_t launch_rotary(const Launch& l, const RotaryArgs& a);

// cache.cu
// A bounded cache: K, V [B, Hkv, T, D] by strides (elements: b, h, slot),
// weights and positions [B, Hkv, T] dense, len / next_pos / counters [B].
struct CacheArgs {
  void *K, *V;
  int64_t kst[3], vst[3];
  float* weights;
  int32_t *positions, *len, *next_pos, *counters;
  bool bf16;
  int B, Hkv, D, budget, n_sink, n_local;
  int64_t T;
};
struct CacheSource {  // rows to compress; weights and positions [B, Hkv, S] dense
  const void *K, *V;
  int64_t kst[3], vst[3];
  const float* weights;
  const int32_t *positions, *len, *next_pos;  // each may be null
  int64_t S;
};
cudaError_t launch_cache_insert(const Launch& l, const CacheArgs& c, const void* k,
                                const int64_t* kst, const void* v, const int64_t* vst);
cudaError_t launch_cache_compress(const Launch& l, const CacheArgs& dst, const CacheSource& s);

// prefix_decode.cu
struct PrefixDecodeArgs {
  bool bf16, out_bf16;
  int B, Hq, Hkv, D, N;
  float scale;
  const void* q;                            // [B, Hq, D]
  const void *Kp, *Vp, *K, *V;
  int64_t kps[3], vps[3], ks[3], vs[3];     // strides: prefix / sequence, head, token
  int64_t Tp, T;
  const int32_t *prefix_len, *group_start, *len, *next_pos;
  void* out;
  float *lse_out, *weights;
  float decay;
  void* workspace;
};
int64_t prefix_decode_workspace_bytes(bool bf16, int B, int Hkv, int G, int D, int N, int64_t Tp,
                                      int64_t T, bool weights, int num_sms);
cudaError_t launch_prefix_decode(const Launch& l, const PrefixDecodeArgs& a, std::string* why);

// decode.cu
int decode_default_parts(bool bf16, int D, int L, int num_sms);
// Merged mode: the last CTA of each unit combines the unit's splits.
struct MergeOut {
  int* counters;   // [B*Hkv], zero on entry, left zero on a normal exit
  void* out;       // [B, Hq, D]
  bool out_bf16;
  float* lse_out;  // [B, Hq] or null
  // bf16 only: full-head units first, then (after the selection kernel that
  // precedes it on the stream completes) the sparse units; the decode is
  // launched with programmatic dependent launch
  bool phased = false;
  // phased: CTAs at the end of the grid that take no full-head work (they
  // start only after the selection's CTAs leave their SMs)
  int late = 0;
  // bf16 hybrid context: gist K/V rows [B, Hkv, C, D] (C = T / L) that every
  // sparse unit attends over next to its selected chunks; null = off.
  // gist_selected: only the gist rows of the unit's selected chunks, else
  // every chunk's gist row
  const void* Kg = nullptr;
  const void* Vg = nullptr;
  bool gist_selected = false;
  // the caller left the number of pieces to the library: steps with few
  // chunks per unit and no full-attention heads may run as one cluster of
  // CTAs per unit (its parts combined in distributed shared memory)
  bool allow_cluster = false;
};
constexpr int kMergedMaxParts = 256;
cudaError_t launch_decode(const Launch& l, const void* q, const void* K, const void* V, bool bf16,
                          const int32_t* idx, const int32_t* count, int kmax,
                          const uint8_t* head_full, int B, int Hq, int Hkv, int D, int64_t T,
                          int L, float scale, int num_parts, int max_splits, float* o_part,
                          float* lse_part, const MergeOut* merge, std::string* why);
cudaError_t launch_merge(const Launch& l, const float* o_part, const float* lse_part, int rows,
                         int max_splits, int D, void* out, bool out_bf16, float* lse_out);

// hostio.cu: bytes / 16 words from src to dst (both 16-byte aligned; src may
// be mapped pinned host memory)
cudaError_t launch_copy16(const Launch& l, const void* src, void* dst, size_t bytes);

// prefill.cu
// skip_empty: units with no chunk write nothing (else their rows get 0).
// dense_k (dense causal mode; idx/count unused): tile t of (b, h) attends
// to chunks 0 .. t when t * 64 < dense_k[b * Hkv + h], else it is empty.
cudaError_t launch_prefill(const Launch& l, const void* Q, const void* K, const void* V,
                           const int32_t* idx, const int32_t* count, int kmax, int B, int S,
                           int Hq, int Hkv, int D, int tile_m, int L, float scale, void* O,
                           std::string* why, bool skip_empty = false,
                           const int32_t* dense_k = nullptr);

// tma_host.cu: 2-D bf16 tensor map over a row-major [rows, cols] matrix with
// `row_stride` elements between rows, box [box_rows, box_cols], 128-byte swizzle.
bool make_tmap_bf16_2d(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                       uint64_t row_stride, uint32_t box_rows, uint32_t box_cols,
                       std::string* why);

// The same over a tensor [n2, n1, rows, cols] with element strides s2, s1 and
// row_stride (any order); box [1, 1, box_rows, box_cols].
bool make_tmap_bf16_4d(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                       uint64_t n1, uint64_t n2, uint64_t row_stride, uint64_t s1, uint64_t s2,
                       uint32_t box_rows, uint32_t box_cols, std::string* why);

// bf16 or fp32 [n1, rows, cols] (n1 = 0: two-dimensional), 128- or 64-byte swizzle.
bool make_tmap_3d(CUtensorMap* map, const void* base, bool f32, uint64_t cols, uint64_t rows,
                  uint64_t n1, uint64_t row_stride, uint64_t s1, uint32_t box_cols,
                  uint32_t box_rows, uint32_t box_n1, int swizzle, std::string* why);

}  // namespace csa
