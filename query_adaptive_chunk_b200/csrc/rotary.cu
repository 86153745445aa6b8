// Rotary positions for queries and keys: both pair layouts, part of the head,
// scaled frequencies, strided views, and the transposed rotation (the
// gradient).
//
// Pair i (i < rot/2) of a token at position p turns by t = p w_i:
//   y_a = A (x_a cos t - x_b sin t),  y_b = A (x_b cos t + x_a sin t),
// (a, b) = (i, i + rot/2) or (2i, 2i + 1); values past rot are copied.
//
// Angles.  cos and sin only need p w_i modulo one turn, so a frequency is
// held as the 64-bit fraction of a turn per position (w / 2 pi * 2^64) and
// p w_i is one integer product that wraps by itself: the table's own frequency
// turns exactly modulo a turn at any 32-bit position (also a negative one).
// The table is formed in 64-bit floats, off by at most (|ln w| + 8) 2^-53 of w
// (a negative own frequency by 2^-54 turns besides): at p = 2^31 an angle is
// within 2^-22 turns of the formula's, 2^-24.3 measured for theta up to 10^8.  The
// top 32 bits, as a float in [-1, 1) half turns, go to sincospif: no range
// reduction, no 64-bit float.
//
// Bound by HBM: 2 * bytes(q, k).  A thread keeps the sines and cosines of
// its V pairs in registers and runs over the heads (stride J), so a token's
// angles are formed once per J heads' worth of threads; loads are up to 16
// bytes, two heads in flight per thread (four leave too few threads: 173
// against 120 us), the first ones under way while the angles are formed.  32K
// tokens of 40 heads of 128 (bf16, a packed projection's views): 113 us, 5.9
// TB/s, 92% of the copy rate; 115 us a call through Python.
#include <algorithm>

#include "internal.h"

namespace csa {
namespace {

constexpr int kRotThreads = 256;

struct RotTensor {
  const void* x;
  void* y;
  int H;
  int64_t xb, xs, xh, yb, ys, yh;  // strides in elements
};

struct RotParams {
  RotTensor t[2];
  uint32_t tokens, S;
  uint32_t J, nrot, ntail;  // threads per token along the heads; V-wide chunks: rotated, copied
  int rot;
  const uint64_t* table;
  float amp, sgn;
  const int32_t* positions;
  int64_t pos_b;
  int64_t pos0;
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

template <typename T>
__device__ __forceinline__ float to_f(T v) { return static_cast<float>(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V elements as one access; 16 bytes go as uint4 (as a struct of eight the
// compiler takes 10% longer over them).
template <typename VT>
__device__ __forceinline__ VT ld_vec(const void* p) {
  if constexpr (sizeof(VT) == 16) {
    const uint4 x = *static_cast<const uint4*>(p);
    return *reinterpret_cast<const VT*>(&x);
  } else {
    return *static_cast<const VT*>(p);
  }
}
template <typename VT>
__device__ __forceinline__ void st_vec(void* p, const VT& v) {
  if constexpr (sizeof(VT) == 16)
    *static_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&v);
  else
    *static_cast<VT*>(p) = v;
}

// HALF: V pairs from two V-wide accesses rot/2 apart; otherwise V/2 pairs
// from one V-wide access.
constexpr int kRotFlight = 2;  // heads in flight per thread

// BLOCKS: per SM at least.
template <typename T, int V, bool HALF, int BLOCKS>
__global__ void __launch_bounds__(kRotThreads, BLOCKS) rotary_kernel(const RotParams p) {
  constexpr int NP = HALF ? V : V / 2;
  constexpr int U = kRotFlight;
  using VT = Vec<T, V>;
  const uint32_t nchunk = p.nrot + p.ntail;
  const uint32_t id = blockIdx.x * kRotThreads + threadIdx.x;  // B S D <= 2^29: fits 32 bits
  const uint32_t slot = id / nchunk, c = id - slot * nchunk;
  const uint32_t tok = slot / p.J;
  const int j = static_cast<int>(slot - tok * p.J), J = static_cast<int>(p.J);
  if (tok >= p.tokens) return;
  const int64_t b = tok / p.S, s = tok % p.S;
  const bool tail = c >= p.nrot;
  const int e0 = static_cast<int>(tail ? p.rot + (c - p.nrot) * V : c * V);  // first element
  const int far = HALF && !tail ? p.rot / 2 : 0;                              // second access
  VT u[U], w[U];
  // heads j, j + J, .. of tensor k
  auto load = [&](const T* x, int64_t step, int h, int H) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (h + i * J < H) {
        u[i] = ld_vec<VT>(x + i * step);
        if (HALF && far) w[i] = ld_vec<VT>(x + i * step + far);
      }
  };
  auto row = [&](const void* base, int64_t sb, int64_t ss, int64_t sh) {
    return static_cast<const T*>(base) + b * sb + s * ss + j * sh + e0;
  };
  // the first rows are on their way while the angles are formed
  const int k0 = p.t[0].H > j ? 0 : 1;
  {
    const RotTensor& t = p.t[k0];
    load(row(t.x, t.xb, t.xs, t.xh), t.xh * J, j, t.H);
  }
  float cs[NP], sn[NP];
  if (!tail) {
    const int64_t pos = p.positions ? static_cast<int64_t>(p.positions[b * p.pos_b + s]) : p.pos0 + s;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint64_t turn = static_cast<uint64_t>(pos) * __ldg(p.table + c * NP + i);
      const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
      float sv, cv;
      sincospif(half_turns, &sv, &cv);
      cs[i] = cv * p.amp;
      sn[i] = sv * p.amp * p.sgn;
    }
  }
#pragma unroll 1
  for (int k = k0; k < 2; ++k) {
    const RotTensor& t = p.t[k];
    const T* x = row(t.x, t.xb, t.xs, t.xh);
    T* y = const_cast<T*>(row(t.y, t.yb, t.ys, t.yh));
    const int64_t xs = t.xh * J, ys = t.yh * J;
#pragma unroll 1
    for (int h = j; h < t.H; h += U * J, x += U * xs, y += U * ys) {
      if (k != k0 || h != j) load(x, xs, h, t.H);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (h + i * J >= t.H) continue;
        if (!tail) {
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            const float a = to_f(HALF ? u[i].v[n] : u[i].v[2 * n]);
            const float d = to_f(HALF ? w[i].v[n] : u[i].v[2 * n + 1]);
            const T ya = from_f<T>(a * cs[n] - d * sn[n]);
            const T yd = from_f<T>(d * cs[n] + a * sn[n]);
            if (HALF) {
              u[i].v[n] = ya;
              w[i].v[n] = yd;
            } else {
              u[i].v[2 * n] = ya;
              u[i].v[2 * n + 1] = yd;
            }
          }
        }
        st_vec(y + i * ys, u[i]);
        if (HALF && far) st_vec(y + i * ys + far, w[i]);
      }
    }
  }
}

struct TableParams {
  int n, rot, scaling;
  double theta, factor, orig_len, low, high;
  const double* freqs;
  uint64_t* table;
};

__global__ void rotary_table_kernel(const TableParams p) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= p.n) return;
  double w;
  if (p.freqs != nullptr) {
    w = p.freqs[i];
  } else {
    const double e = -2.0 * i / p.rot;
    w = pow(p.theta, e);
    double keep = 1.0;  // share of the unscaled frequency
    switch (p.scaling) {
      case ROT_LINEAR:
        keep = 0.0;
        break;
      case ROT_NTK:
        w = p.rot > 2 ? pow(p.theta * pow(p.factor, p.rot / (p.rot - 2.0)), e) : 1.0;
        break;
      case ROT_TURNS:
        keep = (p.orig_len * w / kTwoPi - p.low) / (p.high - p.low);
        break;
      case ROT_RAMP: {
        const double lt = 2.0 * log(p.theta);
        const double lo = fmax(0.0, floor(p.rot * log(p.orig_len / (p.high * kTwoPi)) / lt));
        const double hi = fmin(p.rot - 1.0, ceil(p.rot * log(p.orig_len / (p.low * kTwoPi)) / lt));
        keep = 1.0 - (i - lo) / fmax(hi - lo, 0.001);
        break;
      }
      default:
        break;
    }
    keep = fmin(1.0, fmax(0.0, keep));
    w = w / p.factor * (1.0 - keep) + w * keep;
  }
  double t = w / kTwoPi;
  t -= floor(t);  // whole turns fall away
  const double f = rint(t * 0x1p64);
  p.table[i] = f >= 0x1p64 ? 0ull : static_cast<uint64_t>(f);
}

template <typename T, int V, int BLOCKS>
cudaError_t launch_blocks(const Launch& l, const RotParams& p, bool half, unsigned grid) {
  if (half) {
    rotary_kernel<T, V, true, BLOCKS><<<grid, kRotThreads, 0, l.stream>>>(p);
  } else {
    // a pair is two neighbours: the one-element width does not occur
    if constexpr (V >= 2) rotary_kernel<T, V, false, BLOCKS><<<grid, kRotThreads, 0, l.stream>>>(p);
  }
  return cudaGetLastError();
}

// Four blocks per SM keep more loads in flight over a long run, three spill
// nothing, which counts in a short one (32K tokens of 40 heads 113 against 121
// us, 8K tokens of 56 heads of 64, 3.4 blocks per SM in all, 32.6 against 30.6).
template <typename T, int V>
cudaError_t launch_v(const Launch& l, const RotParams& p, bool half) {
  const int64_t threads = static_cast<int64_t>(p.tokens) * p.J * (p.nrot + p.ntail);
  const unsigned grid = static_cast<unsigned>((threads + kRotThreads - 1) / kRotThreads);
  return grid > 8u * l.num_sms ? launch_blocks<T, V, 4>(l, p, half, grid)
                               : launch_blocks<T, V, 3>(l, p, half, grid);
}

template <typename T>
cudaError_t launch_t(const Launch& l, const RotParams& p, bool half, int V) {
  switch (V) {
    case 8:
      if constexpr (sizeof(T) == 2) return launch_v<T, 8>(l, p, half);
      return cudaErrorInvalidValue;
    case 4: return launch_v<T, 4>(l, p, half);
    case 2: return launch_v<T, 2>(l, p, half);
    default: return launch_v<T, 1>(l, p, half);
  }
}

}  // namespace

cudaError_t launch_rotary_table(const Launch& l, int rot, double theta, int scaling, double factor,
                                double orig_len, double low, double high, const double* freqs,
                                uint64_t* table) {
  const int n = rot / 2;
  TableParams p{n, rot, scaling, theta, factor, orig_len, low, high, freqs, table};
  rotary_table_kernel<<<(n + 127) / 128, 128, 0, l.stream>>>(p);
  return cudaGetLastError();
}

// The widest access that every row, pair half and stride allows.
static int rotary_width(const RotaryArgs& a) {
  int V = a.bf16 ? 8 : 4;
  auto ok = [&](int64_t n) { return n % V == 0; };
  const int64_t edge = a.half ? a.rot / 2 : a.rot;
  for (; V > 1; V /= 2) {
    bool good = ok(edge) && ok(a.D - a.rot);
    for (int k = 0; k < 2; ++k)
      if (a.t[k].H > 0) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(a.t[k].x) | reinterpret_cast<uintptr_t>(a.t[k].y);
        good = good && at % (static_cast<uintptr_t>(V) * (a.bf16 ? 2 : 4)) == 0;
        for (int i = 0; i < 3; ++i) good = good && ok(a.t[k].xst[i]) && ok(a.t[k].yst[i]);
      }
    if (good) break;
  }
  return V;
}

bool rotary_supported(const RotaryArgs& a) { return a.half || rotary_width(a) >= 2; }

cudaError_t launch_rotary(const Launch& l, const RotaryArgs& a) {
  RotParams p{};
  bool in_place = true;
  int H = 0;
  for (int k = 0; k < 2; ++k) {
    const auto& t = a.t[k];
    p.t[k] = RotTensor{t.x,      t.y,      t.H,      t.xst[0], t.xst[1], t.xst[2],
                       t.yst[0], t.yst[1], t.yst[2]};
    H += t.H;
    if (t.H > 0 && t.x != t.y) in_place = false;
  }
  const int V = rotary_width(a);
  p.tokens = static_cast<uint32_t>(a.B * a.S);
  p.S = static_cast<uint32_t>(a.S);
  p.rot = a.rot;
  p.nrot = a.half ? a.rot / 2 / V : a.rot / V;
  p.ntail = in_place ? 0 : (a.D - a.rot) / V;  // in place, the copied part is there already
  p.table = a.table;
  p.amp = a.amplitude;
  p.sgn = a.transpose ? -1.f : 1.f;
  p.positions = a.positions;
  p.pos_b = a.pos_stride_b;
  p.pos0 = a.pos0;
  // Heads side by side: up to four keep a warp's accesses in long runs, but with
  // eight heads a thread at least to share its angles (16K to 200K tokens of 2 to
  // 6 heads: half the time that four side by side take); more when the tokens
  // alone are too few to fill the SMs.
  const int64_t per_token = p.nrot + p.ntail;
  const int64_t want = 1024ll * l.num_sms;
  const int64_t lanes = p.tokens * per_token;
  p.J = static_cast<uint32_t>(std::min<int64_t>(H, std::max<int64_t>(std::max(1, std::min(4, H / 8)), (want + lanes - 1) / lanes)));
  return a.bf16 ? launch_t<__nv_bfloat16>(l, p, a.half, V) : launch_t<float>(l, p, a.half, V);
}

}  // namespace csa
