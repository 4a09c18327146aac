// Expert routing by scores: softmax or sigmoid over the router logits, a bias
// that steers the choice (not the weights), groups of experts of which the best
// take part, top-k, weights renormalised or not, times a scale; and its gradient.
//
//   p_e = exp(l_e) / sum exp(l)  or  1 / (1 + exp(-l_e))        c_e = p_e + b_e
//   group score = sum of the group's group_top largest c; the topk_groups groups
//   with the largest score take part; slots = the k largest c among their experts,
//   (c descending, index ascending); w_j = scale * p_j / (sum of the selected p)
//
// The choice is exact: without a bias the scores' order is that of the FP32
// logits, compared as they are; sums p + b and group scores are formed in FP64
// (two experts 1e-7 apart are then still told apart as the formula tells them;
// FP32 scores would swap about one token in three thousand at 384 experts).
// FP64 vector operations run at the rate of unpacked FP32 ones here.
#include "common.h"
#include "internal.h"
#include "route.h"
#include "tiles.h"

namespace moe {

namespace {

constexpr float kMaskedLogit = -3.3895313892515355e38f;   // BF16's lowest finite value

// A logit that takes part: above the lowest BF16 value (-inf, NaN and the lowest
// finite FP32 value are masks too); +inf counts as the largest finite value.
__device__ __forceinline__ bool takes_part(float l) { return l > kMaskedLogit; }
__device__ __forceinline__ float finite_logit(float l) { return fminf(l, 3.4028234663852886e38f); }

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
  return v;
}
__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, kWave));
  return v;
}

// Monotone map of an FP64 value to 64 bits (-0 folded onto +0); finite values map
// above 2^52, so 0 (taken, or not in a selected group) and 1 (masked) lie below.
__device__ __forceinline__ uint64_t ordered_key64(double d) {
  uint64_t u = static_cast<uint64_t>(__double_as_longlong(d));
  if ((u << 1) == 0) u = 0;
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// The k largest keys of a wave, lane l holding candidates l + 64 i in key[i]:
// returns in lane j < k the index of slot j (key descending, index ascending).
template <int R>
__device__ __forceinline__ int select_topk(uint64_t (&key)[R], int k) {
  const int lane = lane_id();
  int mine = 0;
  for (int r = 0; r < k; ++r) {
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < R; ++i) best = key[i] > best ? key[i] : best;
    const uint32_t hi = wave_max_u32(static_cast<uint32_t>(best >> 32));
    const uint32_t lo = wave_max_u32(static_cast<uint32_t>(best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
    best = (static_cast<uint64_t>(hi) << 32) | lo;
    int sel = 0;
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      const uint64_t b = __ballot(key[i] == best);
      sel = b ? kWave * i + __builtin_ctzll(b) : sel;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) key[i] = (lane + kWave * i == sel) ? 0u : key[i];
    if (lane == r) mine = sel;
  }
  return mine;
}

struct RouteArgs {
  const float* logits;
  const float* bias;
  int T, E, k, groups, topk_groups, group_top;
  bool sigmoid, renorm;
  float scale;
};

}  // namespace

// One wave per token, lane l holding experts l + 64 i.  kChoice: a bias or groups
// are given (FP64 scores); otherwise the order is the logits'.
template <int R, bool kChoice>
__global__ __launch_bounds__(256) void route_scored_kernel(RouteArgs a, int32_t* __restrict__ idx,
                                                           float* __restrict__ w, uint32_t okey) {
  extern __shared__ __align__(16) double lds_c[];        // kChoice with groups: [wave][E]
  const int t0 = blockIdx.x * (blockDim.x / kWave) + wave_id();
  if (t0 >= a.T) return;                                 // (whole waves; no barrier below)
  const int t = permute_item(t0, a.T, okey);
  const int lane = lane_id(), E = a.E, k = a.k;
  const float* lrow = a.logits + static_cast<size_t>(t) * E;
  float v[R];
  bool on[R];
  float top = -INFINITY;                                 // largest logit that takes part
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = lane + kWave * i;
    const float l = e < E ? lrow[e] : -INFINITY;
    on[i] = takes_part(l);
    v[i] = on[i] ? finite_logit(l) : 0.f;
    if (on[i]) top = fmaxf(top, v[i]);
  }
  const bool need_top = !a.sigmoid && (kChoice || !a.renorm);
  if (need_top) top = wave_max_f32(top);
  uint64_t key[R];
  if (!kChoice) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      key[i] = lane + kWave * i >= E ? 0ull
               : on[i] ? (static_cast<uint64_t>(ordered_key(v[i])) << 32) | 2u : 1ull;
  } else {
    double c[R];
    double z = 1.0;
    if (!a.sigmoid) {
      z = 0.0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        c[i] = on[i] ? exp(static_cast<double>(v[i]) - static_cast<double>(top)) : 0.0;
        z += c[i];
      }
      z = wave_sum64(z);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int e = lane + kWave * i;
      c[i] = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(v[i]))) : c[i] / z;
      if (a.bias && on[i]) c[i] += static_cast<double>(a.bias[e]);
    }
    uint64_t taken = ~0ull;                              // bit group * span: the group takes part
    int span = 0, size = E;
    if (a.groups > 1) {
      // span lanes per group: each takes the two largest of its members, then the
      // lanes of a group merge theirs
      double* cw = lds_c + static_cast<size_t>(wave_id()) * E;
      size = E / a.groups;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (lane + kWave * i < E) cw[lane + kWave * i] = on[i] ? c[i] : -INFINITY;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      span = 1;
      while (2 * span * a.groups <= kWave) span *= 2;
      const int g = lane / span, m = lane & (span - 1);
      double b1 = -INFINITY, b2 = -INFINITY;             // largest, second largest
      if (g < a.groups)
        for (int j = m; j < size; j += span) {
          const double x = cw[g * size + j];
          b2 = fmax(b2, fmin(b1, x));
          b1 = fmax(b1, x);
        }
      for (int s = 1; s < span; s *= 2) {
        const double o1 = __shfl_xor(b1, s, kWave), o2 = __shfl_xor(b2, s, kWave);
        b2 = fmax(fmax(b2, o2), fmin(b1, o1));
        b1 = fmax(b1, o1);
      }
      // a group with one expert that takes part scores that expert's c alone
      const double gs = a.group_top > 1 && b2 != -INFINITY ? b1 + b2 : b1;
      const uint64_t gk = ordered_key64(gs);
      int rank = 0;
      for (int o = 0; o < a.groups; ++o) {
        const uint64_t ok = __shfl(gk, o * span, kWave);
        rank += ok > gk || (ok == gk && o < g) ? 1 : 0;
      }
      taken = __ballot(m == 0 && g < a.groups && rank < a.topk_groups);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int e = lane + kWave * i;
      const bool in = e < E && ((taken >> ((e < E ? e / size : 0) * span)) & 1);
      key[i] = !in ? 0ull : !on[i] ? 1ull
               : a.bias ? ordered_key64(c[i])
                        : (static_cast<uint64_t>(ordered_key(v[i])) << 32) | 2u;   // the logits' order
    }
  }
  const int sel = select_topk<R>(key, k);
  // weights of the selected, FP32: lane j < k holds slot j
  float l = lane < k ? lrow[sel] : -INFINITY;
  const bool use = takes_part(l);
  l = use ? finite_logit(l) : 0.f;
  float p;
  if (a.sigmoid) {
    p = use ? 1.0f / (1.0f + expf(-l)) : 0.f;
  } else if (a.renorm) {
    const float m = wave_max_f32(use ? l : -INFINITY);
    p = use ? expf(l - m) : 0.f;
  } else {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) z += on[i] ? expf(v[i] - top) : 0.f;
    z = wave_sum(z);
    p = use ? expf(l - top) / z : 0.f;
  }
  if (a.renorm) {
    const float den = wave_sum(p);
    p = den > 0.f ? p / den : 0.f;
  }
  if (lane < k) {
    idx[static_cast<size_t>(t) * k + lane] = sel;
    w[static_cast<size_t>(t) * k + lane] = a.scale * p;
  }
}

// Gradient of the weights with the selection held fixed: one wave per token.
//   sigmoid, renormalised:  dl_j = scale p_j (1 - p_j) (dw_j - sum w' dw) / sum p
//   sigmoid:                dl_j = scale p_j (1 - p_j) dw_j
//   softmax, renormalised:  dl_j = scale w'_j (dw_j - sum w' dw)
//   softmax:                dl_e = scale p_e (dw_e [selected] - sum p dw)   for every e
// with w' the renormalised scores.  Every logit of the row is written.
template <int R>
__global__ __launch_bounds__(256) void route_scored_backward_kernel(
    RouteArgs a, const int32_t* __restrict__ idx, const float* __restrict__ dw,
    float* __restrict__ dlogits, uint32_t okey) {
  const int t0 = blockIdx.x * (blockDim.x / kWave) + wave_id();
  if (t0 >= a.T) return;
  const int t = permute_item(t0, a.T, okey);
  const int lane = lane_id(), E = a.E, k = a.k;
  const float* lrow = a.logits + static_cast<size_t>(t) * E;
  float* drow = dlogits + static_cast<size_t>(t) * E;
  int e = -1;
  float d = 0.f, l = -INFINITY;
  if (lane < k) {
    e = idx[static_cast<size_t>(t) * k + lane];
    d = dw[static_cast<size_t>(t) * k + lane];
    if (static_cast<unsigned>(e) < static_cast<unsigned>(E)) l = lrow[e];
    else e = -1;
  }
  const bool use = takes_part(l);
  l = use ? finite_logit(l) : 0.f;
  if (!use) d = 0.f;
  float g[R];
#pragma unroll
  for (int i = 0; i < R; ++i) g[i] = 0.f;
  float val;                                             // slot j's own term
  if (a.sigmoid) {
    const float p = use ? 1.0f / (1.0f + expf(-l)) : 0.f;
    const float q = use ? 1.0f / (1.0f + expf(l)) : 0.f;    // 1 - p without cancellation
    if (a.renorm) {
      const float z = wave_sum(p);
      const float mean = wave_sum(p * d) / z;
      val = z > 0.f ? p * q * (d - mean) / z : 0.f;
    } else {
      val = p * q * d;
    }
    val *= a.scale;
  } else if (a.renorm) {
    const float m = wave_max_f32(use ? l : -INFINITY);
    const float x = use ? expf(l - m) : 0.f;
    const float z = wave_sum(x);
    const float p = z > 0.f ? x / z : 0.f;
    val = a.scale * p * (d - wave_sum(p * d));
  } else {
    float v[R], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = lane + kWave * i;
      v[i] = c < E ? lrow[c] : -INFINITY;
      v[i] = takes_part(v[i]) ? finite_logit(v[i]) : -INFINITY;
      top = fmaxf(top, v[i]);
    }
    top = wave_max_f32(top);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      g[i] = v[i] > -INFINITY ? expf(v[i] - top) : 0.f;
      z += g[i];
    }
    z = wave_sum(z);
    const float inv = z > 0.f ? 1.0f / z : 0.f;
    const float p = use ? expf(l - top) * inv : 0.f;
    const float mean = wave_sum(p * d);
#pragma unroll
    for (int i = 0; i < R; ++i) g[i] *= -a.scale * inv * mean;
    val = a.scale * p * d;
  }
  for (int j = 0; j < k; ++j) {
    const int ej = __builtin_amdgcn_readlane(e, j);
    const float vj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(val), j));
#pragma unroll
    for (int i = 0; i < R; ++i) g[i] += lane + kWave * i == ej ? vj : 0.f;
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (lane + kWave * i < E) drow[lane + kWave * i] = g[i];
}

namespace {
constexpr int kPerBlock = 4;                             // tokens (waves) per workgroup
RouteArgs route_args(const float* logits, const float* bias, int T, const ScoredRoute& p) {
  return RouteArgs{logits, bias, T, p.E, p.k, p.groups, p.topk_groups, p.group_top,
                   p.sigmoid, p.renorm, p.scale};
}
}  // namespace

hipError_t launch_route_scored(const float* logits, const float* bias, int T, const ScoredRoute& p,
                               int32_t* idx, float* w, hipStream_t s) {
  const RouteArgs a = route_args(logits, bias, T, p);
  const dim3 grid((T + kPerBlock - 1) / kPerBlock), block(kPerBlock * kWave);
  const bool choice = bias != nullptr || p.groups > 1;
  const size_t lds = p.groups > 1 ? kPerBlock * sizeof(double) * p.E : 0;   // at most 32 KB
  prof_begin(kRoute, s);
#define ROUTE(R)                                                                              \
  do {                                                                                        \
    if (choice) hipLaunchKernelGGL((route_scored_kernel<R, true>), grid, block, lds, s, a, idx, w, order_key()); \
    else hipLaunchKernelGGL((route_scored_kernel<R, false>), grid, block, 0, s, a, idx, w, order_key());         \
  } while (0)
  if (p.E <= 64) ROUTE(1);
  else if (p.E <= 128) ROUTE(2);
  else if (p.E <= 256) ROUTE(4);
  else if (p.E <= 512) ROUTE(8);
  else ROUTE(16);
#undef ROUTE
  prof_end(kRoute, s);
  return hipGetLastError();
}

hipError_t launch_route_scored_backward(const float* logits, const int32_t* idx, const float* dw,
                                        int T, const ScoredRoute& p, float* dlogits, hipStream_t s) {
  const RouteArgs a = route_args(logits, nullptr, T, p);
  const dim3 grid((T + kPerBlock - 1) / kPerBlock), block(kPerBlock * kWave);
  prof_begin(kRouteBackward, s);
#define BWD(R) hipLaunchKernelGGL(route_scored_backward_kernel<R>, grid, block, 0, s, a, idx, dw, dlogits, order_key())
  if (p.E <= 64) BWD(1);
  else if (p.E <= 128) BWD(2);
  else if (p.E <= 256) BWD(4);
  else if (p.E <= 512) BWD(8);
  else BWD(16);
#undef BWD
  prof_end(kRouteBackward, s);
  return hipGetLastError();
}

}  // namespace moe
