// Expert routing by scores: softmax or sigmoid over the router logits, a bias
// that steers the choice (not the weights), groups of experts of which the best
// take part, top-k, weights renormalised or not, times a scale; and its gradient.
//
//   p_e = exp(l_e) / sum exp(l)  or  1 / (1 + exp(-l_e))        c_e = p_e + b_e
//   group score = sum of the group's group_top largest c; the topk_groups groups
//   with the largest score take part; slots = the k largest c among their experts,
//   (c descending, index ascending); w_j = scale * p_j / (sum of the selected p)
//
// The choice is exact: without a bias the scores' order is that of the FP32 logits,
// compared as they are; sums p + b and group scores are compared as in FP64 (scores
// 1e-7 apart are then still told apart as the formula tells them; plain FP32 scores
// would swap about one token in three thousand at 384 experts).  They are formed in
// FP32 first: where neighbours in the resulting order lie further apart than FP32 can
// be wrong, the order is certain; only a token with a closer pair (or an exact tie)
// is done again in FP64, by its wave alone.  16384 x 384, sigmoid, bias, 8 groups:
// FP64 throughout 51 us, this form 25 us (5 us of traffic; bound by its instructions,
// about 700 of the vector unit's a token).  64 x 512, softmax: 4.7 us, one launch.
#include "block.h"
#include "common.h"
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
// One DPP step: the value of the lane that CTRL names (quad_perm [1,0,3,2] and [2,3,0,1],
// row_half_mirror, row_mirror: partners 1, 2, 4 and 8 lanes away in a reduction).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ float lane_of(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
// Wave-wide maximum and sum, on every lane: within rows of 16 lanes, then over the rows.
__device__ __forceinline__ float wave_max_f32(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  return fmaxf(fmaxf(lane_of(v, 0), lane_of(v, 16)), fmaxf(lane_of(v, 32), lane_of(v, 48)));
}
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

// Wave-wide maximum of an integer, uniform: rows of 16 lanes, then rows 0 into 1 and 2
// into 3, then 1 into 3 (row_bcast:15 and :31); lane 63 has seen all.
__device__ __forceinline__ int wave_max_i32(int v) {
  constexpr int kLeast = -0x7FFFFFFF - 1;
  v = max(v, dpp<0xB1>(v));
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  v = max(v, dpp<0x140>(v));
  v = max(v, __builtin_amdgcn_update_dpp(kLeast, v, 0x142, 0xA, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(kLeast, v, 0x143, 0xC, 0xF, false));
  return __builtin_amdgcn_readlane(v, 63);
}

// exp(x), x <= 0, within about 1.5 units in the last place: 2^(x log2 e) with the
// product's rounding error put back (the hardware's 2^h is good to one unit).
__device__ __forceinline__ float exp_close(float x) {
  x = fmaxf(x, -200.0f);                                 // (0 from there on; keeps the products finite)
  constexpr float kL = 1.44269502162933349609375f, kLLow = 1.92596299112661746887e-8f;
  const float h = x * kL;
  const float l = fmaf(x, kL, -h) + x * kLLow;
  return __builtin_amdgcn_exp2f(h) * fmaf(l, 0.693147180559945f, 1.0f);
}

// exp(a - b), a <= b, as close: the difference's own rounding error (half a step of it,
// which at a - b = -70 would be 60 steps of the exponential) is put back too.
__device__ __forceinline__ float exp_diff(float a, float b) {
  const float d = a - b, bb = d - a;
  const float err = (a - (d - bb)) - (b + bb);
  const float p = exp_close(d);
  return d > -200.0f ? fmaf(p, err, p) : 0.f;
}

// FP32 values as integers of the same order, and back.
__device__ __forceinline__ int order_of(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float float_of(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7FFFFFFF)); }

// Monotone map of an FP64 value to 64 bits (-0 folded onto +0); finite values map
// above 2^52, so 0 (taken, or not in a selected group) and 1 (masked) lie below.
__device__ __forceinline__ uint64_t ordered_key64(double d) {
  uint64_t u = static_cast<uint64_t>(__double_as_longlong(d));
  if ((u << 1) == 0) u = 0;
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t wave_max_key(uint32_t v) { return wave_max_u32(v); }
__device__ __forceinline__ uint64_t wave_max_key(uint64_t v) {
  const uint32_t hi = wave_max_u32(static_cast<uint32_t>(v >> 32));
  const uint32_t lo = wave_max_u32(static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

struct RouteArgs {
  const float* logits;
  const float* bias;
  int T, E, k, groups, topk_groups, group_top;
  bool sigmoid, renorm;
  float scale;
};

// Where a wave's candidates live: lane l holds experts first + step * i, i < count.
// Without groups 64 experts a row; with groups, span lanes per group hold its members.
struct Place {
  int first, step, count, span;
};
__device__ __forceinline__ Place place(const RouteArgs& a) {
  const int lane = lane_id();
  if (a.groups == 1) return Place{lane, kWave, lane < a.E ? (a.E - lane + kWave - 1) / kWave : 0, kWave};
  int span = 1;
  while (2 * span * a.groups <= kWave) span *= 2;
  const int size = a.E / a.groups, g = lane / span, m = lane & (span - 1);
  return Place{g * size + m, span, g < a.groups && m < size ? (size - m + span - 1) / span : 0, span};
}

// Integer keys (order_of): candidates lie above kOffKey, masked experts and places
// without a candidate at the bottom of the range.
constexpr int kOffKey = -0x7F7F0000;                     // order_of(-3.3895e38), the mask's own value
constexpr int kMaskedKey = -0x7FC00000;
constexpr int kNone = -0x7FFFFFFF - 1;

__device__ __forceinline__ int lane_value(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ double lane_value(double v, int l) { return __shfl(v, l, kWave); }

// Scores as values of the same order, with a place below -inf (a score like others: a bias
// gives it) for an expert that does not take part: whole numbers for FP32; for FP64, whose
// scores come from FP32 biases and lie far from its ends, -inf is moved to kLeast64.
constexpr double kLeast64 = -1e300;
__device__ __forceinline__ int order_key_of(float c) { return order_of(c); }
__device__ __forceinline__ double order_key_of(double c) { return max(c, kLeast64); }
__device__ __forceinline__ double from_order_key(double k) { return k; }
__device__ __forceinline__ float from_order_key(int k) { return float_of(k); }

// Whether the group that this lane's candidates belong to takes part (C float or
// double).  `close`: set where the FP32 scores do not decide it.
template <int R, typename C>
__device__ __forceinline__ bool group_taken(const RouteArgs& a, const Place& pl, const C (&c)[R],
                                            const bool (&on)[R], float tol, bool& close) {
  typedef decltype(order_key_of(C())) Key;
  constexpr Key kOut = sizeof(C) == 4 ? static_cast<Key>(kNone) : static_cast<Key>(-INFINITY);
  const int g = lane_id() / pl.span;
  Key k1 = kOut, k2 = kOut;                              // largest, second largest
  auto merge = [&](Key o1, Key o2) {
    k2 = max(max(k2, o2), min(k1, o1));
    k1 = max(k1, o1);
  };
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const Key x = on[i] ? order_key_of(c[i]) : kOut;
    k2 = max(k2, min(k1, x));
    k1 = max(k1, x);
  }
  if constexpr (sizeof(C) == 4) {
    if (pl.span >= 2) merge(dpp<0xB1>(k1), dpp<0xB1>(k2));
    if (pl.span >= 4) merge(dpp<0x4E>(k1), dpp<0x4E>(k2));
    if (pl.span >= 8) merge(dpp<0x141>(k1), dpp<0x141>(k2));
    if (pl.span >= 16) merge(dpp<0x140>(k1), dpp<0x140>(k2));
    if (pl.span >= 32) merge(__shfl_xor(k1, 16, kWave), __shfl_xor(k2, 16, kWave));
  } else {
    for (int s = 1; s < pl.span; s *= 2) merge(__shfl_xor(k1, s, kWave), __shfl_xor(k2, s, kWave));
  }
  // a group with one expert that takes part scores that expert's c alone; one without any
  // comes after all others
  const bool live = k1 != kOut;
  C gs = from_order_key(k1);
  if (a.group_top > 1 && k2 != kOut) gs += from_order_key(k2);
  gs += static_cast<C>(0);                               // -0 and +0 tie
  // (a sum with kLeast64 in it is -inf)
  if constexpr (sizeof(C) == 8) gs = gs < 0.5 * kLeast64 ? kLeast64 : gs;
  const Key gk = live ? order_key_of(gs) : kOut;
  int rank = 0;
  for (int o = 0; o < a.groups; ++o) {
    const Key ok = lane_value(gk, o * pl.span);
    rank += ok > gk || (ok == gk && o < g) ? 1 : 0;
  }
  const bool taken = g < a.groups && rank < a.topk_groups;
  if constexpr (sizeof(C) == 4) {
    // Every group in has to lie above every group out by more than both can be off: the
    // scores p by less than tol, each c by half a step of itself (p + b is rounded: 2^-24 |c|,
    // however little of it a sum that cancels leaves), the sum by half a step; twice these
    // roundings here.  A c of -inf is exact; a sum past FP32's range has infinite bounds.
    const float c1 = from_order_key(k1), c2 = a.group_top > 1 && k2 != kOut ? from_order_key(k2) : 0.f;
    const float size = fabsf(c1) + fabsf(c2);
    const bool exact = c1 == -INFINITY || c2 == -INFINITY;
    const float err = exact ? 0.f : tol + 2.4e-7f * size;
    const float lo = exact ? -INFINITY : err < INFINITY ? gs - err : -INFINITY;
    const float hi = exact ? -INFINITY : err < INFINITY ? gs + err : INFINITY;
    const float in = -wave_max_f32(taken && live ? -lo : -INFINITY);
    const float out = wave_max_f32(live && !taken ? hi : -INFINITY);
    if (__ballot(live && !taken) && !(in > out)) close = true;
  }
  return taken;
}

// The k largest keys of a wave in order (key descending, expert ascending): lane j < k
// gets slot j's expert.  Key 0: no candidate, 1: masked.
template <int R, typename K>
__device__ __forceinline__ int select_exact(const RouteArgs& a, const Place& pl, K (&key)[R]) {
  const int lane = lane_id();
  int sel = 0;
  for (int r = 0; r < a.k; ++r) {
    K head = key[0];                                     // the lane's largest key and its expert
    int he = pl.first;
#pragma unroll
    for (int i = 1; i < R; ++i) {
      const bool gt = key[i] > head;
      head = gt ? key[i] : head;
      he = gt ? pl.first + pl.step * i : he;
    }
    const K best = wave_max_key(head);
    const uint32_t low = wave_max_u32(head == best ? ~static_cast<uint32_t>(he) : 0u);   // a tie: the lowest expert
    const int e = static_cast<int>(~low);
    sel = lane == r ? e : sel;
#pragma unroll
    for (int i = 0; i < R; ++i) key[i] = pl.first + pl.step * i == e ? static_cast<K>(0) : key[i];
  }
  return sel;
}

// The same from FP32 values (as integer keys) that may be off by `tol`: each key's low
// bits make room for its place i in the lane, the lane's keys are sorted
// (compare-exchanges of one maximum and one minimum), and each round takes the wave's
// largest head and moves that lane's list up.  Returns false where that does not settle
// the order: two neighbours among the first k + 1 within the keys' error, or a masked
// expert among the k.
template <int R>
__device__ __forceinline__ bool select_fast(const RouteArgs& a, const Place& pl, int (&c)[R], float tol,
                                            int& sel) {
  constexpr int kBits = R <= 8 ? 3 : R <= 16 ? 4 : 5;
  constexpr int kLow = (1 << kBits) - 1;
  const int lane = lane_id();
#pragma unroll
  for (int i = 0; i < R; ++i) c[i] = (c[i] & ~kLow) | i;
#pragma unroll
  for (int p = 1; p < R; p *= 2)                         // odd-even merge sort, largest first
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < R; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < R && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const int hi = max(c[i + j], c[i + j + q]), lo = min(c[i + j], c[i + j + q]);
            c[i + j] = hi;
            c[i + j + q] = lo;
          }
  int mine = kNone, from = 0;                            // lane r: the r-th largest key and its lane
  for (int r = 0; r <= a.k; ++r) {
    const int best = wave_max_i32(c[0]);
    const int win = __builtin_ctzll(__ballot(c[0] == best));   // (equal heads: not settled below)
    mine = lane == r ? best : mine;
    from = lane == r ? win : from;
    if (lane == win) {                                   // (as selects of c[j + 1] or c[j] it would be indexed)
#pragma unroll
      for (int j = 0; j + 1 < R; ++j) c[j] = c[j + 1];
      c[R - 1] = kNone;
    }
  }
  sel = __shfl(pl.first, from, kWave) + pl.step * (mine & kLow);
  const int next = __shfl_down(mine, 1, kWave);
  const float fm = float_of(mine), fn = float_of(next);
  // (1e-30: keys of 0 and next to it, where the low bits alone set the order)
  const float err = tol + 1e-30f + (fabsf(fm) + fabsf(fn)) * (static_cast<float>(1 << kBits) * 1.1920929e-7f + 2.4e-7f);
  const bool bad = lane < a.k && (mine < kOffKey || (next >= kOffKey && !(fm - fn >= err)));
  return __ballot(bad) == 0;
}

}  // namespace

// One wave per token, tokens gridDim.x * 4 apart.  kChoice: a bias or groups are given;
// otherwise the order is the logits'.
template <int R, bool kChoice>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(R <= 8 ? 5 : R <= 16 ? 3 : 1))) void route_scored_kernel(RouteArgs a, int32_t* __restrict__ idx,
                                                           float* __restrict__ w, uint32_t okey) {
  const int lane = lane_id(), E = a.E, k = a.k;
  const Place pl = place(a);
  float bias[R];
  if (kChoice && a.bias) {
#pragma unroll
    for (int i = 0; i < R; ++i) bias[i] = i < pl.count ? a.bias[pl.first + pl.step * i] : 0.f;
  }
  // FP32's error of a score: sigmoid below 2.5e-7 (the exponential's argument and result,
  // the reciprocal), softmax below 2.5e-6 (its sum's relative error, |l - max| up to ln E
  // on average); a bound for the two that a comparison takes, and twice that
  const float tol = a.sigmoid ? 1e-6f : 1e-5f;
  const int step = gridDim.x * (blockDim.x / kWave);
  // (wave-uniform, said so: the row's address then lives in scalar registers)
  for (int t0 = blockIdx.x * (blockDim.x / kWave) + __builtin_amdgcn_readfirstlane(wave_id()); t0 < a.T; t0 += step) {
    const int t = permute_item(t0, a.T, okey);
    const float* lrow = a.logits + static_cast<size_t>(t) * E;
    float v[R];
    bool on[R];
    float top = -INFINITY;                               // largest logit that takes part
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float l = i < pl.count ? lrow[pl.first + pl.step * i] : -INFINITY;
      on[i] = takes_part(l);
      v[i] = on[i] ? finite_logit(l) : -INFINITY;
      top = fmaxf(top, v[i]);
    }
    if (!a.sigmoid && (kChoice || !a.renorm)) top = wave_max_f32(top);
    float zsum = 0.f;                                    // softmax's sum, where the weights need it
    if (!a.sigmoid && !a.renorm) {
#pragma unroll
      for (int i = 0; i < R; ++i) zsum += on[i] ? exp_close(v[i] - top) : 0.f;
      zsum = wave_sum_f32(zsum);
    }
    int sel;
    bool close = false, in = true;
    int ck[R];
    if (kChoice) {
      float c[R];
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (a.sigmoid) c[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-v[i]));
        else c[i] = on[i] ? __expf(v[i] - top) : 0.f;
        z += c[i];
      }
      if (!a.sigmoid) {
        z = __builtin_amdgcn_rcpf(wave_sum_f32(z));
#pragma unroll
        for (int i = 0; i < R; ++i) c[i] *= z;
      }
      if (a.bias) {
#pragma unroll
        for (int i = 0; i < R; ++i) c[i] += bias[i];
      }
      if (a.groups > 1) in = group_taken<R>(a, pl, c, on, tol, close);
#pragma unroll
      for (int i = 0; i < R; ++i) ck[i] = order_of(a.bias ? c[i] : v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) ck[i] = order_of(v[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) ck[i] = i >= pl.count || !in ? kNone : on[i] ? ck[i] : kMaskedKey;
    if (close || !select_fast<R>(a, pl, ck, kChoice && a.bias ? tol : 0.f, sel)) {
      // exactly: on the logits, or on scores and sums in FP64.  The logits and the bias
      // are read again (from the caches): held across this rare path they would cost the
      // common one its registers.
      int again = 0;
      asm volatile("" : "+v"(again));
      const float* lr = lrow + again;
      const float* br = a.bias + again;
      float u[R];
      bool part[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float x = i < pl.count ? lr[pl.first + pl.step * i] : -INFINITY;
        part[i] = takes_part(x);
        u[i] = part[i] ? finite_logit(x) : -INFINITY;
      }
      double d[R];
      if (kChoice) {
        double zd = 0.0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          d[i] = 0.0;
          if (part[i]) d[i] = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(u[i])))
                                        : exp(static_cast<double>(u[i]) - static_cast<double>(top));
          zd += d[i];
          __builtin_amdgcn_sched_barrier(0);             // (one exponential's registers at a time)
        }
        if (!a.sigmoid) {
          zd = wave_sum64(zd);
#pragma unroll
          for (int i = 0; i < R; ++i) d[i] /= zd;
        }
        if (a.bias) {
#pragma unroll
          for (int i = 0; i < R; ++i)
            if (i < pl.count) d[i] += static_cast<double>(br[pl.first + pl.step * i]);
        }
        bool none = false;
        in = true;
        if (a.groups > 1) in = group_taken<R>(a, pl, d, part, 0.f, none);
      }
      if (kChoice && a.bias) {
        uint64_t key[R];
#pragma unroll
        for (int i = 0; i < R; ++i)
          key[i] = i >= pl.count || !in ? 0ull : !part[i] ? 1ull : ordered_key64(d[i]);
        sel = select_exact<R>(a, pl, key);
      } else {
        uint32_t key[R];
#pragma unroll
        for (int i = 0; i < R; ++i) key[i] = i >= pl.count || !in ? 0u : !part[i] ? 1u : ordered_key(u[i]);
        sel = select_exact<R>(a, pl, key);
      }
    }
    // weights of the selected, FP32: lane j < k holds slot j
    float l = lane < k ? lrow[sel] : -INFINITY;
    const bool use = takes_part(l);
    l = use ? finite_logit(l) : 0.f;
    float p;
    if (a.renorm) {
      // relative to the largest: sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)), and the
      // first factor over that of the largest does not vanish however low the logits are
      const float m = wave_max_f32(use ? l : -INFINITY);
      if (a.sigmoid) p = exp_diff(fminf(l, 0.f), fminf(m, 0.f)) * __builtin_amdgcn_rcpf(1.0f + exp_close(-fabsf(l)));
      else p = exp_diff(l, m);
      p = use ? p : 0.f;
      const float den = wave_sum_f32(p);                 // (at least 0.5 where any expert takes part)
      p = den > 0.f ? p * __builtin_amdgcn_rcpf(den) : 0.f;
    } else if (a.sigmoid) {
      const float en = exp_close(-fabsf(l));
      p = use ? (l < 0.f ? en : 1.0f) * __builtin_amdgcn_rcpf(1.0f + en) : 0.f;
    } else {
      p = use ? exp_diff(l, top) / zsum : 0.f;
    }
    if (lane < k) {
      idx[static_cast<size_t>(t) * k + lane] = sel;
      w[static_cast<size_t>(t) * k + lane] = a.scale * p;
    }
  }
}

// Gradient of the weights with the selection held fixed: one wave per token.
//   sigmoid, renormalised:  dl_j = scale w'_j (1 - p_j) (dw_j - sum w' dw)
//   sigmoid:                dl_j = scale p_j (1 - p_j) dw_j
//   softmax, renormalised:  dl_j = scale w'_j (dw_j - sum w' dw)
//   softmax:                dl_e = scale p_e (dw_e [selected] - sum p dw)   for every e
// with w' the renormalised scores.  Every logit of the row is written: one pass over the
// row's memory.  8191 x 256, softmax, not renormalised 7.5 us (17 MB; a launch's start and
// end are most of it); 2048 x 384, sigmoid 4.3 us.
template <int R>
__global__ __launch_bounds__(256) void route_scored_backward_kernel(
    RouteArgs a, const int32_t* __restrict__ idx, const float* __restrict__ dw,
    float* __restrict__ dlogits, uint32_t okey) {
  const int t0 = blockIdx.x * (blockDim.x / kWave) + __builtin_amdgcn_readfirstlane(wave_id());
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
    const float en = exp_close(-fabsf(l)), r = 1.0f / (1.0f + en);
    const float q = (l < 0.f ? 1.0f : en) * r;             // 1 - p without cancellation
    if (a.renorm) {                                        // (the forward's weights)
      const float m = wave_max_f32(use ? l : -INFINITY);
      const float x = use ? exp_diff(fminf(l, 0.f), fminf(m, 0.f)) * r : 0.f;
      const float z = wave_sum_f32(x);
      const float p = z > 0.f ? x / z : 0.f;
      val = p * q * (d - wave_sum_f32(p * d));
    } else {
      val = (l < 0.f ? en : 1.0f) * r * q * d;
    }
    val *= a.scale;
  } else if (a.renorm) {
    const float m = wave_max_f32(use ? l : -INFINITY);
    const float x = use ? exp_diff(l, m) : 0.f;
    const float z = wave_sum_f32(x);
    const float p = z > 0.f ? x / z : 0.f;
    val = a.scale * p * (d - wave_sum_f32(p * d));
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
      g[i] = v[i] > -INFINITY ? exp_diff(v[i], top) : 0.f;
      z += g[i];
    }
    z = wave_sum_f32(z);
    const float inv = z > 0.f ? 1.0f / z : 0.f;
    const float p = use ? exp_diff(l, top) * inv : 0.f;
    const float mean = wave_sum_f32(p * d);
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
                               int32_t* idx, float* w, hipStream_t s, int num_cus) {
  const RouteArgs a = route_args(logits, bias, T, p);
  // 8192 waves at most: what a wave sets up once, and its bias, serve several tokens
  const int blocks = (T + kPerBlock - 1) / kPerBlock;
  const dim3 grid(blocks < 8 * num_cus ? blocks : 8 * num_cus), block(kPerBlock * kWave);
  const bool choice = bias != nullptr || p.groups > 1;
  int cand = (p.E + kWave - 1) / kWave;                    // candidates per lane
  if (p.groups > 1) {
    int span = 1;
    while (2 * span * p.groups <= kWave) span *= 2;
    cand = (p.E / p.groups + span - 1) / span;             // (at most 31: 33 groups of 31)
  }
  prof_begin(kRoute, s);
#define ROUTE(R)                                                                              \
  do {                                                                                        \
    if (choice) hipLaunchKernelGGL((route_scored_kernel<R, true>), grid, block, 0, s, a, idx, w, order_key()); \
    else hipLaunchKernelGGL((route_scored_kernel<R, false>), grid, block, 0, s, a, idx, w, order_key());       \
  } while (0)
  if (cand <= 1) ROUTE(1);
  else if (cand <= 2) ROUTE(2);
  else if (cand <= 4) ROUTE(4);
  else if (cand <= 6) ROUTE(6);
  else if (cand <= 8) ROUTE(8);
  else if (cand <= 16) ROUTE(16);
  else ROUTE(32);
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
