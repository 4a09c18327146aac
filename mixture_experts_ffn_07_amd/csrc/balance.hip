// The router's balance loss and z-loss, the tokens of each expert, and their gradient.
//
// T tokens form S sequences of L = T / S; those whose mask byte is 0 take no part.
//   p[t,e]  = softmax over the experts, or sigmoid scores over their sum
//   P[s,e]  = mean of p over the sequence's N_s tokens     c[s,e] = its routed pairs of expert e
//   f[s,e]  = E c[s,e] / sum_m c[s,m]
//   losses  = (1/S) sum_s sum_e f P,   (1/N) sum_t lse_t^2,  lse_t = log sum_e exp(l[t,e])
//   dl[t,e] = d0 / (S N_s) p_e (f_e - sum_m p_m f_m) (1 - sigma_e for sigmoid scores)
//             + d1 2/N lse_t exp(l_e - lse_t)
// Masked logits (as in moe_route_scored) have p = 0 and no gradient.
#include <cfloat>

#include "block.h"
#include "common.h"
#include "tiles.h"

namespace moe {

namespace {

constexpr float kMaskedLogit = -3.3895313892515355e38f;   // BF16's lowest finite value
constexpr int kRowWaves = 8;                              // waves of a workgroup of rows

inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// exp(x), x <= 0, within two units in the last place: the product x log2(e) in two parts, where
// the hardware's exp2 of the rounded one alone is |x| 2^-25 off.  (0 below -200.)
__device__ __forceinline__ float exp_fine(float x) {
  x = fmaxf(x, -200.f);
  const float h = x * 1.44269502f;
  const float l = fmaf(x, 1.92596300e-8f, fmaf(x, 1.44269502f, -h));
  return __builtin_amdgcn_exp2f(h) * fmaf(l, 0.693147182f, 1.0f);
}
__device__ __forceinline__ float log_fine(float x) { return __builtin_amdgcn_logf(x) * 0.693147182f; }

// Reductions of R values at once over the wave, the results uniform: within rows of 16 lanes by
// lane permutations in the vector unit, then over the four rows.
template <int CTRL>
__device__ __forceinline__ float lanes(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_of(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
template <int R, bool MAX>
__device__ __forceinline__ void reduce_rows(float (&v)[R]) {
#define STEP(CTRL)                                                      \
  _Pragma("unroll") for (int j = 0; j < R; ++j) {                       \
    const float o = lanes<CTRL>(v[j]);                                  \
    v[j] = MAX ? fmaxf(v[j], o) : v[j] + o;                             \
  }
  STEP(0xB1) STEP(0x4E) STEP(0x141) STEP(0x140)
#undef STEP
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const float a = lane_of(v[j], 0), b = lane_of(v[j], 16), c = lane_of(v[j], 32), d = lane_of(v[j], 48);
    v[j] = MAX ? fmaxf(fmaxf(a, b), fmaxf(c, d)) : (a + b) + (c + d);
  }
}

// Experts of a lane: pairs of neighbours (V = 2, even E) or single ones, NV in all.
template <int V>
__device__ __forceinline__ int expert_of(int i) {
  return V == 2 ? 128 * (i >> 1) + 2 * lane_id() + (i & 1) : 64 * i + lane_id();
}

// A row's values, `rest` past its end.
template <int V, int NV>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, float rest, float (&l)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; i += V) {
    const int e = expert_of<V>(i);
    if (V == 2) {
      const float2 v = e < E ? *reinterpret_cast<const float2*>(row + e) : make_float2(rest, rest);
      l[i] = v.x;
      l[i + V - 1] = v.y;
    } else {
      l[i] = e < E ? row[e] : rest;
    }
  }
}

// Scores of R rows: p normalised scores, q softmax, both 0 where masked, slope 1 - sigma (sigmoid
// scores), lse (0 for a row without experts).  Sigmoid scores are taken relative to
// exp(min(largest, 0)), so that they hold their digits however low they are.
template <bool SIG, int R, int NV>
__device__ __forceinline__ void row_scores(float (&l)[R][NV], float (&p)[R][NV], float (&q)[R][NV],
                                           float (&slope)[R][SIG ? NV : 1], float (&lse)[R]) {
  float m[R], z[R], s[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
#pragma unroll
    for (int i = 0; i < NV; ++i)                          // (NaN too is masked)
      l[j][i] = l[j][i] > kMaskedLogit ? fminf(l[j][i], FLT_MAX) : -INFINITY;
    m[j] = l[j][0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m[j] = fmaxf(m[j], l[j][i]);
  }
  reduce_rows<R, true>(m);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const float top = m[j] == -INFINITY ? 0.f : m[j];
    z[j] = s[j] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      q[j][i] = exp_fine(l[j][i] - top);
      z[j] += q[j][i];
    }
    if (SIG) {
      const float t = fminf(top, 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float x = l[j][i], ea = exp_fine(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + ea);
        // sigma(x) = exp(min(x, 0)) / (1 + exp(-|x|))
        p[j][i] = (t < 0.f ? exp_fine(fminf(x, 0.f) - t) : x >= 0.f ? 1.f : ea) * r;
        slope[j][SIG ? i : 0] = (x >= 0.f ? ea : 1.f) * r;
        s[j] += p[j][i];
      }
    }
  }
  reduce_rows<R, false>(z);
  if (SIG) reduce_rows<R, false>(s);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const bool any = m[j] != -INFINITY;
    const float rz = any ? 1.0f / z[j] : 0.f, rs = any ? 1.0f / s[j] : 0.f;
    lse[j] = any ? m[j] + log_fine(z[j]) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      q[j][i] *= rz;
      if (SIG) p[j][i] *= rs;
      else p[j][i] = q[j][i];
    }
  }
}

// What 64 experts of a sequence add to the losses.
struct BalanceShare {
  double dot, z;
  long long total, tokens;
};

// Registers of a lane for E experts, and rows that a wave takes at once (more of short ones, to
// pass the latencies of loads and reductions together).
constexpr int rows_at_once(int nv) { return nv <= 4 ? 4 : nv <= 8 ? 2 : 1; }
inline int lane_values(int E) {
  if (E & 1) return E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16;
  return E <= 128 ? 2 : E <= 256 ? 4 : E <= 384 ? 6 : E <= 512 ? 8 : E <= 768 ? 12 : 16;
}

}  // namespace

BalanceWs balance_ws_layout(int T, int E, int S) {
  BalanceWs L{};
  const int len = T / S;
  // chunks of a sequence's rows, one workgroup each, a step of rows each at least: 1024, four workgroups a CU
  // (32768 x 256 in 8 sequences, us of the rows' kernel / of the gradient's: 256 chunks 16.1 / 29, 512 15.6 / 25,
  // 1024 13.6 / 21.7)
  const int step = kRowWaves * rows_at_once(lane_values(E));
  const int most = S < 1024 ? 1024 / S : 1, want = (len + step - 1) / step;
  const int room = want < 1 ? 1 : want < most ? want : most;   // (does not fall as T grows)
  L.rows = (len + room * step - 1) / (room * step) * step;
  if (L.rows < step) L.rows = step;
  L.chunks = (len + L.rows - 1) / L.rows;
  if (L.chunks < 1) L.chunks = 1;
  const size_t n = static_cast<size_t>(S) * room;
  size_t o = 0;
  L.share = o;   o = align256(o + sizeof(BalanceShare) * S * ((E + 63) / 64));
  L.probs = o;   o = align256(o + sizeof(float) * n * E);
  L.counts = o;  o = align256(o + sizeof(int) * n * E);
  L.z = o;       o = align256(o + sizeof(double) * n);
  L.tokens = o;  o = align256(o + sizeof(int) * n);
  L.total = o;
  return L;
}

// Workgroup = a chunk of a sequence's rows, R rows at a time to each wave; its sums of p, its
// counts, its sum of lse^2 and its tokens go to the workspace, to be joined in chunk order.
// 2048 x 384 sigmoid: 5.6 us, the latency of one pass.  32768 x 256 softmax, k 8: 13.3 to 13.9 us for
// 35 MB, 2.6 TB/s: the vector units issue in 69 % of the CUs' busy cycles (556 instructions a wave:
// an exponential, a product and a sum for each score, reductions, the pairs' counters), and the rest
// is the latency of the one step of four rows that a wave has, 47 % of its time.  With one row at a
// time to a wave the calls took 59 and 30 us, now 14 to 16 and 18.5.
template <bool SIG, int V, int NV>
__global__ __launch_bounds__(kRowWaves * kWave) void balance_rows(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
    int E, int k, int len, int chunks, int rows, float* __restrict__ pp, int* __restrict__ pc,
    double* __restrict__ pz, int* __restrict__ pn, uint32_t okey) {
  constexpr int R = rows_at_once(NV);
  __shared__ float s_p[kRowWaves][NV * 64];
  __shared__ int s_c[NV * 64];
  __shared__ double s_z[kRowWaves];
  __shared__ int s_n[kRowWaves];
  const int wg = permute_item(blockIdx.x, gridDim.x, okey);
  const int s = wg / chunks, c = wg - s * chunks;
  const int tid = threadIdx.x, lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(wave_id());
  for (int i = tid; i < NV * 64; i += kRowWaves * kWave) s_c[i] = 0;
  __syncthreads();
  float acc[NV];
  double z = 0.0;                                         // (squares whose sum may pass FP32's range)
  int n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.f;
  const int r_end = min(len, (c + 1) * rows);
  for (int r = c * rows + wv * R; r < r_end; r += kRowWaves * R) {
    float l[R][NV], p[R][NV], q[R][NV], slope[R][SIG ? NV : 1], lse[R];
    bool on[R];
    int e[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const size_t t = static_cast<size_t>(s) * len + min(r + j, len - 1);
      on[j] = r + j < r_end && (!mask || mask[t] != 0);
      load_row<V, NV>(logits + t * E, E, -INFINITY, l[j]);
      e[j] = lane < k ? idx[t * k + lane] : -1;
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (on[j] && static_cast<unsigned>(e[j]) < static_cast<unsigned>(E)) atomicAdd(&s_c[e[j]], 1);
      if (!on[j])
#pragma unroll
        for (int i = 0; i < NV; ++i) l[j][i] = -INFINITY;
    }
    row_scores<SIG, R, NV>(l, p, q, slope, lse);
#pragma unroll
    for (int j = 0; j < R; ++j) {
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] += p[j][i];
      z = fma(static_cast<double>(lse[j]), static_cast<double>(lse[j]), z);
      n += on[j];
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) s_p[wv][expert_of<V>(i)] = acc[i];
  if (lane == 0) {
    s_z[wv] = z;
    s_n[wv] = n;
  }
  __syncthreads();
  for (int e = tid; e < E; e += kRowWaves * kWave) {
    float v = s_p[0][e];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) v += s_p[w][e];
    pp[static_cast<size_t>(wg) * E + e] = v;
    pc[static_cast<size_t>(wg) * E + e] = s_c[e];
  }
  if (tid == 0) {
    double v = s_z[0];
    int m = s_n[0];
    for (int w = 1; w < kRowWaves; ++w) {
      v += s_z[w];
      m += s_n[w];
    }
    pz[wg] = v;
    pn[wg] = m;
  }
}

// Joins the chunks: workgroup = (sequence, 64 experts), sixteen strips of chunks, in FP64, with the
// share of its experts in sum c P and sum c (and the sequence's sum of lse^2 and its tokens).
__global__ __launch_bounds__(1024) void balance_join(const float* __restrict__ pp, const int* __restrict__ pc,
                                                     const double* __restrict__ pz, const int* __restrict__ pn,
                                                     int E, int chunks, BalanceShare* __restrict__ share,
                                                     float* __restrict__ probs, int* __restrict__ counts,
                                                     int* __restrict__ tokens) {
  __shared__ double s_p[16][64], s_z[16];
  __shared__ int s_c[16][64], s_n[16];
  const int lane = lane_id(), wv = wave_id();
  const int blocks = gridDim.y;
  const int s = blockIdx.x, e = blockIdx.y * 64 + lane, ee = min(e, E - 1);
  const size_t row0 = static_cast<size_t>(s) * chunks;
  double p = 0.0, z = 0.0;
  int c = 0, n = 0;
  for (int j = wv * 64 + lane; j < chunks; j += 1024) {
    n += pn[row0 + j];
    z += pz[row0 + j];
  }
  for (int j = wv; j < chunks; j += 16 * 8) {           // eight chunks' loads in flight
    float pv[8];
    int cv[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const size_t at = (row0 + min(j + 16 * u, chunks - 1)) * E + ee;
      pv[u] = pp[at];
      cv[u] = pc[at];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j + 16 * u < chunks) {
        p += pv[u];
        c += cv[u];
      }
  }
  for (int m = 32; m >= 1; m >>= 1) {
    n += __shfl_xor(n, m, kWave);
    z += __shfl_xor(z, m, kWave);
  }
  s_p[wv][lane] = p;
  s_c[wv][lane] = c;
  if (lane == 0) {
    s_n[wv] = n;
    s_z[wv] = z;
  }
  __syncthreads();
  if (wv == 0) {
    p = z = 0.0;
    c = n = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      p += s_p[w][lane];
      c += s_c[w][lane];
      n += s_n[w];
      z += s_z[w];
    }
    const float mean = static_cast<float>(p / (n > 0 ? n : 1));
    if (e < E) {
      probs[static_cast<size_t>(s) * E + e] = mean;
      counts[static_cast<size_t>(s) * E + e] = c;
    }
    double dot = e < E ? static_cast<double>(c) * mean : 0.0;
    long long total = e < E ? c : 0;
    for (int m = 32; m >= 1; m >>= 1) {
      dot += __shfl_xor(dot, m, kWave);
      total += __shfl_xor(total, m, kWave);
    }
    if (lane == 0) {
      if (blockIdx.y == 0) tokens[s] = n;
      share[s * blocks + blockIdx.y] = BalanceShare{dot, z, total, n};
    }
  }
}

// Both losses, from the shares: one workgroup.  (As the end of the join's last workgroup, found by
// a counter, they took 9.2 us together where these two launches take 6.2 to 7.4: its fence writes the caches
// back.)
__global__ __launch_bounds__(256) void balance_losses(const BalanceShare* __restrict__ share, int E, int S,
                                                      int blocks, float* __restrict__ losses) {
  __shared__ double s_l[4], s_z[4];
  __shared__ long long s_t[4];
  const int lane = lane_id(), wv = wave_id(), tid = threadIdx.x;
  double loss = 0.0, z = 0.0;
  long long n = 0;
  for (int s = tid; s < S; s += 256) {                    // a sequence a thread
    double dot = 0.0;
    long long total = 0;
    for (int y = 0; y < blocks; ++y) {
      dot += share[s * blocks + y].dot;
      total += share[s * blocks + y].total;
    }
    z += share[s * blocks].z;
    n += share[s * blocks].tokens;
    loss += total > 0 ? E * dot / static_cast<double>(total) : 0.0;
  }
  for (int m = 32; m >= 1; m >>= 1) {
    loss += __shfl_xor(loss, m, kWave);
    z += __shfl_xor(z, m, kWave);
    n += __shfl_xor(n, m, kWave);
  }
  if (lane == 0) {
    s_l[wv] = loss;
    s_z[wv] = z;
    s_t[wv] = n;
  }
  __syncthreads();
  if (tid == 0) {
    loss = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
    z = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
    n = s_t[0] + s_t[1] + s_t[2] + s_t[3];
    losses[0] = static_cast<float>(loss / S);
    losses[1] = static_cast<float>(n > 0 ? z / static_cast<double>(n) : 0.0);
  }
}

// Gradient: workgroup = a chunk of a sequence's rows, R rows at a time to each wave; the
// sequence's counts and the sum of tokens are read once.  32768 x 256, added to a given gradient:
// 101 MB in 20-22 us, 4.6-5.1 TB/s, bound by memory; 2048 x 384 7.1 us, a launch and one pass.
template <bool SIG, int V, int NV>
__global__ __launch_bounds__(kRowWaves * kWave) void balance_backward_rows(
    const float* __restrict__ logits, const uint8_t* __restrict__ mask, const int* __restrict__ counts,
    const int* __restrict__ tokens, const float* __restrict__ d_losses, const float* d_add, int E, int S,
    int len, int chunks, int rows, float* dlogits, uint32_t okey) {
  constexpr int R = rows_at_once(NV);
  const int wg = permute_item(blockIdx.x, gridDim.x, okey);
  const int s = wg / chunks, c = wg - s * chunks;
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(wave_id());
  // sum p = 1, so a number taken from every count changes nothing: less their mean (over the experts that
  // have any), level counts are exactly 0, and the rounding of up - dot goes by how far they lie apart
  int cnt[NV], live = 0;
  long long total = 0, n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = expert_of<V>(i);
    cnt[i] = e < E ? counts[static_cast<size_t>(s) * E + e] : 0;
    total += cnt[i];
    live += cnt[i] > 0;
  }
  for (int i = lane; i < S; i += 64) n += tokens[i];
  for (int m = 32; m >= 1; m >>= 1) {
    total += __shfl_xor(total, m, kWave);
    n += __shfl_xor(n, m, kWave);
    live += __shfl_xor(live, m, kWave);
  }
  const int mid = live > 0 ? static_cast<int>(static_cast<double>(total) / live) : 0;
  float up[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) up[i] = static_cast<float>(cnt[i] - mid);
  const int ns = tokens[s];
  const float c0 = total > 0 && ns > 0
      ? static_cast<float>(static_cast<double>(d_losses[0]) * E / (static_cast<double>(S) * ns * static_cast<double>(total))) : 0.f;
  const float c1 = n > 0 ? static_cast<float>(2.0 * d_losses[1] / static_cast<double>(n)) : 0.f;
  const int r_end = min(len, (c + 1) * rows);
  for (int r = c * rows + wv * R; r < r_end; r += kRowWaves * R) {
    float l[R][NV], p[R][NV], q[R][NV], slope[R][SIG ? NV : 1], lse[R], add[R][NV], dot[R];
    bool on[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const size_t t = static_cast<size_t>(s) * len + min(r + j, len - 1);
      on[j] = !mask || mask[t] != 0;
      load_row<V, NV>(logits + t * E, E, -INFINITY, l[j]);
      if (d_add) load_row<V, NV>(d_add + t * E, E, 0.f, add[j]);
      else
#pragma unroll
        for (int i = 0; i < NV; ++i) add[j][i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (!on[j])
#pragma unroll
        for (int i = 0; i < NV; ++i) l[j][i] = -INFINITY;
    row_scores<SIG, R, NV>(l, p, q, slope, lse);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      dot[j] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) dot[j] = fmaf(p[j][i], up[i], dot[j]);
    }
    reduce_rows<R, false>(dot);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (r + j >= r_end) break;
      float* row = dlogits + (static_cast<size_t>(s) * len + r + j) * E;
      float d[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float g = c0 * p[j][i] * (up[i] - dot[j]);
        if (SIG) g *= slope[j][SIG ? i : 0];
        // (lse q first: c1 lse may pass the range, and times a q of 0 would be NaN)
        d[i] = fmaf(c1, lse[j] * q[j][i], g) + add[j][i];
      }
#pragma unroll
      for (int i = 0; i < NV; i += V) {
        const int e = expert_of<V>(i);
        if (e >= E) continue;
        if (V == 2) *reinterpret_cast<float2*>(row + e) = make_float2(d[i], d[i + V - 1]);
        else row[e] = d[i];
      }
    }
  }
}

// F(V, NV) for E experts
#define BALANCE_FORMS(F)                                                       \
  do {                                                                         \
    const int nv_ = lane_values(E);                                            \
    if (E & 1) {                                                               \
      if (nv_ == 1) F(1, 1);                                                   \
      else if (nv_ == 2) F(1, 2);                                              \
      else if (nv_ == 4) F(1, 4);                                              \
      else if (nv_ == 8) F(1, 8);                                              \
      else F(1, 16);                                                           \
    } else {                                                                   \
      if (nv_ == 2) F(2, 2);                                                   \
      else if (nv_ == 4) F(2, 4);                                              \
      else if (nv_ == 6) F(2, 6);                                              \
      else if (nv_ == 8) F(2, 8);                                              \
      else if (nv_ == 12) F(2, 12);                                            \
      else F(2, 16);                                                           \
    }                                                                          \
  } while (0)

hipError_t launch_balance_loss(const float* logits, const int32_t* idx, const uint8_t* mask, int T, int E,
                               int k, int S, bool sigmoid, float* losses, int32_t* counts, float* probs,
                               int32_t* tokens, void* ws, hipStream_t s) {
  const BalanceWs L = balance_ws_layout(T, E, S);
  char* b = static_cast<char*>(ws);
  BalanceShare* share = reinterpret_cast<BalanceShare*>(b + L.share);
  float* pp = reinterpret_cast<float*>(b + L.probs);
  int* pc = reinterpret_cast<int*>(b + L.counts);
  double* pz = reinterpret_cast<double*>(b + L.z);
  int* pn = reinterpret_cast<int*>(b + L.tokens);
  prof_begin(kBalance, s);
#define ROWS(V, NV)                                                                                        \
  do {                                                                                                  \
    if (sigmoid)                                                                                        \
      hipLaunchKernelGGL((balance_rows<true, V, NV>), dim3(S * L.chunks), dim3(kRowWaves * kWave), 0, s,   \
                         logits, idx, mask, E, k, T / S, L.chunks, L.rows, pp, pc, pz, pn, order_key()); \
    else                                                                                                \
      hipLaunchKernelGGL((balance_rows<false, V, NV>), dim3(S * L.chunks), dim3(kRowWaves * kWave), 0, s,  \
                         logits, idx, mask, E, k, T / S, L.chunks, L.rows, pp, pc, pz, pn, order_key()); \
  } while (0)
  BALANCE_FORMS(ROWS);
#undef ROWS
  hipLaunchKernelGGL(balance_join, dim3(S, (E + 63) / 64), dim3(1024), 0, s, pp, pc, pz, pn, E, L.chunks, share,
                     probs, counts, tokens);
  hipLaunchKernelGGL(balance_losses, dim3(1), dim3(256), 0, s, share, E, S, (E + 63) / 64, losses);
  prof_end(kBalance, s);
  return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const float* logits, const uint8_t* mask, const int32_t* counts,
                                        const int32_t* tokens, const float* d_losses, const float* d_add,
                                        int T, int E, int S, bool sigmoid, float* dlogits, hipStream_t s) {
  const BalanceWs L = balance_ws_layout(T, E, S);
  prof_begin(kBalanceBackward, s);
#define ROWS(V, NV)                                                                                        \
  do {                                                                                                  \
    if (sigmoid)                                                                                        \
      hipLaunchKernelGGL((balance_backward_rows<true, V, NV>), dim3(S * L.chunks), dim3(kRowWaves * kWave), 0, s, \
                         logits, mask, counts, tokens, d_losses, d_add, E, S, T / S, L.chunks, L.rows,  \
                         dlogits, order_key());                                                         \
    else                                                                                                \
      hipLaunchKernelGGL((balance_backward_rows<false, V, NV>), dim3(S * L.chunks), dim3(kRowWaves * kWave), 0, s, \
                         logits, mask, counts, tokens, d_losses, d_add, E, S, T / S, L.chunks, L.rows,  \
                         dlogits, order_key());                                                         \
  } while (0)
  BALANCE_FORMS(ROWS);
#undef ROWS
  prof_end(kBalanceBackward, s);
  return hipGetLastError();
}

}  // namespace moe
