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
constexpr int kRowWaves = 4;                              // waves of a workgroup, a row at a time each

inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// exp(x) within two units in the last place: the product x log2(e) in two parts, where the
// hardware's exp2 of the rounded one alone is |x| 2^-25 off.  x <= 0 here.
__device__ __forceinline__ float exp_fine(float x) {
  const float h = x * 1.44269502f;
  const float l = fmaf(x, 1.92596300e-8f, fmaf(x, 1.44269502f, -h));
  return __builtin_amdgcn_exp2f(h) * fmaf(l, 0.693147182f, 1.0f);
}
__device__ __forceinline__ float log_fine(float x) { return __builtin_amdgcn_logf(x) * 0.693147182f; }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, kWave));
  return v;
}

// One row's scores: lane holds experts lane + 64 i in l (masked ones -inf).  p normalised
// scores, q softmax, both 0 where masked; returns lse (0 for a row without experts).
// Sigmoid scores are taken relative to exp(min(largest, 0)), so that they hold their digits
// however low they are.
template <bool SIG, int NV>
__device__ __forceinline__ float row_scores(const float (&l)[NV], float (&p)[NV], float (&q)[NV]) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
  m = wave_max(m);
  if (m == -INFINITY) {
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = q[i] = 0.f;
    return 0.f;
  }
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    q[i] = exp_fine(fmaxf(l[i] - m, -200.f));             // (-200: exp is 0, and so are its parts)
    z += q[i];
  }
  z = wave_sum(z);
  const float rz = 1.0f / z;
#pragma unroll
  for (int i = 0; i < NV; ++i) q[i] *= rz;
  if (SIG) {
    const float t = fminf(m, 0.f);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] = exp_fine(fmaxf(fminf(l[i], 0.f) - t, -200.f)) / (1.0f + exp_fine(fmaxf(-fabsf(l[i]), -200.f)));
      s += p[i];
    }
    s = wave_sum(s);
    const float rs = 1.0f / s;
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] *= rs;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = q[i];
  }
  return m + log_fine(z);
}

template <int NV>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, float (&l)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane_id() + 64 * i;
    l[i] = e < E ? row[e] : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) l[i] = l[i] > kMaskedLogit ? fminf(l[i], FLT_MAX) : -INFINITY;   // (NaN too)
}

}  // namespace

BalanceWs balance_ws_layout(int T, int E, int S) {
  BalanceWs L{};
  const int len = T / S;
  // chunks of a sequence's rows, one workgroup each: as many as fill the GPU, of a row a
  // wave and more
  const int most = S < 1024 ? 1024 / S : 1, want = (len + kRowWaves - 1) / kRowWaves;
  L.chunks = want < most ? want : most;
  if (L.chunks < 1) L.chunks = 1;
  L.rows = (len + L.chunks - 1) / L.chunks;
  const size_t n = static_cast<size_t>(S) * L.chunks;
  size_t o = 0;
  L.probs = o;   o = align256(o + sizeof(float) * n * E);
  L.counts = o;  o = align256(o + sizeof(int) * n * E);
  L.z = o;       o = align256(o + sizeof(float) * n);
  L.tokens = o;  o = align256(o + sizeof(int) * n);
  L.total = o;
  return L;
}

// Workgroup = a chunk of a sequence's rows, a row at a time to each wave; its sums of p, its
// counts, its sum of lse^2 and its tokens go to the workspace, to be joined in chunk order.
template <bool SIG, int NV>
__global__ __launch_bounds__(kRowWaves * kWave) void balance_rows(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
    int E, int k, int len, int chunks, int rows, float* __restrict__ pp, int* __restrict__ pc,
    float* __restrict__ pz, int* __restrict__ pn, uint32_t okey) {
  __shared__ float s_p[kRowWaves][NV * 64];
  __shared__ int s_c[NV * 64];
  __shared__ float s_z[kRowWaves];
  __shared__ int s_n[kRowWaves];
  const int wg = permute_item(blockIdx.x, gridDim.x, okey);
  const int s = wg / chunks, c = wg - s * chunks;
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_id();
  for (int i = tid; i < E; i += blockDim.x) s_c[i] = 0;
  __syncthreads();
  float acc[NV], z = 0.f;
  int n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.f;
  const int r_end = min(len, (c + 1) * rows);
  for (int r = c * rows + wv; r < r_end; r += kRowWaves) {
    const int t = s * len + r;
    if (mask && !mask[t]) continue;
    float l[NV], p[NV], q[NV];
    load_row<NV>(logits + static_cast<size_t>(t) * E, E, l);
    const int e = lane < k ? idx[static_cast<size_t>(t) * k + lane] : -1;
    if (static_cast<unsigned>(e) < static_cast<unsigned>(E)) atomicAdd(&s_c[e], 1);
    const float lse = row_scores<SIG, NV>(l, p, q);
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] += p[i];
    z = fmaf(lse, lse, z);
    ++n;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) s_p[wv][lane + 64 * i] = acc[i];
  if (lane == 0) {
    s_z[wv] = z;
    s_n[wv] = n;
  }
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x) {
    float v = s_p[0][e];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) v += s_p[w][e];
    pp[static_cast<size_t>(wg) * E + e] = v;
    pc[static_cast<size_t>(wg) * E + e] = s_c[e];
  }
  if (tid == 0) {
    float v = s_z[0];
    int m = s_n[0];
    for (int w = 1; w < kRowWaves; ++w) {
      v += s_z[w];
      m += s_n[w];
    }
    pz[wg] = v;
    pn[wg] = m;
  }
}

// Joins a sequence's chunks: workgroup = (sequence, 64 experts), four strips of chunks.
__global__ __launch_bounds__(256) void balance_join(const float* __restrict__ pp, const int* __restrict__ pc,
                                                    const int* __restrict__ pn, int E, int chunks,
                                                    float* __restrict__ probs, int* __restrict__ counts,
                                                    int* __restrict__ tokens) {
  __shared__ double s_p[4][64];
  __shared__ int s_c[4][64];
  __shared__ int s_n[4];
  const int s = blockIdx.x, lane = lane_id(), wv = wave_id(), e = blockIdx.y * 64 + lane;
  double p = 0.0;
  int c = 0, n = 0;
  for (int j = wv; j < chunks; j += 4) {
    const size_t row = static_cast<size_t>(s) * chunks + j;
    if (e < E) {
      p += pp[row * E + e];
      c += pc[row * E + e];
    }
    n += pn[row];
  }
  s_p[wv][lane] = p;
  s_c[wv][lane] = c;
  if (lane == 0) s_n[wv] = n;
  __syncthreads();
  if (wv) return;
  n = s_n[0] + s_n[1] + s_n[2] + s_n[3];
  if (e < E) {
    p = (s_p[0][lane] + s_p[1][lane]) + (s_p[2][lane] + s_p[3][lane]);
    probs[static_cast<size_t>(s) * E + e] = static_cast<float>(p / (n > 0 ? n : 1));
    counts[static_cast<size_t>(s) * E + e] = s_c[0][lane] + s_c[1][lane] + s_c[2][lane] + s_c[3][lane];
  }
  if (blockIdx.y == 0 && lane == 0) tokens[s] = n;
}

// Both losses, in one workgroup: a sequence at a time to each wave.
__global__ __launch_bounds__(1024) void balance_losses(const float* __restrict__ probs,
                                                       const int* __restrict__ counts,
                                                       const int* __restrict__ tokens,
                                                       const float* __restrict__ pz, int E, int S,
                                                       int chunks, float* __restrict__ losses) {
  __shared__ double s_l[16], s_z[16];
  __shared__ long long s_n[16];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_id();
  double loss = 0.0, z = 0.0;
  long long n = 0;
  for (int s = wv; s < S; s += 16) {
    double dot = 0.0;
    long long total = 0;
    for (int e = lane; e < E; e += 64) {
      const int c = counts[static_cast<size_t>(s) * E + e];
      total += c;
      dot += static_cast<double>(c) * probs[static_cast<size_t>(s) * E + e];
    }
    for (int m = 32; m >= 1; m >>= 1) {
      dot += __shfl_xor(dot, m, kWave);
      total += __shfl_xor(total, m, kWave);
    }
    loss += total > 0 ? E * dot / static_cast<double>(total) : 0.0;
    n += tokens[s];
  }
  const size_t parts = static_cast<size_t>(S) * chunks;
  for (size_t i = tid; i < parts; i += 1024) z += pz[i];
  for (int m = 32; m >= 1; m >>= 1) z += __shfl_xor(z, m, kWave);
  if (lane == 0) {
    s_l[wv] = loss;
    s_z[wv] = z;
    s_n[wv] = n;
  }
  __syncthreads();
  if (tid == 0) {
    loss = z = 0.0;
    n = 0;
    for (int w = 0; w < 16; ++w) {
      loss += s_l[w];
      z += s_z[w];
      n += s_n[w];
    }
    losses[0] = static_cast<float>(loss / S);
    losses[1] = static_cast<float>(n > 0 ? z / static_cast<double>(n) : 0.0);
  }
}

// Gradient: workgroup = a chunk of a sequence's rows, a row at a time to each wave; the
// sequence's counts and the sum of tokens are read once.
template <bool SIG, int NV>
__global__ __launch_bounds__(kRowWaves * kWave) void balance_backward_rows(
    const float* __restrict__ logits, const uint8_t* __restrict__ mask, const int* __restrict__ counts,
    const int* __restrict__ tokens, const float* __restrict__ d_losses, const float* d_add, int E, int S,
    int len, int chunks, int rows, float* dlogits, uint32_t okey) {
  const int wg = permute_item(blockIdx.x, gridDim.x, okey);
  const int s = wg / chunks, c = wg - s * chunks;
  const int lane = lane_id(), wv = wave_id();
  float up[NV];
  long long total = 0, n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i, v = e < E ? counts[static_cast<size_t>(s) * E + e] : 0;
    up[i] = static_cast<float>(v);
    total += v;
  }
  for (int i = lane; i < S; i += 64) n += tokens[i];
  for (int m = 32; m >= 1; m >>= 1) {
    total += __shfl_xor(total, m, kWave);
    n += __shfl_xor(n, m, kWave);
  }
  const int ns = tokens[s];
  const float c0 = total > 0 && ns > 0
      ? static_cast<float>(static_cast<double>(d_losses[0]) * E / (static_cast<double>(S) * ns * static_cast<double>(total))) : 0.f;
  const float c1 = n > 0 ? static_cast<float>(2.0 * d_losses[1] / static_cast<double>(n)) : 0.f;
  const int r_end = min(len, (c + 1) * rows);
  for (int r = c * rows + wv; r < r_end; r += kRowWaves) {
    const size_t t = static_cast<size_t>(s) * len + r;
    float d[NV];
    if (mask && !mask[t]) {
#pragma unroll
      for (int i = 0; i < NV; ++i) d[i] = 0.f;
    } else {
      float l[NV], p[NV], q[NV];
      load_row<NV>(logits + t * E, E, l);
      const float lse = row_scores<SIG, NV>(l, p, q);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) dot = fmaf(p[i], up[i], dot);
      dot = wave_sum(dot);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float slope = 1.f;
        if (SIG) {
          const float ea = exp_fine(fmaxf(-fabsf(l[i]), -200.f));
          slope = (l[i] >= 0.f ? ea : 1.f) / (1.f + ea);
        }
        d[i] = fmaf(c0 * p[i] * (up[i] - dot), slope, c1 * lse * q[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E) dlogits[t * E + e] = d[i] + (d_add ? d_add[t * E + e] : 0.f);
    }
  }
}

#define BALANCE_FORMS(F)                                                       \
  do {                                                                         \
    if (E <= 64) F(1);                                                         \
    else if (E <= 128) F(2);                                                   \
    else if (E <= 256) F(4);                                                   \
    else if (E <= 512) F(8);                                                   \
    else F(16);                                                                \
  } while (0)

hipError_t launch_balance_loss(const float* logits, const int32_t* idx, const uint8_t* mask, int T, int E,
                               int k, int S, bool sigmoid, float* losses, int32_t* counts, float* probs,
                               int32_t* tokens, void* ws, hipStream_t s) {
  const BalanceWs L = balance_ws_layout(T, E, S);
  char* b = static_cast<char*>(ws);
  float* pp = reinterpret_cast<float*>(b + L.probs);
  int* pc = reinterpret_cast<int*>(b + L.counts);
  float* pz = reinterpret_cast<float*>(b + L.z);
  int* pn = reinterpret_cast<int*>(b + L.tokens);
  prof_begin(kBalance, s);
#define ROWS(NV)                                                                                        \
  do {                                                                                                  \
    if (sigmoid)                                                                                        \
      hipLaunchKernelGGL((balance_rows<true, NV>), dim3(S * L.chunks), dim3(kRowWaves * kWave), 0, s,   \
                         logits, idx, mask, E, k, T / S, L.chunks, L.rows, pp, pc, pz, pn, order_key()); \
    else                                                                                                \
      hipLaunchKernelGGL((balance_rows<false, NV>), dim3(S * L.chunks), dim3(kRowWaves * kWave), 0, s,  \
                         logits, idx, mask, E, k, T / S, L.chunks, L.rows, pp, pc, pz, pn, order_key()); \
  } while (0)
  BALANCE_FORMS(ROWS);
#undef ROWS
  hipLaunchKernelGGL(balance_join, dim3(S, (E + 63) / 64), dim3(256), 0, s, pp, pc, pn, E, L.chunks, probs,
                     counts, tokens);
  hipLaunchKernelGGL(balance_losses, dim3(1), dim3(1024), 0, s, probs, counts, tokens, pz, E, S, L.chunks, losses);
  prof_end(kBalance, s);
  return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const float* logits, const uint8_t* mask, const int32_t* counts,
                                        const int32_t* tokens, const float* d_losses, const float* d_add,
                                        int T, int E, int S, bool sigmoid, float* dlogits, hipStream_t s) {
  const BalanceWs L = balance_ws_layout(T, E, S);
  prof_begin(kBalanceBackward, s);
#define ROWS(NV)                                                                                        \
  do {                                                                                                  \
    if (sigmoid)                                                                                        \
      hipLaunchKernelGGL((balance_backward_rows<true, NV>), dim3(S * L.chunks), dim3(kRowWaves * kWave), 0, s, \
                         logits, mask, counts, tokens, d_losses, d_add, E, S, T / S, L.chunks, L.rows,  \
                         dlogits, order_key());                                                         \
    else                                                                                                \
      hipLaunchKernelGGL((balance_backward_rows<false, NV>), dim3(S * L.chunks), dim3(kRowWaves * kWave), 0, s, \
                         logits, mask, counts, tokens, d_losses, d_add, E, S, T / S, L.chunks, L.rows,  \
                         dlogits, order_key());                                                         \
  } while (0)
  BALANCE_FORMS(ROWS);
#undef ROWS
  prof_end(kBalanceBackward, s);
  return hipGetLastError();
}

}  // namespace moe
