// Residual sum and root-mean-square norm in front of the experts, with the
// output in the form that they read (BF16, MXFP8, INT8), its backward pass, and
// the INT8 quantization of BF16 rows.
//
//   s = bf16(x + r)     q = 1 / sqrt(mean(s^2) + eps)     y = s q w
//
// s is rounded to BF16 because that is what the residual stream holds; the norm
// is that of the rounded s, so the backward pass, which reads s back, is the
// gradient of exactly what the forward computed.  y is not rounded on its way
// to the 8-bit codes.
#include "block.h"
#include "common.h"
#include "int8.h"
#include "tiles.h"

namespace moe {

namespace {

constexpr int kVec = 8;                            // BF16 values of a 16-byte load

__device__ __forceinline__ void unpack8(i32x4 raw, float (&v)[kVec]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = static_cast<uint32_t>(raw[i]);
    v[2 * i] = __uint_as_float(w << 16);
    v[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
  }
}
__device__ __forceinline__ i32x4 pack8(const float (&v)[kVec]) {
  i32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = static_cast<int>(pack_bf16x2(v[2 * i], v[2 * i + 1]));
  return o;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, kWave));
  return v;
}

// Sum / maximum over the workgroup, the same on every lane: the waves' values in
// wave order (fixed).  `red` holds 16 floats; a second use of the same `red` needs
// another buffer or a barrier in between.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  const int nw = blockDim.x / kWave;
  if (nw == 1) return v;
  if (lane_id() == 0) red[wave_id()] = v;
  __syncthreads();
  float s = red[0];
  for (int i = 1; i < nw; ++i) s += red[i];
  return s;
}
__device__ __forceinline__ float block_max(float v, float* red) {
  v = wave_max(v);
  const int nw = blockDim.x / kWave;
  if (nw == 1) return v;
  if (lane_id() == 0) red[wave_id()] = v;
  __syncthreads();
  float s = red[0];
  for (int i = 1; i < nw; ++i) s = fmaxf(s, red[i]);
  return s;
}

__device__ __forceinline__ uint2 encode_int8(const float (&v)[kVec], float inv) {
  return make_uint2(int8_codes4(v[0], v[1], v[2], v[3], inv), int8_codes4(v[4], v[5], v[6], v[7], inv));
}

}  // namespace

// One row per workgroup of W waves, NV vectors of 8 values to a lane: vector
// v * 64W + tid of the row.  The row stays in registers between its one read and
// its writes, so x, r and the outputs may share memory.  Q: 0 none, 1 MXFP8
// (four lanes hold a block of 32), 2 INT8.  Bound by the memory: 2048 x 7168 with a
// residual and MXFP8 codes 17.3 us (103 MB, 6.0 TB/s), 9001 x 2048 with INT8 codes
// 20.6 us (129 MB, 6.3 TB/s); few rows by the launch: 8 x 4096 3.6 us.
template <int NV, int Q>
__global__ __launch_bounds__(1024) void add_rmsnorm_kernel(
    const uint16_t* x, const uint16_t* r, const uint16_t* __restrict__ w, int T, int H, float eps,
    uint16_t* sum, uint16_t* y, uint8_t* codes, void* scales, uint32_t okey) {
  __shared__ float red[2][16];
  const int t = permute_item(blockIdx.x, T, okey);
  const int64_t row = static_cast<int64_t>(t) * H;
  const int nvec = H / kVec;
  float s[NV][kVec];
  i32x4 xr[NV], rr[NV], wr[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    xr[v] = rr[v] = wr[v] = i32x4{0, 0, 0, 0};
    if (c < nvec) {
      xr[v] = ld16(x + row + c * kVec);
      if (r) rr[v] = ld16(r + row + c * kVec);
      wr[v] = ld16(w + c * kVec);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    unpack8(xr[v], s[v]);
    if (r) {
      float b[kVec];
      unpack8(rr[v], b);
#pragma unroll
      for (int i = 0; i < kVec; ++i) s[v][i] += b[i];
      const i32x4 o = pack8(s[v]);
      if (sum && c < nvec) st16(sum + row + c * kVec, o);
      unpack8(o, s[v]);
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) ss = fmaf(s[v][i], s[v][i], ss);
  }
  ss = block_sum(ss, red[0]);
  const float q = 1.0f / sqrtf(ss / static_cast<float>(H) + eps);
  float amax = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    float g[kVec];
    unpack8(wr[v], g);
#pragma unroll
    for (int i = 0; i < kVec; ++i) s[v][i] = s[v][i] * q * g[i];
    if (y && c < nvec) st16(y + row + c * kVec, pack8(s[v]));
    if (Q == 1) {
      float bm = 0.f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) bm = fmaxf(bm, fabsf(s[v][i]));
      bm = fmaxf(bm, __shfl_xor(bm, 1, kWave));
      bm = fmaxf(bm, __shfl_xor(bm, 2, kWave));
      const int e = mx_scale_exp(bm);
      const float inv = exp2_neg(e);
      if (c < nvec) {
        const uint32_t lo = f32x4_to_e4m3x4(s[v][0] * inv, s[v][1] * inv, s[v][2] * inv, s[v][3] * inv);
        const uint32_t hi = f32x4_to_e4m3x4(s[v][4] * inv, s[v][5] * inv, s[v][6] * inv, s[v][7] * inv);
        *reinterpret_cast<uint2*>(codes + row + c * kVec) = make_uint2(lo, hi);
        if ((c & 3) == 0)
          static_cast<uint8_t*>(scales)[static_cast<int64_t>(t) * (H / 32) + c / 4] = static_cast<uint8_t>(e + 127);
      }
    } else if (Q == 2) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) amax = fmaxf(amax, fabsf(s[v][i]));
    }
  }
  if (Q == 2) {
    amax = block_max(amax, red[1]);
    const float inv = int8_inverse(amax);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = v * blockDim.x + threadIdx.x;
      if (c < nvec) *reinterpret_cast<uint2*>(codes + row + c * kVec) = encode_int8(s[v], inv);
    }
    if (threadIdx.x == 0) static_cast<float*>(scales)[t] = int8_scale(amax);
  }
}

// moe_quantize_int8: one BF16 row per workgroup, the row in registers.
template <int NV>
__global__ __launch_bounds__(1024) void quant_int8_rows(const uint16_t* __restrict__ src,
                                                        int64_t rows, int K,
                                                        uint8_t* __restrict__ codes,
                                                        float* __restrict__ scales, uint32_t okey) {
  __shared__ float red[16];
  const int64_t t = permute_item(blockIdx.x, static_cast<int>(rows), okey);
  const int64_t row = t * K;
  const int nvec = K / kVec;
  float s[NV][kVec];
  float amax = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    i32x4 raw = {0, 0, 0, 0};
    if (c < nvec) raw = ld16(src + row + c * kVec);
    unpack8(raw, s[v]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) amax = fmaxf(amax, fabsf(s[v][i]));
  }
  amax = block_max(amax, red);
  const float inv = int8_inverse(amax);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    if (c < nvec) *reinterpret_cast<uint2*>(codes + row + c * kVec) = encode_int8(s[v], inv);
  }
  if (threadIdx.x == 0) scales[t] = int8_scale(amax);
}

// Backward.  With n = s q (the normed row before the weight),
//   dx = q (w dy - n mean(n w dy)) + ds      dw = sum over rows of n dy
// Workgroup b takes rows b, b + gridDim.x, ...: each lane keeps its columns' share of
// dw in registers and writes it once, into row b of `partial`; norm_dweight adds the
// gridDim.x rows in a fixed order.  The next row is on its way while one is worked on,
// and the two sums of a row share one barrier: 2048 x 7168 with ds 45 -> 23.4 us (117 MB,
// 5.0 TB/s), then norm_dweight 4.0 us.  333 x 6144: 8.2 + 3.2 us, and the second launch.
template <int NV>
__global__ __launch_bounds__(1024) void add_rmsnorm_backward_kernel(
    const uint16_t* s, const uint16_t* __restrict__ w, const uint16_t* dy, const uint16_t* ds,
    int T, int H, float eps, uint16_t* dx, float* __restrict__ partial, uint32_t okey) {
  __shared__ float2 red[2][16];                    // [row parity][wave]
  const int nvec = H / kVec;
  float acc[NV][kVec];
  i32x4 wr[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    wr[v] = i32x4{0, 0, 0, 0};
    if (c < nvec) wr[v] = ld16(w + c * kVec);
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[v][i] = 0.f;
  }
  const int b = permute_item(blockIdx.x, gridDim.x, okey);
  i32x4 sr[NV], dr[NV], er[NV];
  auto fetch = [&](int t) {
    const int64_t row = static_cast<int64_t>(t) * H;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = v * blockDim.x + threadIdx.x;
      sr[v] = dr[v] = er[v] = i32x4{0, 0, 0, 0};
      if (c < nvec) {
        sr[v] = ld16(s + row + c * kVec);
        dr[v] = ld16(dy + row + c * kVec);
        if (ds) er[v] = ld16(ds + row + c * kVec);
      }
    }
  };
  if (b < T) fetch(b);
  int par = 0;
  for (int t = b; t < T; t += gridDim.x, par ^= 1) {
    i32x4 s0[NV], d0[NV], e0[NV];
    float2 sum = {0.f, 0.f};                       // sum s^2, sum s w dy
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      s0[v] = sr[v];
      d0[v] = dr[v];
      e0[v] = er[v];
    }
    // a later row of this workgroup: dx written in place does not reach it
    if (t + static_cast<int>(gridDim.x) < T) fetch(t + gridDim.x);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float a[kVec], d[kVec], g[kVec];
      unpack8(s0[v], a);
      unpack8(d0[v], d);
      unpack8(wr[v], g);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        sum.x = fmaf(a[i], a[i], sum.x);
        sum.y = fmaf(a[i], g[i] * d[i], sum.y);
      }
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
      sum.x += __shfl_xor(sum.x, m, kWave);
      sum.y += __shfl_xor(sum.y, m, kWave);
    }
    const int nw = blockDim.x / kWave;
    if (nw > 1) {
      if (lane_id() == 0) red[par][wave_id()] = sum;
      __syncthreads();
      sum = red[par][0];
      for (int i = 1; i < nw; ++i) {
        sum.x += red[par][i].x;
        sum.y += red[par][i].y;
      }
    }
    const float q = 1.0f / sqrtf(sum.x / static_cast<float>(H) + eps);
    const float m = sum.y * q / static_cast<float>(H);   // mean(n w dy)
    const int64_t row = static_cast<int64_t>(t) * H;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = v * blockDim.x + threadIdx.x;
      float a[kVec], d[kVec], g[kVec], e[kVec];
      unpack8(s0[v], a);
      unpack8(d0[v], d);
      unpack8(wr[v], g);
      unpack8(e0[v], e);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float n = a[i] * q;
        acc[v][i] = fmaf(n, d[i], acc[v][i]);
        e[i] = fmaf(q, fmaf(-n, m, g[i] * d[i]), e[i]);
      }
      if (c < nvec) st16(dx + row + c * kVec, pack8(e));
    }
  }
  const int64_t prow = static_cast<int64_t>(b) * H;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = v * blockDim.x + threadIdx.x;
    if (c < nvec) {
      *reinterpret_cast<f32x4*>(partial + prow + c * kVec) = f32x4{acc[v][0], acc[v][1], acc[v][2], acc[v][3]};
      *reinterpret_cast<f32x4*>(partial + prow + c * kVec + 4) = f32x4{acc[v][4], acc[v][5], acc[v][6], acc[v][7]};
    }
  }
}

// dweight[c] = bf16(sum of `rows` partial rows): 32 columns per workgroup, thread (row
// lane i, four columns) adding rows i, i + 32, ... in order, eight of them in flight,
// then the 32 row lanes' sums in order.
__global__ __launch_bounds__(256) void norm_dweight(const float* __restrict__ partial, int rows,
                                                    int H, uint16_t* __restrict__ dweight) {
  __shared__ f32x4 red[32][8];
  const int quad = threadIdx.x & 7, i0 = threadIdx.x >> 3;
  const float* p = partial + blockIdx.x * 32 + quad * 4;
  f32x4 a = {0.f, 0.f, 0.f, 0.f};
  for (int i = i0; i < rows; i += 32 * 8) {
    f32x4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      v[u] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (i + 32 * u < rows) v[u] = *reinterpret_cast<const f32x4*>(p + static_cast<int64_t>(i + 32 * u) * H);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) a += v[u];
  }
  red[i0][quad] = a;
  __syncthreads();
  if (threadIdx.x < 32) {
    const float* r = reinterpret_cast<const float*>(&red[0][0]) + threadIdx.x;
    float s = r[0];
    for (int i = 1; i < 32; ++i) s += r[32 * i];
    dweight[blockIdx.x * 32 + threadIdx.x] = static_cast<uint16_t>(f32_to_bf16_rne(s));
  }
}

namespace {

// Waves per row and vectors per lane for rows of `nvec` vectors.  `wide`: as many
// lanes as the row has vectors (few rows: the row's latency is what counts).
struct RowShape {
  int nv, threads;
};
RowShape row_shape(int nvec, bool wide) {
  RowShape r;
  r.nv = wide ? 1 : 2;
  while (r.nv < 8 && nvec > r.nv * 1024) r.nv *= 2;
  const int waves = (nvec + r.nv * kWave - 1) / (r.nv * kWave);
  r.threads = waves * kWave;
  return r;
}

}  // namespace

hipError_t launch_add_rmsnorm(const uint16_t* x, const uint16_t* r, const uint16_t* w, int T, int H,
                              float eps, uint16_t* sum, uint16_t* y, int qtype, uint8_t* codes,
                              void* scales, hipStream_t s, int num_cus) {
  const RowShape rs = row_shape(H / kVec, T <= 2 * num_cus);
  prof_begin(kNorm, s);
#define NORM(NV, Q)                                                                         \
  hipLaunchKernelGGL((add_rmsnorm_kernel<NV, Q>), dim3(T), dim3(rs.threads), 0, s, x, r, w, \
                     T, H, eps, sum, y, codes, scales, order_key())
#define NORM_Q(Q) do { if (rs.nv == 1) NORM(1, Q); else NORM(2, Q); } while (0)
  if (qtype == 1) NORM_Q(1);
  else if (qtype == 2) NORM_Q(2);
  else NORM_Q(0);
#undef NORM_Q
#undef NORM
  prof_end(kNorm, s);
  return hipGetLastError();
}

hipError_t launch_quant_int8(const uint16_t* src, int64_t rows, int K, uint8_t* codes, float* scales,
                             hipStream_t s, int num_cus) {
  const RowShape rs = row_shape(K / kVec, rows <= 2 * num_cus);
  prof_begin(kQuant, s);
  for (int64_t r0 = 0; r0 < rows; r0 += kMaxRows - 1) {   // (one launch but for millions of rows)
    const int64_t n = rows - r0 < kMaxRows - 1 ? rows - r0 : kMaxRows - 1;
    const dim3 grid(static_cast<unsigned>(n)), block(rs.threads);
    if (rs.nv == 1)
      hipLaunchKernelGGL(quant_int8_rows<1>, grid, block, 0, s, src + r0 * K, n, K, codes + r0 * K,
                         scales + r0, order_key());
    else
      hipLaunchKernelGGL(quant_int8_rows<2>, grid, block, 0, s, src + r0 * K, n, K, codes + r0 * K,
                         scales + r0, order_key());
  }
  prof_end(kQuant, s);
  return hipGetLastError();
}

// Workgroups of the backward pass: as many as fill 256 CUs with 16 waves each, 1024 at
// most (every workgroup writes a row of partial weight gradients).  Measured, us (256 /
// 512 / 1024 workgroups): 2048 x 7168 25.9 / 31.0 / 36.1; 8192 x 4096 49.6 / 46.6 / 51.3;
// 16384 x 2048 71.6 / 50.0 / 46.5; 16000 x 512 49.2 / 31.4 / 22.0.
int norm_backward_rows(int T, int H) {
  const int waves = row_shape(H / kVec, true).threads / kWave;
  const int grid = waves > 8 ? 256 : waves > 4 ? 512 : 1024;
  return T < grid ? T : grid;
}

hipError_t launch_add_rmsnorm_backward(const uint16_t* sum, const uint16_t* w, const uint16_t* dy,
                                       const uint16_t* ds, int T, int H, float eps, uint16_t* dx,
                                       uint16_t* dweight, float* partial, hipStream_t s) {
  const RowShape rs = row_shape(H / kVec, true);
  const int rows = norm_backward_rows(T, H);
  prof_begin(kNormBackward, s);
  if (rows > 0) {
    if (rs.nv == 1)
      hipLaunchKernelGGL(add_rmsnorm_backward_kernel<1>, dim3(rows), dim3(rs.threads), 0, s, sum, w, dy,
                         ds, T, H, eps, dx, partial, order_key());
    else
      hipLaunchKernelGGL(add_rmsnorm_backward_kernel<2>, dim3(rows), dim3(rs.threads), 0, s, sum, w, dy,
                         ds, T, H, eps, dx, partial, order_key());
  }
  hipLaunchKernelGGL(norm_dweight, dim3(H / 32), dim3(256), 0, s, partial, rows, H,
                     dweight);
  prof_end(kNormBackward, s);
  return hipGetLastError();
}

}  // namespace moe
