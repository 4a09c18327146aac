// Experts in 8-bit integers: both projections of the routed-expert FFN as INT8
// products, with one FP32 scale per token (activations) and per output channel
// (weights).
//
//   g, u = sx[t] sg[e,n] (x[t] . W[e,n])     a = silu(g) u      sh = max|a| / 127 per pair
//   hq = rint(a 127 / max|a|)                y = sh sd[e,n] (hq . Wd[e,n])
//   out[t] = sum over slots j of w[t,j] y[t,j], in slot order, FP32, rounded once
//
// The dot products are exact in INT32 (v_mfma_i32_16x16x64_i8; 127 * 128 * 16384
// stays below 2^31), so any split of a reduction gives the same bits.  Everything
// after them is FP32: a is not rounded before its codes are taken.
//
// Data flow: group_experts (expert-grouped rows, as the other batched forms), the
// gate/up product with SwiGLU into FP32 a, the rows' codes and scales, the down
// product, and the slot sum.  A pair whose expert id lies outside [0, E) has no
// row: it adds nothing to its token.
#include "common.h"
#include "internal.h"
#include "tiles.h"

namespace moe {

namespace {

constexpr int kBM8 = 64;                           // rows (routed pairs) per M-tile
inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int round_up(int v, int m) { return (v + m - 1) / m * m; }

__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

enum { kGateUp8 = 0, kDown8 = 1, kDownFused8 = 2 };

constexpr int kI8C = 256;                          // K stage of the staged codes (two chunks)
constexpr int kI8RS = kI8C + 16;                   // padded LDS row stride (bytes)
constexpr int kI8CH = kI8C / 16;                   // 16-byte code chunks per row per stage

}  // namespace

Int8Ws int8_ws_layout(int T, int H, int I, int E, int k) {
  Int8Ws L{};
  const size_t P = static_cast<size_t>(T) * k;
  L.bm = kBM8;
  L.max_tiles = static_cast<int>(E + (P + L.bm - 1) / L.bm);
  size_t o = 0;
  L.n_tiles = o;   o += 256;
  L.counts = o;    o = align256(o + sizeof(int) * E);
  L.offsets = o;   o = align256(o + sizeof(int) * (E + 1));
  L.tiles = o;     o = align256(o + sizeof(int) * 2 * L.max_tiles);
  L.perm = o;      o = align256(o + sizeof(int) * P);
  L.row_of = o;    o = align256(o + sizeof(int) * P);
  L.act = o;       o = align256(o + sizeof(float) * P * I);
  L.codes = o;     o = align256(o + P * I);
  L.scales = o;    o = align256(o + sizeof(float) * P);
  L.y = o;
  if (k > 1) o = align256(o + sizeof(float) * P * H);
  L.total = o;
  return L;
}

// Batched INT8 projections with a whole-line weight stream: workgroup = (M-tile of
// 64 routed rows, NW waves), each wave owning two groups of 16 weight rows
// (gate_up: 16 neurons' gate and up rows; down: 32 output channels).  A
// 128-position chunk of a row is 128 bytes: the wave reads its 32 rows as four
// loads of 8 rows x 128 contiguous bytes (non-temporal), passes them through a
// wave-private 2 KB LDS tile (16-byte chunks XOR-swizzled by row) and reads back
// two 16-byte operands of the 16x16x64 MFMA: lane (r, g) takes chunks g and 4 + g
// of row r, of the weights and of the activations alike.  The activation codes
// are staged in LDS in 256-position stages, double-buffered and shared by the
// waves.  Rows past the tile's end load the tile's first row; their columns are
// computed and discarded.
template <int KIND, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(4, 8))) void gemm_i8s(
    const uint8_t* __restrict__ act, const float* __restrict__ acts,
    const uint8_t* __restrict__ wt, const float* __restrict__ wts,
    const int* __restrict__ perm, const int2* __restrict__ tiles, const int* __restrict__ n_tiles,
    const int* __restrict__ counts, const int* __restrict__ offsets, const float* __restrict__ w,
    int H, int I, int k, float* __restrict__ y, uint16_t* __restrict__ out, uint32_t okey) {
  constexpr int NT = NW * 64;
  constexpr bool GU = KIND == kGateUp8;
  constexpr int RPW = GU ? 16 : 32;                       // outputs per wave
  constexpr int LPT = kBM8 * kI8CH / NT;                  // 16-byte code loads per thread
  __shared__ __align__(16) uint8_t xl[2][kBM8 * kI8RS];
  __shared__ __align__(16) i32x4 wtl[NW][16 * 8];         // per wave: [16 rows][8 chunks]
  const int K = GU ? H : I;                               // reduction length
  const int N = GU ? I : H;                               // outputs
  const int nblk = N / (NW * RPW);
  const int item0 = real_item(blockIdx.x, nblk, *n_tiles);
  if (item0 < 0) return;
  const int item = permute_item(item0, nblk * *n_tiles, okey);
  const int tile = item / nblk, nb_i = item - tile * nblk;
  const int2 te = tiles[tile];
  const int e = te.x, m0 = te.y;
  const int mcount = min(kBM8, counts[e] - m0);
  const int rbase = offsets[e] + m0;
  const int tid = threadIdx.x, ln = tid & 63, col = ln & 15, grp = ln >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nb = nb_i * NW * RPW + wv * RPW;              // the wave's first output
  const int row0 = nb, row1 = GU ? I + nb : nb + 16;
  const size_t wrows = GU ? 2 * static_cast<size_t>(I) : static_cast<size_t>(N);

  // whole-line loads: lane = (row lr of an 8-row group, 16-byte chunk lc)
  const int lr = ln >> 3, lc = ln & 7;
  const uint8_t* __restrict__ wb = wt + static_cast<size_t>(e) * wrows * K;
  uint32_t ow[4];                                         // group 0 rows 0-7, 8-15, group 1 rows 0-7, 8-15
#pragma unroll
  for (int i = 0; i < 4; ++i)
    ow[i] = static_cast<uint32_t>(((i < 2 ? row0 : row1) + 8 * (i & 1) + lr) * K + lc * 16);
  i32x4* tw = wtl[wv];
  i32x4* wdst = tw + lr * 8 + (lc ^ lr);                  // + 64 for rows 8-15
  const i32x4* asrc = tw + col * 8;
  const int sw = col & 7;

  uint32_t oxl[LPT];
  int lrow[LPT];
#pragma unroll
  for (int i = 0; i < LPT; ++i) {
    const int c = tid + i * NT, r = c / kI8CH, rr = r < mcount ? r : 0;
    lrow[i] = r * kI8RS + (c % kI8CH) * 16;
    const int arow = GU ? perm[rbase + rr] / k : rbase + rr;
    oxl[i] = static_cast<uint32_t>(arow * K + (c % kI8CH) * 16);
  }
  i32x4 xr[LPT];
#pragma unroll
  for (int i = 0; i < LPT; ++i) xr[i] = ld16(act + oxl[i]);
#pragma unroll
  for (int i = 0; i < LPT; ++i) *reinterpret_cast<i32x4*>(&xl[0][lrow[i]]) = xr[i];

  i32x4 acc0[4], acc1[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) acc0[g] = acc1[g] = i32x4{0, 0, 0, 0};
  const int nchunk = K / 128, nstage = K / kI8C;
  i32x4 wA[4], wB[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) wA[i] = ld16_stream(wb + ow[i]);
  __syncthreads();

  auto chunk = [&](const i32x4 (&W)[4], int buf, int cc) {
    const uint8_t* xcur = &xl[buf][col * kI8RS + cc * 128 + 16 * grp];
#pragma unroll
    for (int m = 0; m < 2; ++m) {                         // row group 0, then 1
      wdst[0] = W[2 * m];
      wdst[64] = W[2 * m + 1];
      __builtin_amdgcn_wave_barrier();
      const i32x4 a0 = asrc[grp ^ sw], a1 = asrc[(4 + grp) ^ sw];
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint8_t* p = xcur + (16 * g) * kI8RS;
        const i32x4 b0 = *reinterpret_cast<const i32x4*>(p), b1 = *reinterpret_cast<const i32x4*>(p + 64);
        if (m == 0) acc0[g] = mfma_i8(a1, b1, mfma_i8(a0, b0, acc0[g]));
        else acc1[g] = mfma_i8(a1, b1, mfma_i8(a0, b0, acc1[g]));
      }
    }
  };
  for (int st = 0; st < nstage; ++st) {
    const int buf = st & 1;
    const bool more = st + 1 < nstage;
    if (more) {
#pragma unroll
      for (int i = 0; i < LPT; ++i) xr[i] = ld16(act + oxl[i] + (st + 1) * kI8C);
    }
    // chunks 2st (weights in wA) and 2st+1 (wB); the chunk after each is loaded
    // first (clamped to the last chunk, a harmless repeat: fixed load count)
    const uint32_t k1 = static_cast<uint32_t>((2 * st + 1) * 128);
    const uint32_t k2 = static_cast<uint32_t>(min(2 * st + 2, nchunk - 1) * 128);
#pragma unroll
    for (int i = 0; i < 4; ++i) wB[i] = ld16_stream(wb + ow[i] + k1);
    chunk(wA, buf, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) wA[i] = ld16_stream(wb + ow[i] + k2);
    chunk(wB, buf, 1);
    if (more) {
#pragma unroll
      for (int i = 0; i < LPT; ++i) *reinterpret_cast<i32x4*>(&xl[buf ^ 1][lrow[i]]) = xr[i];
    }
    __syncthreads();
  }
  // lane: outputs row0 + 4grp + i (group 0) and row1 + 4grp + i (group 1) of tile row 16g + col
  const float* ws_e = wts + static_cast<size_t>(e) * wrows;
  const f32x4 s0 = *reinterpret_cast<const f32x4*>(ws_e + row0 + 4 * grp);
  const f32x4 s1 = *reinterpret_cast<const f32x4*>(ws_e + row1 + 4 * grp);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int r = 16 * g + col;
    if (r >= mcount) continue;
    const int pr = perm[rbase + r];
    const float sx = GU ? acts[pr / k] : acts[rbase + r];
    f32x4 v0, v1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v0[i] = static_cast<float>(acc0[g][i]) * sx * s0[i];
      v1[i] = static_cast<float>(acc1[g][i]) * sx * s1[i];
    }
    if (GU) {
      f32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = swiglu(v0[i], v1[i]);
      st16_stream(y + static_cast<size_t>(rbase + r) * I + nb + 4 * grp, o);
    } else if (KIND == kDownFused8) {
      const float wt_ = w[pr];                            // k = 1: pair id == token
      uint16_t* orow = out + static_cast<size_t>(pr) * H + nb + 4 * grp;
      *reinterpret_cast<uint2*>(orow) =
          make_uint2(pack_bf16x2(wt_ * v0[0], wt_ * v0[1]), pack_bf16x2(wt_ * v0[2], wt_ * v0[3]));
      *reinterpret_cast<uint2*>(orow + 16) =
          make_uint2(pack_bf16x2(wt_ * v1[0], wt_ * v1[1]), pack_bf16x2(wt_ * v1[2], wt_ * v1[3]));
    } else {
      float* yr = y + static_cast<size_t>(rbase + r) * H + nb + 4 * grp;
      st16_stream(yr, v0);
      st16_stream(yr + 16, v1);
    }
  }
}

// Codes and scales of the FP32 activations, one grouped row per workgroup (I a
// multiple of 256, at most 16384).  With k = 1 a pair without a row (expert id out
// of range) gets its output row cleared here, as no down tile will write it.
__global__ __launch_bounds__(256) void quant_act_rows(const float* __restrict__ a,
                                                      const int* __restrict__ offsets, int E,
                                                      const int* __restrict__ row_of, int P, int H,
                                                      int I, uint8_t* __restrict__ codes,
                                                      float* __restrict__ scales,
                                                      uint16_t* __restrict__ out, uint32_t okey) {
  __shared__ float red[4];
  const int b = permute_item(blockIdx.x, P, okey);
  if (out && row_of[b] >= P)
    for (int c = threadIdx.x; c < H / 8; c += blockDim.x)
      st16(out + static_cast<size_t>(b) * H + 8 * c, i32x4{0, 0, 0, 0});
  if (b >= offsets[E]) return;
  const float* row = a + static_cast<size_t>(b) * I;
  float amax = 0.f;
  for (int c = threadIdx.x; c < I / 4; c += blockDim.x) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(row + 4 * c);
    amax = fmaxf(fmaxf(fmaxf(amax, fabsf(v[0])), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m, kWave));
  if (lane_id() == 0) red[wave_id()] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float inv = int8_inverse(amax);
  for (int c = threadIdx.x; c < I / 4; c += blockDim.x) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(row + 4 * c);
    *reinterpret_cast<uint32_t*>(codes + static_cast<size_t>(b) * I + 4 * c) =
        int8_codes4(v[0], v[1], v[2], v[3], inv);
  }
  if (threadIdx.x == 0) scales[b] = int8_scale(amax);
}

hipError_t launch_experts_int8(const int8_t* x, const float* xs, const int8_t* wgu,
                               const float* wgus, const int8_t* wd, const float* wds,
                               const int32_t* idx, const float* w, int T, int H, int I, int E,
                               int k, uint16_t* out, void* ws, hipStream_t s, int num_cus) {
  const Int8Ws L = int8_ws_layout(T, H, I, E, k);
  const int P = T * k;
  char* b = static_cast<char*>(ws);
  int* n_tiles = reinterpret_cast<int*>(b + L.n_tiles);
  int* counts = reinterpret_cast<int*>(b + L.counts);
  int* offsets = reinterpret_cast<int*>(b + L.offsets);
  int2* tiles = reinterpret_cast<int2*>(b + L.tiles);
  int* perm = reinterpret_cast<int*>(b + L.perm);
  int* row_of = reinterpret_cast<int*>(b + L.row_of);
  float* act = reinterpret_cast<float*>(b + L.act);
  uint8_t* codes = reinterpret_cast<uint8_t*>(b + L.codes);
  float* scales = reinterpret_cast<float*>(b + L.scales);
  float* y = reinterpret_cast<float*>(b + L.y);
  if (const hipError_t e = launch_group_experts(idx, P, E, L.bm, counts, offsets, tiles, n_tiles,
                                                perm, row_of, s); e != hipSuccess) return e;
  const uint8_t* x8 = reinterpret_cast<const uint8_t*>(x);
  const uint8_t* wgu8 = reinterpret_cast<const uint8_t*>(wgu);
  const uint8_t* wd8 = reinterpret_cast<const uint8_t*>(wd);
  prof_begin(kInt8GateUp, s);
  hipLaunchKernelGGL((gemm_i8s<kGateUp8, 8>), dim3(round_up((I / 128) * L.max_tiles, kXcds)), dim3(512),
                     0, s, x8, xs, wgu8, wgus, perm, tiles, n_tiles, counts, offsets, nullptr, H, I, k,
                     act, nullptr, order_key());
  prof_end(kInt8GateUp, s);
  hipLaunchKernelGGL(quant_act_rows, dim3(P), dim3(256), 0, s, act, offsets, E, row_of, P, H, I, codes,
                     scales, k == 1 ? out : nullptr, order_key());
  prof_begin(kInt8Down, s);
  const dim3 grid(round_up((H / 256) * L.max_tiles, kXcds));
  if (k == 1)
    hipLaunchKernelGGL((gemm_i8s<kDownFused8, 8>), grid, dim3(512), 0, s, codes, scales, wd8, wds, perm,
                       tiles, n_tiles, counts, offsets, w, H, I, k, nullptr, out, order_key());
  else
    hipLaunchKernelGGL((gemm_i8s<kDown8, 8>), grid, dim3(512), 0, s, codes, scales, wd8, wds, perm,
                       tiles, n_tiles, counts, offsets, w, H, I, k, y, nullptr, order_key());
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && k > 1)
    e = launch_combine_slots(y, row_of, w, T, H, k, out, 0, H, H, s, num_cus);
  prof_end(kInt8Down, s);
  return e;
}

}  // namespace moe
