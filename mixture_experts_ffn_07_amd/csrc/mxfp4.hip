// MXFP4 (E2M1 codes with one E8M0 scale per 32 along K): rows to codes and back, and the
// routed experts' products with MXFP4 weights.
//
//   g, u = W_gate_up[e] x[t]        a = silu(g) u         h = MX codes of a, in x's type
//   out[t] = sum over slots j of w[t,j] W_down[e_j] h[t,j], in slot order, FP32, rounded once
//
// Activations are MXFP8 or MXFP4; a is FP32 and goes into its codes unrounded.  Data flow:
// group_experts (expert-grouped rows, as the other batched forms), the gate/up product with
// SwiGLU and the encoding in its epilogue, the down product, the slot sum.  A pair whose
// expert id lies outside [0, E) has no row: it adds nothing to its token.
#include "block.h"
#include "common.h"
#include "mxfp4.h"
#include "tiles.h"

namespace moe {

namespace {

constexpr int kBM4 = 64;                                 // rows (routed pairs) per M-tile
inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int round_up(int v, int m) { return (v + m - 1) / m * m; }

// silu(g) u on the hardware's reciprocal, one unit in the last place off.
__device__ __forceinline__ float swiglu4(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Largest magnitude of the four lanes of a quad, on each of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  const uint32_t a = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, true);   // [1,0,3,2]
  v = v > a ? v : a;
  const uint32_t b = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xF, 0xF, true);   // [2,3,0,1]
  return v > b ? v : b;
}

}  // namespace

// moe_quantize_mxfp4: four lanes per block of 32, eight BF16 values each.  n pieces of eight.
__global__ __launch_bounds__(256) void quant_mx4_rows(const uint16_t* __restrict__ src, int64_t n,
                                                      uint32_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales, int64_t base, uint32_t okey) {
  const int64_t i = base + static_cast<int64_t>(permute_item(blockIdx.x, gridDim.x, okey)) * 256 + threadIdx.x;
  if (i >= n) return;                                     // (n is a multiple of 4: whole quads)
  const i32x4 v = ld16(src + 8 * i);
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t d = static_cast<uint32_t>(v[j]), lo = d << 16 & 0x7FFF0000u, hi = d & 0x7FFF0000u;
    top = max(top, max(lo, hi));
  }
  const int s = mx4_scale_exp(__uint_as_float(quad_max(top)));
  const float inv = exp2_neg(s);
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t d = static_cast<uint32_t>(v[j]);
    f[2 * j] = bf16_to_f32(d & 0xFFFFu) * inv;
    f[2 * j + 1] = __uint_as_float(d & 0xFFFF0000u) * inv;
  }
  codes[i] = f32x4_to_e2m1x4(f[0], f[1], f[2], f[3]) | f32x4_to_e2m1x4(f[4], f[5], f[6], f[7]) << 16;
  if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(s + 127);
}

// moe_dequantize_mxfp4: eight codes a lane.
__global__ __launch_bounds__(256) void dequant_mx4_rows(const uint32_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales, int64_t n,
                                                        uint16_t* __restrict__ dst, int64_t base,
                                                        uint32_t okey) {
  const int64_t i = base + static_cast<int64_t>(permute_item(blockIdx.x, gridDim.x, okey)) * 256 + threadIdx.x;
  if (i >= n) return;
  const uint32_t c = codes[i], sc = scales[i >> 2];
  const float scale = sc == 0 ? __uint_as_float(0x00400000u)
                    : sc == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(sc << 23);
  i32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t m = c >> (8 * j + 4 * q) & 15u, e = m >> 1 & 3u;
      // magnitude: (m & 1) / 2 below 1, else (2 + (m & 1)) 2^(e - 2)
      const float mag = e == 0 ? 0.5f * (m & 1u) : __uint_as_float((126u + e) << 23 | (m & 1u) << 22);
      f[q] = __uint_as_float(__float_as_uint(mag) | (m & 8u) << 28) * scale;
    }
    o[j] = static_cast<int>(pack_bf16x2(f[0], f[1]));
  }
  st16(dst + 8 * i, o);
}

Mx4Ws mx4_ws_layout(int T, int H, int I, int E, int k, bool a4) {
  Mx4Ws L{};
  const size_t P = static_cast<size_t>(T) * k;
  L.bm = kBM4;
  L.max_tiles = static_cast<int>(E + (P + L.bm - 1) / L.bm);
  size_t o = 0;
  L.n_tiles = o;   o += 256;
  L.counts = o;    o = align256(o + sizeof(int) * E);
  L.offsets = o;   o = align256(o + sizeof(int) * (E + 1));
  L.tiles = o;     o = align256(o + sizeof(int) * 2 * L.max_tiles);
  L.perm = o;      o = align256(o + sizeof(int) * P);
  L.row_of = o;    o = align256(o + sizeof(int) * P);
  L.codes = o;     o = align256(o + P * (a4 ? I / 2 : I));
  L.scales = o;    o = align256(o + P * (I / 32));
  L.y = o;
  if (k > 1) o = align256(o + sizeof(float) * P * H);
  L.total = o;
  return L;
}

enum { kGateUp4 = 0, kDown4 = 1, kDownFused4 = 2 };

// Batched products with a whole-line weight stream: workgroup = (M-tile of BM routed rows,
// NW waves), each wave owning two groups of 16 weight rows (gate_up: 16 neurons' gate and up
// rows; down: 32 output channels).  A chunk is 256 positions of K, 128 bytes of a weight
// row: the wave reads its 32 rows as four loads of 8 rows x 128 contiguous bytes
// (non-temporal), passes them through a wave-private 2 KB LDS tile (16-byte pieces
// XOR-swizzled by row), and reads back two operands of the 16x16x128 MFMA: product j takes
// blocks 2g + j of the chunk's eight in lane group g, so a lane's two scales are neighbours.
// The activations are staged in LDS, 256 bytes of each row a stage (two chunks of MXFP4,
// one of MXFP8) with their scales, double-buffered and shared by the waves; the weights of
// the next two chunks are in flight while one multiplies.  Rows past the tile's end load
// the tile's first row; their columns are computed and discarded.
template <int KIND, int NW, int BM, bool A4>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(BM == 64 ? 4 : 2, 8))) void gemm_mx4s(
    const uint8_t* __restrict__ act, const uint8_t* __restrict__ acts,
    const uint8_t* __restrict__ wt, const uint8_t* __restrict__ wts,
    const int* __restrict__ perm, const int2* __restrict__ tiles, const int* __restrict__ n_tiles,
    const int* __restrict__ counts, const int* __restrict__ offsets, const int* __restrict__ row_of,
    const float* __restrict__ w, int H, int I, int k, int P, uint8_t* __restrict__ hq,
    uint8_t* __restrict__ hs, float* __restrict__ y, uint16_t* __restrict__ out, uint32_t okey) {
  constexpr int NT = NW * 64;
  constexpr bool GU = KIND == kGateUp4;
  constexpr int RPW = GU ? 16 : 32;                       // outputs per wave
  constexpr int G = BM / 16;                              // 16-row groups of the tile
  constexpr int CPS = A4 ? 2 : 1;                         // chunks per stage
  constexpr int SB = 256;                                 // activation bytes of a row per stage
  constexpr int RS = SB + 16;                             // padded LDS row stride
  constexpr int CH = SB / 16;                             // 16-byte pieces of a row per stage
  constexpr int LPT = BM * CH / NT;                       // 16-byte code loads per thread
  constexpr int SS = 8 * CPS;                             // scale bytes of a row per stage
  __shared__ __align__(16) uint8_t xl[2][BM * RS];
  __shared__ __align__(16) uint8_t sl[2][BM * SS];
  __shared__ __align__(16) i32x4 wtl[NW][16 * 8];         // per wave: [16 rows][8 pieces]
  __shared__ float s_amax[GU ? NW : 1][BM];
  const int tid = threadIdx.x;
  // one slot: the down product stores whole output rows, those of pairs without a row are
  // cleared here
  if (GU && out)
    for (int b = blockIdx.x; b < P; b += gridDim.x)
      if (row_of[b] >= P)
        for (int c = tid; c < H / 8; c += NT) st16(out + static_cast<size_t>(b) * H + 8 * c, i32x4{0, 0, 0, 0});
  const int K = GU ? H : I;                               // reduction length
  const int N = GU ? I : H;                               // outputs
  const int RB = K / 2, KB = K / 32, AB = A4 ? K / 2 : K; // bytes of a row: weights, scales, activations
  const int nblk = N / (NW * RPW);
  const int item0 = real_item(blockIdx.x, nblk, *n_tiles);
  if (item0 < 0) return;
  const int item = permute_item(item0, nblk * *n_tiles, okey);
  const int tile = item / nblk, nb_i = item - tile * nblk;
  const int nchunk = K / 256, nstage = (nchunk + CPS - 1) / CPS;
  const int2 te = tiles[tile];
  const int e = te.x, m0 = te.y;
  const int mcount = min(BM, counts[e] - m0);
  const int rbase = offsets[e] + m0;
  const int ng = __builtin_amdgcn_readfirstlane((mcount + 15) / 16);   // 16-row groups that hold rows
  const int ln = tid & 63, col = ln & 15, grp = ln >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nb = nb_i * NW * RPW + wv * RPW;              // the wave's first output
  const int row0 = nb, row1 = GU ? I + nb : nb + 16;
  const size_t wrows = GU ? 2 * static_cast<size_t>(I) : static_cast<size_t>(N);

  // whole-line loads: lane = (row lr of an 8-row group, 16-byte piece lc)
  const int lr = ln >> 3, lc = ln & 7;
  const uint8_t* __restrict__ wb = wt + static_cast<size_t>(e) * wrows * RB;
  const uint8_t* __restrict__ wsb = wts + static_cast<size_t>(e) * wrows * KB;
  uint32_t ow[4];                                         // group 0 rows 0-7, 8-15, group 1 rows 0-7, 8-15
#pragma unroll
  for (int i = 0; i < 4; ++i)
    ow[i] = static_cast<uint32_t>(((i < 2 ? row0 : row1) + 8 * (i & 1) + lr) * RB + lc * 16);
  const uint32_t os0 = static_cast<uint32_t>((row0 + col) * KB), os1 = static_cast<uint32_t>((row1 + col) * KB);
  i32x4* tw = wtl[wv];
  i32x4* wdst = tw + lr * 8 + (lc ^ lr);                  // + 64 for rows 8-15
  const i32x4* asrc = tw + col * 8;
  const int sw = col & 7;

  uint32_t oxl[LPT];
  int lrow[LPT], piece[LPT];
#pragma unroll
  for (int i = 0; i < LPT; ++i) {
    const int c = tid + i * NT, r = c / CH, rr = r < mcount ? r : 0;
    piece[i] = (c % CH) * 16;
    lrow[i] = r * RS + piece[i];
    oxl[i] = static_cast<uint32_t>((GU ? perm[rbase + rr] / k : rbase + rr) * AB);
  }
  const bool sload = tid < BM;
  const int srow = tid < mcount ? tid : 0;
  const uint32_t osx = static_cast<uint32_t>(sload ? (GU ? perm[rbase + srow] / k : rbase + srow) * KB : 0);
  i32x4 xr[LPT], wA[4], wB[4];
  uint2 sr[CPS], sA[2], sB[2];
  // activations of stage st (a row's last stage may hold one chunk: its first one again)
  auto fetch = [&](int st) {
    if (st < nstage) {
#pragma unroll
      for (int i = 0; i < LPT; ++i) {
        const int b = st * SB + piece[i];
        xr[i] = ld16(act + oxl[i] + (b < AB ? b : b - 128));
      }
      if (sload)
#pragma unroll
        for (int c = 0; c < CPS; ++c)
          sr[c] = *reinterpret_cast<const uint2*>(acts + osx + 8 * min(st * CPS + c, nchunk - 1));
    }
  };
  auto publish = [&](int st) {
    if (st < nstage) {
#pragma unroll
      for (int i = 0; i < LPT; ++i) *reinterpret_cast<i32x4*>(&xl[st & 1][lrow[i]]) = xr[i];
      if (sload)
#pragma unroll
        for (int c = 0; c < CPS; ++c) *reinterpret_cast<uint2*>(&sl[st & 1][tid * SS + 8 * c]) = sr[c];
    }
    __syncthreads();
  };
  // weights of chunk c and the scales of the lane's rows (past the end the last chunk again)
  auto request = [&](i32x4 (&W)[4], uint2 (&sc)[2], int c) {
    const uint32_t cc = static_cast<uint32_t>(min(c, nchunk - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) W[i] = ld16_stream(wb + ow[i] + 128 * cc);
    sc[0] = *reinterpret_cast<const uint2*>(wsb + os0 + 8 * cc);
    sc[1] = *reinterpret_cast<const uint2*>(wsb + os1 + 8 * cc);
  };
  fetch(0);
  request(wA, sA, 0);
  request(wB, sB, 1);
  f32x4 acc0[G], acc1[G];
#pragma unroll
  for (int g = 0; g < G; ++g) acc0[g] = acc1[g] = f32x4{0.f, 0.f, 0.f, 0.f};
  publish(0);

  // One chunk: the weights through the wave's LDS tile into operands, the chunk after next
  // on its way into the registers they left, then the products.
  auto chunk = [&](i32x4 (&W)[4], uint2 (&sc)[2], int buf, int cc, int next) {
    i32x4 a[4];
    int sa[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      wdst[0] = W[2 * m];
      wdst[64] = W[2 * m + 1];
      __builtin_amdgcn_wave_barrier();
      a[2 * m] = asrc[(2 * grp) ^ sw];
      a[2 * m + 1] = asrc[(2 * grp + 1) ^ sw];
      __builtin_amdgcn_wave_barrier();
      sa[m] = static_cast<int>((grp < 2 ? sc[m].x : sc[m].y) >> (16 * (grp & 1)));
    }
    request(W, sc, next);
    __builtin_amdgcn_sched_barrier(0);                    // (the compiler would sink the loads behind the products)
    const uint8_t* xcur = &xl[buf][col * RS + (A4 ? cc * 128 + 32 * grp : 64 * (grp >> 1) + 16 * (grp & 1))];
    const uint8_t* scur = &sl[buf][col * SS + cc * 8 + 2 * grp];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g && g >= ng) break;                            // (uniform: the tile has no rows there)
      const uint8_t* p = xcur + 16 * g * RS;
      i32x8 b[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(p + (A4 ? 16 : 32) * j);
        const i32x4 hi = A4 ? i32x4{0, 0, 0, 0} : *reinterpret_cast<const i32x4*>(p + 128 + 32 * j);
        b[j] = cat8(lo, hi);
      }
      const int sx = *reinterpret_cast<const uint16_t*>(scur + 16 * g * SS);
      acc0[g] = mfma_mx4_16<A4, 0>(a[0], b[0], sa[0], sx, acc0[g]);
      acc1[g] = mfma_mx4_16<A4, 0>(a[2], b[0], sa[1], sx, acc1[g]);
      acc0[g] = mfma_mx4_16<A4, 1>(a[1], b[1], sa[0], sx, acc0[g]);
      acc1[g] = mfma_mx4_16<A4, 1>(a[3], b[1], sa[1], sx, acc1[g]);
      // (kept at their place: sunk to the end of the stage they would hold every operand live)
      asm volatile("" : "+v"(acc0[g]), "+v"(acc1[g]));
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (int c = 0; c < nchunk; c += 2) {                   // chunk c in wA, c + 1 in wB
    if (A4) {
      fetch(c / 2 + 1);
      chunk(wA, sA, (c / 2) & 1, 0, c + 2);
      if (c + 1 < nchunk) chunk(wB, sB, (c / 2) & 1, 1, c + 3);
      publish(c / 2 + 1);
    } else {
      fetch(c + 1);
      chunk(wA, sA, 0, 0, c + 2);
      publish(c + 1);
      if (c + 1 < nchunk) {
        fetch(c + 2);
        chunk(wB, sB, 1, 0, c + 3);
        publish(c + 2);
      }
    }
  }
  // lane: outputs row0 + 4grp + i (group 0) and row1 + 4grp + i (group 1) of tile row 16g + col
  if (GU) {
    // SwiGLU into acc0; a row's largest magnitude over the wave's 16 neurons, met in LDS with
    // the other half of the 32-neuron block (wave wv ^ 1), gives the block's scale
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc0[g][i] = swiglu4(acc0[g][i], acc1[g][i]);
        top = fmaxf(top, fabsf(acc0[g][i]));
      }
      top = fmaxf(top, __shfl_xor(top, 16, kWave));
      top = fmaxf(top, __shfl_xor(top, 32, kWave));
      if (grp == 0) s_amax[GU ? wv : 0][16 * g + col] = top;
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int r = 16 * g + col;
      if (r >= mcount) continue;
      const float top = fmaxf(s_amax[GU ? wv : 0][r], s_amax[GU ? wv ^ 1 : 0][r]);
      const int s = A4 ? mx4_scale_exp(top) : mx_scale_exp(top);
      const float inv = exp2_neg(s);
      const f32x4 v = acc0[g];
      const size_t row = static_cast<size_t>(rbase + r);
      if (A4)
        *reinterpret_cast<uint16_t*>(hq + row * (I / 2) + (nb + 4 * grp) / 2) =
            static_cast<uint16_t>(f32x4_to_e2m1x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv));
      else
        *reinterpret_cast<uint32_t*>(hq + row * I + nb + 4 * grp) =
            f32x4_to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      if (grp == 0 && (wv & 1) == 0) hs[row * (I / 32) + nb / 32] = static_cast<uint8_t>(s + 127);
    }
    return;
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int r = 16 * g + col;
    if (r >= mcount) continue;
    if (KIND == kDownFused4) {
      const int t = perm[rbase + r];                      // k = 1: pair id == token
      const float wj = w[t];
      uint16_t* orow = out + static_cast<size_t>(t) * H + nb + 4 * grp;
      *reinterpret_cast<uint2*>(orow) = make_uint2(pack_bf16x2(wj * acc0[g][0], wj * acc0[g][1]),
                                                   pack_bf16x2(wj * acc0[g][2], wj * acc0[g][3]));
      *reinterpret_cast<uint2*>(orow + 16) = make_uint2(pack_bf16x2(wj * acc1[g][0], wj * acc1[g][1]),
                                                        pack_bf16x2(wj * acc1[g][2], wj * acc1[g][3]));
    } else {
      float* yr = y + static_cast<size_t>(rbase + r) * H + nb + 4 * grp;
      *reinterpret_cast<f32x4*>(yr) = acc0[g];            // (read back by the slot sum)
      *reinterpret_cast<f32x4*>(yr + 16) = acc1[g];
    }
  }
}

// The MX rows' launches: grids of fewer than 2^32 threads.
constexpr int64_t kMx4Launch = int64_t(1) << 31;

hipError_t launch_quant_mx4(const uint16_t* src, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                            hipStream_t s) {
  const int64_t n = rows * (K / 8);
  prof_begin(kQuant, s);
  for (int64_t base = 0; base < n; base += kMx4Launch) {
    const int64_t m = n - base < kMx4Launch ? n - base : kMx4Launch;
    hipLaunchKernelGGL(quant_mx4_rows, dim3(static_cast<unsigned>((m + 255) / 256)), dim3(256), 0, s, src, n,
                       reinterpret_cast<uint32_t*>(codes), scales, base, order_key());
  }
  prof_end(kQuant, s);
  return hipGetLastError();
}

hipError_t launch_dequant_mx4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K,
                              uint16_t* dst, hipStream_t s) {
  const int64_t n = rows * (K / 8);
  prof_begin(kQuant, s);
  for (int64_t base = 0; base < n; base += kMx4Launch) {
    const int64_t m = n - base < kMx4Launch ? n - base : kMx4Launch;
    hipLaunchKernelGGL(dequant_mx4_rows, dim3(static_cast<unsigned>((m + 255) / 256)), dim3(256), 0, s,
                       reinterpret_cast<const uint32_t*>(codes), scales, n, dst, base, order_key());
  }
  prof_end(kQuant, s);
  return hipGetLastError();
}

hipError_t launch_experts_mx4(const uint8_t* x, const uint8_t* xs, bool a4, const uint8_t* wgu,
                              const uint8_t* wgus, const uint8_t* wd, const uint8_t* wds,
                              const int32_t* idx, const float* w, int T, int H, int I, int E, int k,
                              uint16_t* out, void* ws, hipStream_t s, int num_cus) {
  const Mx4Ws L = mx4_ws_layout(T, H, I, E, k, a4);
  const int P = T * k;
  char* b = static_cast<char*>(ws);
  int* n_tiles = reinterpret_cast<int*>(b + L.n_tiles);
  int* counts = reinterpret_cast<int*>(b + L.counts);
  int* offsets = reinterpret_cast<int*>(b + L.offsets);
  int2* tiles = reinterpret_cast<int2*>(b + L.tiles);
  int* perm = reinterpret_cast<int*>(b + L.perm);
  int* row_of = reinterpret_cast<int*>(b + L.row_of);
  uint8_t* hq = reinterpret_cast<uint8_t*>(b + L.codes);
  uint8_t* hs = reinterpret_cast<uint8_t*>(b + L.scales);
  float* y = reinterpret_cast<float*>(b + L.y);
  if (const hipError_t e = launch_group_experts(idx, P, E, L.bm, counts, offsets, tiles, n_tiles, perm, row_of, s);
      e != hipSuccess) return e;
#define STREAM4(KD, A, AS, W, WS, Y, O, NBLK)                                                    \
  do {                                                                                           \
    const dim3 grid_(round_up((NBLK) * L.max_tiles, kXcds));                                     \
    if (a4)                                                                                      \
      hipLaunchKernelGGL((gemm_mx4s<KD, 8, kBM4, true>), grid_, dim3(512), 0, s, A, AS, W, WS, perm, tiles, \
                         n_tiles, counts, offsets, row_of, w, H, I, k, P, hq, hs, Y, O, order_key()); \
    else                                                                                         \
      hipLaunchKernelGGL((gemm_mx4s<KD, 8, kBM4, false>), grid_, dim3(512), 0, s, A, AS, W, WS, perm, tiles, \
                         n_tiles, counts, offsets, row_of, w, H, I, k, P, hq, hs, Y, O, order_key()); \
  } while (0)
  prof_begin(kMx4GateUp, s);
  STREAM4(kGateUp4, x, xs, wgu, wgus, nullptr, k == 1 ? out : nullptr, I / 128);
  prof_end(kMx4GateUp, s);
  prof_begin(kMx4Down, s);
  if (k == 1) STREAM4(kDownFused4, hq, hs, wd, wds, nullptr, out, H / 256);
  else STREAM4(kDown4, hq, hs, wd, wds, y, nullptr, H / 256);
#undef STREAM4
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && k > 1) e = launch_combine_slots(y, row_of, w, T, H, k, out, 0, H, H, s, num_cus);
  prof_end(kMx4Down, s);
  return e;
}

}  // namespace moe
