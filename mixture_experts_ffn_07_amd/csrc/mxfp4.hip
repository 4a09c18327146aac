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
#include <type_traits>

#include "block.h"
#include "common.h"
#include "gemm_large.h"
#include "mxfp4.h"
#include "tiles.h"

namespace moe {

namespace {

constexpr int kShort4 = 32, kTall4 = 96;                 // rows (routed pairs) per M-tile of the streaming form
inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int round_up(int v, int m) { return (v + m - 1) / m * m; }

// silu(g) u on the hardware's exponential and reciprocal, one unit in the last place each; the
// exponential's argument is rounded before it, which moves it by about |g| 2^-24 of it.  A code of a
// keeps 2^-2 or 2^-4 of it, so this shows only next to the border of two codes.
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

// One slot (k = 1): the output rows of pairs without a row, which no tile of the down product
// stores, are cleared: by the whole grid, a row a wave, 64 pairs looked at together.
__device__ __forceinline__ void clear_rows(uint16_t* __restrict__ out, const int* __restrict__ row_of, int P, int H) {
  const int lane = lane_id(), waves = gridDim.x * (blockDim.x / kWave);
  for (int b0 = (blockIdx.x * (blockDim.x / kWave) + wave_id()) * kWave; b0 < P; b0 += waves * kWave) {
    uint64_t none = __ballot(b0 + lane < P && row_of[b0 + lane] >= P);
    while (none) {
      const int b = b0 + __builtin_ctzll(none);
      none &= none - 1;
      for (int c = lane; c < H / 8; c += kWave) st16(out + static_cast<size_t>(b) * H + 8 * c, i32x4{0, 0, 0, 0});
    }
  }
}

}  // namespace

// moe_quantize_mxfp4: four lanes per block of 32, eight BF16 values each, so that a wave reads
// 1 KB and writes 256 bytes of codes in one piece; the block's scale from the largest of the four
// lanes.  n pieces of eight.  Bound by memory: 16384 x 4096 in 29.7 us, 5.7 TB/s (6.1 from 900 MB on).
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

// moe_dequantize_mxfp4: eight codes a lane.  Bound by memory, above all by its stores, which are
// streaming ones (451 MB, 43520 x 4096: plain 110 us, streaming 88, 5.1 TB/s; 16384 x 4096 41 and 26;
// streaming loads of the codes take the gain back, 105).
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
  st16_stream(dst + 8 * i, o);
}

Mx4Ws mx4_ws_layout(int T, int H, int I, int E, int k, bool a4) {
  Mx4Ws L{};
  const size_t P = static_cast<size_t>(T) * k;
  // 256-row tiles where the products are bound by the matrix cores and LDS: from 192 rows an
  // expert, where an expert's rows times H I reach 3 G (long reductions or many rows, against a
  // tile's start and end and the scales' transposition), with tiles of gate/up for half of the CUs.
  // Measured, us (256-row / 96-row tiles, MXFP4; MXFP8):
  //   H 4096 I 14336 E 8 k 2: 128 rows an expert 298 / 323; 372 / 376, 192 rows 315 / 428; 414 / 486
  //   H 7168 I 2048 E 32 k 4: 192 rows (2.8 G) 393 / 396; 489 / 443, 256 rows 431 / 498; 540 / 563, 512 rows 746 / 853;
  //     924 / 974
  //   H 7168 I 2048 E 6 k 1, MXFP8: 171 rows 116 / 101, 320 rows (112 tiles) 150 / 148
  //   H 2048 I 5632 E 8 k 2: 256 rows MXFP8 154 / 132, 512 rows 187 / 176; 229 / 210
  //   H 4096 I 1024 E 64 k 6: 256 rows MXFP8 429 / 375, 384 rows 477 / 471; 557 / 533, 1536 rows 1555 / 1659
  //   H 4096 I 1024 E 16 k 4: 512 rows 198 / 161, 1024 rows 296 / 287; 342 / 329, 2048 rows 556 / 564; 642 / 651
  //   H 2048 I 768 E 64 k 8: 1024 rows 545 / 522; 620 / 587, 2048 rows 1007 / 1013; 1155 / 1146
  //   H 2048 I 1024 k 4: E 16, 1024 rows 197 / 156; 219 / 181, E 64, 2048 rows 1140 / 1161; 1328 / 1357
  // 96-row tiles from 18 rows an expert, below it 32-row ones (32 / 96):
  //   H 4096 I 1024 E 64 k 6: 19 rows 115 / 103; 121 / 108, 73 rows 265 / 164; 284 / 179
  //   H 2048 I 768 E 128 k 8: 4 rows 65 / 68; 66 / 70, 16 rows 82 / 79; 86 / 84
  //   H 4096 I 14336 E 8 k 2, MXFP8: 16 rows 169 / 184, 32 rows 264 / 195
  //   H 7168 I 2048, MXFP8: E 32 k 4, 6 rows 151 / 156, 12 rows 174 / 163, 19 rows 193 / 167; E 6 k 1, 21 rows
  //     51 / 56
  // (The 32-row figures with MXFP8 activations are from before its gate/up sums were exact: now 2 to 4 % more.
  // 64-row ones lie within 8 % of the better of the two, on both sides, from 16 to 75 rows; 128-row ones leave
  // registers for half as many weight rows a wave: E 64, 73 rows 171; 188, E 16, 1024 rows 179; 215.)
  const bool large = P >= 192 * static_cast<size_t>(E) && P * H * I >= (size_t(3) << 30) * E &&
                     P / kLargeBM * (I / 128) >= 128;
  L.bm = large ? kLargeBM : P >= 18 * static_cast<size_t>(E) ? kTall4 : kShort4;
  L.max_tiles = static_cast<int>(E + (P + L.bm - 1) / L.bm);
  const size_t tile_room = E + (P + kShort4 - 1) / kShort4;     // (as many as any smaller T takes)
  size_t o = 0;
  L.n_tiles = o;   o += 256;
  L.counts = o;    o = align256(o + sizeof(int) * E);
  L.offsets = o;   o = align256(o + sizeof(int) * (E + 1));
  L.tiles = o;     o = align256(o + sizeof(int) * 2 * tile_room);
  L.perm = o;      o = align256(o + sizeof(int) * P);
  L.row_of = o;    o = align256(o + sizeof(int) * P);
  const size_t past = kLargeBM;                            // rows behind the last that a tile may read
  L.codes = o;     o = align256(o + (P + past) * (a4 ? I / 2 : I));
  L.scales = o;    o = align256(o + P * (I / 32) + past * 8);
  L.y = o;
  if (k > 1) o = align256(o + sizeof(float) * P * H);
  L.partial = L.wgu_t = L.wd_t = L.x_t = o;
  if (L.bm == kLargeBM) {
    o = align256(o + sizeof(float) * kLargeMaxSlices * kLargeBM * 256);
    L.wgu_t = o;   o = align256(o + static_cast<size_t>(E) * 2 * I * (H / 32));
    L.wd_t = o;    o = align256(o + static_cast<size_t>(E) * H * (I / 32));
    L.x_t = o;     o = align256(o + P * (H / 32) + past * 8);
  }
  L.total = o;
  return L;
}

enum { kGateUp4 = 0, kDown4 = 1, kDownFused4 = 2 };

// Batched products with a whole-line weight stream: workgroup = (M-tile of BM routed rows,
// 4 waves), each wave owning 2 R groups of 16 weight rows (gate_up: 16 R neurons' gate and up
// rows; down: 32 R output channels).  A chunk is 256 positions of K, 128 bytes of a weight
// row: the wave reads a group as two loads of 8 rows x 128 contiguous bytes
// (non-temporal, KEEP: plain), passes them through a wave-private 2 KB LDS tile (16-byte pieces
// XOR-swizzled by row), and reads back two operands of the 16x16x128 MFMA: product j takes
// blocks 2g + j of the chunk's eight in lane group g, so a lane's two scales are neighbours.
// The activations are staged in LDS, 256 bytes of each row a stage (two chunks of MXFP4,
// one of MXFP8) with their scales, double-buffered and shared by the waves; the next
// chunk's weights and the next stage's activations are in flight while one multiplies, and
// the CU's other workgroups cover what that does not.  Rows past the tile's end load the
// tile's first row; their columns are computed and discarded.
//
// 32-row tiles are bound by the weights' bytes: R = 1, 100-106 registers (gate/up with E4M3
// activations 126), four workgroups a CU (8 experts of 4096 x 14336, 64 tokens: 748 MB in
// 160-169 us, 4.4-4.7 TB/s, 172 with exact sums; 8 waves a workgroup 196, R = 2 198).  96-row
// tiles fill no unit (E 16, 4095 tokens, MXFP8, gate/up and down: matrix cores busy 40 and 29 %
// of the CUs' cycles, LDS 42 and 29, a third of that bank conflicts; a wave waits for memory or a
// barrier a fifth of its time and stands behind instructions issued before for half of it).  Every
// wave reads the whole stage from LDS: R = 2 halves that per product, 246-252 registers, two
// workgroups a CU (the same call: 215 us with R = 1 and 8 waves, 191 with R = 2, 176 to 180 with
// KEEP, 1.15 PFLOP/s).  A second chunk and stage in flight cost the second workgroup and 4 %;
// stages of 128 bytes, twice the barriers, 2-10 %; weights loaded straight to LDS, 3-9 %.
template <int KIND, int BM, int R, bool KEEP, bool A4>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(BM == kShort4 ? 4 : 2, 8))) void gemm_mx4s(
    const uint8_t* __restrict__ act, const uint8_t* __restrict__ acts,
    const uint8_t* __restrict__ wt, const uint8_t* __restrict__ wts,
    const int* __restrict__ perm, const int2* __restrict__ tiles, const int* __restrict__ n_tiles,
    const int* __restrict__ counts, const int* __restrict__ offsets, const int* __restrict__ row_of,
    const float* __restrict__ w, int H, int I, int k, int P, uint8_t* __restrict__ hq,
    uint8_t* __restrict__ hs, float* __restrict__ y, uint16_t* __restrict__ out, uint32_t okey) {
  constexpr int NW = 4, NT = NW * 64;
  constexpr bool GU = KIND == kGateUp4;
  constexpr int RPW = (GU ? 16 : 32) * R;                       // outputs per wave
  constexpr int G = BM / 16;                              // 16-row groups of the tile
  constexpr int CPS = A4 ? 2 : 1;                         // chunks per stage
  constexpr int SB = 256;                                 // activation bytes of a row per stage
  constexpr int RS = SB + 16;                             // padded LDS row stride
  constexpr int CH = SB / 16;                             // 16-byte pieces of a row per stage
  constexpr int LPT = BM * CH / NT;                       // 16-byte code loads per thread
  constexpr int SS = 8 * CPS;                             // scale bytes of a row per stage
  constexpr int BD = 2;                                   // activation operands held
  // gate/up sums of E4M3 activations exact to FP32 (split_e4m3: twice the products), so that no activation
  // takes the other of two codes: where a token's output rests on few of them and the weights' bytes leave
  // the matrix cores room (16 rows an expert, H 2048 I 768 E 128: 85.6 -> 89.0 us; 64 tokens, 8 experts of
  // 4096 x 14336 168 -> 172).  The taller tiles have none (777 tokens 172 -> 256, 4095 179 -> 246; with
  // R = 1, E 6, 256 tokens 64 -> 98).
  constexpr bool EXACT = GU && !A4 && BM == kShort4;
  __shared__ __align__(16) uint8_t xl[2][BM * RS];
  __shared__ __align__(16) uint8_t sl[2][BM * SS];
  __shared__ __align__(16) i32x4 wtl[NW][16 * 8];         // per wave: [16 rows][8 pieces]
  const int tid = threadIdx.x;
  if (GU && out) clear_rows(out, row_of, P, H);           // (one slot: the down product stores whole rows)
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
  // first weight row of group m (gate_up: gate and up rows in turn)
  auto grow = [&](int m) { return GU ? (m & 1) * I + nb + 16 * (m >> 1) : nb + 16 * m; };
  const size_t wrows = GU ? 2 * static_cast<size_t>(I) : static_cast<size_t>(N);

  // whole-line loads: lane = (row lr of an 8-row group, 16-byte piece lc)
  const int lr = ln >> 3, lc = ln & 7;
  const uint8_t* __restrict__ wb = wt + static_cast<size_t>(e) * wrows * RB;
  const uint8_t* __restrict__ wsb = wts + static_cast<size_t>(e) * wrows * KB;
  const uint32_t ow = static_cast<uint32_t>(lr * RB + lc * 16), os = static_cast<uint32_t>(col * KB);
  i32x4* tw = wtl[wv];
  i32x4* wdst = tw + lr * 8 + (lc ^ lr);                  // + 64 for rows 8-15
  const i32x4* asrc = tw + col * 8;
  const int sw = col & 7;

  // activation loads: thread = 16-byte piece tid % CH of rows tid / CH + i NT / CH
  const int piece = (tid % CH) * 16, xrow = tid / CH;
  uint32_t oxl[LPT];
#pragma unroll
  for (int i = 0; i < LPT; ++i) {
    const int r = xrow + i * (NT / CH), rr = r < mcount ? r : 0;
    oxl[i] = static_cast<uint32_t>((GU ? perm[rbase + rr] / k : rbase + rr) * AB + piece);
  }
  const bool sload = tid < BM;
  const int srow = tid < mcount ? tid : 0;
  const uint32_t osx = static_cast<uint32_t>(sload ? (GU ? perm[rbase + srow] / k : rbase + srow) * KB : 0);
  i32x4 xr[LPT], W[4 * R];
  uint2 sr[CPS], sc[2 * R];
  // activations of stage st (a row's last stage may hold one chunk: its first one again)
  auto fetch = [&](int st) {
    if (st < nstage) {
      const int b = st * SB, back = b + piece < AB ? 0 : 128;
#pragma unroll
      for (int i = 0; i < LPT; ++i) xr[i] = ld16(act + oxl[i] + (b - back));
      if (sload)
#pragma unroll
        for (int c = 0; c < CPS; ++c)
          sr[c] = *reinterpret_cast<const uint2*>(acts + osx + 8 * min(st * CPS + c, nchunk - 1));
    }
  };
  auto publish = [&](int st) {
    if (st < nstage) {
      uint8_t* d = &xl[st & 1][xrow * RS + piece];
#pragma unroll
      for (int i = 0; i < LPT; ++i) *reinterpret_cast<i32x4*>(d + i * (NT / CH) * RS) = xr[i];
      if (sload)
#pragma unroll
        for (int c = 0; c < CPS; ++c) *reinterpret_cast<uint2*>(&sl[st & 1][tid * SS + 8 * c]) = sr[c];
    }
    __syncthreads();
  };
  // weights of group m of chunk c and the scales of the lane's row (past the end the last chunk again)
  auto request = [&](int m, int c) {
    const uint32_t cc = static_cast<uint32_t>(min(c, nchunk - 1));
    const uint8_t* p = wb + (static_cast<uint32_t>(grow(m) * RB) + 128 * cc);
    W[2 * m] = KEEP ? ld16(p + ow) : ld16_stream(p + ow);
    W[2 * m + 1] = KEEP ? ld16(p + 8 * RB + ow) : ld16_stream(p + 8 * RB + ow);
    sc[m] = *reinterpret_cast<const uint2*>(wsb + (static_cast<uint32_t>(grow(m) * KB) + 8 * cc) + os);
  };
  fetch(0);
#pragma unroll
  for (int m = 0; m < 2 * R; ++m) request(m, 0);
  f32x4 acc[2 * R][G];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int m = 0; m < 2 * R; ++m) acc[m][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  publish(0);

  // One chunk: the weights through the wave's LDS tile into operands, the next chunk's on their
  // way into the registers they left, then the products.
  auto chunk = [&](int buf, int cc, int next) {
    i32x4 a[4 * R];
    int sa[2 * R];
#pragma unroll
    for (int m = 0; m < 2 * R; ++m) {
      wdst[0] = W[2 * m];
      wdst[64] = W[2 * m + 1];
      __builtin_amdgcn_wave_barrier();
      a[2 * m] = asrc[(2 * grp) ^ sw];
      a[2 * m + 1] = asrc[(2 * grp + 1) ^ sw];
      __builtin_amdgcn_wave_barrier();
      sa[m] = static_cast<int>((grp < 2 ? sc[m].x : sc[m].y) >> (16 * (grp & 1)));
      request(m, next);
    }
    __builtin_amdgcn_sched_barrier(0);                    // (the compiler would sink the loads behind the products)
    const uint8_t* xcur = &xl[buf][col * RS + (A4 ? cc * 128 + 32 * grp : 64 * (grp >> 1) + 16 * (grp & 1))];
    const uint8_t* scur = &sl[buf][col * SS + cc * 8 + 2 * grp];
    int sx[G];
#pragma unroll
    for (int g = 0; g < G; ++g) sx[g] = *reinterpret_cast<const uint16_t*>(scur + 16 * g * SS);
    // operand i = 2 g + j of row group g and product j, read BD - 1 operands ahead
    i32x8 b[BD];
    auto rdb = [&](int i) {
      const uint8_t* p = xcur + 16 * (i >> 1) * RS + (A4 ? 16 : 32) * (i & 1);
      const i32x4 lo = *reinterpret_cast<const i32x4*>(p);
      b[i % BD] = cat8(lo, A4 ? i32x4{0, 0, 0, 0} : *reinterpret_cast<const i32x4*>(p + 128));
    };
#pragma unroll
    for (int i = 0; i < BD - 1 && i < 2 * G; ++i) rdb(i);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g && g >= ng) break;                            // (uniform: the tile has no rows there)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (2 * g + j + BD - 1 < 2 * G) rdb(2 * g + j + BD - 1);
        i32x8 x = b[(2 * g + j) % BD], high;
        if (EXACT)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            int lo, hi;
            split_e4m3(x[i], lo, hi);
            x[i] = lo;
            high[i] = hi;
          }
#pragma unroll
        for (int m = 0; m < 2 * R; ++m) {
          if (j == 0) acc[m][g] = mfma_mx4_16<A4, 0>(a[2 * m], x, sa[m], sx[g], acc[m][g]);
          else acc[m][g] = mfma_mx4_16<A4, 1>(a[2 * m + 1], x, sa[m], sx[g], acc[m][g]);
        }
        if (EXACT)
#pragma unroll
          for (int m = 0; m < 2 * R; ++m) {
            if (j == 0) acc[m][g] = mfma_mx4_16<A4, 0>(a[2 * m], high, sa[m], sx[g], acc[m][g]);
            else acc[m][g] = mfma_mx4_16<A4, 1>(a[2 * m + 1], high, sa[m], sx[g], acc[m][g]);
          }
        // (kept at their place: sunk to the end of the stage they would hold every operand live)
#pragma unroll
        for (int m = 0; m < 2 * R; ++m) asm volatile("" : "+v"(acc[m][g]));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  for (int st = 0; st < nstage; ++st) {
    fetch(st + 1);
    chunk(st & 1, 0, st * CPS + 1);
    if (CPS == 2 && 2 * st + 1 < nchunk) chunk(st & 1, 1, 2 * st + 2);
    publish(st + 1);
  }
  // lane: outputs 4 grp + i of every weight group and tile row 16 g + col
  if (GU) {
    // SwiGLU into the gate groups; a row's largest magnitude over the block of 32 neurons gives
    // its scale: the wave's own two groups, or its one and, through LDS, that of wave wv ^ 1
    float* s_amax = reinterpret_cast<float*>(xl[0]);      // (every wave is done with the stages)
    float top[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      top[g] = 0.f;
#pragma unroll
      for (int m = 0; m < 2 * R; m += 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[m][g][i] = swiglu4(acc[m][g][i], acc[m + 1][g][i]);
          top[g] = fmaxf(top[g], fabsf(acc[m][g][i]));
        }
      top[g] = fmaxf(top[g], __shfl_xor(top[g], 16, kWave));
      top[g] = fmaxf(top[g], __shfl_xor(top[g], 32, kWave));
      if (R == 1 && grp == 0) s_amax[wv * BM + 16 * g + col] = top[g];
    }
    if (R == 1) __syncthreads();
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int r = 16 * g + col;
      if (r >= mcount) continue;
      const int s = [&](float m) { return A4 ? mx4_scale_exp(m) : mx_scale_exp(m); }(
          R == 1 ? fmaxf(top[g], s_amax[(wv ^ 1) * BM + r]) : top[g]);
      const float inv = exp2_neg(s);
      const size_t row = static_cast<size_t>(rbase + r);
#pragma unroll
      for (int m = 0; m < 2 * R; m += 2) {
        const f32x4 v = acc[m][g];
        const int n = nb + 8 * m + 4 * grp;
        if (A4)
          *reinterpret_cast<uint16_t*>(hq + row * (I / 2) + n / 2) =
              static_cast<uint16_t>(f32x4_to_e2m1x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv));
        else
          *reinterpret_cast<uint32_t*>(hq + row * I + n) =
              f32x4_to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      }
      if (grp == 0 && (R == 2 || (wv & 1) == 0)) hs[row * (I / 32) + nb / 32] = static_cast<uint8_t>(s + 127);
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
#pragma unroll
      for (int m = 0; m < 2 * R; ++m)
        *reinterpret_cast<uint2*>(orow + 16 * m) = make_uint2(pack_bf16x2(wj * acc[m][g][0], wj * acc[m][g][1]),
                                                              pack_bf16x2(wj * acc[m][g][2], wj * acc[m][g][3]));
    } else {
      float* yr = y + static_cast<size_t>(rbase + r) * H + nb + 4 * grp;
#pragma unroll
      for (int m = 0; m < 2 * R; ++m) *reinterpret_cast<f32x4*>(yr + 16 * m) = acc[m][g];
    }
  }
}

// ---------------------------------------------------------------------------
// Large groups (hundreds of routed rows per expert and more): the products are bound by the
// matrix cores and by LDS, and run as an LDS-tiled GEMM.  Workgroup tile 256 rows x 256
// weight rows (gate_up: 128 gate + 128 up rows of one expert, so that the epilogue finds g
// and u in one lane); 4 waves of 128 x 128 with the block-scaled 32x32x64 MFMA, accumulators
// in AGPRs; both tiles staged in LDS, two stages, 16-byte pieces XOR-swizzled by row; global
// loads one stage ahead of the LDS writes, which run one stage ahead of the fragment reads.
//
// A step of 256 positions is four MFMA K steps.  MXFP4 activations: one LDS stage of 128
// bytes of either row; K step ks takes blocks 4 hi + ks in lane half hi, so a lane's four
// scale bytes are one dword and ks selects its byte.  MXFP8 activations (a stage of 256
// positions would not fit): two stages of 128 bytes of activation and 64 of weight row; K
// step ks of stage st takes blocks 2 hi + (ks & 1) of the stage's four, and the scale bytes
// are stored in the order that makes these a dword too (scale_place).
//
// The scales come straight to registers, a dword a row and step, from copies with the step
// outside and the row inside (mx4_scales_t; the gate/up epilogue writes h's that way): from
// rows as they are given, a wave's load would touch 32 lines.
//
// Measured, 16384 rows, 6 experts, H 7168, I 2048: MXFP4 gate/up 275 us, 3.5 PFLOP/s (matrix
// cores busy half of the time), down 199, 2.4 (8 steps a tile against its start, and 235 MB of
// output).  With two stages of loads in flight instead of one the whole call took 536 us for 530.
namespace {
constexpr int kLTile = kLargeBM * 128;                   // bytes of an operand's stage

// Place, within a row's 8 scale bytes of a step, of the byte of block b.
template <bool A4>
__host__ __device__ constexpr int scale_place(int b) {
  return A4 ? b : 4 * (b >> 1 & 1) + 2 * (b >> 2) + (b & 1);
}

template <bool A4>
constexpr size_t large4_lds() {
  return A4 ? 2 * 2 * kLTile : 2 * (kLTile + kLTile / 2);
}
constexpr size_t kLSide = 2 * sizeof(int) * kLargeBM;    // (down: the rows' pair ids and weights)

// 32x32x64 with weights w (E2M1) and activations x (E2M1 or E4M3); XW: the activation rows
// along the result's registers and the weight rows along its lanes, else the other way.
template <bool A4, bool XW, int SEL>
__device__ __forceinline__ f32x16 mfma_mx4_32(i32x4 w, i32x8 x, uint32_t sw, uint32_t sx, f32x16 c) {
  const i32x8 w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
  if (XW)
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, w8, c, A4 ? 4 : 0, 4, SEL, static_cast<int>(sx),
                                                           SEL, static_cast<int>(sw));
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, x, c, 4, A4 ? 4 : 0, SEL, static_cast<int>(sw),
                                                         SEL, static_cast<int>(sx));
}

// SwiGLU and the MX codes of two 32-neuron blocks of one row: the lanes (l32, hi = 0 / 1) of
// a row hold neurons 8q + 4hi + t in register 4q + t; each encodes its half of both blocks,
// and the lanes exchange halves, so that lane hi stores block hi, n + 32 hi on.
template <bool A4>
__device__ __forceinline__ void mx4_store_row(const f32x16 (&g)[2], const f32x16 (&u)[2], int r, int mcount,
                                              int rbase, int n, int hi, int I, int P,
                                              uint8_t* __restrict__ hq, uint8_t* __restrict__ hs) {
  uint32_t c[2][4];
  int sx[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    float v[16], top = 0.f;
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      v[x] = swiglu4(g[b][x], u[b][x]);
      top = fmaxf(top, fabsf(v[x]));
    }
    top = fmaxf(top, __shfl_xor(top, 32, kWave));
    sx[b] = A4 ? mx4_scale_exp(top) : mx_scale_exp(top);
    const float inv = exp2_neg(sx[b]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float a0 = v[4 * q] * inv, a1 = v[4 * q + 1] * inv, a2 = v[4 * q + 2] * inv, a3 = v[4 * q + 3] * inv;
      c[b][q] = A4 ? f32x4_to_e2m1x4(a0, a1, a2, a3) : f32x4_to_e4m3x4(a0, a1, a2, a3);
    }
  }
  // what the other lane stores goes there; bytes of quad q: those of lane hi = 0, then of 1
  uint32_t own[4], got[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    own[q] = hi ? c[1][q] : c[0][q];
    got[q] = hi ? c[0][q] : c[1][q];
  }
  if (A4) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(got[2 * p] | got[2 * p + 1] << 16), 32, kWave));
      got[2 * p] = o & 0xFFFFu;
      got[2 * p + 1] = o >> 16;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) got[q] = static_cast<uint32_t>(__shfl_xor(static_cast<int>(got[q]), 32, kWave));
  }
  if (r >= mcount) return;
  const int nb = n + 32 * hi;
  const size_t row = static_cast<size_t>(rbase + r);
  if (A4) {
    i32x4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = static_cast<int>(hi ? got[q] | own[q] << 16 : own[q] | got[q] << 16);
    st16(hq + row * (I / 2) + nb / 2, o);
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      i32x4 o;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        o[2 * z] = static_cast<int>(hi ? got[2 * p + z] : own[2 * p + z]);
        o[2 * z + 1] = static_cast<int>(hi ? own[2 * p + z] : got[2 * p + z]);
      }
      st16(hq + row * I + nb + 16 * p, o);
    }
  }
  hs[(static_cast<size_t>(nb / 256) * P + row) * 8 + scale_place<A4>(nb / 32 % 8)] =
      static_cast<uint8_t>((hi ? sx[1] : sx[0]) + 127);
}

// Two lanes that hold neighbouring columns (even, odd) and the values of two rows (v0, v1)
// exchange one value each: the even lane returns both columns of the first row, the odd
// lane both of the second, as two BF16 (the lower column in the low half).
__device__ __forceinline__ uint32_t pair_rows_bf16(float v0, float v1, int odd) {
  const float give = odd ? v0 : v1;
  const float got = __int_as_float(__builtin_amdgcn_update_dpp(
      0, __float_as_int(give), 0xB1, 0xF, 0xF, true));              // quad_perm [1,0,3,2]
  return odd ? pack_bf16x2(got, v1) : pack_bf16x2(v0, got);
}
}  // namespace

// act / acts: the activations' codes and their scales [K/256][rows][8] (grouped rows); wt / wts:
// the weights' codes and their scales [E][K/256][weight rows][8].  See above.
template <int KIND, bool A4>
__global__ __launch_bounds__(256) void gemm_large_mx4(
    const uint8_t* __restrict__ act, const uint32_t* __restrict__ acts,
    const uint8_t* __restrict__ wt, const uint32_t* __restrict__ wts, const int* __restrict__ perm,
    const int2* __restrict__ tiles, const int* __restrict__ n_tiles, const int* __restrict__ counts,
    const int* __restrict__ offsets, const float* __restrict__ w, int H, int I, int k, int P,
    uint8_t* __restrict__ hq, uint8_t* __restrict__ hs, float* __restrict__ y,
    uint16_t* __restrict__ out, float* __restrict__ partial, int ncu, uint32_t okey) {
  extern __shared__ __align__(16) uint8_t ldl[];         // [stage][weights, activations]
  constexpr bool GU = KIND == kGateUp4;
  constexpr int WB = A4 ? 128 : 64;                      // bytes of a weight row per stage
  constexpr int kWTile = kLargeBM * WB, kStage = kWTile + kLTile;
  constexpr int NW = WB / 16, NS = NW + 8;               // 16-byte loads per thread and stage: weights, all
  constexpr int KS = A4 ? 4 : 2;                         // MFMA K steps per stage
  constexpr int PER = NS / KS;                           // loads and LDS writes per K step
  const int K = GU ? H : I;
  const int RB = K / 2, AB = A4 ? K / 2 : K;             // bytes of a row: weights, activations
  const int nblk = GU ? I / 128 : H / 256;
  const int nk = K / 256;
  const int nt = *n_tiles;
  const TailPlan plan = tail_plan(nblk * nt, ncu, nk);
  const int L = blockIdx.x;
  const int tid = threadIdx.x, wv = tid >> 6, ln = tid & 63, l32 = ln & 31, hi = ln >> 5;
  const int wm = wv & 1, wn = wv >> 1;
  int item, kb = 0, ke = nk, slot = -1;                  // slot >= 0: a slice of a tile of the last round
  if (plan.S > 1 && L < plan.full) {
    item = permute_item(round_item(L, plan.full, ncu), plan.full, okey);
  } else if (plan.S > 1) {
    if (L - plan.full >= plan.rem * plan.S) return;
    slot = permute_item(L - plan.full, plan.rem * plan.S, okey);
    item = plan.full + slot % plan.rem;
    const int sl = slot / plan.rem;
    kb = sl * nk / plan.S;
    ke = (sl + 1) * nk / plan.S;
  } else {
    item = round_real_item(L, nblk, nt, ncu);
    if (item < 0) return;
    item = permute_item(item, nblk * nt, okey);
  }
  int tile, nb;
  large_coords(item, nblk, nt, tile, nb);
  const int2 te = tiles[tile];
  const int e = te.x, m0 = te.y;
  const int mcount = min(kLargeBM, counts[e] - m0);
  const int rbase = offsets[e] + m0;
  const int n0 = nb * 128;

  // loaders.  Activations (and weights of 128 bytes a stage): rows wv*64 + 8j + (ln >> 3), piece
  // ln & 7; weights of 64 bytes: rows wv*64 + 16j + (ln >> 2), piece ln & 3
  const int lrow = ln >> 3, lc = ln & 7;
  const int wrow = A4 ? lrow : ln >> 2, wc = A4 ? lc : ln & 3;
  const size_t wrows = GU ? 2 * static_cast<size_t>(I) : static_cast<size_t>(H);
  const uint8_t* __restrict__ abase = wt + static_cast<size_t>(e) * wrows * RB;
  const int arow = GU ? (wv < 2 ? n0 + wv * 64 : I + n0 + (wv - 2) * 64) : nb * 256 + wv * 64;
  const uint32_t ao = static_cast<uint32_t>((arow + wrow) * RB + wc * 16);
  // gate_up: the tokens' rows, the tile's first one past its end; down: grouped rows, the next ones (or,
  // behind the last, up to 255 rows of the workspace) past its end.  Columns of rows past the end are
  // computed and discarded.
  uint32_t bo[GU ? 8 : 1];
#pragma unroll
  for (int j = 0; j < (GU ? 8 : 1); ++j) {
    const int r = wv * 64 + 8 * j + lrow;
    bo[j] = static_cast<uint32_t>((GU ? perm[rbase + (r < mcount ? r : 0)] / k : r) * AB + lc * 16);
  }
  const uint8_t* __restrict__ actb = GU ? act : act + static_cast<size_t>(rbase) * AB;
  // LDS: piece c of row r of 128 bytes at c ^ (r >> 1 & 7), of 64 bytes at c ^ (r >> 2 & 3): the
  // 16 rows that a read serves at once lie in 64 different banks
  const int lx0 = (wv * 64 + lrow) * 128 + ((lc ^ (lrow >> 1)) * 16);      // even j; odd j: the piece ^ 4
  const int lx1 = lx0 ^ 64;
  const int lw0 = A4 ? lx0 : (wv * 64 + wrow) * 64 + ((wc ^ (wrow >> 2 & 3)) * 16);
  int fa[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    fa[i] = (GU ? (i >> 1) * 128 + wn * 64 + (i & 1) * 32 : wn * 128 + 32 * i) + l32;
  const int fb = wm * 128 + l32;
  const int swx = l32 >> 1 & 7, sww = A4 ? swx : l32 >> 2 & 3;
  // scales: dword hi of the wave's weight rows and of its activation rows, the first blocks' (the
  // others' lie a fixed distance on; past the tile's end the next rows', as above)
  const uint32_t osa = static_cast<uint32_t>(GU ? n0 + wn * 64 + l32 : nb * 256 + wn * 128 + l32) * 2 + hi;
  const uint32_t osb = static_cast<uint32_t>(rbase + fb) * 2 + hi;
  const uint32_t* __restrict__ sab = wts + static_cast<size_t>(e) * nk * wrows * 2;

  i32x4 stg[NS];   // [0, NW) weight rows, [NW, NS) activation rows
  // stage s covers step s / 2 (MXFP8) or s (MXFP4); past the end the last one again
  const int s_end = A4 ? ke : 2 * ke;
  auto gload = [&](int q, int s) {
    const int ss = min(s, s_end - 1);
    if (q < NW) stg[q] = ld16(abase + ao + static_cast<uint32_t>(q * (A4 ? 8 : 16)) * RB + static_cast<uint32_t>(ss * WB));
    else stg[q] = ld16(actb + bo[GU ? (q - NW) & 7 : 0] + (GU ? 0u : static_cast<uint32_t>((q - NW) * 8) * AB) + static_cast<uint32_t>(ss * 128));
  };
  auto lwrite = [&](int q, int s) {
    uint8_t* st = ldl + (s & 1) * kStage;
    if (q < NW) *reinterpret_cast<i32x4*>(st + (A4 ? (q & 1 ? lx1 : lx0) + q * 8 * 128 : lw0 + q * 16 * 64)) = stg[q];
    else *reinterpret_cast<i32x4*>(st + kWTile + (q & 1 ? lx1 : lx0) + ((q - NW) & 7) * 8 * 128) = stg[q];
  };
  // fragments: weights of this and of the next K step, activations of this one, each replaced by
  // the next K step's once its products are issued
  i32x4 fa0[4], fa1[4];
  i32x8 fx[4];
  // weight fragment g, activation fragment g of K step ks of stage s
  auto rda = [&](i32x4 (&f)[4], int g, int s, int ks) {
    const uint8_t* st = ldl + (s & 1) * kStage;
    f[g] = *reinterpret_cast<const i32x4*>(st + fa[g] * WB + (((A4 ? 4 * hi + ks : 2 * hi + ks) ^ sww) * 16));
  };
  auto rdb = [&](int g, int s, int ks) {
    const uint8_t* st = ldl + (s & 1) * kStage + kWTile + (fb + 32 * g) * 128;
    if (A4) {
      fx[g] = cat8(*reinterpret_cast<const i32x4*>(st + ((4 * hi + ks) ^ swx) * 16), i32x4{0, 0, 0, 0});
    } else {
      fx[g] = cat8(*reinterpret_cast<const i32x4*>(st + ((2 * ks + hi) ^ swx) * 16),
                   *reinterpret_cast<const i32x4*>(st + ((4 + 2 * ks + hi) ^ swx) * 16));
    }
  };
  uint32_t sa[4], sb[4], na[4], nbs[4];
  auto sload = [&](int kt) {
    const uint32_t kk = static_cast<uint32_t>(min(kt, ke - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      na[i] = sab[kk * static_cast<uint32_t>(2 * wrows) + (GU ? (i >> 1) * 2 * I + (i & 1) * 64 : 64 * i) + osa];
#pragma unroll
    for (int j = 0; j < 4; ++j) nbs[j] = acts[static_cast<size_t>(kk) * (2 * static_cast<size_t>(P)) + 64 * j + osb];
  };
  f32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  // One MFMA K step on weight fragments f (scale byte SEL): 8 groups of 2 MFMAs; the first groups read
  // the weight fragments of K step rks of stage rs into n, every second one its activation fragment for
  // that step, and the first PER write a staged piece of stage ws to LDS and reload it from stage ws + 1.
  // sched_barrier keeps this order.
  auto phase = [&](auto sel, i32x4 (&f)[4], i32x4 (&n)[4], int rs, int rks, int ws, int q0) {
    constexpr int SEL = decltype(sel)::value;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const int j = g >> 1, i = (g & 1) * 2;
#pragma unroll
      for (int z = 0; z < 2; ++z)
        acc[i + z][j] = mfma_mx4_32<A4, !GU, SEL>(f[i + z], fx[j], sa[i + z], sb[j], acc[i + z][j]);
      __builtin_amdgcn_sched_barrier(0);
      if (g < 4) rda(n, g, rs, rks);
      if (g & 1) rdb(j, rs, rks);
      if (g < PER) {
        lwrite(q0 + g, ws);
        gload(q0 + g, ws + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // The LDS writes of stage s + 1 are spread over the K steps that may write its buffer: the last
  // one of stage s - 1 (the last PER pieces, after the barrier that ends the reads of stage s - 1)
  // and all but the last of stage s (before the barrier that publishes stage s + 1).
  const int s0 = A4 ? kb : 2 * kb;
  sload(kb);
#pragma unroll
  for (int q = 0; q < NS; ++q) gload(q, s0);
#pragma unroll
  for (int q = 0; q < NS; ++q) lwrite(q, s0);
#pragma unroll
  for (int q = 0; q < NS; ++q) gload(q, s0 + 1);
#pragma unroll
  for (int q = NS - PER; q < NS; ++q) {
    lwrite(q, s0 + 1);
    gload(q, s0 + 2);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sa[i] = na[i];
    sb[i] = nbs[i];
  }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    rda(fa0, g, s0, 0);
    rdb(g, s0, 0);
  }
  // the epilogue's data (tile row tid's pair and weight)
  const int my_pr = GU ? 0 : perm[rbase + min(tid, mcount - 1)];
  float my_w = 0.f;
  auto publish = [&]() {
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
  };
  using std::integral_constant;
  for (int kt = kb; kt < ke; ++kt) {
    sload(kt + 1);
    if (A4) {
      phase(integral_constant<int, 0>{}, fa0, fa1, kt, 1, kt + 1, 0);
      phase(integral_constant<int, 1>{}, fa1, fa0, kt, 2, kt + 1, PER);
      phase(integral_constant<int, 2>{}, fa0, fa1, kt, 3, kt + 1, 2 * PER);
      publish();
      // In the loop on purpose: a loop of one basic block would keep a copy of the accumulators
      // outside the AGPRs for the code after it.
      if (KIND == kDownFused4 && kt == kb) my_w = w[my_pr];          // k = 1: pair id == token
      phase(integral_constant<int, 3>{}, fa1, fa0, kt + 1, 0, kt + 2, 3 * PER);
    } else {
      phase(integral_constant<int, 0>{}, fa0, fa1, 2 * kt, 1, 2 * kt + 1, 0);
      publish();
      phase(integral_constant<int, 1>{}, fa1, fa0, 2 * kt + 1, 0, 2 * kt + 2, PER);
      if (KIND == kDownFused4 && kt == kb) my_w = w[my_pr];
      phase(integral_constant<int, 2>{}, fa0, fa1, 2 * kt + 1, 1, 2 * kt + 2, 0);
      publish();
      phase(integral_constant<int, 3>{}, fa1, fa0, 2 * kt + 2, 0, 2 * kt + 3, PER);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sa[i] = na[i];
      sb[i] = nbs[i];
    }
  }
  if (slot >= 0) {
    // tail slice: FP32 partial tile in register order, [64 x f32x4][256 threads]
    f32x4* pp = reinterpret_cast<f32x4*>(partial) + static_cast<size_t>(slot) * 64 * 256 + tid;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
        for (int q = 0; q < 4; ++q)
          pp[((i * 4 + j) * 4 + q) * 256] =
              f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      }
    return;
  }
  if (GU) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) asm volatile("" : "+a"(acc[i][j]));
      const f32x16 g[2] = {acc[0][j], acc[1][j]}, u[2] = {acc[2][j], acc[3][j]};
      mx4_store_row<A4>(g, u, wm * 128 + 32 * j + l32, mcount, rbase, n0 + wn * 64, hi, I, P, hq, hs);
      __builtin_amdgcn_sched_barrier(0);
    }
    return;
  }
  // Lane (l32, hi), register 4q + t of block (i, j): output column l32 of weight block i, tile row
  // 8q + 4hi + t of row block j: a store instruction writes 128 consecutive bytes of two rows (FP32),
  // or 64 of four (BF16, columns paired over lanes).
  int* s_pr = reinterpret_cast<int*>(ldl + large4_lds<A4>());
  float* s_w = reinterpret_cast<float*>(ldl + large4_lds<A4>()) + kLargeBM;
  s_pr[tid] = my_pr;
  s_w[tid] = my_w;
  __syncthreads();
  auto store = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q == 0)
#pragma unroll
          for (int i = 0; i < 4; ++i) asm volatile("" : "+a"(acc[i][j]));
        __builtin_amdgcn_sched_barrier(0);
        const int r0 = wm * 128 + 32 * j + 8 * q + 4 * hi;
        if (!kWhole && r0 >= mcount) continue;
        if (KIND == kDownFused4) {
          const i32x4 pr = *reinterpret_cast<const i32x4*>(s_pr + r0);
          const f32x4 wt4 = *reinterpret_cast<const f32x4*>(s_w + r0);
          const int odd = l32 & 1;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint16_t* orow = out + static_cast<size_t>(odd ? pr[2 * h + 1] : pr[2 * h]) * H + nb * 256 + wn * 128 + l32 - odd;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t o = pair_rows_bf16(wt4[2 * h] * acc[i][j][4 * q + 2 * h],
                                                wt4[2 * h + 1] * acc[i][j][4 * q + 2 * h + 1], odd);
              if (kWhole || r0 + 2 * h + odd < mcount) *reinterpret_cast<uint32_t*>(orow + 32 * i) = o;
            }
          }
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            if (!kWhole && r0 + t >= mcount) continue;
            float* yr = y + static_cast<size_t>(rbase + r0 + t) * H + nb * 256 + wn * 128 + l32;
#pragma unroll
            for (int i = 0; i < 4; ++i) yr[32 * i] = acc[i][j][4 * q + t];
          }
        }
      }
  };
  if (mcount == kLargeBM) store(std::true_type{});
  else store(std::false_type{});
}

// Tail fix-up: the slices of a tile of the last round, added in slice order, and the epilogue.
// gate_up: workgroup (tail item, row block j), a GEMM thread's blocks of that j each; down:
// element-parallel, an f32x4 of the partial tile to a thread.
template <bool A4>
__global__ __launch_bounds__(256) void gemm_large_mx4_fixup_gate_up(
    const int2* __restrict__ tiles, const int* __restrict__ n_tiles, const int* __restrict__ counts,
    const int* __restrict__ offsets, int H, int I, int P, uint8_t* __restrict__ hq,
    uint8_t* __restrict__ hs, const float* __restrict__ partial, int ncu, uint32_t okey) {
  const int nblk = I / 128;
  const TailPlan plan = tail_plan(nblk * *n_tiles, ncu, H / 256);
  const int g = permute_item(blockIdx.x, gridDim.x, okey);
  const int b = g >> 2, j = g & 3;
  if (plan.S == 1 || b >= plan.rem) return;
  int tile, nb;
  large_coords(plan.full + b, nblk, *n_tiles, tile, nb);
  const int2 te = tiles[tile];
  const int e = te.x, m0 = te.y;
  const int mcount = min(kLargeBM, counts[e] - m0);
  const int rbase = offsets[e] + m0;
  const int tid = threadIdx.x, wv = tid >> 6, ln = tid & 63, l32 = ln & 31, hi = ln >> 5;
  const int wm = wv & 1, wn = wv >> 1;
  if (wm * 128 + 32 * j >= mcount) return;               // (uniform in the wave)
  f32x16 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[i][q] = 0.f;
  for (int sl = 0; sl < plan.S; ++sl) {
    const f32x4* pp = reinterpret_cast<const f32x4*>(partial) + static_cast<size_t>(sl * plan.rem + b) * 64 * 256 + tid;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 v = pp[((i * 4 + j) * 4 + q) * 256];
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][4 * q + t] += v[t];
      }
  }
  const f32x16 gg[2] = {acc[0], acc[1]}, uu[2] = {acc[2], acc[3]};
  mx4_store_row<A4>(gg, uu, wm * 128 + 32 * j + l32, mcount, rbase, nb * 128 + wn * 64, hi, I, P, hq, hs);
}

template <int KIND>
__global__ __launch_bounds__(256) void gemm_large_mx4_fixup_down(
    const int* __restrict__ perm, const int2* __restrict__ tiles, const int* __restrict__ n_tiles,
    const int* __restrict__ counts, const int* __restrict__ offsets, const float* __restrict__ w, int H,
    int I, float* __restrict__ y, uint16_t* __restrict__ out, const float* __restrict__ partial, int ncu,
    uint32_t okey) {
  const int nblk = H / 256;
  const TailPlan plan = tail_plan(nblk * *n_tiles, ncu, I / 256);
  const int g = permute_item(blockIdx.x, gridDim.x, okey) * 256 + threadIdx.x;
  const int b = g >> 14;                                  // 64 x 256 threads per tail item
  if (plan.S == 1 || b >= plan.rem) return;
  const int f = g & 16383;                                // f32x4 index within the tile
  const int tid = f & 255, ijq = f >> 8;
  const int i = ijq >> 4, j = (ijq >> 2) & 3, q = ijq & 3;
  int tile, nb;
  large_coords(plan.full + b, nblk, *n_tiles, tile, nb);
  const int2 te = tiles[tile];
  const int e = te.x, m0 = te.y;
  const int mcount = min(kLargeBM, counts[e] - m0);
  const int rbase = offsets[e] + m0;
  const int wv = tid >> 6, ln = tid & 63, l32 = ln & 31, hi = ln >> 5;
  const int wm = wv & 1, wn = wv >> 1;
  const int r0 = wm * 128 + 32 * j + 8 * q + 4 * hi;      // rows r0 .. r0 + 3, one column
  if (r0 >= mcount) return;
  const f32x4* pp = reinterpret_cast<const f32x4*>(partial) + f;
  f32x4 a = {0.f, 0.f, 0.f, 0.f};
  for (int sl = 0; sl < plan.S; ++sl) a += pp[static_cast<size_t>(sl * plan.rem + b) * 64 * 256];
  const int n = nb * 256 + wn * 128 + 32 * i + l32;
  for (int t = 0; t < 4 && r0 + t < mcount; ++t) {
    const int row = rbase + r0 + t;
    if (KIND == kDownFused4) {
      const int pr = perm[row];
      out[static_cast<size_t>(pr) * H + n] = static_cast<uint16_t>(f32_to_bf16_rne(w[pr] * a[t]));
    } else {
      y[static_cast<size_t>(row) * H + n] = a[t];
    }
  }
}

// Scales with the step of 256 positions outside and the row inside, 8 bytes each in the order of
// scale_place, of both weights and of the routed activations (gathered into grouped order):
// workgroup = 64 rows x 32 steps through LDS, reads and writes along their own rows.  With one
// slot, output rows of pairs without an expert are cleared here.  (16384 rows, 6 experts, H 7168,
// I 2048: 12 MB in and out in 13 us.)
template <bool A4>
__global__ __launch_bounds__(256) void mx4_scales_t(
    const uint2* __restrict__ wgus, const uint2* __restrict__ wds, const uint2* __restrict__ xs,
    const int* __restrict__ perm, const int* __restrict__ row_of, const int* __restrict__ offsets, int H,
    int I, int E, int k, int P, uint2* __restrict__ wgu_t, uint2* __restrict__ wd_t, uint2* __restrict__ x_t,
    uint16_t* __restrict__ out, uint32_t okey) {
  __shared__ uint2 tile[32][65];
  const int tid = threadIdx.x;
  if (out) clear_rows(out, row_of, P, H);
  const int nh = H / 256, ni = I / 256;                   // steps of a row
  const int ch = (nh + 31) / 32, ci = (ni + 31) / 32;     // blocks of 32 steps
  const int gu = 2 * I / 64, dn = H / 64;                 // blocks of 64 rows (H and I multiples of 256)
  int b = permute_item(blockIdx.x, gridDim.x, okey);
  const uint2* src;
  uint2* dst;
  int rows, steps, r0, s0, limit;
  bool gather = false;
  if (b < E * gu * ch) {
    const int e = b / (gu * ch), m = b - e * gu * ch;
    rows = 2 * I, steps = nh, r0 = m / ch * 64, s0 = m % ch * 32, limit = rows;
    src = wgus + static_cast<size_t>(e) * rows * steps;
    dst = wgu_t + static_cast<size_t>(e) * rows * steps;
  } else if ((b -= E * gu * ch) < E * dn * ci) {
    const int e = b / (dn * ci), m = b - e * dn * ci;
    rows = H, steps = ni, r0 = m / ci * 64, s0 = m % ci * 32, limit = rows;
    src = wds + static_cast<size_t>(e) * rows * steps;
    dst = wd_t + static_cast<size_t>(e) * rows * steps;
  } else {
    b -= E * dn * ci;
    rows = P, steps = nh, r0 = b / ch * 64, s0 = b % ch * 32, limit = offsets[E];
    src = xs;
    dst = x_t;
    gather = true;
  }
  if (r0 >= limit) return;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int r = u * 8 + (tid >> 5), s = tid & 31;
    if (r0 + r < limit && s0 + s < steps) {
      const size_t row = gather ? perm[r0 + r] / k : r0 + r;
      uint2 v = src[row * steps + s0 + s];
      if (!A4)                                            // blocks 0, 1, 4, 5 and 2, 3, 6, 7 (scale_place)
        v = make_uint2((v.x & 0xFFFFu) | v.y << 16, v.x >> 16 | (v.y & 0xFFFF0000u));
      tile[s][r] = v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int s = u * 4 + (tid >> 6), r = tid & 63;
    if (r0 + r < limit && s0 + s < steps) dst[static_cast<size_t>(s0 + s) * rows + r0 + r] = tile[s][r];
  }
}

hipError_t mx4_set_attributes() {
  hipError_t e = hipSuccess;
#define LDS(F, A4)                                                                              \
  if (e == hipSuccess)                                                                          \
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(F), hipFuncAttributeMaxDynamicSharedMemorySize, \
                            static_cast<int>(large4_lds<A4>() + kLSide))
  LDS((gemm_large_mx4<kGateUp4, true>), true);
  LDS((gemm_large_mx4<kDown4, true>), true);
  LDS((gemm_large_mx4<kDownFused4, true>), true);
  LDS((gemm_large_mx4<kGateUp4, false>), false);
  LDS((gemm_large_mx4<kDown4, false>), false);
  LDS((gemm_large_mx4<kDownFused4, false>), false);
#undef LDS
  return e;
}

// ---------------------------------------------------------------------------
// Few pairs (a decode step): two launches, every routed pair on its own, its weights straight
// from HBM into the operands of the 16x16x128 MFMA, whose 16 activation columns all hold the
// pair's one row.  Blocks, chunks and products follow in the order of the streaming form's 32-row
// tiles, gate/up sums of E4M3 activations in two parts too (one token, 8 of 128 experts 10.6 ->
// 11.0 us), so a pair has the bits that it has there.  The step is bound by the latency of two
// dependent passes over memory and needs no grouping; pairs that share an expert read its weights
// from the L2 the second time.  One token, 8 of 128 experts, H 2048, I 768: 20 MB of weights in
// 6.8 + 5.2 us of kernels, 12.3 us a call (grouped and streamed 21); 8 of 384 experts, H 7168,
// I 2048: 187 MB in 45 us, 4.1 TB/s.
namespace {
// 16 (ROWS 8: 8, each twice) weight rows on their way into operands: U chunks of 256 positions,
// loaded as 8 rows x 128 contiguous bytes (lane = row ln >> 3, piece ln & 7) and passed through
// the wave's 2 KB of LDS, 16-byte pieces XOR-swizzled by row.  w, ws: row 0's codes and scales.
template <bool A4, int ROWS, int U>
struct PairRows {
  static constexpr int L = ROWS / 8;                     // loads per chunk
  i32x4 a[U][L];
  int sa[U];
  __device__ __forceinline__ void request(const uint8_t* __restrict__ w, const uint8_t* __restrict__ ws, int RB,
                                          int KB, int c0, int nchunk) {
    const int ln = lane_id(), lr = ln >> 3, lc = ln & 7, row = ln & (ROWS - 1) & 15, grp = ln >> 4;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u < nchunk) {
#pragma unroll
        for (int i = 0; i < L; ++i)
          a[u][i] = ld16_stream(w + static_cast<uint32_t>((lr + 8 * i) * RB) + 128 * (c0 + u) + 16 * lc);
        sa[u] = *reinterpret_cast<const uint16_t*>(ws + static_cast<uint32_t>(row * KB) + 8 * (c0 + u) + 2 * grp);
      }
  }
  // times one activation row (x, xs: its codes and scales in global memory or LDS; high > 0: the codes of
  // 2 and above lie that far behind x, split_e4m3), added to acc: register i of lane (c, g) holds row 4 g + i
  __device__ __forceinline__ f32x4 times(const uint8_t* x, const uint8_t* xs, int c0, int nchunk, i32x4* tile,
                                         f32x4 acc, int high = 0) {
    const int ln = lane_id(), lr = ln >> 3, lc = ln & 7, row = ln & (ROWS - 1) & 15, grp = ln >> 4;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u < nchunk) {
        const uint8_t* p = x + (A4 ? 128 * (c0 + u) + 32 * grp : 256 * (c0 + u) + 64 * (grp >> 1) + 16 * (grp & 1));
        const int sx = *reinterpret_cast<const uint16_t*>(xs + 8 * (c0 + u) + 2 * grp);
        i32x8 b[2], h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          b[j] = cat8(*reinterpret_cast<const i32x4*>(p + (A4 ? 16 : 32) * j),
                      A4 ? i32x4{0, 0, 0, 0} : *reinterpret_cast<const i32x4*>(p + 128 + 32 * j));
          if (high)
            h[j] = cat8(*reinterpret_cast<const i32x4*>(p + high + 32 * j),
                        *reinterpret_cast<const i32x4*>(p + high + 128 + 32 * j));
        }
#pragma unroll
        for (int i = 0; i < L; ++i) tile[(lr + 8 * i) * 8 + (lc ^ lr)] = a[u][i];
        __builtin_amdgcn_wave_barrier();
        const i32x4 a0 = tile[row * 8 + ((2 * grp) ^ (row & 7))], a1 = tile[row * 8 + ((2 * grp + 1) ^ (row & 7))];
        __builtin_amdgcn_wave_barrier();
        acc = mfma_mx4_16<A4, 0>(a0, b[0], sa[u], sx, acc);
        if (high) acc = mfma_mx4_16<A4, 0>(a0, h[0], sa[u], sx, acc);
        acc = mfma_mx4_16<A4, 1>(a1, b[1], sa[u], sx, acc);
        if (high) acc = mfma_mx4_16<A4, 1>(a1, h[1], sa[u], sx, acc);
      }
    return acc;
  }
};
constexpr int kPairsMax4 = 48;                           // pairs up to which this form may be taken
constexpr int kPairCols4 = 8;                            // output columns per workgroup of the down pass
constexpr int kPairWaves4 = 8;
// Taken for 48 pairs at most, while the weights that it reads more than once (pairs that share an
// expert; expected number of distinct experts E (1 - (1 - k/E)^T)) stay below 60 MB, about the
// 8 to 12 us that grouping and its launches cost the streaming form, and all that it reads below 350 MB,
// where that form's higher rate has made up for them.  Measured, us (this / streaming), MXFP8:
// H 2048 I 768 E 128 k 8, T 1 13.3 / 21.3, T 6 29 / 32; H 2048 I 1024 E 8 k 2, T 8 14.9 / 22.7, T 24
// (133 MB again) 29 / 23; H 7168 I 2048 E 32 k 4, T 2 43 / 50, T 4 (65 MB again) 78 / 70; H 7168 I 2048
// E 384 k 8, T 1 44 / 52, T 2 (374 MB) 79 / 80; H 4096 I 1024 E 4 k 1, T 40 46 / 27.
inline bool use_pairs4(int T, int H, int I, int E, int k) {
  const int64_t P = static_cast<int64_t>(T) * k;
  if (P > kPairsMax4) return false;
  double miss = 1.0;                                     // (1 - k/E)^T
  for (int t = 0; t < T; ++t) miss *= 1.0 - static_cast<double>(k) / E;
  const double bytes = 3.0 * H * I * 17 / 32, again = static_cast<double>(P) - E * (1.0 - miss);
  return again * bytes <= 60e6 && P * bytes <= 350e6;
}
}  // namespace

// Gate/up, SwiGLU and the codes of one block: workgroup (pair, 32 neurons); waves 0, 1 the gate
// rows, 2, 3 the up rows.
template <bool A4>
__global__ __launch_bounds__(256) void pairs_gate_up_mx4(
    const uint8_t* __restrict__ x, const uint8_t* __restrict__ xs, const uint8_t* __restrict__ wgu,
    const uint8_t* __restrict__ wgus, const int32_t* __restrict__ idx, int H, int I, int E, int k, int P,
    uint8_t* __restrict__ hq, uint8_t* __restrict__ hs, uint32_t okey) {
  extern __shared__ __align__(16) uint8_t ldp[];         // the token's codes (MXFP8: low, high), then its scales
  __shared__ __align__(16) float s_v[2][32];
  __shared__ __align__(16) i32x4 s_tile[4][16 * 8];
  const int nblk = I / 32, AB = A4 ? H / 2 : H, KB = H / 32;
  const int high = A4 ? 0 : AB;
  uint8_t* lds = ldp + AB + high;
  const int item = permute_item(blockIdx.x, nblk * P, okey);
  const int p = item / nblk, n0 = (item - p * nblk) * 32;
  const int e = idx[p];
  if (static_cast<unsigned>(e) >= static_cast<unsigned>(E)) return;
  const int t = p / k, tid = threadIdx.x, ln = lane_id(), col = ln & 15, grp = ln >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(wave_id());
  const int nchunk = H / 256;
  const size_t row = static_cast<size_t>(e) * 2 * I + (wv >> 1) * I + n0 + (wv & 1) * 16;
  const uint8_t *wr = wgu + row * (H / 2), *wsr = wgus + row * KB;
  constexpr int U = 8;
  PairRows<A4, 16, U> r;
  r.request(wr, wsr, H / 2, KB, 0, nchunk);              // on their way while the token is staged
  __builtin_amdgcn_sched_barrier(0);
  for (int c = 16 * tid; c < AB; c += 16 * 256) {
    i32x4 v = ld16(x + static_cast<size_t>(t) * AB + c), hi;
    if (!A4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int l, h;
        split_e4m3(v[i], l, h);
        v[i] = l;
        hi[i] = h;
      }
      st16(ldp + AB + c, hi);
    }
    st16(ldp + c, v);
  }
  for (int c = 8 * tid; c < KB; c += 8 * 256)
    *reinterpret_cast<uint2*>(lds + c) = *reinterpret_cast<const uint2*>(xs + static_cast<size_t>(t) * KB + c);
  __syncthreads();
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
  for (int c0 = 0; c0 < nchunk; c0 += U) {
    if (c0) r.request(wr, wsr, H / 2, KB, c0, nchunk);
    d = r.times(ldp, lds, c0, nchunk, s_tile[wv], d, high);
  }
  if (col == 0) *reinterpret_cast<f32x4*>(&s_v[wv >> 1][(wv & 1) * 16 + 4 * grp]) = d;
  __syncthreads();
  if (tid >= 8) return;                                  // eight lanes of four neurons
  const f32x4 g = *reinterpret_cast<const f32x4*>(&s_v[0][4 * tid]), u = *reinterpret_cast<const f32x4*>(&s_v[1][4 * tid]);
  float v[4], top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = swiglu4(g[i], u[i]);
    top = fmaxf(top, fabsf(v[i]));
  }
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, kWave));
  const int s = A4 ? mx4_scale_exp(top) : mx_scale_exp(top);
  const float inv = exp2_neg(s);
  const size_t at = static_cast<size_t>(p) * I + n0 + 4 * tid;
  if (A4)
    *reinterpret_cast<uint16_t*>(hq + at / 2) =
        static_cast<uint16_t>(f32x4_to_e2m1x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(hq + at) = f32x4_to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
  if (tid == 0) hs[at / 32] = static_cast<uint8_t>(s + 127);
}

// Down and the weighted sum: workgroup = 8 output columns, a wave per pair in turn (the operand's
// rows 8 to 15 repeat them); then out[t] from the pairs' values in slot order.
template <bool A4>
__global__ __launch_bounds__(kPairWaves4 * kWave) void pairs_down_mx4(
    const uint8_t* __restrict__ hq, const uint8_t* __restrict__ hs, const uint8_t* __restrict__ wd,
    const uint8_t* __restrict__ wds, const int32_t* __restrict__ idx, const float* __restrict__ w, int H, int I,
    int E, int k, int P, uint16_t* __restrict__ out, uint32_t okey) {
  __shared__ __align__(16) float val[kPairsMax4 * kPairCols4];
  __shared__ float s_w[kPairsMax4];
  __shared__ bool s_on[kPairsMax4];
  __shared__ __align__(16) i32x4 s_tile[kPairWaves4][8 * 8];
  const int tid = threadIdx.x, ln = lane_id(), col = ln & 15, grp = ln >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(wave_id());
  const int n0 = permute_item(blockIdx.x, gridDim.x, okey) * kPairCols4;
  const int nchunk = I / 256, KB = I / 32;
  if (tid < P) {
    s_on[tid] = static_cast<unsigned>(idx[tid]) < static_cast<unsigned>(E);
    s_w[tid] = w[tid];
  }
  for (int p = wv; p < P; p += kPairWaves4) {
    const int e = idx[p];
    if (static_cast<unsigned>(e) >= static_cast<unsigned>(E)) continue;
    const size_t row = static_cast<size_t>(e) * H + n0;
    const uint8_t *x = hq + static_cast<size_t>(p) * (A4 ? I / 2 : I), *xs = hs + static_cast<size_t>(p) * KB;
    constexpr int U = 4;
    PairRows<A4, 8, U> r;
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < nchunk; c0 += U) {
      r.request(wd + row * (I / 2), wds + row * KB, I / 2, KB, c0, nchunk);
      d = r.times(x, xs, c0, nchunk, s_tile[wv], d);
    }
    if (col == 0 && grp < 2) *reinterpret_cast<f32x4*>(&val[p * kPairCols4 + 4 * grp]) = d;
  }
  __syncthreads();
  const int T = P / k;
  for (int i = tid; i < T * kPairCols4; i += kPairWaves4 * kWave) {
    const int t = i / kPairCols4, c = i % kPairCols4;
    float o = 0.f;
    for (int j = 0; j < k; ++j) {
      const int p = t * k + j;
      // (one slot: the weighted value itself, the sign of a zero included, as in the other forms)
      if (s_on[p]) o = k == 1 ? s_w[p] * val[p * kPairCols4 + c] : fmaf(s_w[p], val[p * kPairCols4 + c], o);
    }
    out[static_cast<size_t>(t) * H + n0 + c] = static_cast<uint16_t>(f32_to_bf16_rne(o));
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
  if (use_pairs4(T, H, I, E, k)) {
#define PAIRS4(A4)                                                                                \
  do {                                                                                            \
    prof_begin(kMx4GateUp, s);                                                                    \
    hipLaunchKernelGGL(pairs_gate_up_mx4<A4>, dim3(I / 32 * P), dim3(256), (A4 ? H / 2 : 2 * H) + H / 32, s, x, xs, \
                       wgu, wgus, idx, H, I, E, k, P, hq, hs, order_key());                       \
    prof_end(kMx4GateUp, s);                                                                      \
    prof_begin(kMx4Down, s);                                                                      \
    hipLaunchKernelGGL(pairs_down_mx4<A4>, dim3(H / kPairCols4), dim3(kPairWaves4 * kWave), 0, s, hq, hs, wd, wds, \
                       idx, w, H, I, E, k, P, out, order_key());                                  \
    prof_end(kMx4Down, s);                                                                        \
  } while (0)
    if (a4) PAIRS4(true);
    else PAIRS4(false);
#undef PAIRS4
    return hipGetLastError();
  }
  if (const hipError_t e = launch_group_experts(idx, P, E, L.bm, counts, offsets, tiles, n_tiles, perm, row_of, s);
      e != hipSuccess) return e;
  if (L.bm == kLargeBM) {
    float* partial = reinterpret_cast<float*>(b + L.partial);
    uint8_t *wgu_t = reinterpret_cast<uint8_t*>(b + L.wgu_t), *wd_t = reinterpret_cast<uint8_t*>(b + L.wd_t),
            *x_t = reinterpret_cast<uint8_t*>(b + L.x_t);
    // grid: every item whole, plus room for the tail slices (rem * S - rem < ncu)
    auto grid = [&](int nblk) { return dim3(round_up(nblk * L.max_tiles + num_cus, kXcds)); };
    const int ch = (H / 256 + 31) / 32, ci = (I / 256 + 31) / 32;
    const dim3 tgrid(E * (2 * I / 64) * ch + E * (H / 64) * ci + (P + 63) / 64 * ch);
#define LARGE4(A4, KD, A, AS, W, WS, Y, O, NBLK)                                                  \
  hipLaunchKernelGGL((gemm_large_mx4<KD, A4>), grid(NBLK), dim3(256), large4_lds<A4>() + kLSide, s, A, \
                     reinterpret_cast<const uint32_t*>(AS), W, reinterpret_cast<const uint32_t*>(WS), perm, \
                     tiles, n_tiles, counts, offsets, w, H, I, k, P, hq, hs, Y, O, partial, num_cus, order_key())
#define LAYER4(A4)                                                                                \
  do {                                                                                            \
    prof_begin(kMx4GateUp, s);                                                                    \
    hipLaunchKernelGGL(mx4_scales_t<A4>, tgrid, dim3(256), 0, s, reinterpret_cast<const uint2*>(wgus), \
                       reinterpret_cast<const uint2*>(wds), reinterpret_cast<const uint2*>(xs), perm, row_of, \
                       offsets, H, I, E, k, P, reinterpret_cast<uint2*>(wgu_t), reinterpret_cast<uint2*>(wd_t), \
                       reinterpret_cast<uint2*>(x_t), k == 1 ? out : nullptr, order_key());       \
    LARGE4(A4, kGateUp4, x, x_t, wgu, wgu_t, nullptr, nullptr, I / 128);                          \
    hipLaunchKernelGGL(gemm_large_mx4_fixup_gate_up<A4>, dim3(num_cus / 2 * 4), dim3(256), 0, s, tiles, n_tiles, \
                       counts, offsets, H, I, P, hq, hs, partial, num_cus, order_key());          \
    prof_end(kMx4GateUp, s);                                                                      \
    prof_begin(kMx4Down, s);                                                                      \
    if (k == 1) LARGE4(A4, kDownFused4, hq, hs, wd, wd_t, nullptr, out, H / 256);                 \
    else LARGE4(A4, kDown4, hq, hs, wd, wd_t, y, nullptr, H / 256);                               \
  } while (0)
    if (a4) LAYER4(true);
    else LAYER4(false);
#undef LAYER4
#undef LARGE4
#define FIXUP4(KD)                                                                                \
  hipLaunchKernelGGL(gemm_large_mx4_fixup_down<KD>, dim3(num_cus / 2 * 64), dim3(256), 0, s, perm, tiles, n_tiles, \
                     counts, offsets, w, H, I, y, out, partial, num_cus, order_key())
    if (k == 1) FIXUP4(kDownFused4);
    else FIXUP4(kDown4);
#undef FIXUP4
  } else {
    // 96-row tiles: R = 1 gives twice the workgroups where R = 2 would leave half of the CUs idle (us, R = 1 for
    // few / R = 2: E 8, H 4096, I 14336, 64 tokens 184 / 207; E 6, H 7168, I 2048, 256 tokens 62 / 78; with 192
    // tiles of the down product, E 8, H 2048, I 5632, 1024 tokens 135 / 126)
    // KEEP: from 64 rows an expert some have several tiles, and the caches keep the weights for the others (us,
    // streamed / kept, MXFP8: E 64, H 2048, I 768, 50 rows an expert 71 / 75, 75 rows 80 / 83, 100 rows 101 / 100;
    // E 64, H 4096, I 1024, 60 rows 166 / 161, 73 rows 179 / 169, 192 rows 341 / 296; E 16, H 2048, I 1024, 1024 rows
    // 191 / 176)
    const bool keep = P >= static_cast<int64_t>(64) * E;
    const int64_t each = P / (kTall4 * E) + 1;                // about as many tiles an expert
#define STREAM4_(KD, BM, R, KEEP, A4, A, AS, W, WS, Y, O, N)                                     \
  hipLaunchKernelGGL((gemm_mx4s<KD, BM, R, KEEP, A4>), dim3(round_up((N) / (128 * (R)) * L.max_tiles, kXcds)), \
                     dim3(256), 0, s, A, AS, W, WS, perm, tiles, n_tiles, counts, offsets, row_of, w, H, I, k, P, \
                     hq, hs, Y, O, order_key())
#define STREAM4R(KD, BM, R, KEEP, A, AS, W, WS, Y, O, N)                                         \
  do {                                                                                           \
    if (a4) STREAM4_(KD, BM, R, KEEP, true, A, AS, W, WS, Y, O, N);                              \
    else STREAM4_(KD, BM, R, KEEP, false, A, AS, W, WS, Y, O, N);                                \
  } while (0)
#define STREAM4(KD, A, AS, W, WS, Y, O, N)                                                       \
  do {                                                                                           \
    if (L.bm == kShort4) STREAM4R(KD, kShort4, 1, false, A, AS, W, WS, Y, O, N);                 \
    else if (each * E * ((N) / 256) <= 128) STREAM4R(KD, kTall4, 1, false, A, AS, W, WS, Y, O, N); \
    else if (keep) STREAM4R(KD, kTall4, 2, true, A, AS, W, WS, Y, O, N);                         \
    else STREAM4R(KD, kTall4, 2, false, A, AS, W, WS, Y, O, N);                                  \
  } while (0)
    prof_begin(kMx4GateUp, s);
    STREAM4(kGateUp4, x, xs, wgu, wgus, nullptr, k == 1 ? out : nullptr, 2 * I);
    prof_end(kMx4GateUp, s);
    prof_begin(kMx4Down, s);
    if (k == 1) STREAM4(kDownFused4, hq, hs, wd, wds, nullptr, out, H);
    else STREAM4(kDown4, hq, hs, wd, wds, y, nullptr, H);
#undef STREAM4
#undef STREAM4R
#undef STREAM4_
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && k > 1) e = launch_combine_slots(y, row_of, w, T, H, k, out, 0, H, H, s, num_cus);
  prof_end(kMx4Down, s);
  return e;
}

}  // namespace moe
