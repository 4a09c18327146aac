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
#include <type_traits>

#include "block.h"
#include "common.h"
#include "gemm_large.h"
#include "int8.h"
#include "tiles.h"

namespace moe {

namespace {

constexpr int kBM8 = 64;                           // rows (routed pairs) per M-tile
constexpr int kTall8 = 128;                        // experts averaging 40 rows and more
inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int round_up(int v, int m) { return (v + m - 1) / m * m; }

__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

enum { kGateUp8 = 0, kDown8 = 1, kDownFused8 = 2 };

// silu(g) u on the hardware's reciprocal (one unit in the last place): an exact division
// takes ten instructions more, and the 256-row tiles' epilogue is bound by them.  Every
// form uses this one, so a pair's activations have the same bits in all of them.
__device__ __forceinline__ float swiglu8(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Slices of a streaming product's reduction: where its tiles (nblk column blocks each)
// leave half the CUs or more without a workgroup, as many as those have room for, of at
// least three 256-code stages.  The slices' INT32 sums are exact and are added by the
// kernel that reads them next.  Measured, us (split / whole): T 100 H 7168 I 2048 E 4 k 2
// 64 / 87; T 40 H 4096 I 1024 E 6 k 4 37 / 47; T 14 H 2560 I 1792 E 5 k 5 39 / 45.  Room
// for half as many again: T 128 H 3584 I 1024 E 8 k 8 57 against 59, but T 809 H 3840 I 512
// E 4 k 2 68 against 55.  Slices of one stage: T 2000 H 1024 I 512 E 4 k 1 55 against 36
// whole; of two: T 40 H 4096 40 against 37 of three.
constexpr int kSplitGroups = 256, kSplitStages = 3;
inline int slices(size_t P, int E, int bm, int nblk, int nstage) {
  const size_t tiles = (P < static_cast<size_t>(E) ? P : E) + P / bm;   // (about; each expert ends one early)
  const size_t groups = tiles * nblk;                    // (0 for sizes that the layer refuses)
  const size_t room = groups ? kSplitGroups / groups : 1, most = nstage / kSplitStages;
  const size_t s = room < most ? room : most;
  return s < 2 ? 1 : static_cast<int>(s);
}
// Bytes that the slices of T k = P rows or fewer take, `row` bytes of INT32 sums each: at most
// `most` slices a row, and 2^25 bytes however many rows (slices * tiles * nblk <= 256, P <
// 128 * tiles, row = 1024 nblk for both products).  It does not fall as P grows, where the
// slices themselves come and go.
inline size_t slice_bytes(size_t P, int nstage, size_t row) {
  const size_t most = nstage / kSplitStages, cap = size_t(1) << 25;
  if (most < 2) return 0;
  const size_t rows = most * P;
  return row && rows > cap / row ? cap : rows * row;
}

}  // namespace

Int8Ws int8_ws_layout(int T, int H, int I, int E, int k) {
  Int8Ws L{};
  const size_t P = static_cast<size_t>(T) * k;
  // 256-row tiles where the products are bound by the matrix cores: 360 rows an expert,
  // tiles for half of the CUs, and reductions long enough to pay for a tile's start and
  // end.  Measured, us (256-row / 128-row tiles):
  //   H 7168 I 2048 E 6 k 1: 320 rows an expert 198 / 201, 400 208 / 239, 1500 532 / 713
  //   H 4096 I 1024 E 32 k 6: 320 rows 301 / 292, 400 326 / 378, 1500 1087 / 1312
  //   H 2048 I 768 E 64 k 8: 320 rows 279 / 261, 400 307 / 328, 1500 1070 / 1148
  //   H 1024 I 512 E 16 k 4: 400 rows 95 / 51, 1500 180 / 134
  //   H 4096 I 1024 E 4 k 2: 400 rows (50 tiles of gate/up) 99 / 68, 600 (75) 96 / 92, 1500 (187) 152 / 184
  // 128-row tiles from 40 rows an expert, where about half the experts would need two of
  // 64 rows (their weights streamed twice): H 4096 I 1024 E 64 k 6, 37 rows 200 / 200,
  // 73 rows 262 / 319 (128-row / 64-row).
  const bool mfma_bound = P >= 360 * static_cast<size_t>(E) && P / kLargeBM * (I / 128) >= 128 &&
                          static_cast<size_t>(H) * I >= (size_t(3) << 19);
  L.bm = mfma_bound ? kLargeBM : P >= 40 * static_cast<size_t>(E) ? kTall8 : kBM8;
  L.max_tiles = static_cast<int>(E + (P + L.bm - 1) / L.bm);
  const bool split = L.bm != kLargeBM;
  L.slices_gu = split ? slices(P, E, L.bm, I / 128, H / 256) : 1;
  L.slices_down = split ? slices(P, E, L.bm, H / 256, I / 256) : 1;
  // Each part holds what any smaller T takes, so that a workspace for the largest batch serves
  // every batch (tiles: as many as of the least rows).
  const size_t tile_room = E + (P + kBM8 - 1) / kBM8;
  size_t o = 0;
  L.n_tiles = o;   o += 256;
  L.counts = o;    o = align256(o + sizeof(int) * E);
  L.offsets = o;   o = align256(o + sizeof(int) * (E + 1));
  L.tiles = o;     o = align256(o + sizeof(int) * 2 * tile_room);
  L.perm = o;      o = align256(o + sizeof(int) * P);
  L.row_of = o;    o = align256(o + sizeof(int) * P);
  L.act = o;       o = align256(o + sizeof(float) * P * I);
  L.codes = o;     o = align256(o + P * I);
  L.scales = o;    o = align256(o + sizeof(float) * P);
  L.y = o;
  if (k > 1) o = align256(o + sizeof(float) * P * H);
  L.partial = o;
  const size_t gu = slice_bytes(P, H / 256, sizeof(int) * 2 * I), down = slice_bytes(P, I / 256, sizeof(int) * H);
  const size_t tail = L.bm == kLargeBM ? sizeof(int) * kLargeMaxSlices * kLargeBM * 256 : 0;
  o = align256(o + (tail > gu ? tail > down ? tail : down : gu > down ? gu : down));
  L.total = o;
  return L;
}

// Batched INT8 projections with a whole-line weight stream: workgroup = (M-tile of BM
// routed rows, NW waves), each wave owning two groups of 16 weight rows (gate_up: 16
// neurons' gate and up rows; down: 32 output channels).  A 128-position chunk of a row
// is 128 bytes: the wave reads its 32 rows as four loads of 8 rows x 128 contiguous
// bytes (non-temporal), passes them through a wave-private 2 KB LDS tile (16-byte
// chunks XOR-swizzled by row) and reads back two 16-byte operands of the 16x16x64
// MFMA: lane (r, g) takes chunks g and 4 + g of row r, of the weights and of the
// activations alike.  The activation codes are staged in LDS in stages of two chunks,
// double-buffered and shared by the waves; the weights of the next two chunks are in
// flight while one multiplies.  Rows past the tile's end load the tile's first row; their
// columns are computed and discarded.  Bound by the stream of weights and the latency of
// its way through LDS: 777 tokens, 64 experts, k 6, H 4096 I 1024 (73 rows an expert):
// gate/up 127 us (537 MB, 4.2 TB/s), down 76 us (268 MB of weights and 76 MB of slot
// values).  The 16 bytes of an operand straight from memory, without LDS, read half lines:
// 253 us for that layer instead of 226.  PART: the workgroup takes one of S slices of the
// reduction and stores its INT32 sums in part[S][P][weight rows of an expert].
template <int KIND, int NW, int BM, bool PART>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(BM == 64 ? 4 : 2, 8))) void gemm_i8s(
    const uint8_t* __restrict__ act, const float* __restrict__ acts,
    const uint8_t* __restrict__ wt, const float* __restrict__ wts,
    const int* __restrict__ perm, const int2* __restrict__ tiles, const int* __restrict__ n_tiles,
    const int* __restrict__ counts, const int* __restrict__ offsets, const float* __restrict__ w,
    int H, int I, int k, float* __restrict__ y, uint16_t* __restrict__ out, int P,
    int S, int* __restrict__ part, uint32_t okey) {
  constexpr int NT = NW * 64;
  constexpr bool GU = KIND == kGateUp8;
  constexpr int RPW = GU ? 16 : 32;                       // outputs per wave
  constexpr int G = BM / 16;                              // 16-row groups of the tile
  constexpr int SB = 256;                                 // bytes of a row per stage (two chunks)
  constexpr int RS = SB + 16;                             // padded LDS row stride
  constexpr int CH = SB / 16;                             // 16-byte pieces of a row per stage
  constexpr int LPT = BM * CH / NT;                       // 16-byte code loads per thread
  __shared__ __align__(16) uint8_t xl[2][BM * RS];
  __shared__ __align__(16) i32x4 wtl[NW][16 * 8];         // per wave: [16 rows][8 chunks]
  const int K = GU ? H : I;                               // reduction length
  const int N = GU ? I : H;                               // outputs
  const int nblk = N / (NW * RPW), nitem = PART ? nblk * S : nblk;
  const int item0 = real_item(blockIdx.x, nitem, *n_tiles);
  if (item0 < 0) return;
  const int item = permute_item(item0, nitem * *n_tiles, okey);
  const int tile = item / nitem, in_tile = item - tile * nitem;
  const int slice = PART ? in_tile / nblk : 0, nb_i = in_tile - slice * nblk;
  // the stages [st0, st0 + nstage) of the reduction
  const int st0 = PART ? slice * (K / SB) / S : 0;
  const int nstage = PART ? (slice + 1) * (K / SB) / S - st0 : K / SB, nchunk = 2 * nstage;
  const int2 te = tiles[tile];
  const int e = te.x, m0 = te.y;
  const int mcount = min(BM, counts[e] - m0);
  const int rbase = offsets[e] + m0;
  const int ng = __builtin_amdgcn_readfirstlane((mcount + 15) / 16);   // 16-row groups that hold rows
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
    ow[i] = static_cast<uint32_t>(((i < 2 ? row0 : row1) + 8 * (i & 1) + lr) * K + lc * 16 + st0 * SB);
  i32x4* tw = wtl[wv];
  i32x4* wdst = tw + lr * 8 + (lc ^ lr);                  // + 64 for rows 8-15
  const i32x4* asrc = tw + col * 8;
  const int sw = col & 7;

  uint32_t oxl[LPT];
  int lrow[LPT];
#pragma unroll
  for (int i = 0; i < LPT; ++i) {
    const int c = tid + i * NT, r = c / CH, rr = r < mcount ? r : 0;
    lrow[i] = r * RS + (c % CH) * 16;
    const int arow = GU ? perm[rbase + rr] / k : rbase + rr;
    oxl[i] = static_cast<uint32_t>(arow * K + (c % CH) * 16 + st0 * SB);
  }
  i32x4 xr[LPT], wA[4], wB[4];
#pragma unroll
  for (int i = 0; i < LPT; ++i) xr[i] = ld16(act + oxl[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) wA[i] = ld16_stream(wb + ow[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) wB[i] = ld16_stream(wb + ow[i] + 128);
  // the epilogue's data (tile row tid's pair and scale, output tid's weight scale): its
  // latency passes during the products, and it goes through LDS after them
  const float* ws_e = wts + static_cast<size_t>(e) * wrows;
  const int my_pr = PART ? 0 : perm[rbase + (tid < mcount ? tid : 0)];
  const float my_sx = PART ? 0.f : GU ? acts[my_pr / k] : acts[rbase + (tid < mcount ? tid : 0)];
  const int my_n = nb_i * NW * RPW;
  const float my_ws = !PART && tid < 32 * NW ? ws_e[GU && tid >= 16 * NW ? I + my_n + tid - 16 * NW : my_n + tid] : 0.f;
#pragma unroll
  for (int i = 0; i < LPT; ++i) *reinterpret_cast<i32x4*>(&xl[0][lrow[i]]) = xr[i];

  i32x4 acc0[G], acc1[G];
#pragma unroll
  for (int g = 0; g < G; ++g) acc0[g] = acc1[g] = i32x4{0, 0, 0, 0};
  __syncthreads();

  // One chunk: the weights through the wave's LDS tile into operands (both row groups
  // before the products, so that each activation operand is read once), the chunk
  // after next on its way into the registers they left, then the products.
  auto chunk = [&](i32x4 (&W)[4], int buf, int cc, int next) {
    const uint8_t* xcur = &xl[buf][col * RS + cc * 128 + 16 * grp];
    i32x4 a[4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      wdst[0] = W[2 * m];
      wdst[64] = W[2 * m + 1];
      __builtin_amdgcn_wave_barrier();
      a[2 * m] = asrc[grp ^ sw];
      a[2 * m + 1] = asrc[(4 + grp) ^ sw];
      __builtin_amdgcn_wave_barrier();
    }
    const uint32_t ko = static_cast<uint32_t>(min(next, nchunk - 1) * 128);   // (a harmless repeat past the end)
#pragma unroll
    for (int i = 0; i < 4; ++i) W[i] = ld16_stream(wb + ow[i] + ko);
    __builtin_amdgcn_sched_barrier(0);                    // (the compiler would sink the loads behind the products)
    i32x4 b[2][2];                                        // the next row group's operand is read a group ahead
    b[0][0] = *reinterpret_cast<const i32x4*>(xcur);
    b[0][1] = *reinterpret_cast<const i32x4*>(xcur + 64);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g && g >= ng) break;                            // (uniform: the tile has no rows there)
      if (g + 1 < G) {
        const uint8_t* p = xcur + (16 * (g + 1)) * RS;
        b[(g + 1) & 1][0] = *reinterpret_cast<const i32x4*>(p);
        b[(g + 1) & 1][1] = *reinterpret_cast<const i32x4*>(p + 64);
      }
      acc0[g] = mfma_i8(a[0], b[g & 1][0], acc0[g]);
      acc1[g] = mfma_i8(a[2], b[g & 1][0], acc1[g]);
      acc0[g] = mfma_i8(a[1], b[g & 1][1], acc0[g]);
      acc1[g] = mfma_i8(a[3], b[g & 1][1], acc1[g]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // activations of stage st + 1, on their way while stage st multiplies
  auto fetch = [&](int st) {
    if (st < nstage) {
#pragma unroll
      for (int i = 0; i < LPT; ++i) xr[i] = ld16(act + oxl[i] + st * SB);
    }
  };
  auto publish = [&](int st) {
    if (st < nstage) {
#pragma unroll
      for (int i = 0; i < LPT; ++i) *reinterpret_cast<i32x4*>(&xl[st & 1][lrow[i]]) = xr[i];
    }
    __syncthreads();
  };
  for (int st = 0; st < nstage; ++st) {                   // weights in wA and wB
    fetch(st + 1);
    chunk(wA, st & 1, 0, 2 * st + 2);
    chunk(wB, st & 1, 1, 2 * st + 3);
    publish(st + 1);
  }
  // lane: outputs row0 + 4grp + i (group 0) and row1 + 4grp + i (group 1) of tile row 16g + col
  if (PART) {
    int* pt = part + (static_cast<size_t>(slice) * P + rbase + col) * wrows + 4 * grp;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (16 * g + col >= mcount) continue;
      int* pr = pt + static_cast<size_t>(16 * g) * wrows;
      *reinterpret_cast<i32x4*>(pr + row0) = acc0[g];
      *reinterpret_cast<i32x4*>(pr + row1) = acc1[g];
    }
    return;
  }
  int* s_pr = reinterpret_cast<int*>(xl[0]);              // (every wave is done with the stages)
  float* s_sx = reinterpret_cast<float*>(xl[0]) + BM;
  float* s_ws = reinterpret_cast<float*>(xl[0]) + 2 * BM;
  if (tid < BM) {
    s_pr[tid] = my_pr;
    s_sx[tid] = my_sx;
  }
  if (tid < 32 * NW) s_ws[tid] = my_ws;
  __syncthreads();
  const int c0 = wv * RPW + 4 * grp;
  const f32x4 s0 = *reinterpret_cast<const f32x4*>(s_ws + c0);
  const f32x4 s1 = *reinterpret_cast<const f32x4*>(s_ws + c0 + (GU ? 16 * NW : 16));
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int r = 16 * g + col;
    if (r >= mcount) continue;
    const int pr = s_pr[r];
    const float sx = s_sx[r];
    f32x4 v0, v1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v0[i] = static_cast<float>(acc0[g][i]) * sx * s0[i];
      v1[i] = static_cast<float>(acc1[g][i]) * sx * s1[i];
    }
    if (GU) {
      f32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = swiglu8(v0[i], v1[i]);
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
      *reinterpret_cast<f32x4*>(yr) = v0;                 // (read back by the slot sum: plain stores, 1% faster)
      *reinterpret_cast<f32x4*>(yr + 16) = v1;
    }
  }
}

// ---------------------------------------------------------------------------
// Large groups (360 routed rows per expert and more on average): the products are
// bound by the matrix cores, and run as an LDS-tiled GEMM.  Workgroup tile 256 rows
// x 256 weight rows (gate_up: 128 gate + 128 up rows of one expert, so that the
// epilogue finds g and u in one lane), K in stages of 128 codes; 4 waves of 128 x
// 128 with v_mfma_i32_32x32x32_i8, accumulators in AGPRs; both tiles staged in LDS
// (2 stages x 2 x 32 KB, 16-byte chunks XOR-swizzled by row), global loads one
// stage ahead of the LDS writes, which run one stage ahead of the fragment reads.
// Lane (l32, hi) takes 16-byte chunk 2 ks + hi of its row at K step ks, of both
// operands.  16384 rows, 6 experts, H 7168 I 2048: gate/up 460 us (2.09 POP/s), down 302
// us (1.59 POP/s: 16 stages a tile, its start and its stores not hidden by products).
// Workgroups that keep their CU and load the next tile's first stages during a tile's
// last ones: gate/up level, down 79 -> 90 us at 8000 rows, 4 experts (the loads wait
// behind the stores).
namespace {
constexpr int k8BK = 128;                                // K per stage
constexpr int k8Tile = kLargeBM * k8BK;                  // bytes per operand stage
constexpr int k8Stages = 2 * 2 * k8Tile;                 // 128 KB
constexpr size_t k8Lds = k8Stages + 3 * 4 * kLargeBM;    // and the rows' scales, pair ids and weights
typedef int i32x16 __attribute__((__vector_size__(16 * sizeof(int))));

__device__ __forceinline__ i32x16 mfma32_i8(i32x4 a, i32x4 b, i32x16 c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

// Two lanes that hold neighbouring columns (even, odd) and the values of two rows
// (v0, v1) exchange one value each: the even lane returns both columns of the first
// row, the odd lane both of the second, as two BF16 (the lower column in the low half).
__device__ __forceinline__ uint32_t pair_rows_bf16(float v0, float v1, int odd) {
  const float give = odd ? v0 : v1;
  const float got = __int_as_float(__builtin_amdgcn_update_dpp(
      0, __float_as_int(give), 0xB1, 0xF, 0xF, true));            // quad_perm [1,0,3,2]
  return odd ? pack_bf16x2(got, v1) : pack_bf16x2(v0, got);
}
}  // namespace

template <int KIND>
__global__ __launch_bounds__(256) void gemm_large_i8(
    const uint8_t* __restrict__ act, const float* __restrict__ acts,
    const uint8_t* __restrict__ wt, const float* __restrict__ wts, const int* __restrict__ perm,
    const int2* __restrict__ tiles, const int* __restrict__ n_tiles,
    const int* __restrict__ counts, const int* __restrict__ offsets, const float* __restrict__ w,
    int H, int I, int k, float* __restrict__ y, uint16_t* __restrict__ out,
    int* __restrict__ partial, int ncu, uint32_t okey) {
  extern __shared__ __align__(16) uint8_t lds8[];        // [stage][A, B][256 x 128]
  constexpr bool GU = KIND == kGateUp8;
  const int K = GU ? H : I;
  const int nblk = GU ? I / 128 : H / 256;
  const int nk = K / k8BK;
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

  // loader: thread covers tile rows wv*64 + 8j + (ln >> 3), j = 0..7, of both operands,
  // 16-byte chunk ln & 7 of each 128-byte row segment
  const int lrow = ln >> 3, lc = ln & 7;
  const size_t wrows = GU ? 2 * static_cast<size_t>(I) : static_cast<size_t>(H);
  const uint8_t* __restrict__ abase = wt + static_cast<size_t>(e) * wrows * K;
  const int arow = GU ? (wv < 2 ? n0 + wv * 64 : I + n0 + (wv - 2) * 64) : nb * 256 + wv * 64;
  const uint32_t ao = static_cast<uint32_t>((arow + lrow) * K + lc * 16);
  uint32_t bo[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = wv * 64 + 8 * j + lrow;
    const int rr = r < mcount ? r : 0;
    bo[j] = static_cast<uint32_t>((GU ? perm[rbase + rr] / k : rbase + rr) * K + lc * 16);
  }
  // LDS: row r, chunk c at r*128 + ((c ^ ((r >> 1) & 7)) * 16): the 16 rows that a read
  // serves at once then lie in 64 different banks (two rows span them all, so rows r and
  // r + 2 must differ); of a thread's rows 8j + lrow the odd j's chunk is c ^ 4
  const int lw0 = (wv * 64 + lrow) * k8BK + ((lc ^ (lrow >> 1)) * 16);
  const int lw1 = lw0 ^ 64;
  int fa[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    fa[i] = ((GU ? (i >> 1) * 128 + wn * 64 + (i & 1) * 32 : wn * 128 + 32 * i) + l32) * k8BK;
  const int fb = (wm * 128 + l32) * k8BK;
  const int swz = (l32 >> 1) & 7;

  i32x4 stg[16];   // [0..7] weight rows, [8..15] activation rows
  // (past the end the last stage again)
#define GLOAD(Q, KT) do {                                                               \
    const uint32_t kk_ = static_cast<uint32_t>(min((KT), ke - 1) * k8BK);               \
    if ((Q) < 8) stg[Q] = ld16(abase + ao + static_cast<uint32_t>((Q) * 8) * K + kk_);  \
    else stg[Q] = ld16(act + bo[(Q) - 8] + kk_);                                        \
  } while (0)
#define LWRITE(Q, KT) do {                                                              \
    uint8_t* st_ = lds8 + ((KT) & 1) * 2 * k8Tile + ((Q) < 8 ? 0 : k8Tile);             \
    *reinterpret_cast<i32x4*>(&st_[((Q) & 1 ? lw1 : lw0) + ((Q) & 7) * 8 * k8BK]) = stg[Q]; \
  } while (0)
#define RDF(PTR) (*reinterpret_cast<const i32x4*>(PTR))
  // One MFMA K step on fragments (A, B): 8 groups of 2 MFMAs; groups 0..3 then read
  // fragments A g and B g of the next K step (stage RKT, step RKS) and write staged
  // chunk Q0+g of stage WKT to LDS and reload it from stage WKT+1.  sched_barrier
  // keeps this order.
#define PHASE(A, B, NA, NB, RKT, RKS, WKT, Q0) do {                                     \
    const uint8_t* at_ = lds8 + ((RKT) & 1) * 2 * k8Tile;                               \
    const uint8_t* bt_ = at_ + k8Tile;                                                  \
    const int so_ = (((2 * (RKS) + hi) ^ swz) * 16);                                    \
    _Pragma("unroll") for (int g = 0; g < 8; ++g) {                                     \
      const int i_ = g >> 1, j0_ = (g & 1) * 2;                                         \
      acc[i_][j0_] = mfma32_i8(B[j0_], A[i_], acc[i_][j0_]);                            \
      acc[i_][j0_ + 1] = mfma32_i8(B[j0_ + 1], A[i_], acc[i_][j0_ + 1]);                \
      __builtin_amdgcn_sched_barrier(0);                                                \
      if (g < 4) {                                                                      \
        NA[g] = RDF(&at_[fa[g] + so_]);                                                 \
        NB[g] = RDF(&bt_[fb + 32 * g * k8BK + so_]);                                    \
        LWRITE((Q0) + g, WKT);                                                          \
        GLOAD((Q0) + g, (WKT) + 1);                                                     \
      }                                                                                 \
      __builtin_amdgcn_sched_barrier(0);                                                \
    }                                                                                   \
  } while (0)

  // The LDS writes of stage s+1 are spread over the four K steps that may write its
  // buffer: the last step of stage s-1 (chunks 12..15, after the barrier that ends
  // the reads of stage s-1) and the first three of stage s (chunks 0..11, before the
  // barrier that publishes stage s+1).
#pragma unroll
  for (int q = 0; q < 16; ++q) GLOAD(q, kb);
#pragma unroll
  for (int q = 0; q < 16; ++q) LWRITE(q, kb);
#pragma unroll
  for (int q = 0; q < 16; ++q) GLOAD(q, kb + 1);
#pragma unroll
  for (int q = 12; q < 16; ++q) { LWRITE(q, kb + 1); GLOAD(q, kb + 2); }
  __syncthreads();
  i32x4 a0[4], b0[4], a1[4], b1[4];
  {
    const uint8_t* at = lds8 + (kb & 1) * 2 * k8Tile;
    const int so = (hi ^ swz) * 16;
#pragma unroll
    for (int g = 0; g < 4; ++g) a0[g] = RDF(&at[fa[g] + so]);
#pragma unroll
    for (int g = 0; g < 4; ++g) b0[g] = RDF(&at[k8Tile + fb + 32 * g * k8BK + so]);
  }
  // the epilogue's data (tile row tid's scale, pair and weight; the columns' scales),
  // requested here: its latency passes during the products
  const int my_row = rbase + min(tid, mcount - 1);
  const int my_pr = perm[my_row];
  float my_sx = 0.f, my_w = 0.f;
  float ws[4];
  const float* wse = wts + static_cast<size_t>(e) * wrows;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    ws[i] = wse[GU ? (i >> 1) * I + n0 + wn * 64 + (i & 1) * 32 + l32 : nb * 256 + wn * 128 + 32 * i + l32];
  i32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
  for (int kt = kb; kt < ke; ++kt) {
    PHASE(a0, b0, a1, b1, kt, 1, kt + 1, 0);
    PHASE(a1, b1, a0, b0, kt, 2, kt + 1, 4);
    PHASE(a0, b0, a1, b1, kt, 3, kt + 1, 8);
    // stage kt+1 is in LDS for every wave, and every wave is done reading stage kt
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    // In the loop on purpose: a loop of one basic block keeps a copy of the accumulators
    // outside the AGPRs for the code after it, made again every stage (16384 rows, 6
    // experts 929 us instead of 848).
    if (kt == kb) {
      my_sx = GU ? acts[my_pr / k] : acts[my_row];
      if (KIND == kDownFused8) my_w = w[my_pr];          // k = 1: pair id == token
    }
    PHASE(a1, b1, a0, b0, kt + 1, 0, kt + 2, 12);
  }
  if (slot >= 0) {
    // tail slice: INT32 partial tile in register order, [64 x i32x4][256 threads]
    i32x4* pp = reinterpret_cast<i32x4*>(partial) + static_cast<size_t>(slot) * 64 * 256 + tid;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
        for (int q = 0; q < 4; ++q)
          pp[((i * 4 + j) * 4 + q) * 256] =
              i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      }
    return;
  }
  // Lane (l32, hi), register 4q + t of block (i, j): output column l32 of weight block
  // i, tile row 8q + 4hi + t of row block j - a store instruction writes 128
  // consecutive bytes of two rows (FP32), or 64 of four (BF16, columns paired over
  // lanes).  The rows' scales, pair ids and weights go through LDS, four rows a read.
  float* s_sx = reinterpret_cast<float*>(lds8 + k8Stages);
  int* s_pr = reinterpret_cast<int*>(lds8 + k8Stages) + kLargeBM;
  float* s_w = reinterpret_cast<float*>(lds8 + k8Stages) + 2 * kLargeBM;
  s_sx[tid] = my_sx;
  s_pr[tid] = my_pr;
  s_w[tid] = my_w;
  __syncthreads();
  // whole tiles (the most of them) without the checks of each row
  auto store = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q == 0)                                      // (read from the AGPRs here, not all at once: 876 -> 848 us)
#pragma unroll
          for (int i = 0; i < 4; ++i) asm volatile("" : "+a"(acc[i][j]));
        __builtin_amdgcn_sched_barrier(0);               // (one group of rows at a time: fewer registers live)
        const int r0 = wm * 128 + 32 * j + 8 * q + 4 * hi;
        if (!kWhole && r0 >= mcount) continue;
        const f32x4 sx = *reinterpret_cast<const f32x4*>(s_sx + r0);
        if (KIND == kDownFused8) {
          const i32x4 pr = *reinterpret_cast<const i32x4*>(s_pr + r0);
          const f32x4 wt4 = *reinterpret_cast<const f32x4*>(s_w + r0);
          const int odd = l32 & 1;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint16_t* orow = out + static_cast<size_t>(odd ? pr[2 * h + 1] : pr[2 * h]) * H + nb * 256 + wn * 128 + l32 - odd;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v[2];
#pragma unroll
              for (int t = 0; t < 2; ++t)
                v[t] = wt4[2 * h + t] * (static_cast<float>(acc[i][j][4 * q + 2 * h + t]) * sx[2 * h + t] * ws[i]);
              const uint32_t o = pair_rows_bf16(v[0], v[1], odd);   // (both lanes of a pair take part)
              if (kWhole || r0 + 2 * h + odd < mcount) *reinterpret_cast<uint32_t*>(orow + 32 * i) = o;
            }
          }
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            if (!kWhole && r0 + t >= mcount) continue;
            float* yr = y + static_cast<size_t>(rbase + r0 + t) * (GU ? I : H) +
                        (GU ? n0 + wn * 64 : nb * 256 + wn * 128) + l32;
#pragma unroll
            for (int i = 0; i < (GU ? 2 : 4); ++i) {
              const float v = static_cast<float>(acc[i][j][4 * q + t]) * sx[t] * ws[i];
              yr[32 * i] = GU ? swiglu8(v, static_cast<float>(acc[(i + 2) & 3][j][4 * q + t]) * sx[t] * ws[(i + 2) & 3]) : v;
            }
          }
        }
      }
  };
  if (mcount == kLargeBM) store(std::true_type{});
  else store(std::false_type{});
#undef GLOAD
#undef LWRITE
#undef RDF
#undef PHASE
}

// Tail fix-up, element-parallel: thread g of the grid takes one i32x4 of the partial
// tile of tail item full + g / per_item (register order of the GEMM's thread), adds it
// over the S slices and applies that piece of the epilogue.
template <int KIND>
__global__ __launch_bounds__(256) void gemm_large_i8_fixup(
    const float* __restrict__ acts, const float* __restrict__ wts, const int* __restrict__ perm,
    const int2* __restrict__ tiles, const int* __restrict__ n_tiles,
    const int* __restrict__ counts, const int* __restrict__ offsets, const float* __restrict__ w,
    int H, int I, int k, float* __restrict__ y, uint16_t* __restrict__ out,
    const int* __restrict__ partial, int ncu, uint32_t okey) {
  constexpr bool GU = KIND == kGateUp8;
  constexpr int kPerItem = GU ? 32 * 256 : 64 * 256;     // threads per tail item
  const int nblk = GU ? I / 128 : H / 256;
  const TailPlan plan = tail_plan(nblk * *n_tiles, ncu, (GU ? H : I) / k8BK);
  const int g = permute_item(blockIdx.x, gridDim.x, okey) * 256 + threadIdx.x;
  const int b = g / kPerItem;
  if (plan.S == 1 || b >= plan.rem) return;
  const int f = g - b * kPerItem;                        // i32x4 index within the tile
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
  const i32x4* pp = reinterpret_cast<const i32x4*>(partial) + f;
  i32x4 a = {0, 0, 0, 0}, u = {0, 0, 0, 0};
  for (int sl = 0; sl < plan.S; ++sl) {
    const size_t base = static_cast<size_t>(sl * plan.rem + b) * 64 * 256;
    a += pp[base];
    if (GU) u += pp[base + 2 * 16 * 256];                // up block i + 2
  }
  const int n = (GU ? nb * 128 + wn * 64 : nb * 256 + wn * 128) + 32 * i + l32;
  const float* wse = wts + static_cast<size_t>(e) * (GU ? 2 * static_cast<size_t>(I) : static_cast<size_t>(H));
  const float wa = wse[n], wu = GU ? wse[I + n] : 0.f;
  for (int t = 0; t < 4 && r0 + t < mcount; ++t) {
    const int row = rbase + r0 + t, pr = perm[row];
    const float sx = GU ? acts[pr / k] : acts[row];
    const float v = static_cast<float>(a[t]) * sx * wa;
    if (GU) y[static_cast<size_t>(row) * I + n] = swiglu8(v, static_cast<float>(u[t]) * sx * wu);
    else if (KIND == kDownFused8) out[static_cast<size_t>(pr) * H + n] = static_cast<uint16_t>(f32_to_bf16_rne(w[pr] * v));
    else y[static_cast<size_t>(row) * H + n] = v;
  }
}

hipError_t int8_set_attributes() {
  const int bytes = static_cast<int>(k8Lds);
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(gemm_large_i8<kGateUp8>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess)
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(gemm_large_i8<kDown8>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess)
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(gemm_large_i8<kDownFused8>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e;
}

// What joins the slices of a product: part[S][P][N] INT32 and the scales of both operands.
struct Int8Parts {
  const int* part;
  int S, k;
  const int* perm;
  const int32_t* idx;
  const float *acts, *wts;
};

// Codes and scales of the FP32 activations, one grouped row per workgroup (I a
// multiple of 256, at most 1024 NV), the row in registers between its one read and its
// write (PART: made here from the slices of a split gate/up product).  16384 x 2048: 31 us
// (134 MB read, 34 written, 5.4 TB/s).  With k = 1 a pair without a row (expert id out of range) gets its output row
// cleared here, as no down tile will write it.
template <int NV, bool PART>
__global__ __launch_bounds__(256) void quant_act_rows(const float* __restrict__ a,
                                                      const Int8Parts sum,
                                                      const int* __restrict__ offsets, int E,
                                                      const int* __restrict__ row_of, int P, int H,
                                                      int I, uint8_t* __restrict__ codes,
                                                      float* __restrict__ scales,
                                                      uint16_t* __restrict__ out, uint32_t okey) {
  __shared__ float red[4];
  const int b = permute_item(blockIdx.x, P, okey);
  const float* row = a + static_cast<size_t>(b) * I;
  const int tid = threadIdx.x;
  f32x4 v[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {                          // (rows of the workspace: in bounds for every b < P)
    const int c = 4 * (u * 256 + tid);
    v[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!PART && c < I) v[u] = *reinterpret_cast<const f32x4*>(row + c);
  }
  if (out && row_of[b] >= P)
    for (int c = tid; c < H / 8; c += 256) st16(out + static_cast<size_t>(b) * H + 8 * c, i32x4{0, 0, 0, 0});
  if (b >= offsets[E]) return;
  if (PART) {
    const int pr = sum.perm[b];
    const float sx = sum.acts[pr / sum.k];
    const float* ws = sum.wts + static_cast<size_t>(sum.idx[pr]) * 2 * I;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = 4 * (u * 256 + tid);
      if (c >= I) continue;
      const f32x4 sg = *reinterpret_cast<const f32x4*>(ws + c), su = *reinterpret_cast<const f32x4*>(ws + I + c);
      i32x4 g = {0, 0, 0, 0}, up = {0, 0, 0, 0};
      const int* p = sum.part + static_cast<size_t>(b) * 2 * I + c;
#pragma unroll 4
      for (int sl = 0; sl < sum.S; ++sl, p += static_cast<size_t>(P) * 2 * I) {
        g += *reinterpret_cast<const i32x4*>(p);
        up += *reinterpret_cast<const i32x4*>(p + I);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[u][i] = swiglu8(static_cast<float>(g[i]) * sx * sg[i], static_cast<float>(up[i]) * sx * su[i]);
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int u = 0; u < NV; ++u)
    amax = fmaxf(fmaxf(fmaxf(amax, fabsf(v[u][0])), fabsf(v[u][1])), fmaxf(fabsf(v[u][2]), fabsf(v[u][3])));
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m, kWave));
  if (lane_id() == 0) red[wave_id()] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float inv = int8_inverse(amax);
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = 4 * (u * 256 + tid);
    if (c < I)
      *reinterpret_cast<uint32_t*>(codes + static_cast<size_t>(b) * I + c) =
          int8_codes4(v[u][0], v[u][1], v[u][2], v[u][3], inv);
  }
  if (tid == 0) scales[b] = int8_scale(amax);
}

// Slot sum over the slices of a split down product: the same values and the same order as
// one product and combine_slots (with k = 1 the weighted value itself, its sign included).
__global__ __launch_bounds__(256) void combine_parts(const Int8Parts sum, const int* __restrict__ row_of,
                                                     const float* __restrict__ w, int T, int H,
                                                     uint16_t* __restrict__ out, uint32_t okey) {
  const int t = permute_item(blockIdx.x, gridDim.x, okey);
  const int k = sum.k, P = T * k;
  const int c = blockIdx.y * 1024 + 4 * threadIdx.x;
  if (c >= H) return;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < k; j0 += 8) {                     // eight slots' loads in flight, then their sum in order
    i32x4 v[8], next[8];
    float wj[8], sh[8];
    f32x4 sd[8];
    const int* p[8];
    bool in[8];
    // (loads without conditions, which would wait for each: a slot without a row, or past the
    // last, reads row 0 and is left out below)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int pr = t * k + min(j0 + j, k - 1), row = row_of[pr], e = sum.idx[pr];
      const bool any = static_cast<unsigned>(row) < static_cast<unsigned>(P);
      in[j] = any && j0 + j < k;
      wj[j] = w[pr];
      sh[j] = sum.acts[any ? row : 0];
      sd[j] = *reinterpret_cast<const f32x4*>(sum.wts + static_cast<size_t>(any ? e : 0) * H + c);
      p[j] = sum.part + static_cast<size_t>(any ? row : 0) * H + c;
      v[j] = *reinterpret_cast<const i32x4*>(p[j]);
    }
    for (int sl = 1; sl < sum.S; ++sl) {
#pragma unroll
      for (int j = 0; j < 8; ++j) next[j] = *reinterpret_cast<const i32x4*>(p[j] + static_cast<size_t>(sl) * P * H);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += next[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (in[j]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = static_cast<float>(v[j][i]) * sh[j] * sd[j][i];
          acc[i] = k == 1 ? wj[j] * y : fmaf(wj[j], y, acc[i]);
        }
      }
  }
  uint2 o;
  o.x = pack_bf16x2(acc[0], acc[1]);
  o.y = pack_bf16x2(acc[2], acc[3]);
  *reinterpret_cast<uint2*>(out + static_cast<size_t>(t) * H + c) = o;
}

// ---------------------------------------------------------------------------
// Few pairs (a decode step): two launches, every routed pair on its own, its weights
// straight from HBM into v_dot4 operands.  A wave reads 8 weight rows x 128
// contiguous bytes a load, lane (row ln >> 3, 16-byte chunk ln & 7), and keeps up to
// 16 such loads in flight: the step is bound by the latency of its two dependent
// passes over memory, not by arithmetic, and needs no grouping.  Pairs that share an
// expert read its weights from the L2 the second time.  One token, k 8, H 2048 I 768:
// 6.4 us (25 MB) and 7.0 us (13 MB).
namespace {
// Dot product of 16 codes with 16 codes, added to c.
__device__ __forceinline__ int dot16(i32x4 a, i32x4 b, int c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_sdot4(a[i], b[i], c, false);
  return c;
}
// Sum over the 8 lanes of a row (ln & 7), on each of them.
__device__ __forceinline__ int sum8(int v) {
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}
// Dot products of 8 weight rows (lane (ln >> 3, ln & 7): wrow = its row + 16 (ln & 7))
// with the codes at x + 16 (ln & 7), K a multiple of 128: U loads of each in flight.
template <int U>
__device__ __forceinline__ int rows_dot(const uint8_t* wrow, const uint8_t* x, int K) {
  int acc = 0;
  for (int k0 = 0; k0 < K; k0 += 128 * U) {
    i32x4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + 128 * u < K) a[u] = ld16_stream(wrow + k0 + 128 * u);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + 128 * u < K) b[u] = *reinterpret_cast<const i32x4*>(x + k0 + 128 * u);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + 128 * u < K) acc = dot16(a[u], b[u], acc);
  }
  return sum8(acc);
}
constexpr int kPairsMax = 48;                            // pairs up to which this form may be taken
constexpr size_t kPairsLds = 64 << 10;                   // LDS that a kernel may use without an attribute
constexpr int kPairCols = 8;                             // output columns per workgroup of the down pass
constexpr int kPairWaves = 8;
inline size_t pairs_lds(int P, int I) {
  return static_cast<size_t>(kPairWaves) * I + sizeof(float) * kPairCols * P;
}
// Taken while the weights that it reads more than once (pairs that share an expert;
// expected number of distinct experts E (1 - (1 - k/E)^T)) stay below 120 MB: about
// the 20 us that grouping and its launches cost the other form; and for 48 pairs at
// most, which a wave of the down pass takes eight apart, one after the other.  Measured,
// us (this / grouped): H 2048 I 768 E 128 k 8, T 1 13.8 / 27.4, T 8 (64 pairs) 60 / 61,
// T 12 86 / 70; H 7168 I 2048 E 32 k 4, T 2 71 / 70, T 4 (122 MB) 124 / 106; H 2048 I 1024
// E 8 k 2, T 12 (102 MB) 25 / 30; H 1024 I 512 E 8 k 2, T 20 18.5 / 23.5, T 30 (60 pairs)
// 25.0 / 23.4; H 768 I 512 E 64 k 8, T 12 (96 pairs) 44 / 27.
inline bool use_pairs(int T, int H, int I, int E, int k) {
  const int64_t P = static_cast<int64_t>(T) * k;
  if (P > kPairsMax || pairs_lds(static_cast<int>(P), I) > kPairsLds) return false;
  double miss = 1.0;                                     // (1 - k/E)^T
  for (int t = 0; t < T; ++t) miss *= 1.0 - static_cast<double>(k) / E;
  const double again = static_cast<double>(P) - E * (1.0 - miss);
  return again * 3.0 * H * I <= 120e6;
}
}  // namespace

// Gate/up and SwiGLU: workgroup (pair, 16 neurons); waves 0, 1 the gate rows, 2, 3 the
// up rows.  a[pair][I] FP32.
__global__ __launch_bounds__(256) void pairs_gate_up(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, const uint8_t* __restrict__ wgu,
    const float* __restrict__ wgus, const int32_t* __restrict__ idx, int H, int I, int E, int k,
    int P, float* __restrict__ a, uint32_t okey) {
  __shared__ int s_dot[32];
  const int nblk = I / 16;
  const int item = permute_item(blockIdx.x, nblk * P, okey);
  const int p = item / nblk, n0 = (item - p * nblk) * 16;
  const int e = idx[p];
  if (static_cast<unsigned>(e) >= static_cast<unsigned>(E)) return;
  const int t = p / k, ln = lane_id(), wv = wave_id();
  const int row = (wv >> 1) * I + n0 + (wv & 1) * 8 + (ln >> 3);
  const int d = rows_dot<16>(wgu + static_cast<size_t>(e) * 2 * I * H + static_cast<uint32_t>(row) * H + 16 * (ln & 7),
                             x + static_cast<size_t>(t) * H + 16 * (ln & 7), H);
  if ((ln & 7) == 0) s_dot[wv * 8 + (ln >> 3)] = d;
  __syncthreads();
  const int c = threadIdx.x;
  if (c < 16) {
    const float sx = xs[t];
    const float* ws = wgus + static_cast<size_t>(e) * 2 * I + n0 + c;
    const float g = static_cast<float>(s_dot[c]) * sx * ws[0];
    const float u = static_cast<float>(s_dot[16 + c]) * sx * ws[I];
    a[static_cast<size_t>(p) * I + n0 + c] = swiglu8(g, u);
  }
}

// Down and the weighted sum: workgroup = 8 output columns, a wave per pair in turn (its
// activations' codes in the wave's I bytes of LDS, made from a[pair] by the wave
// itself); then out[t] from the pairs' values in slot order.
__global__ __launch_bounds__(kPairWaves * kWave) void pairs_down(
    const float* __restrict__ a, const uint8_t* __restrict__ wd, const float* __restrict__ wds,
    const int32_t* __restrict__ idx, const float* __restrict__ w, int H, int I, int E, int k, int P,
    uint16_t* __restrict__ out, uint32_t okey) {
  extern __shared__ __align__(16) uint8_t lds8[];        // [wave][I] codes, then [P][8] values
  float* val = reinterpret_cast<float*>(lds8 + kPairWaves * I);
  const int ln = lane_id(), wv = wave_id();
  const int n0 = permute_item(blockIdx.x, gridDim.x, okey) * kPairCols;
  uint8_t* codes = lds8 + wv * I;
  for (int p = wv; p < P; p += kPairWaves) {
    const int e = idx[p];
    if (static_cast<unsigned>(e) >= static_cast<unsigned>(E)) continue;
    const float* row = a + static_cast<size_t>(p) * I;
    const uint8_t* wrow = wd + static_cast<size_t>(e) * H * I + static_cast<uint32_t>(n0 + (ln >> 3)) * I + 16 * (ln & 7);
    // the first 16 loads of the weights, in flight while the codes are made
    i32x4 wr[16];
#pragma unroll
    for (int u = 0; u < 16; ++u)
      if (128 * u < I) wr[u] = ld16_stream(wrow + 128 * u);
    f32x4 v[8];                                          // the first 2048 activations
    float amax = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = 4 * (u * kWave + ln);
      v[u] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (c < I) v[u] = *reinterpret_cast<const f32x4*>(row + c);
      amax = fmaxf(fmaxf(fmaxf(amax, fabsf(v[u][0])), fabsf(v[u][1])), fmaxf(fabsf(v[u][2]), fabsf(v[u][3])));
    }
    for (int c = 2048 + 4 * ln; c < I; c += 4 * kWave) {
      const f32x4 z = *reinterpret_cast<const f32x4*>(row + c);
      amax = fmaxf(fmaxf(fmaxf(amax, fabsf(z[0])), fabsf(z[1])), fmaxf(fabsf(z[2]), fabsf(z[3])));
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m, kWave));
    const float inv = int8_inverse(amax);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = 4 * (u * kWave + ln);
      if (c < I) *reinterpret_cast<uint32_t*>(codes + c) = int8_codes4(v[u][0], v[u][1], v[u][2], v[u][3], inv);
    }
    for (int c = 2048 + 4 * ln; c < I; c += 4 * kWave) {
      const f32x4 z = *reinterpret_cast<const f32x4*>(row + c);
      *reinterpret_cast<uint32_t*>(codes + c) = int8_codes4(z[0], z[1], z[2], z[3], inv);
    }
    // the wave's own codes: its LDS operations complete in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    int acc = 0;
#pragma unroll
    for (int u = 0; u < 16; ++u)
      if (128 * u < I) acc = dot16(wr[u], *reinterpret_cast<const i32x4*>(codes + 128 * u + 16 * (ln & 7)), acc);
    acc = sum8(acc);
    if (I > 2048) acc += rows_dot<16>(wrow + 2048, codes + 2048 + 16 * (ln & 7), I - 2048);
    if ((ln & 7) == 0) {
      const int c = ln >> 3;
      val[p * kPairCols + c] = static_cast<float>(acc) * int8_scale(amax) * wds[static_cast<size_t>(e) * H + n0 + c];
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  const int T = P / k;
  for (int i = threadIdx.x; i < T * kPairCols; i += blockDim.x) {
    const int t = i / kPairCols, c = i % kPairCols;
    float o = 0.f;
    for (int j = 0; j < k; ++j) {
      const int p = t * k + j;
      // (one slot: the weighted value itself, the sign of a zero included, as in the other forms)
      if (static_cast<unsigned>(idx[p]) < static_cast<unsigned>(E))
        o = k == 1 ? w[p] * val[p * kPairCols + c] : fmaf(w[p], val[p * kPairCols + c], o);
    }
    out[static_cast<size_t>(t) * H + n0 + c] = static_cast<uint16_t>(f32_to_bf16_rne(o));
  }
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
  const uint8_t* x8 = reinterpret_cast<const uint8_t*>(x);
  const uint8_t* wgu8 = reinterpret_cast<const uint8_t*>(wgu);
  const uint8_t* wd8 = reinterpret_cast<const uint8_t*>(wd);
  if (use_pairs(T, H, I, E, k)) {
    prof_begin(kInt8GateUp, s);
    hipLaunchKernelGGL(pairs_gate_up, dim3(I / 16 * P), dim3(256), 0, s, x8, xs, wgu8, wgus, idx, H, I, E,
                       k, P, act, order_key());
    prof_end(kInt8GateUp, s);
    prof_begin(kInt8Down, s);
    hipLaunchKernelGGL(pairs_down, dim3(H / kPairCols), dim3(kPairWaves * kWave), pairs_lds(P, I), s, act,
                       wd8, wds, idx, w, H, I, E, k, P, out, order_key());
    prof_end(kInt8Down, s);
    return hipGetLastError();
  }
  if (const hipError_t e = launch_group_experts(idx, P, E, L.bm, counts, offsets, tiles, n_tiles,
                                                perm, row_of, s); e != hipSuccess) return e;
  int* partial = reinterpret_cast<int*>(b + L.partial);
  const bool large = L.bm == kLargeBM;
  // grid of the large tiles: every item whole, plus room for the tail slices (rem * S - rem < ncu)
  auto large_grid = [&](int nblk) { return dim3(round_up(nblk * L.max_tiles + num_cus, kXcds)); };
#define ARGS perm, tiles, n_tiles, counts, offsets, w, H, I, k
#define LARGE8(KD, A, AS, W, WS, Y, O, NBLK, PER)                                              \
  hipLaunchKernelGGL(gemm_large_i8<KD>, large_grid(NBLK), dim3(256), k8Lds, s, A, AS, W, WS,  \
                     ARGS, Y, O, partial, num_cus, order_key());                              \
  hipLaunchKernelGGL(gemm_large_i8_fixup<KD>, dim3(num_cus / 2 * PER), dim3(256), 0, s, AS, WS, \
                     ARGS, Y, O, partial, num_cus, order_key())
#define STREAM8(KD, PART, A, AS, W, WS, Y, O, NBLK, S)                                        \
  do {                                                                                        \
    const dim3 grid_(round_up((NBLK) * (S) * L.max_tiles, kXcds));                            \
    if (L.bm == kTall8)                                                                       \
      hipLaunchKernelGGL((gemm_i8s<KD, 8, kTall8, PART>), grid_, dim3(512), 0, s, A, AS, W, WS, \
                         ARGS, Y, O, P, S, partial, order_key());                             \
    else                                                                                      \
      hipLaunchKernelGGL((gemm_i8s<KD, 8, kBM8, PART>), grid_, dim3(512), 0, s, A, AS, W, WS, \
                         ARGS, Y, O, P, S, partial, order_key());                             \
  } while (0)
  prof_begin(kInt8GateUp, s);
  if (large) { LARGE8(kGateUp8, x8, xs, wgu8, wgus, act, nullptr, I / 128, 32); }
  else if (L.slices_gu > 1) STREAM8(kGateUp8, true, x8, xs, wgu8, wgus, nullptr, nullptr, I / 128, L.slices_gu);
  else STREAM8(kGateUp8, false, x8, xs, wgu8, wgus, act, nullptr, I / 128, 1);
  prof_end(kInt8GateUp, s);
  const Int8Parts gu{partial, L.slices_gu, k, perm, idx, xs, wgus};
  const Int8Parts down{partial, L.slices_down, k, perm, idx, scales, wds};
  uint16_t* const clear = k == 1 && L.slices_down == 1 ? out : nullptr;
#define QUANT8(NV)                                                                            \
  do {                                                                                        \
    if (L.slices_gu > 1)                                                                      \
      hipLaunchKernelGGL((quant_act_rows<NV, true>), dim3(P), dim3(256), 0, s, nullptr, gu, offsets, E, \
                         row_of, P, H, I, codes, scales, clear, order_key());                 \
    else                                                                                      \
      hipLaunchKernelGGL((quant_act_rows<NV, false>), dim3(P), dim3(256), 0, s, act, gu, offsets, E, \
                         row_of, P, H, I, codes, scales, clear, order_key());                 \
  } while (0)
  if (I <= 1024) QUANT8(1);
  else if (I <= 2048) QUANT8(2);
  else if (I <= 4096) QUANT8(4);
  else QUANT8(16);
#undef QUANT8
  prof_begin(kInt8Down, s);
  if (large && k == 1) { LARGE8(kDownFused8, codes, scales, wd8, wds, nullptr, out, H / 256, 64); }
  else if (large) { LARGE8(kDown8, codes, scales, wd8, wds, y, nullptr, H / 256, 64); }
  else if (L.slices_down > 1) STREAM8(kDown8, true, codes, scales, wd8, wds, nullptr, nullptr, H / 256, L.slices_down);
  else if (k == 1) STREAM8(kDownFused8, false, codes, scales, wd8, wds, nullptr, out, H / 256, 1);
  else STREAM8(kDown8, false, codes, scales, wd8, wds, y, nullptr, H / 256, 1);
#undef ARGS
#undef LARGE8
#undef STREAM8
  if (L.slices_down > 1)
    hipLaunchKernelGGL(combine_parts, dim3(T, (H + 1023) / 1024), dim3(256), 0, s, down, row_of, w, T, H, out,
                       order_key());
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && k > 1 && L.slices_down == 1)
    e = launch_combine_slots(y, row_of, w, T, H, k, out, 0, H, H, s, num_cus);
  prof_end(kInt8Down, s);
  return e;
}

}  // namespace moe
