// What the 256 x 256-tiled grouped GEMMs share (gemm_large.hip, int8.hip): the split
// of the last round's tiles along K, the order of the tiles, and their way to the XCDs.
#pragma once

#include "common.h"
#include "internal.h"
#include "tiles.h"

namespace moe {

// Tail split.  One workgroup fills a CU, so n items run in ceil(n / ncu)
// rounds; when the last round would leave more than half of the CUs idle, its
// items are cut along K into S slices that run side by side.  Each slice
// writes its FP32 partial tile to the workspace and gemm_large_fixup adds the
// S partials of an item in slice order (fixed, so results stay bit-identical
// run to run) before the usual epilogue.  Items before `full` run whole.
struct TailPlan {
  int full, rem, S;
};
__device__ __forceinline__ TailPlan tail_plan(int n_real, int ncu, int nk) {
  TailPlan p;
  const int rounds = n_real / ncu;
  p.rem = n_real - rounds * ncu;
  p.S = 1;
  if (p.rem > 0 && 2 * p.rem <= ncu && ncu % kXcds == 0)
    p.S = max(1, min(min(8, ncu / p.rem), min(nk / 2, kLargeMaxSlices / p.rem)));
  p.full = p.S > 1 ? rounds * ncu : n_real;
  return p;
}

// Item order.  Items are (M-tile, N-block) pairs; an XCD runs a contiguous run
// of item numbers, 32 at a time.  Numbering N-blocks fastest would make those
// 32 one or two M-tiles against ~32 different weight blocks (about 34 distinct
// operand blocks per K stage in the XCD's L2); numbering groups of
// kLargeGroupM M-tiles with the M-tile fastest makes them 8 M-tiles x 4
// N-blocks (12 distinct blocks), so each staged block is shared by more CUs.
// (Measured over group sizes 2, 4, 6, 8 and 16: 8 is best for MXFP8 and level
// with 4 for BF16.)
constexpr int kLargeGroupM = 8;
__device__ __forceinline__ void large_coords(int item, int nblk, int n_tiles, int& tile, int& nb) {
  const int grp = item / (kLargeGroupM * nblk);
  const int r = item - grp * kLargeGroupM * nblk;
  const int t0 = grp * kLargeGroupM;
  const int gm = min(kLargeGroupM, n_tiles - t0);
  nb = r / gm;
  tile = t0 + (r - nb * gm);
}

// Workgroup -> item across XCDs.  One workgroup fills a CU, so the ncu
// workgroups resident at a time are consecutive; mapping each such round to one
// contiguous run of items (XCD x, = L mod 8, taking the x-th chunk of it) keeps
// every CU on the same one or two experts at a time, whose operands then stay in
// the last-level cache (spreading the XCDs over the whole item range put six
// experts' weights, 352 MB on the BF16 EP share, in flight at once).  n is a
// multiple of 8; a last partial round keeps the contiguous-per-XCD split.
__device__ __forceinline__ int round_item(int L, int n, int ncu) {
  if (ncu < kXcds || ncu % kXcds) return xcd_item(L, n);
  const int full = n / ncu * ncu;
  if (L < full) {
    const int r = L / ncu, w = L - r * ncu;
    return r * ncu + (w % kXcds) * (ncu / kXcds) + w / kXcds;
  }
  return full + xcd_item(L - full, n - full);
}
__device__ __forceinline__ int round_real_item(int L, int nblk, int n_tiles, int ncu) {
  const int n_real = (nblk * n_tiles + kXcds - 1) / kXcds * kXcds;
  if (L >= n_real) return -1;
  const int item = round_item(L, n_real, ncu);
  return item / nblk < n_tiles ? item : -1;
}

// s_waitcnt with only the LDS/scalar counter constrained to 0
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

}  // namespace moe
