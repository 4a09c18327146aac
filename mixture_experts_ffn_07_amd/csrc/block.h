// Launch wrappers of the operators around the routed experts (norm.hip,
// route_scored.hip, int8.hip, mxfp4.hip, balance.hip), between the C ABI (abi.cpp) and
// their kernels.
// Arguments have been validated by the caller; each returns hipGetLastError()
// after its launches.
#pragma once

#include "internal.h"

namespace moe {

// Kernel ids of the timing hook, after internal.h's.
enum BlockKernelId { kNorm = kKernelCount, kNormBackward, kRouteBackward, kInt8GateUp, kInt8Down,
                     kMx4GateUp, kMx4Down, kBalance, kBalanceBackward, kAllKernelCount };

// Rows of one launch with a workgroup of up to 1024 threads each: a grid holds fewer than
// 2^32 threads.
constexpr int kMaxRows = 1 << 22;

// Routing by scores (route_scored.hip).
struct ScoredRoute {
  int E, k, groups, topk_groups, group_top;
  bool sigmoid, renorm;
  float scale;
};
hipError_t launch_route_scored(const float* logits, const float* bias, int T, const ScoredRoute& p,
                               int32_t* idx, float* w, hipStream_t s, int num_cus);
hipError_t launch_route_scored_backward(const float* logits, const int32_t* idx, const float* dw,
                                        int T, const ScoredRoute& p, float* dlogits, hipStream_t s);

// Residual sum + RMS norm (norm.hip).  qtype: MOE_BF16 (no 8-bit output), MOE_MXFP8, MOE_INT8.
constexpr int kNormMaxH = 16384;           // a row is held in one workgroup's registers
int norm_backward_rows(int T, int H);      // workgroups (rows of partial weight gradients)
hipError_t launch_add_rmsnorm(const uint16_t* x, const uint16_t* r, const uint16_t* w, int T, int H,
                              float eps, uint16_t* sum, uint16_t* y, int qtype, uint8_t* codes,
                              void* scales, hipStream_t s, int num_cus);
hipError_t launch_add_rmsnorm_backward(const uint16_t* sum, const uint16_t* w, const uint16_t* dy,
                                       const uint16_t* ds, int T, int H, float eps, uint16_t* dx,
                                       uint16_t* dweight, float* partial, hipStream_t s);
hipError_t launch_quant_int8(const uint16_t* src, int64_t rows, int K, uint8_t* codes, float* scales,
                             hipStream_t s, int num_cus);

// INT8 experts (int8.hip): byte layout of the workspace, and the whole layer.
struct Int8Ws {
  size_t n_tiles, counts, offsets, tiles, perm, row_of, act, codes, scales, y, partial, total;
  int max_tiles, bm, slices_gu, slices_down;   // slices of the two reductions
};
Int8Ws int8_ws_layout(int T, int H, int I, int E, int k);
hipError_t launch_experts_int8(const int8_t* x, const float* xs, const int8_t* wgu,
                               const float* wgus, const int8_t* wd, const float* wds,
                               const int32_t* idx, const float* w, int T, int H, int I, int E,
                               int k, uint16_t* out, void* ws, hipStream_t s, int num_cus);

// MXFP4 rows, and the experts with MXFP4 weights (mxfp4.hip): byte layout of the workspace,
// and the whole layer.  a4: MXFP4 activations, else MXFP8.
hipError_t launch_quant_mx4(const uint16_t* src, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                            hipStream_t s);
hipError_t launch_dequant_mx4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K,
                              uint16_t* dst, hipStream_t s);
struct Mx4Ws {
  size_t n_tiles, counts, offsets, tiles, perm, row_of, codes, scales, y, partial, wgu_t, wd_t, x_t, total;
  int max_tiles, bm;
};
Mx4Ws mx4_ws_layout(int T, int H, int I, int E, int k, bool a4);
hipError_t launch_experts_mx4(const uint8_t* x, const uint8_t* xs, bool a4, const uint8_t* wgu,
                              const uint8_t* wgus, const uint8_t* wd, const uint8_t* wds,
                              const int32_t* idx, const float* w, int T, int H, int I, int E, int k,
                              uint16_t* out, void* ws, hipStream_t s, int num_cus);

// The router's balance loss (balance.hip): S sequences of T / S tokens, cut into chunks of
// `rows` rows, `chunks` to a sequence.
constexpr int kMaxSeqs = 4096;
struct BalanceWs {
  size_t share, probs, counts, z, tokens, total;
  int chunks, rows;
};
BalanceWs balance_ws_layout(int T, int E, int S);
hipError_t launch_balance_loss(const float* logits, const int32_t* idx, const uint8_t* mask, int T, int E,
                               int k, int S, bool sigmoid, float* losses, int32_t* counts, float* probs,
                               int32_t* tokens, void* ws, hipStream_t s);
hipError_t launch_balance_loss_backward(const float* logits, const uint8_t* mask, const int32_t* counts,
                                        const int32_t* tokens, const float* d_losses, const float* d_add,
                                        int T, int E, int S, bool sigmoid, float* dlogits, hipStream_t s);

// combine_slots over the columns [col0, col0 + cols) (batched.hip).
hipError_t launch_combine_slots(const float* y, const int* row_of, const float* w, int T, int H,
                                int k, uint16_t* out, int col0, int cols, int ldy, hipStream_t s,
                                int num_cus);

}  // namespace moe
