// C ABI of the library: host-side validation, workspace sizing and dispatch.
// Every check runs before any HIP call, so the checks work on a host without
// a GPU.  The HIP runtime is first touched by the first valid launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

#include "../../include/moe_mi355x.h"
#include "block.h"
#include "internal.h"

namespace moe {
hipError_t decode_set_attributes();
hipError_t batched_set_attributes();
hipError_t backward_set_attributes();
hipError_t int8_set_attributes();
hipError_t mx4_set_attributes();

ProfileHook& profile_hook() {
  thread_local ProfileHook hook;
  return hook;
}

DebugOptions& debug_options() {
  thread_local DebugOptions opts;
  return opts;
}
}  // namespace moe

static_assert(MOE_STATIC_SCRATCH_BYTES == moe::kStaticScratchBytes,
              "the header's scratch size must match the array's");
static_assert(MOE_DEBUG_PERMUTE_ORDER == moe::kDebugPermute &&
              MOE_DEBUG_DECODE_FUSED == moe::kDebugDecodeFused, "debug option bits");
static_assert(MOE_KERNEL_COUNT == moe::kAllKernelCount &&
              MOE_KERNEL_NORM == moe::kNorm && MOE_KERNEL_INT8_DOWN == moe::kInt8Down &&
              MOE_KERNEL_BALANCE_BACKWARD == moe::kBalanceBackward, "kernel ids");

namespace {

thread_local std::string g_last_error;

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return status;
}

int ok() {
  g_last_error.clear();
  return MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device properties and one-time kernel attributes, per device.
struct DeviceInfo {
  int num_cus = 0;
  bool ready = false;
  void* scratch = nullptr;   // this device's copy of the library-owned scratch array
};
std::mutex g_mu;
DeviceInfo g_dev[moe::kMaxDevices];

int device_info(int* num_cus, void** scratch = nullptr) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= moe::kMaxDevices) return fail(MOE_ERR_UNSUPPORTED, "device ordinal %d", dev);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
    if (std::string(prop.gcnArchName).rfind("gfx950", 0) != 0)
      return fail(MOE_ERR_UNSUPPORTED, "device %d is %s; this library is built for gfx950", dev,
                  prop.gcnArchName);
    e = moe::decode_set_attributes();
    if (e == hipSuccess) e = moe::batched_set_attributes();
    if (e == hipSuccess) e = moe::backward_set_attributes();
    if (e == hipSuccess) e = moe::int8_set_attributes();
    if (e == hipSuccess) e = moe::mx4_set_attributes();
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipFuncSetAttribute: %s", hipGetErrorString(e));
    // the device address of this device's scratch array (the device is current)
    e = moe::static_scratch(dev, &d.scratch);
    if (e != hipSuccess) return fail(MOE_ERR_HIP, "hipGetSymbolAddress: %s", hipGetErrorString(e));
    d.num_cus = prop.multiProcessorCount;
    d.ready = true;
  }
  *num_cus = d.num_cus;
  if (scratch) *scratch = d.scratch;
  return MOE_OK;
}

int hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

int check_common(int T, int H, int I, int E, int k, int hmul, int imul) {
  if (T < 0) return fail(MOE_ERR_SHAPE, "T=%d < 0", T);
  if (E < 1 || E > 1024) return fail(MOE_ERR_SHAPE, "E=%d outside [1, 1024]", E);
  if (k < 1 || k > E || k > 32) return fail(MOE_ERR_SHAPE, "k=%d outside [1, min(E=%d, 32)]", k, E);
  if (H <= 0 || H % hmul) return fail(MOE_ERR_SHAPE, "H=%d is not a positive multiple of %d", H, hmul);
  if (I <= 0 || I % imul) return fail(MOE_ERR_SHAPE, "I=%d is not a positive multiple of %d", I, imul);
  return MOE_OK;
}

// Element offsets the kernels form in 32-bit arithmetic: rows of x (T*H), of
// the routed-pair buffers h and y (T*k*I, T*k*H) and of one expert's weights
// (2I*H).  Each must stay below 2^31.
int check_offsets(int T, int H, int I, int k) {
  const long long lim = 1LL << 31;
  if (static_cast<long long>(T) * H >= lim) return fail(MOE_ERR_SHAPE, "T*H reaches 2^31");
  if (static_cast<long long>(T) * k * H >= lim) return fail(MOE_ERR_SHAPE, "T*k*H reaches 2^31");
  if (static_cast<long long>(T) * k * I >= lim) return fail(MOE_ERR_SHAPE, "T*k*I reaches 2^31");
  if (2LL * I * H >= lim) return fail(MOE_ERR_SHAPE, "2*I*H reaches 2^31");
  return MOE_OK;
}

}  // namespace

extern "C" {

const char* moe_status_string(int status) {
  switch (status) {
    case MOE_OK: return "ok";
    case MOE_ERR_NULL: return "null pointer";
    case MOE_ERR_SHAPE: return "invalid shape";
    case MOE_ERR_ALIGN: return "misaligned pointer";
    case MOE_ERR_WORKSPACE: return "workspace missing or too small";
    case MOE_ERR_UNSUPPORTED: return "unsupported";
    case MOE_ERR_HIP: return "HIP runtime error";
    default: return "unknown status";
  }
}

const char* moe_last_error(void) { return g_last_error.c_str(); }

int moe_profile_kernel(int kernel, void* start_event, void* stop_event) {
  if (kernel < 0 || kernel >= moe::kAllKernelCount)
    return fail(MOE_ERR_SHAPE, "unknown kernel id %d", kernel);
  moe::ProfileHook& h = moe::profile_hook();
  h.kernel = (start_event && stop_event) ? kernel : 0;
  h.start = static_cast<hipEvent_t>(start_event);
  h.stop = static_cast<hipEvent_t>(stop_event);
  return ok();
}

int moe_set_debug_options(unsigned flags, uint32_t seed) {
  if (flags & ~(MOE_DEBUG_PERMUTE_ORDER | MOE_DEBUG_DECODE_FUSED))
    return fail(MOE_ERR_SHAPE, "unknown debug option bits 0x%x", flags);
  moe::DebugOptions& o = moe::debug_options();
  o.flags = flags;
  o.seed = seed;
  return ok();
}

int moe_route_topk(const float* logits, int T, int E, int k, int32_t* topk_idx, float* topk_w,
                   void* stream) {
  if (T < 0) return fail(MOE_ERR_SHAPE, "T=%d < 0", T);
  if (E < 1 || E > 1024) return fail(MOE_ERR_SHAPE, "E=%d outside [1, 1024]", E);
  if (k < 1 || k > E || k > 32) return fail(MOE_ERR_SHAPE, "k=%d outside [1, min(E=%d, 32)]", k, E);
  if (T == 0) return ok();
  if (!logits || !topk_idx || !topk_w) return fail(MOE_ERR_NULL, "logits, topk_idx and topk_w are required");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_route_topk(logits, T, E, k, topk_idx, topk_w,
                                           static_cast<hipStream_t>(stream)),
                    "moe_route_topk launch");
}

size_t moe_decode_workspace_bytes(int T, int H, int I, int E, int k) {
  if (T < 1 || T > 64 || H <= 0 || I <= 0 || E < 1 || k < 1) return 0;
  return moe::decode_ws_layout(T, H, I, E, k).total;
}

int moe_decode_forward(const uint16_t* x, const float* logits, const uint16_t* w_gate_up,
                       const uint16_t* w_down, int T, int H, int I, int E, int k, uint16_t* out,
                       int32_t* topk_idx, float* topk_w, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (int st = check_common(T, H, I, E, k, 256, 256)) return st;
  if (T == 0) return fail(MOE_ERR_SHAPE, "T=0: nothing to decode");
  if (T > 64) return fail(MOE_ERR_UNSUPPORTED, "T=%d > 64: use the batched calls", T);
  if (I > 2048) return fail(MOE_ERR_UNSUPPORTED, "I=%d > 2048: use the batched calls", I);
  if (int st = check_offsets(T, H, I, k)) return st;
  if (!x || !logits || !w_gate_up || !w_down || !out)
    return fail(MOE_ERR_NULL, "x, logits, w_gate_up, w_down and out are required");
  if (!workspace) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = moe::decode_ws_layout(T, H, I, E, k).total;
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(w_down) || !aligned16(out) ||
      !aligned16(workspace) || !aligned16(logits) || (topk_idx && !aligned16(topk_idx)) ||
      (topk_w && !aligned16(topk_w)))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_decode(x, logits, w_gate_up, w_down, T, H, I, E, k, out, topk_idx,
                                       topk_w, workspace, static_cast<hipStream_t>(stream), cus),
                    "moe_decode_forward launch");
}

int moe_decode_forward_noalloc(const uint16_t* x, const float* logits, const uint16_t* w_gate_up,
                               const uint16_t* w_down, int T, int H, int I, int E, int k,
                               uint16_t* out, int32_t* topk_idx, float* topk_w, void* stream) {
  if (int st = check_common(T, H, I, E, k, 256, 256)) return st;
  if (T == 0) return fail(MOE_ERR_SHAPE, "T=0: nothing to decode");
  if (T > 64) return fail(MOE_ERR_UNSUPPORTED, "T=%d > 64: use the batched calls", T);
  if (I > 2048) return fail(MOE_ERR_UNSUPPORTED, "I=%d > 2048: use the batched calls", I);
  if (int st = check_offsets(T, H, I, k)) return st;
  const size_t need = moe::decode_ws_layout(T, H, I, E, k).total;
  if (need > moe::kStaticScratchBytes)
    return fail(MOE_ERR_UNSUPPORTED,
                "workspace of %zu bytes exceeds the library's %zu-byte scratch (T*k*I too "
                "large): use moe_decode_forward with a caller workspace",
                need, moe::kStaticScratchBytes);
  if (!x || !logits || !w_gate_up || !w_down || !out)
    return fail(MOE_ERR_NULL, "x, logits, w_gate_up, w_down and out are required");
  if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(w_down) || !aligned16(out) ||
      !aligned16(logits) || (topk_idx && !aligned16(topk_idx)) || (topk_w && !aligned16(topk_w)))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  void* ws = nullptr;
  if (int st = device_info(&cus, &ws)) return st;
  return hip_status(moe::launch_decode(x, logits, w_gate_up, w_down, T, H, I, E, k, out, topk_idx,
                                       topk_w, ws, static_cast<hipStream_t>(stream), cus),
                    "moe_decode_forward_noalloc launch");
}

size_t moe_workspace_bytes(int T, int H, int I, int E, int k, moe_dtype dtype) {
  if (T < 1 || H <= 0 || I <= 0 || E < 1 || k < 1 || (dtype != MOE_BF16 && dtype != MOE_MXFP8))
    return 0;
  return moe::batched_ws_layout(T, H, I, E, k, dtype).total;
}

int moe_quantize_mxfp8(const uint16_t* src, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                       void* stream) {
  if (rows < 0) return fail(MOE_ERR_SHAPE, "rows=%lld < 0", static_cast<long long>(rows));
  if (K <= 0 || K % 32) return fail(MOE_ERR_SHAPE, "K=%d is not a positive multiple of 32", K);
  if (rows == 0) return ok();
  if (!src || !codes || !scales) return fail(MOE_ERR_NULL, "src, codes and scales are required");
  if (!aligned16(src) || !aligned16(codes) || !aligned16(scales))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_quant_mx(src, rows, K, codes, scales,
                                         static_cast<hipStream_t>(stream)),
                    "moe_quantize_mxfp8 launch");
}

static int check_batched(int T, int H, int I, int E, int k, moe_dtype dtype, const void* ws,
                         size_t ws_bytes) {
  if (int st = check_common(T, H, I, E, k, 256, 256)) return st;
  if (T < 1) return fail(MOE_ERR_SHAPE, "T=%d < 1", T);
  if (dtype != MOE_BF16 && dtype != MOE_MXFP8) return fail(MOE_ERR_SHAPE, "dtype=%d", dtype);
  if (static_cast<long long>(T) * k > (1LL << 30)) return fail(MOE_ERR_SHAPE, "T*k too large");
  // the kernels form 32-bit element offsets into x, h, y and one expert's weights
  if (int st = check_offsets(T, H, I, k)) return st;
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = moe::batched_ws_layout(T, H, I, E, k, dtype).total;
  if (ws_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", ws_bytes, need);
  if (!aligned16(ws)) return fail(MOE_ERR_ALIGN, "workspace must be 16-byte aligned");
  return MOE_OK;
}

int moe_gate_up_3d_batched(const void* x, const uint8_t* x_scales, const void* w_gate_up,
                           const uint8_t* w_gate_up_scales, const int32_t* topk_idx, int T, int H,
                           int I, int E, int k, moe_dtype dtype, void* h, uint8_t* h_scales,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_batched(T, H, I, E, k, dtype, workspace, workspace_bytes)) return st;
  if (!x || !w_gate_up || !topk_idx || !h)
    return fail(MOE_ERR_NULL, "x, w_gate_up, topk_idx and h are required");
  if (dtype == MOE_MXFP8 && (!x_scales || !w_gate_up_scales || !h_scales))
    return fail(MOE_ERR_NULL, "MXFP8 needs x_scales, w_gate_up_scales and h_scales");
  if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(topk_idx) || !aligned16(h) ||
      (dtype == MOE_MXFP8 &&
       (!aligned16(x_scales) || !aligned16(w_gate_up_scales) || !aligned16(h_scales))))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_gate_up_batched(x, x_scales, w_gate_up, w_gate_up_scales, topk_idx,
                                                T, H, I, E, k, dtype, h, h_scales, workspace,
                                                static_cast<hipStream_t>(stream), cus),
                    "moe_gate_up_3d_batched launch");
}

int moe_down_3d_batched(const void* h, const uint8_t* h_scales, const void* w_down,
                        const uint8_t* w_down_scales, const int32_t* topk_idx,
                        const float* topk_w, int T, int H, int I, int E, int k, moe_dtype dtype,
                        uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_batched(T, H, I, E, k, dtype, workspace, workspace_bytes)) return st;
  if (!h || !w_down || !topk_idx || !topk_w || !out)
    return fail(MOE_ERR_NULL, "h, w_down, topk_idx, topk_w and out are required");
  if (dtype == MOE_MXFP8 && (!h_scales || !w_down_scales))
    return fail(MOE_ERR_NULL, "MXFP8 needs h_scales and w_down_scales");
  if (!aligned16(h) || !aligned16(w_down) || !aligned16(topk_idx) || !aligned16(topk_w) ||
      !aligned16(out) || (dtype == MOE_MXFP8 && (!aligned16(h_scales) || !aligned16(w_down_scales))))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_down_batched(h, h_scales, w_down, w_down_scales, topk_idx, topk_w,
                                             T, H, I, E, k, dtype, out, workspace,
                                             static_cast<hipStream_t>(stream), cus),
                    "moe_down_3d_batched launch");
}

size_t moe_backward_workspace_bytes(int T, int H, int I, int E, int k) {
  if (T < 1 || H <= 0 || I <= 0 || E < 1 || k < 1) return 0;
  return moe::backward_ws_layout(T, H, I, E, k).total;
}

int moe_backward_batched(const uint16_t* x, const uint16_t* w_gate_up, const uint16_t* w_down,
                         const int32_t* topk_idx, const float* topk_w, const uint16_t* dout,
                         const float* gu_saved, int T, int H, int I, int E, int k,
                         uint16_t* dx, uint16_t* dw_gate_up,
                         uint16_t* dw_down, float* d_topk_w, float* dlogits, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (int st = check_common(T, H, I, E, k, 256, 256)) return st;
  if (T < 1) return fail(MOE_ERR_SHAPE, "T=%d < 1", T);
  if (static_cast<long long>(T) * k > (1LL << 24))
    return fail(MOE_ERR_SHAPE, "T*k=%lld > 2^24", static_cast<long long>(T) * k);
  if (static_cast<long long>(T) * k * H >= (1LL << 31) ||
      static_cast<long long>(T) * k * 2 * I >= (1LL << 31) ||
      2LL * I * H >= (1LL << 31))
    return fail(MOE_ERR_SHAPE, "T*k*H, T*k*2I or 2I*H reaches 2^31");
  if (!x || !w_gate_up || !w_down || !topk_idx || !topk_w || !dout || !dx || !dw_gate_up ||
      !dw_down || !d_topk_w || !dlogits)
    return fail(MOE_ERR_NULL, "every input and output pointer is required");
  if (!workspace) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = moe::backward_ws_layout(T, H, I, E, k).total;
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(w_down) || !aligned16(topk_idx) ||
      !aligned16(topk_w) || !aligned16(dout) || !aligned16(dx) || !aligned16(dw_gate_up) ||
      !aligned16(dw_down) || !aligned16(d_topk_w) || !aligned16(dlogits) ||
      !aligned16(workspace) || (gu_saved && !aligned16(gu_saved)))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_backward(x, w_gate_up, w_down, topk_idx, topk_w, dout, gu_saved,
                                         T, H, I, E, k, dx, dw_gate_up, dw_down, d_topk_w,
                                         dlogits, workspace, static_cast<hipStream_t>(stream), cus),
                    "moe_backward_batched launch");
}

size_t moe_backward_mxfp8_workspace_bytes(int T, int H, int I, int E, int k) {
  if (T < 1 || H <= 0 || I <= 0 || E < 1 || k < 1) return 0;
  return moe::mx_backward_ws_layout(T, H, I, E, k).total;
}

int moe_backward_batched_mxfp8(const uint16_t* x, const uint8_t* w_gate_up,
                               const uint8_t* w_gate_up_scales, const uint8_t* w_down,
                               const uint8_t* w_down_scales, const int32_t* topk_idx,
                               const float* topk_w, const uint16_t* dout, int T, int H, int I,
                               int E, int k, uint16_t* dx, uint16_t* dw_gate_up, uint16_t* dw_down,
                               float* d_topk_w, float* dlogits, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (int st = check_common(T, H, I, E, k, 256, 256)) return st;
  if (T < 1) return fail(MOE_ERR_SHAPE, "T=%d < 1", T);
  if (static_cast<long long>(T) * k > (1LL << 24))
    return fail(MOE_ERR_SHAPE, "T*k=%lld > 2^24", static_cast<long long>(T) * k);
  if (int st = check_offsets(T, H, I, k)) return st;
  if (static_cast<long long>(T) * k * 2 * I >= (1LL << 31))
    return fail(MOE_ERR_SHAPE, "T*k*2I reaches 2^31");
  // pair-axis operands: rows x (routed pairs, each expert padded to 128) below 2^31
  {
    const size_t cols = static_cast<size_t>(T) * k + static_cast<size_t>(128) * E;
    const size_t rows = static_cast<size_t>(H > 2 * I ? H : 2 * I);
    if (rows * cols >= (static_cast<size_t>(1) << 31))
      return fail(MOE_ERR_SHAPE, "max(H, 2I) * (T*k + 128*E) reaches 2^31");
  }
  if (!x || !w_gate_up || !w_gate_up_scales || !w_down || !w_down_scales || !topk_idx ||
      !topk_w || !dout || !dx || !dw_gate_up || !dw_down || !d_topk_w || !dlogits)
    return fail(MOE_ERR_NULL, "every input and output pointer is required");
  if (!workspace) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = moe::mx_backward_ws_layout(T, H, I, E, k).total;
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(w_gate_up_scales) ||
      !aligned16(w_down) || !aligned16(w_down_scales) || !aligned16(topk_idx) ||
      !aligned16(topk_w) || !aligned16(dout) || !aligned16(dx) || !aligned16(dw_gate_up) ||
      !aligned16(dw_down) || !aligned16(d_topk_w) || !aligned16(dlogits) || !aligned16(workspace))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_backward_mx(x, w_gate_up, w_gate_up_scales, w_down, w_down_scales,
                                            topk_idx, topk_w, dout, T, H, I, E, k, dx, dw_gate_up,
                                            dw_down, d_topk_w, dlogits, workspace,
                                            static_cast<hipStream_t>(stream), cus),
                    "moe_backward_batched_mxfp8 launch");
}

int moe_gate_up_3d_batched_train(const uint16_t* x, const uint16_t* w_gate_up,
                                 const int32_t* topk_idx, int T, int H, int I, int E, int k,
                                 uint16_t* h, float* gu, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (int st = check_batched(T, H, I, E, k, MOE_BF16, workspace, workspace_bytes)) return st;
  if (!x || !w_gate_up || !topk_idx || !h || !gu)
    return fail(MOE_ERR_NULL, "x, w_gate_up, topk_idx, h and gu are required");
  if (static_cast<long long>(T) * k * 2 * I >= (1LL << 31))
    return fail(MOE_ERR_SHAPE, "T*k*2I reaches 2^31");
  if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(topk_idx) || !aligned16(h) ||
      !aligned16(gu))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_gate_up_batched(x, nullptr, w_gate_up, nullptr, topk_idx, T, H, I,
                                                E, k, MOE_BF16, h, nullptr, workspace,
                                                static_cast<hipStream_t>(stream), cus, gu),
                    "moe_gate_up_3d_batched_train launch");
}

static int check_norm(int T, int H, float eps) {
  if (T < 0 || T >= moe::kMaxRows) return fail(MOE_ERR_SHAPE, "T=%d outside [0, %d)", T, moe::kMaxRows);
  if (H < 32 || H % 32 || H > moe::kNormMaxH)
    return fail(MOE_ERR_SHAPE, "H=%d is not a multiple of 32 in [32, %d]", H, moe::kNormMaxH);
  if (!(eps > 0.0f) || !std::isfinite(eps))
    return fail(MOE_ERR_SHAPE, "eps=%g is not finite and above 0", static_cast<double>(eps));
  return MOE_OK;
}

int moe_add_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int T,
                    int H, float eps, uint16_t* residual_out, uint16_t* y, moe_dtype qtype,
                    void* codes, void* scales, void* stream) {
  if (int st = check_norm(T, H, eps)) return st;
  if (qtype != MOE_BF16 && qtype != MOE_MXFP8 && qtype != MOE_INT8)
    return fail(MOE_ERR_SHAPE, "qtype=%d", qtype);
  if (residual_out && !residual)
    return fail(MOE_ERR_NULL, "residual_out needs a residual (without one the sum is x)");
  if (T == 0) return ok();
  if (!x || !weight) return fail(MOE_ERR_NULL, "x and weight are required");
  const bool q = qtype != MOE_BF16;
  if (q && (!codes || !scales)) return fail(MOE_ERR_NULL, "8-bit output needs codes and scales");
  if (!q && !y) return fail(MOE_ERR_NULL, "y is required without 8-bit output");
  if (y && y == residual_out) return fail(MOE_ERR_UNSUPPORTED, "y and residual_out are the same buffer");
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) ||
      !aligned16(y) || (q && (!aligned16(codes) || !aligned16(scales))))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_add_rmsnorm(x, residual, weight, T, H, eps, residual_out, y, qtype,
                                            static_cast<uint8_t*>(codes), scales,
                                            static_cast<hipStream_t>(stream), cus),
                    "moe_add_rmsnorm launch");
}

size_t moe_add_rmsnorm_backward_workspace_bytes(int T, int H) {
  if (T < 0 || H <= 0) return 0;
  const size_t rows = static_cast<size_t>(moe::norm_backward_rows(T, H));
  return (rows > 0 ? rows : 1) * static_cast<size_t>(H) * sizeof(float);
}

int moe_add_rmsnorm_backward(const uint16_t* s, const uint16_t* weight, const uint16_t* dy,
                             const uint16_t* ds, int T, int H, float eps, uint16_t* dx,
                             uint16_t* dweight, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (int st = check_norm(T, H, eps)) return st;
  if (!dweight || (T > 0 && (!s || !weight || !dy || !dx)))
    return fail(MOE_ERR_NULL, "s, weight, dy, dx and dweight are required");
  if (!workspace) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = moe_add_rmsnorm_backward_workspace_bytes(T, H);
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  if (!aligned16(s) || !aligned16(weight) || !aligned16(dy) || !aligned16(ds) || !aligned16(dx) ||
      !aligned16(dweight) || !aligned16(workspace))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_add_rmsnorm_backward(s, weight, dy, ds, T, H, eps, dx, dweight,
                                                     static_cast<float*>(workspace),
                                                     static_cast<hipStream_t>(stream)),
                    "moe_add_rmsnorm_backward launch");
}

static int check_scored(int T, int E, int k, moe_score score, float scale) {
  if (T < 0 || T >= moe::kMaxRows) return fail(MOE_ERR_SHAPE, "T=%d outside [0, %d)", T, moe::kMaxRows);
  if (E < 1 || E > 1024) return fail(MOE_ERR_SHAPE, "E=%d outside [1, 1024]", E);
  if (k < 1 || k > E || k > 32) return fail(MOE_ERR_SHAPE, "k=%d outside [1, min(E=%d, 32)]", k, E);
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_SHAPE, "score=%d", score);
  if (!std::isfinite(scale)) return fail(MOE_ERR_SHAPE, "scale is not finite");
  return MOE_OK;
}

int moe_route_scored(const float* logits, const float* bias, int T, int E, int k, int n_groups,
                     int topk_groups, int group_top, moe_score score, int renormalize, float scale,
                     int32_t* topk_idx, float* topk_w, void* stream) {
  if (int st = check_scored(T, E, k, score, scale)) return st;
  if (n_groups < 1 || n_groups > 64 || E % n_groups)
    return fail(MOE_ERR_SHAPE, "n_groups=%d is not a divisor of E=%d in [1, 64]", n_groups, E);
  if (topk_groups < 1 || topk_groups > n_groups)
    return fail(MOE_ERR_SHAPE, "topk_groups=%d outside [1, n_groups=%d]", topk_groups, n_groups);
  if (group_top != 1 && group_top != 2) return fail(MOE_ERR_SHAPE, "group_top=%d is not 1 or 2", group_top);
  if (k > topk_groups * (E / n_groups))
    return fail(MOE_ERR_SHAPE, "k=%d > %d experts in the selected groups", k, topk_groups * (E / n_groups));
  if (T == 0) return ok();
  if (!logits || !topk_idx || !topk_w)
    return fail(MOE_ERR_NULL, "logits, topk_idx and topk_w are required");
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(topk_idx) || !aligned16(topk_w))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  const moe::ScoredRoute p{E, k, n_groups, topk_groups, group_top, score == MOE_SCORE_SIGMOID,
                           renormalize != 0, scale};
  return hip_status(moe::launch_route_scored(logits, bias, T, p, topk_idx, topk_w,
                                             static_cast<hipStream_t>(stream), cus),
                    "moe_route_scored launch");
}

int moe_route_scored_backward(const float* logits, const int32_t* topk_idx, const float* d_topk_w,
                              int T, int E, int k, moe_score score, int renormalize, float scale,
                              float* dlogits, void* stream) {
  if (int st = check_scored(T, E, k, score, scale)) return st;
  if (T == 0) return ok();
  if (!logits || !topk_idx || !d_topk_w || !dlogits)
    return fail(MOE_ERR_NULL, "logits, topk_idx, d_topk_w and dlogits are required");
  if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(d_topk_w) || !aligned16(dlogits))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  const moe::ScoredRoute p{E, k, 1, 1, 1, score == MOE_SCORE_SIGMOID, renormalize != 0, scale};
  return hip_status(moe::launch_route_scored_backward(logits, topk_idx, d_topk_w, T, p, dlogits,
                                                      static_cast<hipStream_t>(stream)),
                    "moe_route_scored_backward launch");
}

int moe_quantize_int8(const uint16_t* src, int64_t rows, int K, int8_t* codes, float* scales,
                      void* stream) {
  if (rows < 0 || rows >= (1LL << 29))
    return fail(MOE_ERR_SHAPE, "rows=%lld outside [0, 2^29)", static_cast<long long>(rows));
  if (K < 32 || K % 32 || K > moe::kNormMaxH)
    return fail(MOE_ERR_SHAPE, "K=%d is not a multiple of 32 in [32, %d]", K, moe::kNormMaxH);
  if (rows == 0) return ok();
  if (!src || !codes || !scales) return fail(MOE_ERR_NULL, "src, codes and scales are required");
  if (!aligned16(src) || !aligned16(codes) || !aligned16(scales))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_quant_int8(src, rows, K, reinterpret_cast<uint8_t*>(codes), scales,
                                           static_cast<hipStream_t>(stream), cus),
                    "moe_quantize_int8 launch");
}

size_t moe_experts_int8_workspace_bytes(int T, int H, int I, int E, int k) {
  if (T < 1 || H <= 0 || I <= 0 || E < 1 || k < 1) return 0;
  return moe::int8_ws_layout(T, H, I, E, k).total;
}

int moe_experts_int8(const int8_t* x, const float* x_scales, const int8_t* w_gate_up,
                     const float* w_gate_up_scales, const int8_t* w_down,
                     const float* w_down_scales, const int32_t* topk_idx, const float* topk_w,
                     int T, int H, int I, int E, int k, uint16_t* out, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (int st = check_common(T, H, I, E, k, 256, 256)) return st;
  if (H > moe::kNormMaxH || I > moe::kNormMaxH)
    return fail(MOE_ERR_SHAPE, "H=%d or I=%d above %d", H, I, moe::kNormMaxH);
  if (int st = check_offsets(T, H, I, k)) return st;
  if (T == 0) return ok();
  if (!x || !x_scales || !w_gate_up || !w_gate_up_scales || !w_down || !w_down_scales ||
      !topk_idx || !topk_w || !out)
    return fail(MOE_ERR_NULL, "every input and output pointer is required");
  if (!workspace) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = moe::int8_ws_layout(T, H, I, E, k).total;
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  if (!aligned16(x) || !aligned16(x_scales) || !aligned16(w_gate_up) ||
      !aligned16(w_gate_up_scales) || !aligned16(w_down) || !aligned16(w_down_scales) ||
      !aligned16(topk_idx) || !aligned16(topk_w) || !aligned16(out) || !aligned16(workspace))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_experts_int8(x, x_scales, w_gate_up, w_gate_up_scales, w_down,
                                             w_down_scales, topk_idx, topk_w, T, H, I, E, k, out,
                                             workspace, static_cast<hipStream_t>(stream), cus),
                    "moe_experts_int8 launch");
}

static int check_mx4_rows(int64_t rows, int K) {
  if (K <= 0 || K % 32) return fail(MOE_ERR_SHAPE, "K=%d is not a positive multiple of 32", K);
  if (rows < 0 || rows >= (1LL << 40) / K)
    return fail(MOE_ERR_SHAPE, "rows=%lld is negative, or rows * K reaches 2^40", static_cast<long long>(rows));
  return MOE_OK;
}

int moe_quantize_mxfp4(const uint16_t* src, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                       void* stream) {
  if (int st = check_mx4_rows(rows, K)) return st;
  if (rows == 0) return ok();
  if (!src || !codes || !scales) return fail(MOE_ERR_NULL, "src, codes and scales are required");
  if (!aligned16(src) || !aligned16(codes) || !aligned16(scales))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_quant_mx4(src, rows, K, codes, scales, static_cast<hipStream_t>(stream)),
                    "moe_quantize_mxfp4 launch");
}

int moe_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, uint16_t* dst,
                         void* stream) {
  if (int st = check_mx4_rows(rows, K)) return st;
  if (rows == 0) return ok();
  if (!codes || !scales || !dst) return fail(MOE_ERR_NULL, "codes, scales and dst are required");
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(dst))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_dequant_mx4(codes, scales, rows, K, dst, static_cast<hipStream_t>(stream)),
                    "moe_dequantize_mxfp4 launch");
}

// Sizes that moe_experts_mxfp4 serves (T and k aside, those of its limits).
static int check_mx4(int T, int H, int I, int E, int k, moe_dtype xtype) {
  if (int st = check_common(T, H, I, E, k, 256, 256)) return st;
  if (H > moe::kNormMaxH || I > moe::kNormMaxH)
    return fail(MOE_ERR_SHAPE, "H=%d or I=%d above %d", H, I, moe::kNormMaxH);
  if (xtype != MOE_MXFP8 && xtype != MOE_MXFP4) return fail(MOE_ERR_SHAPE, "xtype=%d", xtype);
  return check_offsets(T, H, I, k);
}

size_t moe_experts_mxfp4_workspace_bytes(int T, int H, int I, int E, int k, moe_dtype xtype) {
  if (T < 1 || check_mx4(T, H, I, E, k, xtype) != MOE_OK) return 0;
  return moe::mx4_ws_layout(T, H, I, E, k, xtype == MOE_MXFP4).total;
}

int moe_experts_mxfp4(const uint8_t* x, const uint8_t* x_scales, moe_dtype xtype,
                      const uint8_t* w_gate_up, const uint8_t* w_gate_up_scales,
                      const uint8_t* w_down, const uint8_t* w_down_scales, const int32_t* topk_idx,
                      const float* topk_w, int T, int H, int I, int E, int k, uint16_t* out,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_mx4(T, H, I, E, k, xtype)) return st;
  if (T == 0) return ok();
  if (!x || !x_scales || !w_gate_up || !w_gate_up_scales || !w_down || !w_down_scales || !topk_idx ||
      !topk_w || !out)
    return fail(MOE_ERR_NULL, "every input and output pointer is required");
  if (!workspace) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = moe::mx4_ws_layout(T, H, I, E, k, xtype == MOE_MXFP4).total;
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  if (!aligned16(x) || !aligned16(x_scales) || !aligned16(w_gate_up) || !aligned16(w_gate_up_scales) ||
      !aligned16(w_down) || !aligned16(w_down_scales) || !aligned16(topk_idx) || !aligned16(topk_w) ||
      !aligned16(out) || !aligned16(workspace))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_experts_mx4(x, x_scales, xtype == MOE_MXFP4, w_gate_up, w_gate_up_scales,
                                            w_down, w_down_scales, topk_idx, topk_w, T, H, I, E, k, out,
                                            workspace, static_cast<hipStream_t>(stream), cus),
                    "moe_experts_mxfp4 launch");
}

static int check_balance(int T, int E, int k, int n_seqs, moe_score score) {
  if (int st = check_scored(T, E, k, score, 1.0f)) return st;
  if (n_seqs < 1 || n_seqs > moe::kMaxSeqs || T % n_seqs)
    return fail(MOE_ERR_SHAPE, "n_seqs=%d is not a divisor of T=%d in [1, %d]", n_seqs, T, moe::kMaxSeqs);
  return MOE_OK;
}

size_t moe_balance_loss_workspace_bytes(int T, int E, int n_seqs) {
  if (T < 0 || T >= moe::kMaxRows || E < 1 || E > 1024 || n_seqs < 1 || n_seqs > moe::kMaxSeqs) return 0;
  return moe::balance_ws_layout(T, E, n_seqs).total;
}

int moe_balance_loss(const float* logits, const int32_t* topk_idx, const uint8_t* token_mask, int T,
                     int E, int k, int n_seqs, moe_score score, float* losses, int32_t* counts,
                     float* probs, int32_t* tokens, void* workspace, size_t workspace_bytes,
                     void* stream) {
  if (int st = check_balance(T, E, k, n_seqs, score)) return st;
  if ((T > 0 && (!logits || !topk_idx)) || !losses || !counts || !probs || !tokens)
    return fail(MOE_ERR_NULL, "logits, topk_idx, losses, counts, probs and tokens are required");
  if (!workspace) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
  const size_t need = moe_balance_loss_workspace_bytes(T, E, n_seqs);
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(token_mask) || !aligned16(losses) ||
      !aligned16(counts) || !aligned16(probs) || !aligned16(tokens) || !aligned16(workspace))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_balance_loss(logits, topk_idx, token_mask, T, E, k, n_seqs,
                                             score == MOE_SCORE_SIGMOID, losses, counts, probs, tokens,
                                             workspace, static_cast<hipStream_t>(stream)),
                    "moe_balance_loss launch");
}

int moe_balance_loss_backward(const float* logits, const uint8_t* token_mask, const int32_t* counts,
                              const int32_t* tokens, const float* d_losses, const float* d_add, int T,
                              int E, int n_seqs, moe_score score, float* dlogits, void* stream) {
  if (int st = check_balance(T, E, 1, n_seqs, score)) return st;
  if (T == 0) return ok();
  if (!logits || !counts || !tokens || !d_losses || !dlogits)
    return fail(MOE_ERR_NULL, "logits, counts, tokens, d_losses and dlogits are required");
  if (!aligned16(logits) || !aligned16(token_mask) || !aligned16(counts) || !aligned16(tokens) ||
      !aligned16(d_losses) || !aligned16(d_add) || !aligned16(dlogits))
    return fail(MOE_ERR_ALIGN, "device pointers must be 16-byte aligned");
  int cus = 0;
  if (int st = device_info(&cus)) return st;
  return hip_status(moe::launch_balance_loss_backward(logits, token_mask, counts, tokens, d_losses, d_add,
                                                      T, E, n_seqs, score == MOE_SCORE_SIGMOID, dlogits,
                                                      static_cast<hipStream_t>(stream)),
                    "moe_balance_loss_backward launch");
}

}  // extern "C"
