// C ABI of libawq: argument checks, workspace planning, dispatch to the kernels.
// Declarations and the meaning of every argument: include/awq.h.
#include <cuda_runtime.h>

#include <mutex>

#include "../../include/awq.h"
#include "awq_internal.h"

namespace awq {
namespace {

__device__ int g_device_error = 0;  // id of the last bounded device wait that expired (0 = none)

constexpr int kMaxDevices = 64;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Compute capability 10.3 check, cached per device.
awq_status check_arch() {
  static int cached[kMaxDevices] = {0};  // 0 unknown, 1 ok, -1 wrong arch
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return AWQ_ECUDA;
  if (dev < 0 || dev >= kMaxDevices) return AWQ_ECUDA;
  if (cached[dev] == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return AWQ_ECUDA;
    cached[dev] = (major == 10 && minor == 3) ? 1 : -1;
  }
  return cached[dev] == 1 ? AWQ_OK : AWQ_EARCH;
}

awq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? AWQ_OK : AWQ_ECUDA; }

awq_status check_workspace(size_t need, const void* ws, size_t have) {
  if (need == 0) return AWQ_OK;
  if (ws == nullptr || have < need) return AWQ_EWORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return AWQ_EALIGN;
  return AWQ_OK;
}

}  // namespace

int* device_error_ptr() {
  static int* ptrs[kMaxDevices] = {nullptr};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
    ptrs[dev] = static_cast<int*>(p);
  }
  return ptrs[dev];
}

}  // namespace awq

using namespace awq;

extern "C" {

const char* awq_status_string(awq_status status) {
  switch (status) {
    case AWQ_OK: return "AWQ_OK";
    case AWQ_EINVAL: return "AWQ_EINVAL: size or shape argument out of range";
    case AWQ_EALIGN: return "AWQ_EALIGN: pointer not 16-byte aligned (workspace: 256-byte)";
    case AWQ_EARCH: return "AWQ_EARCH: current device is not compute capability 10.3";
    case AWQ_ECUDA: return "AWQ_ECUDA: CUDA runtime call or kernel launch failed";
    case AWQ_ETIMEOUT: return "AWQ_ETIMEOUT: a bounded device-side wait expired";
    case AWQ_EWORKSPACE: return "AWQ_EWORKSPACE: workspace missing or too small";
    case AWQ_ENULL: return "AWQ_ENULL: required pointer is NULL";
    default: return "AWQ: unknown status";
  }
}

awq_status awq_pack(const uint8_t* q, int64_t rows, int64_t n, int32_t* packed, awq_stream_t stream) {
  if (rows < 0 || n < 0 || n % 8 != 0) return AWQ_EINVAL;
  if (rows == 0 || n == 0) return AWQ_OK;
  if (!q || !packed) return AWQ_ENULL;
  if (!aligned16(q) || !aligned16(packed)) return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_pack(q, rows, n, reinterpret_cast<uint32_t*>(packed), (cudaStream_t)stream));
}

awq_status awq_unpack(const int32_t* packed, int64_t rows, int64_t n, uint8_t* q, awq_stream_t stream) {
  if (rows < 0 || n < 0 || n % 8 != 0) return AWQ_EINVAL;
  if (rows == 0 || n == 0) return AWQ_OK;
  if (!q || !packed) return AWQ_ENULL;
  if (!aligned16(q) || !aligned16(packed)) return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_unpack(reinterpret_cast<const uint32_t*>(packed), rows, n, q, (cudaStream_t)stream));
}

awq_status awq_pack_order(const uint8_t* q, int64_t rows, int64_t n, awq_order order, int32_t* packed,
                          awq_stream_t stream) {
  if (order != AWQ_ORDER_OLD && order != AWQ_ORDER_NEW) return AWQ_EINVAL;
  if (rows < 0 || n < 0 || n % 8 != 0) return AWQ_EINVAL;
  if (rows == 0 || n == 0) return AWQ_OK;
  if (!q || !packed) return AWQ_ENULL;
  if (!aligned16(q) || !aligned16(packed)) return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_pack(q, rows, n, reinterpret_cast<uint32_t*>(packed), (cudaStream_t)stream,
                               order == AWQ_ORDER_NEW));
}

awq_status awq_unpack_order(const int32_t* packed, int64_t rows, int64_t n, awq_order order, uint8_t* q,
                            awq_stream_t stream) {
  if (order != AWQ_ORDER_OLD && order != AWQ_ORDER_NEW) return AWQ_EINVAL;
  if (rows < 0 || n < 0 || n % 8 != 0) return AWQ_EINVAL;
  if (rows == 0 || n == 0) return AWQ_OK;
  if (!q || !packed) return AWQ_ENULL;
  if (!aligned16(q) || !aligned16(packed)) return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_unpack(reinterpret_cast<const uint32_t*>(packed), rows, n, q, (cudaStream_t)stream,
                                 order == AWQ_ORDER_NEW));
}

awq_status awq_dequant(const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales, int64_t K,
                       int64_t N, int32_t group_size, uint16_t* w, awq_stream_t stream) {
  if (group_size != 32 && group_size != 64 && group_size != 128 && group_size != 256) return AWQ_EINVAL;
  if (K < 0 || N < 0 || K % group_size != 0 || N % 8 != 0) return AWQ_EINVAL;
  if (K == 0 || N == 0) return AWQ_OK;
  if (!qweight || !scales || !w) return AWQ_ENULL;
  if (!aligned16(qweight) || !aligned16(scales) || !aligned16(w) || (qzeros && !aligned16(qzeros)))
    return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_dequant(reinterpret_cast<const uint32_t*>(qweight),
                                  reinterpret_cast<const uint32_t*>(qzeros), scales, K, N, group_size, w,
                                  (cudaStream_t)stream));
}

awq_status awq_dequant_bf16(const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales, int64_t K,
                            int64_t N, int32_t group_size, uint16_t* w, awq_stream_t stream) {
  if (group_size != 32 && group_size != 64 && group_size != 128 && group_size != 256) return AWQ_EINVAL;
  if (K < 0 || N < 0 || K % group_size != 0 || N % 8 != 0) return AWQ_EINVAL;
  if (K == 0 || N == 0) return AWQ_OK;
  if (!qweight || !scales || !w) return AWQ_ENULL;
  if (!aligned16(qweight) || !aligned16(scales) || !aligned16(w) || (qzeros && !aligned16(qzeros)))
    return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_dequant(reinterpret_cast<const uint32_t*>(qweight),
                                  reinterpret_cast<const uint32_t*>(qzeros), scales, K, N, group_size, w,
                                  (cudaStream_t)stream, true));
}

static bool gemv_shape_ok(int64_t M, int64_t K, int64_t N, int32_t group_size, int32_t split_k) {
  return M >= 0 && M <= kGemvMaxM && K > 0 && K % kGroup == 0 && N > 0 && N % 32 == 0 && group_size == kGroup &&
         split_k >= 0 && K <= (int64_t)1 << 30 && N <= (int64_t)1 << 30;
}
static bool gemm_shape_ok(int64_t M, int64_t K, int64_t N, int32_t split_k) {
  return M >= 0 && M <= (int64_t)1 << 24 && K > 0 && K % kGroup == 0 && K <= (int64_t)1 << 30 && N > 0 &&
         N % 32 == 0 && N <= (int64_t)1 << 30 && split_k >= 0 && M * N < ((int64_t)1 << 40);
}

// W4A8 with at most 16 tokens runs on the GEMV (exact products, int32 reduction) when its plan
// keeps every CTA's rows of a tile within 16384; otherwise, and for more tokens, on the GEMM.
static bool w4a8_on_gemv(int64_t M, int64_t K, int64_t N, int32_t split_k, GemvPlan* plan) {
  if (M < 1 || M > kGemvMaxM) return false;
  *plan = gemv_plan(M, K, N, split_k);
  return gemv_w4a8_ok(*plan, M);
}
// counters | fp16 copy of the codes | GEMV partials (16 token rows per slot; the 8-token instance uses 8)
static size_t w4a8_gemv_workspace_bytes(const GemvPlan& p, int64_t M, int64_t K, int64_t N) {
  const size_t part = gemv_workspace_bytes(p, 16, N);
  return kCounterBytes + align256((size_t)M * (size_t)K * 2) + (part ? part - kCounterBytes : 0);
}

size_t awq_workspace_bytes(awq_op op, int64_t M, int64_t K, int64_t N, int32_t split_k) {
  switch (op) {
    case AWQ_OP_GEMV:
      if (!gemv_shape_ok(M, K, N, kGroup, split_k) || M == 0) return 0;
      return gemv_workspace_bytes(gemv_plan(M, K, N, split_k), M, N);
    case AWQ_OP_GEMM:
      if (!gemm_shape_ok(M, K, N, split_k) || M == 0) return 0;
      return gemm_workspace_bytes(gemm_plan(M, K, N, split_k, kModeZeroPoint), M, K, N, kModeZeroPoint);
    case AWQ_OP_GEMV_BF16:  // sized for the 16-token instance's partials (the 8-token one needs half)
      if (!gemv_shape_ok(M, K, N, kGroup, split_k) || M == 0) return 0;
      return gemv_workspace_bytes(gemv_plan(M, K, N, split_k), 16, N);
    case AWQ_OP_GEMM_BF16:
      if (!gemm_shape_ok(M, K, N, split_k) || M == 0) return 0;
      return gemm_workspace_bytes(gemm_plan(M, K, N, split_k, kModeZeroPointBF16), M, K, N, kModeZeroPointBF16);
    case AWQ_OP_W4A8_GROUPED:
      if (!gemm_shape_ok(M, K, N, split_k) || M == 0) return 0;
      return gemm_workspace_bytes(gemm_plan(M, K, N, split_k, kModeW4A8G), M, K, N, kModeW4A8G);
    case AWQ_OP_GEMV_PREPACKED:
      if (!gemv_shape_ok(M, K, N, kGroup, split_k) || M == 0 || M > 8) return 0;
      return gemv_pp_workspace_bytes(gemv_pp_plan(M, K, N, split_k));
    case AWQ_OP_W4A8_GEMM: {
      if (!gemm_shape_ok(M, K, N, split_k) || M == 0) return 0;
      GemvPlan gp;
      if (w4a8_on_gemv(M, K, N, split_k, &gp)) return w4a8_gemv_workspace_bytes(gp, M, K, N);
      return gemm_workspace_bytes(gemm_plan(M, K, N, split_k, kModeW4A8), M, K, N, kModeW4A8);
    }
    default:
      return 0;
  }
}

awq_status awq_gemv(const uint16_t* x, const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales,
                    uint16_t* y, int64_t M, int64_t K, int64_t N, int32_t group_size, int32_t split_k,
                    void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  if (!gemv_shape_ok(M, K, N, group_size, split_k)) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !qweight || !scales || !y) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(qweight) || !aligned16(scales) || !aligned16(y) || (qzeros && !aligned16(qzeros)))
    return AWQ_EALIGN;
  const GemvPlan plan = gemv_plan(M, K, N, split_k);
  awq_status st = check_workspace(gemv_workspace_bytes(plan, M, N), workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  return from_cuda(launch_gemv(x, reinterpret_cast<const uint32_t*>(qweight), reinterpret_cast<const uint32_t*>(qzeros),
                               scales, y, M, K, N, plan, workspace, err, (cudaStream_t)stream));
}

size_t awq_prepacked_bytes(int64_t K, int64_t N) {
  if (!gemv_shape_ok(1, K, N, kGroup, 0)) return 0;
  return prepacked_bytes(K, N);
}

awq_status awq_prepack_gemv(const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales, int64_t K,
                            int64_t N, int32_t group_size, void* packed, size_t packed_bytes, awq_stream_t stream) {
  if (!gemv_shape_ok(1, K, N, group_size, 0)) return AWQ_EINVAL;
  if (!qweight || !scales || !packed) return AWQ_ENULL;
  if (!aligned16(qweight) || !aligned16(scales) || !aligned16(packed) || (qzeros && !aligned16(qzeros)))
    return AWQ_EALIGN;
  if (packed_bytes < prepacked_bytes(K, N)) return AWQ_EINVAL;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_prepack(reinterpret_cast<const uint32_t*>(qweight), reinterpret_cast<const uint32_t*>(qzeros),
                                  scales, K, N, static_cast<uint8_t*>(packed), (cudaStream_t)stream));
}

awq_status awq_unprepack_gemv(const void* packed, int64_t K, int64_t N, int32_t* qweight, int32_t* qzeros,
                              uint16_t* scales, awq_stream_t stream) {
  if (!gemv_shape_ok(1, K, N, kGroup, 0)) return AWQ_EINVAL;
  if (!packed || !qweight || !scales) return AWQ_ENULL;
  if (!aligned16(packed) || !aligned16(qweight) || !aligned16(scales) || (qzeros && !aligned16(qzeros)))
    return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_unprepack(static_cast<const uint8_t*>(packed), K, N, reinterpret_cast<uint32_t*>(qweight),
                                    reinterpret_cast<uint32_t*>(qzeros), scales, (cudaStream_t)stream));
}

awq_status awq_gemv_prepacked(const uint16_t* x, const void* packed, uint16_t* y, int64_t M, int64_t K, int64_t N,
                              int32_t split_k, void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  if (!gemv_shape_ok(M, K, N, kGroup, split_k) || M > 8) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !packed || !y) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(packed) || !aligned16(y)) return AWQ_EALIGN;
  const GemvPlan plan = gemv_pp_plan(M, K, N, split_k);
  awq_status st = check_workspace(gemv_pp_workspace_bytes(plan), workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  return from_cuda(launch_gemv_prepacked(x, static_cast<const uint8_t*>(packed), y, M, K, N, plan, workspace, err,
                                         (cudaStream_t)stream));
}

awq_status awq_gemv_bf16(const uint16_t* x, const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales,
                         uint16_t* y, int64_t M, int64_t K, int64_t N, int32_t group_size, int32_t split_k,
                         void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  if (!gemv_shape_ok(M, K, N, group_size, split_k)) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !qweight || !scales || !y) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(qweight) || !aligned16(scales) || !aligned16(y) || (qzeros && !aligned16(qzeros)))
    return AWQ_EALIGN;
  const GemvPlan plan = gemv_plan(M, K, N, split_k);
  awq_status st = check_workspace(gemv_workspace_bytes(plan, 16, N), workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  return from_cuda(launch_gemv(x, reinterpret_cast<const uint32_t*>(qweight), reinterpret_cast<const uint32_t*>(qzeros),
                               scales, y, M, K, N, plan, workspace, err, (cudaStream_t)stream, true));
}

awq_status awq_gemm_bf16(const uint16_t* x, const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales,
                         uint16_t* y, int64_t M, int64_t K, int64_t N, int32_t group_size, int32_t split_k,
                         void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  if (!gemm_shape_ok(M, K, N, split_k) || group_size != kGroup) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !qweight || !scales || !y) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(qweight) || !aligned16(scales) || !aligned16(y) || (qzeros && !aligned16(qzeros)))
    return AWQ_EALIGN;
  const int mode = qzeros ? kModeZeroPointBF16 : kModeSymmetricBF16;
  const GemmPlan plan = gemm_plan(M, K, N, split_k, mode);
  awq_status st = check_workspace(gemm_workspace_bytes(plan, M, K, N, mode), workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  void* part = nullptr;
  int* counters = nullptr;
  if (plan.split > 1) {
    if ((int64_t)plan.n_tiles * plan.m_tiles > kMaxCounters) return AWQ_EINVAL;
    counters = static_cast<int*>(workspace);
    part = static_cast<char*>(workspace) + kCounterBytes;
  }
  return from_cuda(launch_gemm(mode, x, reinterpret_cast<const uint32_t*>(qweight),
                               reinterpret_cast<const uint32_t*>(qzeros), scales, nullptr, nullptr, y, nullptr, M,
                               K, N, plan, part, counters, err, (cudaStream_t)stream));
}

awq_status awq_gemm(const uint16_t* x, const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales,
                    uint16_t* y, int64_t M, int64_t K, int64_t N, int32_t group_size, int32_t split_k,
                    void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  if (!gemm_shape_ok(M, K, N, split_k) || group_size != kGroup) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !qweight || !scales || !y) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(qweight) || !aligned16(scales) || !aligned16(y) || (qzeros && !aligned16(qzeros)))
    return AWQ_EALIGN;
  const int mode = qzeros ? kModeZeroPoint : kModeSymmetric;
  const GemmPlan plan = gemm_plan(M, K, N, split_k, mode);
  awq_status st = check_workspace(gemm_workspace_bytes(plan, M, K, N, mode), workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  void* part = nullptr;
  int* counters = nullptr;
  if (plan.split > 1) {
    if ((int64_t)plan.n_tiles * plan.m_tiles > kMaxCounters) return AWQ_EINVAL;
    counters = static_cast<int*>(workspace);
    part = static_cast<char*>(workspace) + kCounterBytes;
  }
  return from_cuda(launch_gemm(mode, x, reinterpret_cast<const uint32_t*>(qweight),
                               reinterpret_cast<const uint32_t*>(qzeros), scales, nullptr, nullptr, y, nullptr, M,
                               K, N, plan, part, counters, err, (cudaStream_t)stream));
}

awq_status w4a8_quant_act(const uint16_t* x, int8_t* xq, float* s_tok, int64_t M, int64_t K, awq_stream_t stream) {
  if (M < 0 || K <= 0 || K % 8 != 0 || M > 0x7FFFFFFF || K > ((int64_t)1 << 30)) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !xq || !s_tok) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(xq)) return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_quant_act(x, xq, s_tok, M, K, (cudaStream_t)stream));
}

}  // extern "C"

// The W4A8 product once `fill` has written the fp16 codes of the activations into the workspace
// (from int8 codes, or by quantizing fp16 activations): the GEMV (up to 16 tokens) or the GEMM, as planned.
template <class Fill>
static awq_status w4a8_product(Fill fill, const float* s_tok, const int32_t* wq, const uint16_t* s_ch, uint16_t* y,
                               int32_t* acc_out, int64_t M, int64_t K, int64_t N, int32_t split_k, void* workspace,
                               size_t workspace_bytes, awq_stream_t stream) {
  GemvPlan gp;
  const bool on_gemv = w4a8_on_gemv(M, K, N, split_k, &gp);
  const GemmPlan plan = gemm_plan(M, K, N, split_k, kModeW4A8);
  const size_t need = on_gemv ? w4a8_gemv_workspace_bytes(gp, M, K, N) : gemm_workspace_bytes(plan, M, K, N, kModeW4A8);
  awq_status st = check_workspace(need, workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  if (!on_gemv && plan.split > 1 && (int64_t)plan.n_tiles * plan.m_tiles > kMaxCounters) return AWQ_EINVAL;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  char* ws = static_cast<char*>(workspace);
  uint16_t* x16 = reinterpret_cast<uint16_t*>(ws + kCounterBytes);
  const cudaStream_t s = (cudaStream_t)stream;
  if (fill(x16, s) != cudaSuccess) return AWQ_ECUDA;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(wq);
  if (on_gemv) return from_cuda(launch_gemv_w4a8(x16, w, s_tok, s_ch, y, acc_out, M, K, N, gp, workspace, err, s));
  void* part = nullptr;
  int* counters = nullptr;
  if (plan.split > 1) {
    counters = reinterpret_cast<int*>(ws);
    part = ws + kCounterBytes + align256((size_t)M * (size_t)K * 2);
  }
  return from_cuda(launch_gemm(kModeW4A8, x16, w, nullptr, nullptr, s_tok, s_ch, y, acc_out, M, K, N, plan, part,
                               counters, err, s));
}

extern "C" {

awq_status w4a8_gemm(const int8_t* xq, const float* s_tok, const int32_t* wq, const uint16_t* s_ch, uint16_t* y,
                     int32_t* acc_out, int64_t M, int64_t K, int64_t N, int32_t split_k, void* workspace,
                     size_t workspace_bytes, awq_stream_t stream) {
  if (!gemm_shape_ok(M, K, N, split_k)) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!xq || !s_tok || !wq || !s_ch || !y) return AWQ_ENULL;
  if (!aligned16(xq) || !aligned16(wq) || !aligned16(s_ch) || !aligned16(y) || (acc_out && !aligned16(acc_out)))
    return AWQ_EALIGN;
  auto widen = [&](uint16_t* x16, cudaStream_t s) { return launch_i8_to_f16(xq, x16, M * K, s); };
  return w4a8_product(widen, s_tok, wq, s_ch, y, acc_out, M, K, N, split_k, workspace, workspace_bytes, stream);
}

awq_status w4a8_linear(const uint16_t* x, const int32_t* wq, const uint16_t* s_ch, uint16_t* y, int32_t* acc_out,
                       int8_t* xq_out, float* s_tok, int64_t M, int64_t K, int64_t N, int32_t split_k,
                       void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  if (!gemm_shape_ok(M, K, N, split_k)) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !s_tok || !wq || !s_ch || !y) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(s_ch) || !aligned16(y) || (acc_out && !aligned16(acc_out)) ||
      (xq_out && !aligned16(xq_out)))
    return AWQ_EALIGN;
  auto quantize = [&](uint16_t* x16, cudaStream_t s) { return launch_quant_act(x, xq_out, s_tok, M, K, s, x16); };
  return w4a8_product(quantize, s_tok, wq, s_ch, y, acc_out, M, K, N, split_k, workspace, workspace_bytes, stream);
}

}  // extern "C"

// The per-group W4A8 product once `fill` has written the fp16 codes of the activations into the workspace:
// the tensor-core GEMM with 1024-row exact chunks (every token count).
template <class Fill>
static awq_status w4a8_grouped_product(Fill fill, const float* s_tok, const int32_t* wq, const uint16_t* s3,
                                       const uint16_t* s2, uint16_t* y, int32_t* acc_out, int64_t M, int64_t K,
                                       int64_t N, int32_t split_k, void* workspace, size_t workspace_bytes,
                                       awq_stream_t stream) {
  const GemmPlan plan = gemm_plan(M, K, N, split_k, kModeW4A8G);
  awq_status st = check_workspace(gemm_workspace_bytes(plan, M, K, N, kModeW4A8G), workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  if (plan.split > 1 && (int64_t)plan.n_tiles * plan.m_tiles > kMaxCounters) return AWQ_EINVAL;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  char* ws = static_cast<char*>(workspace);
  uint16_t* x16 = reinterpret_cast<uint16_t*>(ws + kCounterBytes);
  const cudaStream_t s = (cudaStream_t)stream;
  if (fill(x16, s) != cudaSuccess) return AWQ_ECUDA;
  void* part = nullptr;
  int* counters = nullptr;
  if (plan.split > 1) {
    counters = reinterpret_cast<int*>(ws);
    part = ws + kCounterBytes + align256((size_t)M * (size_t)K * 2);
  }
  return from_cuda(launch_gemm(kModeW4A8G, x16, reinterpret_cast<const uint32_t*>(wq), nullptr, s3, s_tok, s2, y,
                               acc_out, M, K, N, plan, part, counters, err, s));
}

extern "C" {

awq_status w4a8_gemm_grouped(const int8_t* xq, const float* s_tok, const int32_t* wq, const uint16_t* s3,
                             const uint16_t* s2, uint16_t* y, int32_t* acc_out, int64_t M, int64_t K, int64_t N,
                             int32_t group_size, int32_t split_k, void* workspace, size_t workspace_bytes,
                             awq_stream_t stream) {
  if (!gemm_shape_ok(M, K, N, split_k) || group_size != kGroup) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!xq || !s_tok || !wq || !s3 || !s2 || !y) return AWQ_ENULL;
  if (!aligned16(xq) || !aligned16(wq) || !aligned16(s3) || !aligned16(s2) || !aligned16(y) ||
      (acc_out && !aligned16(acc_out)))
    return AWQ_EALIGN;
  auto widen = [&](uint16_t* x16, cudaStream_t s) { return launch_i8_to_f16(xq, x16, M * K, s); };
  return w4a8_grouped_product(widen, s_tok, wq, s3, s2, y, acc_out, M, K, N, split_k, workspace, workspace_bytes,
                              stream);
}

awq_status w4a8_linear_grouped(const uint16_t* x, const int32_t* wq, const uint16_t* s3, const uint16_t* s2,
                               uint16_t* y, int32_t* acc_out, int8_t* xq_out, float* s_tok, int64_t M, int64_t K,
                               int64_t N, int32_t group_size, int32_t split_k, void* workspace,
                               size_t workspace_bytes, awq_stream_t stream) {
  if (!gemm_shape_ok(M, K, N, split_k) || group_size != kGroup) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !s_tok || !wq || !s3 || !s2 || !y) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(s3) || !aligned16(s2) || !aligned16(y) ||
      (acc_out && !aligned16(acc_out)) || (xq_out && !aligned16(xq_out)))
    return AWQ_EALIGN;
  auto quantize = [&](uint16_t* x16, cudaStream_t s) { return launch_quant_act(x, xq_out, s_tok, M, K, s, x16); };
  return w4a8_grouped_product(quantize, s_tok, wq, s3, s2, y, acc_out, M, K, N, split_k, workspace, workspace_bytes,
                              stream);
}

static awq_status rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* res_out,
                          uint16_t* y, int8_t* xq, float* s_tok, int64_t M, int64_t K, int64_t x_stride,
                          int64_t res_stride, float eps, awq_dtype dtype, awq_stream_t stream) {
  if (M < 0 || M > INT32_MAX || K < 8 || K > kNormMaxK || K % 8 != 0 || x_stride < K || x_stride % 8 != 0 ||
      !(eps >= 0.f) || (dtype != AWQ_FP16 && dtype != AWQ_BF16))
    return AWQ_EINVAL;
  if (residual && (res_stride < K || res_stride % 8 != 0)) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !weight) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(res_out) || !aligned16(y) ||
      !aligned16(xq) || (reinterpret_cast<uintptr_t>(s_tok) & 3u) != 0)
    return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_rmsnorm(x, residual, weight, res_out, y, xq, s_tok, M, K, x_stride, res_stride, eps,
                                  dtype == AWQ_BF16, (cudaStream_t)stream));
}

awq_status w4a8_rmsnorm_quant(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* res_out,
                              uint16_t* y, int8_t* xq, float* s_tok, int64_t M, int64_t K, int64_t x_stride,
                              int64_t res_stride, float eps, awq_dtype dtype, awq_stream_t stream) {
  if (M > 0 && (!xq || !s_tok)) return AWQ_ENULL;
  return rmsnorm(x, residual, weight, res_out, y, xq, s_tok, M, K, x_stride, res_stride, eps, dtype, stream);
}

awq_status awq_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* res_out,
                       uint16_t* y, int64_t M, int64_t K, int64_t x_stride, int64_t res_stride, float eps,
                       awq_dtype dtype, awq_stream_t stream) {
  if (M > 0 && !y) return AWQ_ENULL;
  return rmsnorm(x, residual, weight, res_out, y, nullptr, nullptr, M, K, x_stride, res_stride, eps, dtype, stream);
}

static bool kv4_shape_ok(int64_t num_pages, int32_t kv_heads, int32_t dim, int32_t page_size) {
  return num_pages >= 0 && num_pages <= INT32_MAX && kv_heads >= 1 && kv_heads <= 1024 && (dim == 64 || dim == 128) &&
         page_size >= 16 && page_size <= 1024 && page_size % 16 == 0 && (64 % page_size == 0 || page_size % 64 == 0);
}

size_t kv4_cache_bytes(int64_t num_pages, int32_t kv_heads, int32_t head_dim, int32_t page_size) {
  if (!kv4_shape_ok(num_pages, kv_heads, head_dim, page_size)) return 0;
  return (size_t)num_pages * kv_heads * (page_size / kKv4Unit) * kv4_unit_bytes(head_dim);
}

awq_status kv4_append(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t q_stride, int64_t k_stride,
                      int64_t v_stride, const int32_t* positions, const int64_t* slots, const float* table,
                      int64_t max_pos, int32_t rot_dim, int32_t interleaved, uint16_t* q_out, int64_t q_out_stride,
                      void* cache, int64_t num_pages, int64_t T, int32_t heads, int32_t kv_heads, int32_t head_dim,
                      int32_t page_size, awq_dtype dtype, awq_stream_t stream) {
  if (heads < 0 || heads > 1024 || kv_heads < 0 || !kv4_shape_ok(num_pages, kv_heads ? kv_heads : 1, head_dim, page_size))
    return AWQ_EINVAL;
  if (T < 0 || T > INT32_MAX || rot_dim < 0 || rot_dim > head_dim || rot_dim % 8 != 0 || max_pos < 0 ||
      (dtype != AWQ_FP16 && dtype != AWQ_BF16))
    return AWQ_EINVAL;
  const int64_t qw = (int64_t)heads * head_dim, kw = (int64_t)kv_heads * head_dim;
  if (heads && (q_stride < qw || q_stride % 8 != 0 || q_out_stride < qw || q_out_stride % 8 != 0)) return AWQ_EINVAL;
  if (kv_heads && (k_stride < kw || k_stride % 8 != 0 || v_stride < kw || v_stride % 8 != 0)) return AWQ_EINVAL;
  if (T == 0 || heads + kv_heads == 0) return AWQ_OK;
  if ((heads && (!q || !q_out)) || (kv_heads && (!k || !v || !slots || !cache)) || (rot_dim && (!positions || !table)))
    return AWQ_ENULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(cache) || !aligned16(table) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u) != 0 || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
    return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  const Kv4Rope rope{positions, table, max_pos, rot_dim, interleaved != 0};
  return from_cuda(launch_kv4_append(q, k, v, q_stride, k_stride, v_stride, slots, rope, q_out, q_out_stride,
                                     static_cast<uint8_t*>(cache), Kv4Shape{num_pages, kv_heads, head_dim, page_size}, T,
                                     heads, dtype == AWQ_BF16, (cudaStream_t)stream));
}

awq_status kv4_gather(const void* cache, const int64_t* slots, uint16_t* k, uint16_t* v, int64_t num_pages, int64_t T,
                      int32_t kv_heads, int32_t head_dim, int32_t page_size, awq_dtype dtype, awq_stream_t stream) {
  if (!kv4_shape_ok(num_pages, kv_heads, head_dim, page_size) || T < 0 || T > INT32_MAX ||
      (dtype != AWQ_FP16 && dtype != AWQ_BF16))
    return AWQ_EINVAL;
  if (T == 0 || (!k && !v)) return AWQ_OK;
  if (!cache || !slots) return AWQ_ENULL;
  if (!aligned16(cache) || !aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
    return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_kv4_gather(static_cast<const uint8_t*>(cache), slots, k, v,
                                     Kv4Shape{num_pages, kv_heads, head_dim, page_size}, T, dtype == AWQ_BF16,
                                     (cudaStream_t)stream));
}

static bool kv4_attention_shape_ok(int64_t T, int64_t B, int32_t max_q, int32_t heads, int32_t kv_heads, int32_t dim) {
  return T >= 0 && T <= INT32_MAX && B >= 0 && B <= kKv4MaxSeqs && max_q >= 1 && heads >= 1 && heads <= 1024 &&
         kv_heads >= 1 && heads % kv_heads == 0 && (dim == 64 || dim == 128) &&
         (max_q < T ? max_q : T) * (heads / kv_heads) <= kKv4MaxRows;
}

size_t kv4_attention_workspace_bytes(int64_t T, int64_t B, int32_t max_q, int32_t heads, int32_t kv_heads,
                                     int32_t head_dim) {
  if (!kv4_attention_shape_ok(T, B, max_q, heads, kv_heads, head_dim)) return 0;
  return kv4_attention_workspace(T, B, max_q, heads, kv_heads, head_dim);
}

awq_status kv4_attention(const uint16_t* q, int64_t q_stride, const void* cache, const int32_t* block_table,
                         int64_t table_stride, const int32_t* kv_len, const int32_t* q_start, uint16_t* out, float* lse,
                         int64_t T, int64_t B, int32_t max_q, int32_t heads, int32_t kv_heads, int32_t head_dim,
                         int64_t num_pages, int32_t page_size, int32_t max_pages, float scale, int32_t window,
                         awq_dtype dtype, void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  if (!kv4_attention_shape_ok(T, B, max_q, heads, kv_heads, head_dim) ||
      !kv4_shape_ok(num_pages, kv_heads, head_dim, page_size) || num_pages < 1)
    return AWQ_EINVAL;
  if (q_stride < (int64_t)heads * head_dim || q_stride % 8 != 0 || max_pages < 1 || table_stride < max_pages ||
      (int64_t)max_pages * page_size > (1 << 30) || !(scale - scale == 0.f) || window < 0 ||
      (dtype != AWQ_FP16 && dtype != AWQ_BF16))
    return AWQ_EINVAL;
  if (!q_start && (T != B || max_q != 1)) return AWQ_EINVAL;
  if (T == 0 || B == 0) return AWQ_OK;
  if (!q || !cache || !block_table || !kv_len || !out) return AWQ_ENULL;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || (reinterpret_cast<uintptr_t>(block_table) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(kv_len) & 3u) != 0 || (reinterpret_cast<uintptr_t>(q_start) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return AWQ_EALIGN;
  awq_status st = check_workspace(kv4_attention_workspace(T, B, max_q, heads, kv_heads, head_dim), workspace,
                                  workspace_bytes);
  if (st != AWQ_OK) return st;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  // one that no sequence can outgrow is none: the kernels' positions less a window stay within 32 bits
  if (window >= (int64_t)max_pages * page_size) window = 0;
  const Kv4AttnArgs a{q,     q_stride, static_cast<const uint8_t*>(cache), block_table, table_stride, kv_len,
                      q_start, out,    lse,                                T,           (int)B,       max_q,
                      heads, kv_heads, num_pages,                          page_size,   max_pages,    scale,
                      window};
  return from_cuda(launch_kv4_attention(a, head_dim, dtype == AWQ_BF16, workspace, err, (cudaStream_t)stream));
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
static bool is_dtype(awq_dtype d) { return d == AWQ_FP16 || d == AWQ_BF16; }
// Whether `bytes` from p on share any with n rows of row_bytes each, `stride` bytes apart (>= row_bytes), from `rows` on.
static bool overlaps(const void* p, int64_t bytes, const void* rows, int64_t n, int64_t row_bytes, int64_t stride) {
  const int64_t begin = (int64_t)(reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(rows)), end = begin + bytes;
  const int64_t first = begin < row_bytes ? 0 : (begin - row_bytes) / stride + 1;  // the first row that ends behind `begin`
  return first < n && first * stride < end;
}

awq_status awq_moe_plan(const int32_t* ids, int64_t R, int32_t experts, int32_t* offsets, int32_t* order, int32_t* place,
                        awq_stream_t stream) {
  if (R < 0 || R > kMoeMaxRows || experts < 1 || experts > kMoeMaxExperts) return AWQ_EINVAL;
  if (!offsets || (R > 0 && (!ids || !order || !place))) return AWQ_ENULL;
  if (!aligned4(ids) || !aligned4(offsets) || !aligned4(order) || !aligned4(place)) return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_moe_plan(ids, R, experts, offsets, order, place, (cudaStream_t)stream));
}

awq_status awq_moe_route(const void* logits, int64_t logits_stride, int64_t T, int32_t experts, int32_t top_k,
                         int32_t normalize, awq_logits_type type, int32_t* ids, float* weights, int32_t* offsets,
                         int32_t* order, int32_t* place, awq_stream_t stream) {
  if (experts < 1 || experts > kMoeMaxExperts || top_k < 1 || top_k > experts || top_k > kMoeMaxTopK || T < 0 ||
      T > kMoeMaxRows / top_k || logits_stride < experts ||
      (type != AWQ_LOGITS_FP16 && type != AWQ_LOGITS_BF16 && type != AWQ_LOGITS_FP32))
    return AWQ_EINVAL;
  if (T > 0 && (!logits || !ids || !weights)) return AWQ_ENULL;
  if (T > 0 && ((offsets != nullptr) != (order != nullptr) || (offsets != nullptr) != (place != nullptr))) return AWQ_ENULL;
  const uintptr_t element = type == AWQ_LOGITS_FP32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(logits) & (element - 1)) != 0 || !aligned4(ids) || !aligned4(weights) ||
      !aligned4(offsets) || !aligned4(order) || !aligned4(place))
    return AWQ_EALIGN;
  if (T == 0 && !offsets) return AWQ_OK;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_moe_route(logits, logits_stride, T, experts, top_k, normalize != 0, (int)type, ids, weights,
                                    offsets, order, place, (cudaStream_t)stream));
}

static bool moe_shape_ok(int32_t experts, int64_t K, int64_t N, int32_t gated) {
  return experts >= 1 && experts <= kMoeMaxExperts && K >= kGroup && K <= kMoeMaxSize && K % kGroup == 0 && N >= 1 &&
         N <= kMoeMaxSize && N % (gated ? 64 : 32) == 0;
}

size_t awq_moe_prepacked_bytes(int32_t experts, int64_t K, int64_t N, int32_t gated) {
  if (!moe_shape_ok(experts, K, N, gated)) return 0;
  return (size_t)experts * (size_t)moe_tiles(N, gated != 0) * (size_t)(K / kGroup) * kMoeUnitBytes;
}

awq_status awq_moe_prepack(const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales, int32_t experts, int64_t K,
                           int64_t N, int32_t group_size, int32_t gated, void* packed, size_t packed_bytes,
                           awq_stream_t stream) {
  const size_t need = awq_moe_prepacked_bytes(experts, K, N, gated);
  if (need == 0 || group_size != kGroup || packed_bytes < need) return AWQ_EINVAL;
  if (!qweight || !scales || !packed) return AWQ_ENULL;
  if (!aligned16(qweight) || !aligned16(qzeros) || !aligned16(scales) || !aligned16(packed)) return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_moe_prepack(reinterpret_cast<const uint32_t*>(qweight), reinterpret_cast<const uint32_t*>(qzeros),
                                      scales, experts, K, N, gated != 0, static_cast<uint8_t*>(packed),
                                      (cudaStream_t)stream));
}

awq_status awq_moe_unprepack(const void* packed, int32_t experts, int64_t K, int64_t N, int32_t gated, int32_t* qweight,
                             int32_t* qzeros, uint16_t* scales, awq_stream_t stream) {
  if (!moe_shape_ok(experts, K, N, gated)) return AWQ_EINVAL;
  if (!qweight || !scales || !packed) return AWQ_ENULL;
  if (!aligned16(qweight) || !aligned16(qzeros) || !aligned16(scales) || !aligned16(packed)) return AWQ_EALIGN;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_moe_unprepack(static_cast<const uint8_t*>(packed), experts, K, N, gated != 0,
                                        reinterpret_cast<uint32_t*>(qweight), reinterpret_cast<uint32_t*>(qzeros), scales,
                                        (cudaStream_t)stream));
}

size_t awq_moe_gemm_workspace_bytes(int64_t R, int32_t experts, int64_t K, int64_t N, int32_t gated) {
  if (R < 1 || R > kMoeMaxRows || !moe_shape_ok(experts, K, N, gated)) return 0;
  return moe_gemm_workspace(R, experts, K, true);
}

awq_status awq_moe_gemm(const uint16_t* x, int64_t x_stride, int64_t x_rows, const void* packed, const int32_t* offsets,
                        const int32_t* order, int32_t top_k, void* y, int32_t y_fp32, int64_t R, int32_t experts, int64_t K,
                        int64_t N, int32_t gated, awq_dtype dtype, void* workspace, size_t workspace_bytes,
                        awq_stream_t stream) {
  if (R < 0 || R > kMoeMaxRows || x_rows < (R > 0 ? 1 : 0) || x_rows > kMoeMaxRows || !moe_shape_ok(experts, K, N, gated) ||
      x_stride < K || x_stride % 8 != 0 || !is_dtype(dtype) || (order && (top_k < 1 || top_k > kMoeMaxTopK)))
    return AWQ_EINVAL;
  if (R == 0) return AWQ_OK;
  if (!packed || !offsets || !y || !x) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(packed) || !aligned16(y) || !aligned4(offsets) || !aligned4(order)) return AWQ_EALIGN;
  awq_status st = check_workspace(moe_gemm_workspace(R, experts, K, true), workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  if (overlaps(y, R * (gated ? N / 2 : N) * (y_fp32 ? 4 : 2), x, x_rows, K * 2, x_stride * 2)) return AWQ_EINVAL;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  const MoeGemmArgs a{x, x_stride, x_rows, static_cast<const uint8_t*>(packed), offsets, order, order ? top_k : 1,
                      y, R,        experts, K, N, (int)moe_tiles(N, gated != 0), false};
  return from_cuda(launch_moe_gemm(a, gated != 0, y_fp32 != 0, dtype == AWQ_BF16, workspace, err, (cudaStream_t)stream));
}

// Results [T, H] may be the residual itself, piece by piece, or have no memory in common with it.
static bool may_add_to(const uint16_t* out, const uint16_t* residual, int64_t T, int64_t H, int64_t res_stride) {
  return !residual || (out == residual && (res_stride == H || T == 1)) || !overlaps(out, T * H * 2, residual, T, H * 2, res_stride * 2);
}

awq_status awq_moe_combine(const void* y, int32_t y_fp32, const int32_t* place, const float* weights, const uint16_t* residual,
                           int64_t res_stride, uint16_t* out, int64_t T, int32_t top_k, int64_t H, int64_t R,
                           awq_dtype dtype, awq_stream_t stream) {
  if (top_k < 1 || top_k > kMoeMaxTopK || T < 0 || T > kMoeMaxRows / top_k || R < 0 || R > kMoeMaxRows || H < 8 ||
      H > kMoeMaxSize || H % 8 != 0 || !is_dtype(dtype))
    return AWQ_EINVAL;
  if (residual && (res_stride < H || res_stride % 8 != 0)) return AWQ_EINVAL;
  if (T == 0) return AWQ_OK;
  if ((R > 0 && !y) || !place || !weights || !out) return AWQ_ENULL;
  if (!aligned16(y) || !aligned16(residual) || !aligned16(out) || !aligned4(place) || !aligned4(weights)) return AWQ_EALIGN;
  if (overlaps(out, T * H * 2, y, R, H * (y_fp32 ? 4 : 2), H * (y_fp32 ? 4 : 2)) || !may_add_to(out, residual, T, H, res_stride))
    return AWQ_EINVAL;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_moe_combine(y, y_fp32 != 0, place, weights, residual, res_stride, out, T, top_k, H, R, dtype == AWQ_BF16,
                                      (cudaStream_t)stream));
}

// Workspace of the whole layer: what the products need | rows between up and down | rows between down and the sum.
struct MoeLayout {
  size_t product, rows, bytes;
};
static bool moe_layout(int64_t T, int32_t top_k, int32_t experts, int64_t K, int64_t inner, int64_t H, MoeLayout& l) {
  if (top_k < 1 || top_k > kMoeMaxTopK || T < 0 || T > kMoeMaxRows / top_k || inner < 1 || inner > kMoeMaxSize / 2 ||
      !moe_shape_ok(experts, K, 2 * inner, 1) || !moe_shape_ok(experts, inner, H, 0))
    return false;
  const int64_t R = T * top_k;
  const size_t up = moe_gemm_workspace(R, experts, K, true), down = moe_gemm_workspace(R, experts, inner, false);
  l.product = align256(up > down ? up : down);
  l.rows = align256((size_t)R * (size_t)inner * 2);
  l.bytes = l.product + l.rows + (size_t)R * (size_t)H * 4;
  return true;
}

size_t awq_moe_workspace_bytes(int64_t T, int32_t top_k, int32_t experts, int64_t K, int64_t inner, int64_t H) {
  MoeLayout l;
  return moe_layout(T, top_k, experts, K, inner, H, l) && T > 0 ? l.bytes : 0;
}

awq_status awq_moe(const uint16_t* x, int64_t x_stride, const void* up, const void* down, const int32_t* offsets,
                   const int32_t* order, const int32_t* place, const float* weights, const uint16_t* residual,
                   int64_t res_stride, uint16_t* out, int64_t T, int32_t top_k, int32_t experts, int64_t K, int64_t inner,
                   int64_t H, awq_dtype dtype, void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  MoeLayout l;
  if (!moe_layout(T, top_k, experts, K, inner, H, l) || x_stride < K || x_stride % 8 != 0 || !is_dtype(dtype)) return AWQ_EINVAL;
  if (residual && (res_stride < H || res_stride % 8 != 0)) return AWQ_EINVAL;
  if (T == 0) return AWQ_OK;
  if (!x || !up || !down || !offsets || !order || !place || !weights || !out) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(up) || !aligned16(down) || !aligned16(residual) || !aligned16(out) || !aligned4(offsets) ||
      !aligned4(order) || !aligned4(place) || !aligned4(weights))
    return AWQ_EALIGN;
  awq_status st = check_workspace(l.bytes, workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  if (!may_add_to(out, residual, T, H, res_stride)) return AWQ_EINVAL;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  const cudaStream_t s = (cudaStream_t)stream;
  const bool bf16 = dtype == AWQ_BF16;
  const int64_t R = T * top_k;
  uint16_t* h = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + l.product);
  float* y = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + l.product + l.rows);
  const MoeGemmArgs first{x, x_stride, T, static_cast<const uint8_t*>(up), offsets, order, top_k,
                          h, R,        experts, K, 2 * inner, (int)moe_tiles(2 * inner, true), false};
  if (launch_moe_gemm(first, true, false, bf16, workspace, err, s) != cudaSuccess) return AWQ_ECUDA;
  // up has waited for what wrote the plan: down reads it, and its weights, while up runs
  const MoeGemmArgs second{h, inner, R, static_cast<const uint8_t*>(down), offsets, nullptr, 1,
                           y, R,     experts, inner, H, (int)moe_tiles(H, false), true};
  if (launch_moe_gemm(second, false, true, bf16, workspace, err, s) != cudaSuccess) return AWQ_ECUDA;
  return from_cuda(launch_moe_combine(y, true, place, weights, residual, res_stride, out, T, top_k, H, R, bf16, s));
}

// ---- e4m3 linear layers

static bool fp8_shape_ok(int64_t M, int64_t K, int64_t N) {
  return M >= 0 && M <= kMoeMaxRows && K >= 16 && K <= kMoeMaxSize && K % 16 == 0 && N >= 8 && N <= kMoeMaxSize && N % 8 == 0;
}

awq_status awq_fp8_quant_act(const uint16_t* x, int64_t x_stride, uint8_t* xq, float* s_x, int64_t M, int64_t K,
                             awq_dtype dtype, awq_stream_t stream) {
  if (!fp8_shape_ok(M, K, 8) || x_stride < K || x_stride % 8 != 0 || !is_dtype(dtype)) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !xq || !s_x) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(xq) || !aligned4(s_x)) return AWQ_EALIGN;
  if (overlaps(xq, M * K, x, M, K * 2, x_stride * 2)) return AWQ_EINVAL;
  awq_status st = check_arch();
  if (st != AWQ_OK) return st;
  return from_cuda(launch_fp8_quant(x, x_stride, xq, s_x, M, K, dtype == AWQ_BF16, (cudaStream_t)stream));
}

size_t awq_fp8_gemm_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  return fp8_shape_ok(M, K, N) && M > 0 ? fp8_gemm_workspace(M, K, N) : 0;
}

awq_status awq_fp8_gemm(const uint8_t* xq, const float* s_x, const uint8_t* wq, const float* s_w, uint16_t* y, int64_t M,
                        int64_t K, int64_t N, awq_dtype dtype, void* workspace, size_t workspace_bytes,
                        awq_stream_t stream) {
  if (!fp8_shape_ok(M, K, N) || !is_dtype(dtype)) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!xq || !s_x || !wq || !s_w || !y) return AWQ_ENULL;
  if (!aligned16(xq) || !aligned16(wq) || !aligned16(y) || !aligned4(s_x) || !aligned4(s_w)) return AWQ_EALIGN;
  awq_status st = check_workspace(fp8_gemm_workspace(M, K, N), workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  if (overlaps(y, M * N * 2, xq, M, K, K)) return AWQ_EINVAL;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  return from_cuda(launch_fp8_gemm(Fp8GemmArgs{nullptr, 0, xq, s_x, wq, s_w, y, M, K, N}, dtype == AWQ_BF16, workspace, err,
                                   (cudaStream_t)stream));
}

// The product's own workspace, whose counters no other call's codes may fall on, then codes and scales.
static size_t fp8_codes_offset(int64_t M, int64_t K, int64_t N) {
  const size_t own = align256(fp8_gemm_workspace(M, K, N));
  return own < kCounterBytes ? kCounterBytes : own;
}
size_t awq_fp8_linear_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (!fp8_shape_ok(M, K, N) || M == 0) return 0;
  return fp8_codes_offset(M, K, N) + align256((size_t)M * (size_t)K) + (size_t)M * (size_t)((K + kGroup - 1) / kGroup) * 4;
}

awq_status awq_fp8_linear(const uint16_t* x, int64_t x_stride, const uint8_t* wq, const float* s_w, uint16_t* y, int64_t M,
                          int64_t K, int64_t N, awq_dtype dtype, void* workspace, size_t workspace_bytes,
                          awq_stream_t stream) {
  if (!fp8_shape_ok(M, K, N) || x_stride < K || x_stride % 8 != 0 || !is_dtype(dtype)) return AWQ_EINVAL;
  if (M == 0) return AWQ_OK;
  if (!x || !wq || !s_w || !y) return AWQ_ENULL;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(y) || !aligned4(s_w)) return AWQ_EALIGN;
  awq_status st = check_workspace(awq_fp8_linear_workspace_bytes(M, K, N), workspace, workspace_bytes);
  if (st != AWQ_OK) return st;
  st = check_arch();
  if (st != AWQ_OK) return st;
  int* err = device_error_ptr();
  if (!err) return AWQ_ECUDA;
  uint8_t* xq = static_cast<uint8_t*>(workspace) + fp8_codes_offset(M, K, N);
  float* s_x = reinterpret_cast<float*>(xq + align256((size_t)M * (size_t)K));
  const cudaStream_t s = (cudaStream_t)stream;
  const bool bf16 = dtype == AWQ_BF16;
  // the form of few tokens reads x to the end of the launch that writes y
  if (M <= kFp8FusedTokens && !overlaps(y, M * N * 2, x, M, K * 2, x_stride * 2))
    return from_cuda(launch_fp8_gemm(Fp8GemmArgs{x, x_stride, nullptr, nullptr, wq, s_w, y, M, K, N}, bf16, workspace, err, s));
  if (launch_fp8_quant(x, x_stride, xq, s_x, M, K, bf16, s) != cudaSuccess) return AWQ_ECUDA;
  return from_cuda(launch_fp8_gemm(Fp8GemmArgs{nullptr, 0, xq, s_x, wq, s_w, y, M, K, N}, bf16, workspace, err, s));
}

awq_status awq_last_device_error(int32_t* code) {
  if (!code) return AWQ_ENULL;
  *code = 0;
  int* p = device_error_ptr();
  if (!p) return AWQ_ECUDA;
  if (cudaDeviceSynchronize() != cudaSuccess) return AWQ_ECUDA;
  int v = 0;
  if (cudaMemcpy(&v, p, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return AWQ_ECUDA;
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpy(p, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return AWQ_ECUDA;
  }
  *code = v;
  return v ? AWQ_ETIMEOUT : AWQ_OK;
}

}  // extern "C"
