// C entry points of the operators around a recurrent layer (declared in
// include/kda.h): host-side validation and kernel dispatch.  Nothing here
// allocates or synchronises.
#include <cstdint>

#include "../../include/kda_testing.h"
#include "kda_layer.cuh"

namespace {

constexpr size_t kStatusBytes = 256;  // DeviceStatus + reserve, as in kda_fwd's workspace
constexpr int kMaxChannels = 1 << 20;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool dtype_ok(kda_dtype_t dt) { return dt == KDA_F32 || dt == KDA_BF16; }
int esize(kda_dtype_t dt) { return dt == KDA_BF16 ? 2 : 4; }
kda_status_t result(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// Whether the dense `out` of `rows` rows of `width` elements shares memory with `rows`
// rows of `in_width` elements, `ld` apart.  (Between the rows of a slice it may lie.)
bool shares(const void* out, int64_t width, const void* in, int64_t in_width, int64_t ld, int64_t rows, kda_dtype_t dt) {
  if (!out || !in || rows <= 0) return false;
  const __int128 start = (__int128)reinterpret_cast<uintptr_t>(out) - (__int128)reinterpret_cast<uintptr_t>(in);
  const __int128 end = start + (__int128)rows * width * esize(dt);
  const __int128 step = (__int128)ld * esize(dt), row = (__int128)in_width * esize(dt);
  if (start >= (rows - 1) * step + row) return false;  // behind the last row
  const __int128 first = start < row ? 0 : (start - row) / step + 1;  // the first row that ends behind `start`
  return first * step < end;
}

kda_status_t check_conv(const void* x, int64_t ldx, const float* weight, const float* bias, const void* out, int C,
                        int K, kda_act_t act, kda_dtype_t dt, bool empty) {
  if (C <= 0 || ldx < C || !dtype_ok(dt)) return KDA_ERR_INVALID_ARG;
  if (act != KDA_ACT_NONE && act != KDA_ACT_SILU) return KDA_ERR_INVALID_ARG;
  if (K < 2 || K > 4 || C > kMaxChannels) return KDA_ERR_UNSUPPORTED;
  if (!weight || (!empty && (!x || !out))) return KDA_ERR_INVALID_ARG;
  if (!aligned_to(x, esize(dt))) return KDA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)weight, (const void*)bias, out})
    if (!aligned16(p)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_status_t check_ssm(const void* x, int64_t ldx, const void* b, int64_t ldb, const void* c, int64_t ldc,
                       const float* delta, const float* A_log, const float* D, const float* dt_bias, const void* out,
                       int H, int G, int dk, int dv, kda_dtype_t dt, bool empty) {
  if (H <= 0 || G <= 0 || H % G != 0 || !dtype_ok(dt)) return KDA_ERR_INVALID_ARG;
  if (!dim_ok(dk) || !dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
  if (ldx < (int64_t)H * dv || ldb < (int64_t)G * dk || ldc < (int64_t)G * dk) return KDA_ERR_INVALID_ARG;
  for (int64_t ld : {ldx, ldb, ldc})
    if (ld * esize(dt) % 16 != 0) return KDA_ERR_INVALID_ARG;
  if (!A_log) return KDA_ERR_INVALID_ARG;
  if (!empty && (!x || !b || !c || !delta || !out)) return KDA_ERR_INVALID_ARG;
  if (!aligned_to(delta, 4)) return KDA_ERR_INVALID_ARG;
  for (const void* p : {x, b, c, (const void*)A_log, (const void*)D, (const void*)dt_bias, out})
    if (!aligned16(p)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

// The same of the scan's token inputs: heads and tokens are done in any order.
bool shares_any(const void* out, const void* x, int64_t ldx, const void* b, int64_t ldb, const void* c, int64_t ldc, int H,
                int G, int dk, int dv, int64_t rows, kda_dtype_t dt) {
  const int64_t width = (int64_t)H * dv, keys = (int64_t)G * dk;
  return shares(out, width, x, width, ldx, rows, dt) || shares(out, width, b, keys, ldb, rows, dt) ||
         shares(out, width, c, keys, ldc, rows, dt);
}

kda_status_t ssm_fwd(const void* x, int64_t ldx, const void* b, int64_t ldb, const void* c, int64_t ldc,
                     const float* delta, const float* A_log, const float* D, const float* dt_bias,
                     const float* init_state, void* out, float* final_state, int B, int64_t T, int H, int G,
                     int dk, int dv, const int32_t* cu_seqlens, void* stream, kda_dtype_t dt, void* workspace,
                     size_t workspace_bytes, uint64_t wait_ns = kda::SSM_WAIT_NS, int stop_at = kda::SSM_NO_STOP) {
  if (B < 0 || T < 0) return KDA_ERR_INVALID_ARG;
  if (T > (int64_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;
  const int64_t tokens = cu_seqlens ? T : (int64_t)B * T;
  if (tokens > (int64_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;
  const kda_status_t st =
      check_ssm(x, ldx, b, ldb, c, ldc, delta, A_log, D, dt_bias, out, H, G, dk, dv, dt, tokens == 0 || B == 0);
  if (st != KDA_OK) return st;
  for (const void* p : {(const void*)init_state, (const void*)final_state, (const void*)cu_seqlens})
    if (!aligned16(p)) return KDA_ERR_INVALID_ARG;
  if ((int64_t)B * H > (int64_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < kda_ssm_fwd_workspace_size(B, T, H, G, dk, dv, cu_seqlens != nullptr, dt))
    return KDA_ERR_WORKSPACE;
  if (B > 0 && shares_any(out, x, ldx, b, ldb, c, ldc, H, G, dk, dv, tokens, dt)) return KDA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  kda::DeviceStatus* status = reinterpret_cast<kda::DeviceStatus*>(workspace);
  if (cudaMemsetAsync(status, 0, sizeof(kda::DeviceStatus), s) != cudaSuccess) return KDA_ERR_CUDA;
  if (B == 0) return KDA_OK;
  const kda::SsmArgs a{x, ldx, b, ldb, c, ldc, delta, A_log, D, dt_bias, init_state, out, final_state,
                       B, T, H, G, dk, dv, cu_seqlens, status};
  if (tokens == 0) {  // nothing to walk: the states alone
    if (!final_state) return KDA_OK;
    const size_t bytes = (size_t)B * H * dk * dv * sizeof(float);
    if (!init_state) return result(cudaMemsetAsync(final_state, 0, bytes, s));
    if (final_state == init_state) return KDA_OK;
    return result(cudaMemcpyAsync(final_state, init_state, bytes, cudaMemcpyDeviceToDevice, s));
  }
  if (kda::ssm_tc_supported(dk, dv, dt == KDA_BF16)) return result(kda::launch_ssm_fwd_tc(a, workspace, s, wait_ns, stop_at));
  return result(kda::launch_ssm_fwd_simt(a, workspace, dt == KDA_BF16, s));
}

}  // namespace

extern "C" {

kda_status_t kda_conv_fwd(const void* x, int64_t ldx, const float* weight, const float* bias, const void* init_state,
                          void* out, void* final_state, int B, int64_t T, int C, int K, const int32_t* cu_seqlens,
                          kda_act_t act, void* stream, kda_dtype_t dt) {
  if (B < 0 || T < 0) return KDA_ERR_INVALID_ARG;
  const int64_t tokens = cu_seqlens ? T : (T > INT32_MAX ? T : (int64_t)B * T);
  if (T > (int64_t)INT32_MAX || tokens > (int64_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;
  const kda_status_t st = check_conv(x, ldx, weight, bias, out, C, K, act, dt, tokens == 0 || B == 0);
  if (st != KDA_OK) return st;
  for (const void* p : {init_state, (const void*)final_state, (const void*)cu_seqlens})
    if (!aligned16(p)) return KDA_ERR_INVALID_ARG;
  if (shares(out, C, x, C, ldx, tokens, dt)) return KDA_ERR_INVALID_ARG;  // a token reads the ones before it
  if (B == 0) return KDA_OK;
  const kda::ConvArgs a{x, ldx, weight, bias, init_state, out, final_state, B, T, C, K, cu_seqlens, act};
  return result(kda::launch_conv_fwd(a, dt == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status_t kda_conv_step(const void* x, int64_t ldx, const float* weight, const float* bias, void* state, void* out,
                           int B, int C, int K, kda_act_t act, void* stream, kda_dtype_t dt) {
  if (B < 0) return KDA_ERR_INVALID_ARG;
  const kda_status_t st = check_conv(x, ldx, weight, bias, out, C, K, act, dt, B == 0);
  if (st != KDA_OK) return st;
  if ((B > 0 && !state) || !aligned16(state)) return KDA_ERR_INVALID_ARG;
  if (shares(out, C, x, C, ldx, B, dt)) return KDA_ERR_INVALID_ARG;  // sequences in any order
  if (B == 0) return KDA_OK;
  const kda::ConvArgs a{x, ldx, weight, bias, nullptr, out, state, B, 1, C, K, nullptr, act};
  return result(kda::launch_conv_step(a, dt == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_ssm_fwd_workspace_size(int B, int64_t T, int H, int G, int dk, int dv, int packed, kda_dtype_t dt) {
  if (B <= 0 || T <= 0 || H <= 0 || G <= 0 || H % G != 0 || !dim_ok(dk) || !dim_ok(dv)) return kStatusBytes;
  return kda::ssm_tc_supported(dk, dv, dt == KDA_BF16) ? kda::ssm_tc_workspace(B, T, H, G, dk, dv, packed != 0)
                                                       : kda::ssm_simt_workspace(B, T, H, dk, dv, packed != 0);
}

kda_status_t kda_ssm_fwd(const void* x, int64_t ldx, const void* b, int64_t ldb, const void* c, int64_t ldc,
                         const float* delta, const float* A_log, const float* D, const float* dt_bias,
                         const float* init_state, void* out, float* final_state, int B, int64_t T, int H, int G,
                         int dk, int dv, const int32_t* cu_seqlens, void* stream, kda_dtype_t dt, void* workspace,
                         size_t workspace_bytes) {
  return ssm_fwd(x, ldx, b, ldb, c, ldc, delta, A_log, D, dt_bias, init_state, out, final_state, B, T, H, G, dk, dv,
                 cu_seqlens, stream, dt, workspace, workspace_bytes);
}

// (test hook, include/kda_testing.h)
kda_status_t kda_testing_ssm_fwd(const void* x, int64_t ldx, const void* b, int64_t ldb, const void* c, int64_t ldc,
                                 const float* delta, const float* A_log, const float* D, const float* dt_bias,
                                 const float* init_state, void* out, float* final_state, int B, int64_t T, int H,
                                 int G, int dk, int dv, const int32_t* cu_seqlens, void* stream, kda_dtype_t dt,
                                 void* workspace, size_t workspace_bytes, uint64_t wait_ns, int stop_at) {
  if (!kda::ssm_tc_supported(dk, dv, dt == KDA_BF16)) return KDA_ERR_UNSUPPORTED;
  return ssm_fwd(x, ldx, b, ldb, c, ldc, delta, A_log, D, dt_bias, init_state, out, final_state, B, T, H, G, dk, dv,
                 cu_seqlens, stream, dt, workspace, workspace_bytes, wait_ns, stop_at);
}

kda_status_t kda_ssm_step(const void* x, int64_t ldx, const void* b, int64_t ldb, const void* c, int64_t ldc,
                          const float* delta, const float* A_log, const float* D, const float* dt_bias, float* state,
                          void* out, int B, int H, int G, int dk, int dv, void* stream, kda_dtype_t dt) {
  if (B < 0) return KDA_ERR_INVALID_ARG;
  const kda_status_t st =
      check_ssm(x, ldx, b, ldb, c, ldc, delta, A_log, D, dt_bias, out, H, G, dk, dv, dt, B == 0);
  if (st != KDA_OK) return st;
  if ((B > 0 && !state) || !aligned16(state)) return KDA_ERR_INVALID_ARG;
  if ((int64_t)B * H > (int64_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if (shares_any(out, x, ldx, b, ldb, c, ldc, H, G, dk, dv, B, dt)) return KDA_ERR_INVALID_ARG;
  if (B == 0) return KDA_OK;
  const kda::SsmArgs a{x, ldx, b, ldb, c, ldc, delta, A_log, D, dt_bias, nullptr, out, nullptr,
                       B, 1, H, G, dk, dv, nullptr, nullptr};
  return result(kda::launch_ssm_step(a, state, dt == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status_t kda_group_norm(const void* x, int64_t ldx, const void* gate, int64_t ldg, const float* weight,
                            const float* bias, void* out, int64_t rows, int groups, int width, int shared, float eps,
                            int center, kda_act_t act, int gate_first, void* stream, kda_dtype_t dt) {
  if (rows < 0 || groups <= 0 || width <= 0 || !dtype_ok(dt) || !(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
  if (act != KDA_ACT_NONE && act != KDA_ACT_SILU && act != KDA_ACT_SIGMOID) return KDA_ERR_INVALID_ARG;
  if (gate_first && !gate && rows > 0) return KDA_ERR_INVALID_ARG;
  const int64_t C = (int64_t)groups * width;
  if (ldx < C || (gate && ldg < C)) return KDA_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !out)) return KDA_ERR_INVALID_ARG;
  if (!aligned_to(x, esize(dt)) || !aligned_to(gate, esize(dt))) return KDA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)weight, (const void*)bias, (const void*)out})
    if (!aligned16(p) && p != x && p != gate) return KDA_ERR_INVALID_ARG;
  // An output that is also an input is dense, so that every thread writes where it has read.
  if (rows > 1 && ((out == x && ldx != C) || (out == gate && gate && ldg != C))) return KDA_ERR_INVALID_ARG;
  if (width > kda::NORM_MAX_WIDTH || rows > (int64_t)INT32_MAX / groups) return KDA_ERR_UNSUPPORTED;
  if ((out != x && shares(out, C, x, C, ldx, rows, dt)) || (out != gate && shares(out, C, gate, C, ldg, rows, dt)))
    return KDA_ERR_INVALID_ARG;
  if (rows == 0) return KDA_OK;
  const kda::NormArgs a{x, ldx, gate, ldg, weight, bias, out, rows, groups, width, shared ? 1 : 0,
                        eps, center ? 1 : 0, act, gate_first ? 1 : 0};
  return result(kda::launch_group_norm(a, dt == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
