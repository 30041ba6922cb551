// Shared pieces of the operators around a recurrent layer (short convolution,
// selective scan, group norm): vector loads and stores of 16-byte pieces, the
// activations, and the launchers that the C entry points call.
#pragma once
#include "kda_internal.cuh"

namespace kda {

// N elements of T moved as one access of N * sizeof(T) bytes.
template <typename T, int N>
struct alignas(N * sizeof(T)) Vec {
  T v[N];
};

template <typename T, int N>
__device__ __forceinline__ void unpack(const Vec<T, N>& r, float (&f)[N]) {
  if constexpr (sizeof(T) == 2 && N % 2 == 0) {  // a bf16 is the upper half of the fp32 with its value
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f32(r.v[i]);
  }
}
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> pack(const float (&f)[N]) {
  Vec<T, N> r;
  if constexpr (sizeof(T) == 2 && N % 2 == 0) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = from_f32<T>(f[i]);
  }
  return r;
}

// Elementwise arithmetic, two lanes of the fp32 pipe at a time where N is even:
// a * b, a * s, a * b + c.
template <int N>
__device__ __forceinline__ void vmul(float (&a)[N], const float (&b)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
      a[i] = v.x; a[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] *= b[i];
  }
}
template <int N>
__device__ __forceinline__ void vscale(float (&a)[N], float s) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(s, s));
      a[i] = v.x; a[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] *= s;
  }
}
template <int N>
__device__ __forceinline__ void vadd(float (&a)[N], const float (&b)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = __fadd2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
      a[i] = v.x; a[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] += b[i];
  }
}
template <int N>
__device__ __forceinline__ void vfma(float (&c)[N], const float (&a)[N], const float (&b)[N]) {  // c += a b
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(c[i], c[i + 1]));
      c[i] = v.x; c[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = fmaf(a[i], b[i], c[i]);
  }
}

// N neighbouring fp32 parameters; 16-byte loads where N is a multiple of 4 (their
// offset is then one of 16 bytes, and parameters start on such a boundary).
template <int N>
__device__ __forceinline__ void load_params(const float* p, float (&f)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __ldg(p + i);
  }
}

// s = sigmoid(x) = 1 / (1 + e^-x), elementwise, by the hardware's base-2
// exponential and reciprocal (2 steps each, and |x| / 2 steps from the exponent's
// rounding).  e^-x overflows to infinity below x = -88, where the quotient is
// zero as it should be.
template <int N>
__device__ __forceinline__ void vsigmoid(const float (&x)[N], float (&s)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = x[i];
  vscale(s, -1.4426950408889634f);
#pragma unroll
  for (int i = 0; i < N; ++i) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s[i]) : "f"(s[i]));
  float one[N];
#pragma unroll
  for (int i = 0; i < N; ++i) one[i] = 1.f;
  vadd(s, one);
#pragma unroll
  for (int i = 0; i < N; ++i) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s[i]) : "f"(s[i]));
}

// log(1 + e) for e in [0, 1], relative error within 4 steps: with z = e / (2 + e)
// <= 1/3, log(1 + e) = 2 atanh(z) = 2 z (1 + z^2/3 + z^4/5 + ...); the first
// term left out, z^14/15, is below 1.5e-8.
__device__ __forceinline__ float log1p_unit(float e) {
  const float z = __fdividef(e, 2.f + e), q = z * z;
  float p = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  p = fmaf(q, p, 1.f / 9.f);
  p = fmaf(q, p, 1.f / 7.f);
  p = fmaf(q, p, 1.f / 5.f);
  p = fmaf(q, p, 1.f / 3.f);
  return fmaf(2.f * z * q, p, 2.f * z);
}

// softplus(d) = log(1 + e^d) without overflow: max(d, 0) + log(1 + e^-|d|).
__device__ __forceinline__ float softplus_f32(float d) { return fmaxf(d, 0.f) + log1p_unit(expf(-fabsf(d))); }

// exp(A_log), kept where its product with log2(e) is finite: with an infinite rate a step
// of zero, which leaves the state as it is, would make it no number.  Not a number stays so.
__device__ __forceinline__ float decay_rate(float A_log) {
  const float r = expf(A_log);
  return r > 2e38f ? 2e38f : r;
}

// Sequences of a token tensor: N of T tokens each, or packed by offsets.
// Offsets are cut off at the tensor's T tokens, so that bad ones never lead
// outside it.
struct Seqs {
  const int32_t* cu;
  int N;
  int64_t T;  // tokens per sequence, or in total when packed
  __device__ __forceinline__ int64_t tokens() const { return cu ? T : (int64_t)N * T; }
  __device__ __forceinline__ int64_t begin(int n) const {
    if (!cu) return (int64_t)n * T;
    const int64_t v = cu[n];
    return v < 0 ? 0 : (v < T ? v : T);
  }
  __device__ __forceinline__ int64_t end(int n) const { return cu ? begin(n + 1) : (int64_t)(n + 1) * T; }
  // The sequence that holds token t: the last n with begin(n) <= t (-1 when
  // t lies before all of them; t >= end(n) when it lies behind the last).
  __device__ __forceinline__ int find(int64_t t) const {
    if (!cu) return (int)(t / T);
    int lo = 0, hi = N;  // begin(lo - 1) <= t < begin(hi), taking begin(-1) = -inf
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (begin(mid) <= t) lo = mid + 1; else hi = mid;
    }
    return lo - 1;
  }
};

struct ConvArgs {
  const void* x;
  int64_t ldx;
  const float *weight, *bias;
  const void* init;
  void *out, *fin;
  int N;
  int64_t T;
  int C, K;
  const int32_t* cu;
  int act;
};
cudaError_t launch_conv_fwd(const ConvArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_conv_step(const ConvArgs& a, bool bf16, cudaStream_t s);  // N sequences; fin: the state, in place

struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* gate;
  int64_t ldg;
  const float *weight, *bias;
  void* out;
  int64_t rows;
  int groups, width, shared;
  float eps;
  int center, act, gate_first;
};
constexpr int NORM_MAX_WIDTH = 16384;
cudaError_t launch_group_norm(const NormArgs& a, bool bf16, cudaStream_t s);

struct SsmArgs {
  const void* x;
  int64_t ldx;
  const void* b;
  int64_t ldb;
  const void* c;
  int64_t ldc;
  const float *delta, *A_log, *D, *dt_bias, *init;
  void* out;
  float* fin;
  int N;      // sequences
  int64_t T;  // tokens per sequence, or in total when packed
  int H, G, dk, dv;
  const int32_t* cu;
  DeviceStatus* status;
};
// Prompts: workspace bytes (with the status word) and launches of the two paths.
size_t ssm_simt_workspace(int N, int64_t T, int H, int dk, int dv, bool packed);
cudaError_t launch_ssm_fwd_simt(const SsmArgs& a, void* workspace, bool bf16, cudaStream_t s);
bool ssm_tc_supported(int dk, int dv, bool bf16);
size_t ssm_tc_workspace(int N, int64_t T, int H, int G, int dk, int dv, bool packed);
constexpr uint64_t SSM_WAIT_NS = 2000000000;  // limit of a device-side wait, and the most that can be asked for
constexpr int SSM_NO_STOP = INT32_MAX;
cudaError_t launch_ssm_fwd_tc(const SsmArgs& a, void* workspace, cudaStream_t s, uint64_t wait_ns = SSM_WAIT_NS,
                              int stop_at = SSM_NO_STOP);
cudaError_t launch_ssm_step(const SsmArgs& a, float* state, bool bf16, cudaStream_t s);

// True when every row of `p` starts on a boundary of `bytes` (a power of two).
inline bool rows_aligned(const void* p, int64_t ld, int esz, int bytes) {
  return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld * esz) % bytes == 0);
}

}  // namespace kda
