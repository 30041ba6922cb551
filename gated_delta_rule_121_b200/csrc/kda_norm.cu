// Group norm over the channels of each row, channels last, with an activation
// (Kimi K3 digest, "Full-rank output gate": y = W_o[sigmoid(W_g x) * RMSNorm(o)],
// the RMSNorm per head; the form with the gate first is the one that
// state-space layers use).
//
// Every element is read once and written once: a team of TPG threads holds a
// group in registers, takes the mean and then the mean of the centred squares
// (two passes over registers, so no cancellation), and writes the result.  HBM
// bandwidth bounds it: 6 bytes per bf16 element with a gate, 4 without.
#include "kda_layer.cuh"

namespace kda {
namespace {

template <int TPG>
__device__ __forceinline__ float team_sum(float v, float* red) {
  constexpr int W = TPG < 32 ? TPG : 32;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPG > 32) {
    constexpr int NW = TPG / 32;
    __syncthreads();  // the previous sum has been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) v += red[i];
  }
  return v;
}

// TPG threads per group, NV pieces of VEC elements per thread.
template <typename T, int VEC, int TPG, int NV>
__global__ void __launch_bounds__(TPG > 256 ? TPG : 256)
    group_norm_kernel(const NormArgs a) {
  using V = Vec<T, VEC>;
  constexpr int THREADS = TPG > 256 ? TPG : 256;
  __shared__ float red[TPG > 32 ? TPG / 32 : 1];
  const int lane = threadIdx.x % TPG;
  const int64_t units = a.rows * a.groups;
  const int64_t u = (int64_t)blockIdx.x * (THREADS / TPG) + threadIdx.x / TPG;
  const bool live = u < units;  // every thread stays for the team's sums
  const int64_t row = live ? u / a.groups : 0;
  const int g = live ? (int)(u - row * a.groups) : 0;
  const int64_t col = (int64_t)g * a.width;
  const T* x = (const T*)a.x + row * a.ldx + col;
  const T* z = a.gate ? (const T*)a.gate + row * a.ldg + col : nullptr;

  V xr[NV], zr[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * TPG + lane) * VEC;
    if (live && e < a.width) {
      xr[v] = *reinterpret_cast<const V*>(x + e);
      if (z) zr[v] = *reinterpret_cast<const V*>(z + e);
    }
  }
  float f[NV][VEC];
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * TPG + lane) * VEC;
    const bool in = live && e < a.width;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      f[v][i] = in ? to_f32(xr[v].v[i]) : 0.f;
      if (in && z && a.gate_first) f[v][i] *= activate(to_f32(zr[v].v[i]), a.act);
      sum += f[v][i];
    }
  }
  const float inv = 1.f / (float)a.width;
  const float mu = a.center ? team_sum<TPG>(sum, red) * inv : 0.f;
  float sq = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const bool in = live && (v * TPG + lane) * VEC < a.width;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      f[v][i] -= mu;
      if (in) sq = fmaf(f[v][i], f[v][i], sq);
    }
  }
  const float r = rsqrtf(team_sum<TPG>(sq, red) * inv + a.eps);
  if (!live) return;
  const int64_t pcol = a.shared ? 0 : col;
  T* out = (T*)a.out + row * ((int64_t)a.groups * a.width) + col;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * TPG + lane) * VEC;
    if (e >= a.width) continue;
    float o[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float n = f[v][i] * r;
      if (a.weight) n *= a.weight[pcol + e + i];
      if (a.bias) n += a.bias[pcol + e + i];
      if (!z) n = activate(n, a.act);
      else if (!a.gate_first) n *= activate(to_f32(zr[v].v[i]), a.act);
      o[i] = n;
    }
    *reinterpret_cast<V*>(out + e) = pack<T, VEC>(o);
  }
}

template <typename T, int VEC, int TPG, int NV>
cudaError_t go(const NormArgs& a, cudaStream_t s) {
  constexpr int THREADS = TPG > 256 ? TPG : 256, TEAMS = THREADS / TPG;
  const int64_t units = a.rows * a.groups;
  const unsigned blocks = (unsigned)((units + TEAMS - 1) / TEAMS);
  group_norm_kernel<T, VEC, TPG, NV><<<blocks, THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

// The smallest team that holds a group in few registers.
template <typename T, int VEC>
cudaError_t by_width(const NormArgs& a, cudaStream_t s) {
  const int pieces = (a.width + VEC - 1) / VEC;
  if (pieces <= 4) return go<T, VEC, 4, 1>(a, s);
  if (pieces <= 8) return go<T, VEC, 8, 1>(a, s);
  if (pieces <= 16) return go<T, VEC, 16, 1>(a, s);
  if (pieces <= 32) return go<T, VEC, 32, 1>(a, s);
  if (pieces <= 64) return go<T, VEC, 32, 2>(a, s);
  if (pieces <= 128) return go<T, VEC, 32, 4>(a, s);
  if (pieces <= 256) return go<T, VEC, 256, 1>(a, s);
  if (pieces <= 512) return go<T, VEC, 256, 2>(a, s);
  if (pieces <= 1024) return go<T, VEC, 512, 2>(a, s);
  if (pieces <= 2048) return go<T, VEC, 512, 4>(a, s);
  if constexpr (VEC <= 4) {
    if (pieces <= 4096) return go<T, VEC, 512, 8>(a, s);
  }
  if constexpr (VEC == 1) return go<T, VEC, 512, 32>(a, s);
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t by_type(const NormArgs& a, cudaStream_t s) {
  constexpr int WIDE = 16 / sizeof(T);
  const int64_t C = (int64_t)a.groups * a.width;
  auto fits = [&](int vec) {
    const int bytes = vec * (int)sizeof(T);
    return a.width % vec == 0 && rows_aligned(a.x, a.ldx, sizeof(T), bytes) &&
           rows_aligned(a.gate, a.ldg, sizeof(T), bytes) && rows_aligned(a.out, C, sizeof(T), bytes);
  };
  return fits(WIDE) ? by_width<T, WIDE>(a, s) : by_width<T, 1>(a, s);
}

}  // namespace

cudaError_t launch_group_norm(const NormArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? by_type<__nv_bfloat16>(a, s) : by_type<float>(a, s);
}

}  // namespace kda
