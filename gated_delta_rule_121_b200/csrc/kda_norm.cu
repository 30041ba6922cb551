// Group norm over the channels of each row, channels last, with an activation
// (Kimi K3 digest, "Full-rank output gate": y = W_o[sigmoid(W_g x) * RMSNorm(o)],
// the RMSNorm per head; the form with the gate first is the one that
// state-space layers use).
//
// Every element is read once and written once: a team of TPG threads holds a
// group in registers, takes the mean and then the mean of the centred squares
// (two passes over registers, so no cancellation), and writes the result.  HBM
// bandwidth bounds it: 6 bytes per bf16 element with a gate, 4 without.
// Measured: 64K rows of 96 groups of 128, bf16 with a gate, 0.71 to 0.81 ms (by where
// the buffers lie), 6.0 to 6.8 TB/s, a copy's rate; 512 rows of one group of 6144 8
// us, most of it the launch.  Groups or rows off 16-byte boundaries are taken element
// by element, which is bound by the accesses: 16K rows of 96 groups of 128 take 188 us,
// of 100 465.
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

// v *= act(g), or v = act(v): one branch per vector.
template <int N>
__device__ __forceinline__ void times_act(float (&v)[N], const float (&g)[N], int act) {
  if (act != KDA_ACT_SIGMOID) vmul(v, g);
  if (act != KDA_ACT_NONE) {
    float s[N];
    vsigmoid(g, s);
    vmul(v, s);
  }
}
template <int N>
__device__ __forceinline__ void to_act(float (&v)[N], int act) {
  if (act == KDA_ACT_NONE) return;
  float s[N];
  vsigmoid(v, s);
  if (act == KDA_ACT_SILU) {
    vmul(v, s);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = s[i];
  }
}

// TPG threads per group, NV pieces of VEC elements per thread, U rows per team
// (the same group of each: its parameters are loaded once, and the rows' loads
// are in flight together).  FULL: every thread's pieces lie inside the group, and
// every team's rows inside the tensor.
template <typename T, int VEC, int TPG, int NV, int U, bool FULL>
__global__ void __launch_bounds__(TPG > 256 ? TPG : 256)
    group_norm_kernel(const NormArgs a) {
  using V = Vec<T, VEC>;
  constexpr int THREADS = TPG > 256 ? TPG : 256;
  __shared__ float red[TPG > 32 ? TPG / 32 : 1];
  const int lane = threadIdx.x % TPG;
  const int64_t team = (int64_t)blockIdx.x * (THREADS / TPG) + threadIdx.x / TPG;
  const int64_t block = team / a.groups;  // of U rows
  const int g = (int)(team - block * a.groups);
  const int64_t row0 = block * U, col = (int64_t)g * a.width;
  auto inside = [&](int u, int v) {
    return FULL || (row0 + u < a.rows && (v * TPG + lane) * VEC < a.width);
  };
  V xr[U][NV], zr[U][NV];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * TPG + lane) * VEC;
      if (inside(u, v)) {
        xr[u][v] = *reinterpret_cast<const V*>((const T*)a.x + (row0 + u) * a.ldx + col + e);
        if (a.gate) zr[u][v] = *reinterpret_cast<const V*>((const T*)a.gate + (row0 + u) * a.ldg + col + e);
      }
    }
  }
  const int64_t pcol = a.shared ? 0 : col;
  const float inv = 1.f / (float)a.width;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // (a team's threads stay for its sums, whatever they hold)
    float f[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (inside(u, v)) {
        unpack(xr[u][v], f[v]);
        if (a.gate_first) {
          float z[VEC];
          unpack(zr[u][v], z);
          times_act(f[v], z, a.act);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[v][i] = 0.f;
      }
    }
    if (a.center) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum += f[v][i];
      const float mu = team_sum<TPG>(sum, red) * inv;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (inside(u, v)) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) f[v][i] -= mu;
        }
    }
    float part[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) part[i] = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) vfma(part, f[v], f[v]);
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) sq += part[i];
    const float r = rsqrtf(team_sum<TPG>(sq, red) * inv + a.eps);
    T* out = (T*)a.out + (row0 + u) * ((int64_t)a.groups * a.width) + col;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * TPG + lane) * VEC;
      if (!inside(u, v)) continue;
      float p[VEC];
      vscale(f[v], r);
      if (a.weight) {
        load_params(a.weight + pcol + e, p);
        vmul(f[v], p);
      }
      if (a.bias) {
        load_params(a.bias + pcol + e, p);
        vadd(f[v], p);
      }
      if (!a.gate) {
        to_act(f[v], a.act);
      } else if (!a.gate_first) {
        unpack(zr[u][v], p);
        times_act(f[v], p, a.act);
      }
      *reinterpret_cast<V*>(out + e) = pack<T, VEC>(f[v]);
    }
  }
}

template <typename T, int VEC, int TPG, int NV, int U>
cudaError_t go_rows(const NormArgs& a, cudaStream_t s) {
  constexpr int THREADS = TPG > 256 ? TPG : 256, TEAMS = THREADS / TPG;
  const int64_t teams = (a.rows + U - 1) / U * a.groups;
  const unsigned blocks = (unsigned)((teams + TEAMS - 1) / TEAMS);
  if (a.width == TPG * NV * VEC && a.rows % U == 0 && teams % TEAMS == 0)
    group_norm_kernel<T, VEC, TPG, NV, U, true><<<blocks, THREADS, 0, s>>>(a);
  else
    group_norm_kernel<T, VEC, TPG, NV, U, false><<<blocks, THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

// Four rows per team where a warp or less holds a group in one piece per thread
// and enough blocks remain, else one.
template <typename T, int VEC, int TPG, int NV>
cudaError_t go(const NormArgs& a, cudaStream_t s) {
  if constexpr (TPG <= 32 && NV == 1) {
    if (a.rows * a.groups / (256 / TPG) >= 4 * 148 * 8) return go_rows<T, VEC, TPG, NV, 4>(a, s);
  }
  return go_rows<T, VEC, TPG, NV, 1>(a, s);
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
