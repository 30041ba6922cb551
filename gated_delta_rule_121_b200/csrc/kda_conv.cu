// Short depthwise causal convolution with an activation (Kimi K3 digest,
// "Kimi Delta Attention" section: a convolution of kernel size 4 and a Swish
// on q, k and v before the recurrence), for prompts and for single tokens.
//
//   out_t[c] = act(bias[c] + sum_{j<K} weight[c][j] x_{t-K+1+j}[c])
//
// A prompt moves 2 elements per K multiply-adds, so HBM bandwidth bounds it.
// A thread owns VEC neighbouring channels and RUN consecutive tokens: the RUN
// loads are issued before the first product, the K - 1 inputs before the run
// stay in registers, and a warp's accesses are 32 * VEC contiguous elements.
// Threads of a block take consecutive runs of the same channels, so that the
// inputs before a run come from L1.
#include "kda_layer.cuh"

namespace kda {
namespace {

constexpr int RUN = 8;    // tokens per thread
constexpr int WARPS = 8;  // runs per block

template <typename T, int VEC, int K>
struct Taps {
  float w[VEC][K], b[VEC];
  __device__ __forceinline__ void load(const float* weight, const float* bias, int c) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
      for (int j = 0; j < K; ++j) w[i][j] = weight[(int64_t)(c + i) * K + j];
      b[i] = bias ? bias[c + i] : 0.f;
    }
  }
  // rows: the K - 1 inputs before this one (oldest first), then this one
  __device__ __forceinline__ Vec<T, VEC> apply(const Vec<T, VEC>* const (&rows)[K], int act) const {
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = b[i];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float f[VEC];
      unpack(*rows[j], f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w[i][j], f[i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = activate(acc[i], act);
    return pack<T, VEC>(acc);
  }
};

// Row `pos` (negative: before the sequence) of sequence n starting at token t0.
template <typename T, int VEC, int K>
__device__ __forceinline__ Vec<T, VEC> input_row(const T* x, int64_t ldx, const T* init, int64_t t0, int n,
                                                 int64_t pos, int C, int c) {
  using V = Vec<T, VEC>;
  if (pos >= 0) return *reinterpret_cast<const V*>(x + (t0 + pos) * ldx + c);
  if (init) return *reinterpret_cast<const V*>(init + ((int64_t)n * (K - 1) + (pos + K - 1)) * C + c);
  V z;
#pragma unroll
  for (int i = 0; i < VEC; ++i) z.v[i] = from_f32<T>(0.f);
  return z;
}

// The state after sequence n: its last K - 1 inputs.  All rows are read before
// the first is written, so the state may be the initial one.
template <typename T, int VEC, int K>
__device__ __forceinline__ void final_rows(const T* x, int64_t ldx, const T* init, T* fin, const Seqs& q, int n,
                                           int C, int c) {
  using V = Vec<T, VEC>;
  const int64_t t0 = q.begin(n);
  int64_t L = q.end(n) - t0;
  if (L < 0) L = 0;
  V r[K - 1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) r[j] = input_row<T, VEC, K>(x, ldx, init, t0, n, L - (K - 1) + j, C, c);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) *reinterpret_cast<V*>(fin + ((int64_t)n * (K - 1) + j) * C + c) = r[j];
}

// Blocks [0, run_blocks) in y: the runs; the blocks behind them: final states.
template <typename T, int VEC, int K>
__global__ void __launch_bounds__(32 * WARPS)
    conv_fwd_kernel(const T* __restrict__ x, int64_t ldx, const float* __restrict__ weight,
                    const float* __restrict__ bias, const T* init, T* __restrict__ out, T* fin, Seqs q, int C,
                    int act, int run_blocks) {
  using V = Vec<T, VEC>;
  const int c = (blockIdx.y * 32 + (threadIdx.x & 31)) * VEC;
  if (c >= C) return;
  const int warp = threadIdx.x >> 5;
  if ((int)blockIdx.x >= run_blocks) {
    const int n = ((int)blockIdx.x - run_blocks) * WARPS + warp;
    if (n < q.N) final_rows<T, VEC, K>(x, ldx, init, fin, q, n, C, c);
    return;
  }
  const int64_t t0 = ((int64_t)blockIdx.x * WARPS + warp) * RUN, Ttot = q.tokens();
  if (t0 >= Ttot) return;
  int n = q.find(t0);
  int64_t s0 = n >= 0 ? q.begin(n) : 0, s1 = n >= 0 ? q.end(n) : q.begin(0);
  Taps<T, VEC, K> taps;
  if (n >= 0 && t0 + RUN <= s1) {  // the whole run lies in one sequence
    V r[K - 1 + RUN];
#pragma unroll
    for (int j = 0; j < RUN; ++j) r[K - 1 + j] = *reinterpret_cast<const V*>(x + (t0 + j) * ldx + c);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j] = input_row<T, VEC, K>(x, ldx, init, s0, n, t0 - s0 - (K - 1) + j, C, c);
    taps.load(weight, bias, c);
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      const V* rows[K];
#pragma unroll
      for (int i = 0; i < K; ++i) rows[i] = &r[j + i];
      *reinterpret_cast<V*>(out + (t0 + j) * C + c) = taps.apply(rows, act);
    }
    return;
  }
  taps.load(weight, bias, c);
#pragma unroll 1
  for (int64_t t = t0; t < t0 + RUN && t < Ttot; ++t) {
    while (t >= s1 && n + 1 < q.N) {  // the next sequence that is not empty
      ++n;
      s0 = q.begin(n);
      s1 = q.end(n);
    }
    if (n < 0 || t < s0 || t >= s1) continue;  // behind the last sequence, or before the first
    V r[K];
    const V* rows[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      r[j] = input_row<T, VEC, K>(x, ldx, init, s0, n, t - s0 - (K - 1) + j, C, c);
      rows[j] = &r[j];
    }
    *reinterpret_cast<V*>(out + t * C + c) = taps.apply(rows, act);
  }
}

// One token: the K - 1 state rows and the input make the output; the state
// moves up by one row.
template <typename T, int VEC, int K>
__global__ void __launch_bounds__(128)
    conv_step_kernel(const T* __restrict__ x, int64_t ldx, const float* __restrict__ weight,
                     const float* __restrict__ bias, T* __restrict__ state, T* __restrict__ out, int N, int C, int act) {
  using V = Vec<T, VEC>;
  const int c = (blockIdx.y * 128 + threadIdx.x) * VEC;
  if (c >= C) return;
  const int n = blockIdx.x;
  V r[K];
  T* st = state + (int64_t)n * (K - 1) * C + c;
#pragma unroll
  for (int j = 0; j < K - 1; ++j) r[j] = *reinterpret_cast<const V*>(st + (int64_t)j * C);
  r[K - 1] = *reinterpret_cast<const V*>(x + n * ldx + c);
  Taps<T, VEC, K> taps;
  taps.load(weight, bias, c);
  const V* rows[K];
#pragma unroll
  for (int j = 0; j < K; ++j) rows[j] = &r[j];
  *reinterpret_cast<V*>(out + (int64_t)n * C + c) = taps.apply(rows, act);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) *reinterpret_cast<V*>(st + (int64_t)j * C) = r[j + 1];
}

template <typename T, int VEC, int K>
cudaError_t conv_fwd(const ConvArgs& a, cudaStream_t s) {
  const Seqs q{a.cu, a.N, a.T};
  const int64_t tokens = a.cu ? a.T : (int64_t)a.N * a.T;
  const unsigned cb = (unsigned)((a.C + 32 * VEC - 1) / (32 * VEC));
  const int runs = (int)((tokens + RUN * WARPS - 1) / (RUN * WARPS));
  const int fins = a.fin ? (a.N + WARPS - 1) / WARPS : 0;
  const T *x = (const T*)a.x, *init = (const T*)a.init;
  auto go = [&](int run_blocks, int fin_blocks) {
    if (run_blocks + fin_blocks == 0) return;
    conv_fwd_kernel<T, VEC, K><<<dim3(run_blocks + fin_blocks, cb), 32 * WARPS, 0, s>>>(
        x, a.ldx, a.weight, a.bias, init, (T*)a.out, (T*)a.fin, q, a.C, a.act, run_blocks);
  };
  // A state written over the initial one waits for the outputs that read it.
  if (a.fin && a.fin == a.init) {
    go(runs, 0);
    go(0, fins);
  } else {
    go(runs, fins);
  }
  return cudaGetLastError();
}

template <typename T, int VEC, int K>
cudaError_t conv_step(const ConvArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.N, (unsigned)((a.C + 128 * VEC - 1) / (128 * VEC)));
  conv_step_kernel<T, VEC, K><<<grid, 128, 0, s>>>((const T*)a.x, a.ldx, a.weight, a.bias, (T*)a.fin, (T*)a.out, a.N,
                                                   a.C, a.act);
  return cudaGetLastError();
}

template <bool STEP, typename T, int VEC>
cudaError_t conv_k(const ConvArgs& a, cudaStream_t s) {
  switch (a.K) {
    case 2: return STEP ? conv_step<T, VEC, 2>(a, s) : conv_fwd<T, VEC, 2>(a, s);
    case 3: return STEP ? conv_step<T, VEC, 3>(a, s) : conv_fwd<T, VEC, 3>(a, s);
    case 4: return STEP ? conv_step<T, VEC, 4>(a, s) : conv_fwd<T, VEC, 4>(a, s);
  }
  return cudaErrorInvalidValue;
}

// 16-byte accesses where the channel count and the row stride allow them in
// every row, single elements otherwise.
template <bool STEP, typename T>
cudaError_t conv_t(const ConvArgs& a, cudaStream_t s) {
  constexpr int VEC = 16 / sizeof(T);
  if (a.C % VEC == 0 && rows_aligned(a.x, a.ldx, sizeof(T), 16)) return conv_k<STEP, T, VEC>(a, s);
  return conv_k<STEP, T, 1>(a, s);
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? conv_t<false, __nv_bfloat16>(a, s) : conv_t<false, float>(a, s);
}
cudaError_t launch_conv_step(const ConvArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? conv_t<true, __nv_bfloat16>(a, s) : conv_t<true, float>(a, s);
}

}  // namespace kda
