// Short depthwise causal convolution with an activation (Kimi K3 digest,
// "Kimi Delta Attention" section: a convolution of kernel size 4 and a Swish
// on q, k and v before the recurrence), for prompts and for single tokens.
//
//   out_t[c] = act(bias[c] + sum_{j<K} weight[c][j] x_{t-K+1+j}[c])
//
// A prompt moves 2 elements per K multiply-adds, so HBM bandwidth bounds it.  A
// thread owns VEC neighbouring channels and walks RUN tokens at a time: the RUN
// loads go out before the first product, the K - 1 inputs before them stay in
// registers, and the weights are loaded once for all its runs.  A block spans up
// to 256 threads' channels of the same tokens, whole DRAM pages of a row.  A run
// that a sequence's border cuts is done token by token, and so is a thread's run
// behind one that ended with its sequence (64K tokens of 1112 channels: 82 us as one
// sequence, 89 in sequences of 64, 247 in sequences of 16).
// Measured: 64K tokens of 12288 bf16 channels 577 us, 5.6 TB/s, 85 % of a copy's
// rate, and 606 us as a slice of rows three times as wide; the rest is latency
// between a thread's batches (requesting the next batch's rows one by one as this
// one's are used was slower, 790 us).  Channels that 4 does not divide are taken
// one by one: 1110 of them 100 us, 44 % of a copy's rate, where 1112 take 82.
#include "kda_layer.cuh"

namespace kda {
namespace {

// Channels per thread and access, and tokens per batch of loads.  Four channels by
// sixteen tokens: of the same bytes in flight, eight by eight took 627 us for 64K
// tokens of 12288 bf16 channels where this takes 576.
constexpr int WIDE = 4;
template <int VEC>
constexpr int run_tokens = VEC == 1 ? 8 : 16;
constexpr int THREADS = 256;  // per block: `lanes` along the channels, the others along the tokens

// VEC channels' weights (by tap, so that neighbouring channels are neighbours)
// and biases.
template <int VEC, int K>
struct Taps {
  float w[K][VEC], b[VEC];
  __device__ __forceinline__ void load(const float* weight, const float* bias, int c) {
    float f[VEC * K];
    load_params(weight + (int64_t)c * K, f);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      b[i] = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][i] = f[i * K + j];
    }
    if (bias) load_params(bias + c, b);
  }
};

// One output: rows[0..K-2] the inputs before, rows[K-1] the token's own.
template <typename T, int VEC, int K, int ACT>
__device__ __forceinline__ Vec<T, VEC> taps_apply(const Taps<VEC, K>& taps, const float (&rows)[K][VEC]) {
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = taps.b[i];
#pragma unroll
  for (int j = 0; j < K; ++j) vfma(acc, taps.w[j], rows[j]);
  if constexpr (ACT == KDA_ACT_SILU) {
    float s[VEC];
    vsigmoid(acc, s);
    vmul(acc, s);
  }
  return pack<T, VEC>(acc);
}

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

// Blocks [0, run_blocks) in x: `runs` runs per thread; the blocks behind them: final states.
template <typename T, int VEC, int K, int ACT>
__global__ void __launch_bounds__(THREADS, 2)
    conv_fwd_kernel(const T* __restrict__ x, int64_t ldx, const float* __restrict__ weight,
                    const float* __restrict__ bias, const T* init, T* __restrict__ out, T* fin, Seqs q, int C,
                    int run_blocks, int runs, int lanes) {
  using V = Vec<T, VEC>;
  constexpr int RUN = run_tokens<VEC>;
  const int group = threadIdx.x / lanes, groups = THREADS / lanes;
  const int c = (blockIdx.y * lanes + threadIdx.x % lanes) * VEC;
  if (c >= C) return;
  if ((int)blockIdx.x >= run_blocks) {
    const int n = ((int)blockIdx.x - run_blocks) * groups + group;
    if (n < q.N) final_rows<T, VEC, K>(x, ldx, init, fin, q, n, C, c);
    return;
  }
  const int64_t Ttot = q.tokens();
  int64_t t = ((int64_t)blockIdx.x * groups + group) * (RUN * runs);
  if (t >= Ttot) return;
  Taps<VEC, K> taps;
  taps.load(weight, bias, c);
  int n = q.find(t);
  int64_t s0 = n >= 0 ? q.begin(n) : 0, s1 = n >= 0 ? q.end(n) : q.begin(0);
  float before[K - 1][VEC];  // the inputs before token t, where `carried`
  bool carried = false;
#pragma unroll 1
  for (int run = 0; run < runs && t < Ttot; ++run, t += RUN) {
    if (n >= 0 && t >= s0 && t + RUN <= s1) {  // the whole run lies in one sequence
      const T* xt = x + t * ldx + c;
      V r[RUN];
#pragma unroll
      for (int j = 0; j < RUN; ++j) r[j] = *reinterpret_cast<const V*>(xt + j * ldx);
      if (!carried) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) unpack(input_row<T, VEC, K>(x, ldx, init, s0, n, t - s0 - (K - 1) + j, C, c), before[j]);
      }
      T* ot = out + t * C + c;
#pragma unroll
      for (int j = 0; j < RUN; ++j) {
        float rows[K][VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
          for (int k = 0; k < K - 1; ++k) rows[k][i] = before[k][i];
        }
        unpack(r[j], rows[K - 1]);
        *reinterpret_cast<V*>(ot + (int64_t)j * C) = taps_apply<T, VEC, K, ACT>(taps, rows);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
          for (int k = 0; k < K - 1; ++k) before[k][i] = rows[k + 1][i];
        }
      }
      carried = true;
      continue;
    }
    carried = false;
#pragma unroll 1
    for (int64_t u = t; u < t + RUN && u < Ttot; ++u) {
      while (u >= s1 && n + 1 < q.N) {  // the next sequence that is not empty
        ++n;
        s0 = q.begin(n);
        s1 = q.end(n);
      }
      if (n < 0 || u < s0 || u >= s1) continue;  // behind the last sequence, or before the first
      float rows[K][VEC];
#pragma unroll
      for (int j = 0; j < K; ++j) unpack(input_row<T, VEC, K>(x, ldx, init, s0, n, u - s0 - (K - 1) + j, C, c), rows[j]);
      *reinterpret_cast<V*>(out + u * C + c) = taps_apply<T, VEC, K, ACT>(taps, rows);
    }
    while (t + RUN >= s1 && n + 1 < q.N) {  // where the next run starts
      if (t + RUN < q.begin(n + 1)) break;
      ++n;
      s0 = q.begin(n);
      s1 = q.end(n);
    }
  }
}

// One token: the K - 1 state rows and the input make the output; the state
// moves up by one row.  A thread takes `per` sequences with one load of its
// weights, which are as many bytes as a sequence's rows; two are in flight.
constexpr int STEP_THREADS = 128;
template <typename T, int VEC, int K, int ACT>
__global__ void __launch_bounds__(STEP_THREADS)
    conv_step_kernel(const T* __restrict__ x, int64_t ldx, const float* __restrict__ weight,
                     const float* __restrict__ bias, T* __restrict__ state, T* __restrict__ out, int N, int C, int per) {
  using V = Vec<T, VEC>;
  const int c = (blockIdx.y * STEP_THREADS + threadIdx.x) * VEC;
  if (c >= C) return;
  const int n0 = blockIdx.x * per, n1 = min(n0 + per, N);
  Taps<VEC, K> taps;
  taps.load(weight, bias, c);
#pragma unroll 2
  for (int n = n0; n < n1; ++n) {
    V r[K];
    T* st = state + (int64_t)n * (K - 1) * C + c;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j] = *reinterpret_cast<const V*>(st + (int64_t)j * C);
    r[K - 1] = *reinterpret_cast<const V*>(x + n * ldx + c);
    float rows[K][VEC];
#pragma unroll
    for (int j = 0; j < K; ++j) unpack(r[j], rows[j]);
    *reinterpret_cast<V*>(out + (int64_t)n * C + c) = taps_apply<T, VEC, K, ACT>(taps, rows);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) *reinterpret_cast<V*>(st + (int64_t)j * C) = r[j + 1];
  }
}

constexpr int64_t BLOCKS = 148 * 8;  // blocks that keep every SM busy

template <typename T, int VEC, int K, int ACT>
cudaError_t conv_fwd(const ConvArgs& a, cudaStream_t s) {
  const Seqs q{a.cu, a.N, a.T};
  const int64_t tokens = a.cu ? a.T : (int64_t)a.N * a.T;
  constexpr int RUN = run_tokens<VEC>;
  const int pieces = (a.C + VEC - 1) / VEC;
  int lanes = 32;  // neighbouring blocks of tokens share their inputs in L2, neighbouring lanes a DRAM page
  while (lanes < THREADS && lanes < pieces) lanes *= 2;
  const int groups = THREADS / lanes;
  const unsigned cb = (unsigned)((pieces + lanes - 1) / lanes);
  // as many runs per thread (up to 8) as leave enough blocks
  const int64_t blocks = (tokens + RUN * groups - 1) / (RUN * groups);
  int runs = 1;
  while (runs < 8 && blocks * cb / (2 * runs) >= BLOCKS) runs *= 2;
  const int run_blocks = (int)((tokens + (int64_t)RUN * groups * runs - 1) / ((int64_t)RUN * groups * runs));
  const int fins = a.fin ? (a.N + groups - 1) / groups : 0;
  const T *x = (const T*)a.x, *init = (const T*)a.init;
  auto go = [&](int rb, int fb) {
    if (rb + fb == 0) return;
    conv_fwd_kernel<T, VEC, K, ACT><<<dim3(rb + fb, cb), THREADS, 0, s>>>(x, a.ldx, a.weight, a.bias, init, (T*)a.out,
                                                                        (T*)a.fin, q, a.C, rb, runs, lanes);
  };
  // A state written over the initial one waits for the outputs that read it.
  if (a.fin && a.fin == a.init) {
    go(run_blocks, 0);
    go(0, fins);
  } else {
    go(run_blocks, fins);
  }
  return cudaGetLastError();
}

template <typename T, int VEC, int K, int ACT>
cudaError_t conv_step(const ConvArgs& a, cudaStream_t s) {
  const unsigned cb = (unsigned)((a.C + STEP_THREADS * VEC - 1) / (STEP_THREADS * VEC));
  int per = 1;
  while (per < 8 && (int64_t)a.N * cb / (2 * per) >= BLOCKS) per *= 2;
  const dim3 grid((unsigned)((a.N + per - 1) / per), cb);
  conv_step_kernel<T, VEC, K, ACT><<<grid, STEP_THREADS, 0, s>>>((const T*)a.x, a.ldx, a.weight, a.bias, (T*)a.fin,
                                                                (T*)a.out, a.N, a.C, per);
  return cudaGetLastError();
}

template <bool STEP, typename T, int VEC, int K>
cudaError_t conv_act(const ConvArgs& a, cudaStream_t s) {
  if (a.act == KDA_ACT_SILU)
    return STEP ? conv_step<T, VEC, K, KDA_ACT_SILU>(a, s) : conv_fwd<T, VEC, K, KDA_ACT_SILU>(a, s);
  return STEP ? conv_step<T, VEC, K, KDA_ACT_NONE>(a, s) : conv_fwd<T, VEC, K, KDA_ACT_NONE>(a, s);
}

template <bool STEP, typename T, int VEC>
cudaError_t conv_k(const ConvArgs& a, cudaStream_t s) {
  switch (a.K) {
    case 2: return conv_act<STEP, T, VEC, 2>(a, s);
    case 3: return conv_act<STEP, T, VEC, 3>(a, s);
    case 4: return conv_act<STEP, T, VEC, 4>(a, s);
  }
  return cudaErrorInvalidValue;
}

// Wide accesses where the channel count and the row stride allow them in every
// row, single elements otherwise.
template <bool STEP, typename T>
cudaError_t conv_t(const ConvArgs& a, cudaStream_t s) {
  if (a.C % WIDE == 0 && rows_aligned(a.x, a.ldx, sizeof(T), WIDE * sizeof(T))) return conv_k<STEP, T, WIDE>(a, s);
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
