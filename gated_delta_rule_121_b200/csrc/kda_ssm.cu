// Selective state-space scan with a scalar decay per head, on CUDA cores: the
// prompt form for fp32 inputs and for the sizes that the tensor-core kernel
// does not take, and the single-token form for all of them.
//
//   D_t = softplus(delta_t + dt_bias),  a_t = exp(-exp(A_log) D_t)
//   S_t = a_t S_{t-1} + D_t b_t x_t^T,  y_t = S_t^T c_t + D x_t
//
// Prompt: a block owns PV value columns of one head's state and walks its piece
// of a sequence (kda_ssm_pieces.cuh) token by token.  A thread keeps NR rows of
// one column in registers; the RG row groups of a column are neighbouring lanes,
// so y is a sum over RG lanes.  TB tokens at a time are staged in shared memory
// as fp32 while the next ones are on their way to registers.
//   Over a stage the state is kept without its decay: with G_t the sum of log
// decays from the stage's start, S_t = e^{G_t} Z_t, Z_t = Z_{t-1} + e^{-G_t} D_t b_t
// x_t^T, y_t = e^{G_t} Z_t^T c_t + D x_t.  That is one multiply-add per element
// less, and one rounding of the state's decay per stage in place of one per
// token (over thousands of slowly decaying tokens those add up to 1e-6).  Where
// a stage decays by more than 2^-20 the plain recurrence runs instead.
//   Each thread's chain of multiply-adds and the shared-memory reads beside it
// bound it (two float4 for eight multiply-adds; 4 dk dv flops per token and head).
// fp32: 2 x 1000 tokens, 4 heads, 16 x 16 states, 33 us; 2 x 4096 tokens, 8 heads,
// 128 x 64, 324 us, 6.6 TFLOP/s, with the shared-memory pipe 68 % and the issue slots
// 47 % busy.  bf16, 4 x 8192 tokens, 48 heads: 32 x 64 1.80 ms, 16 x 64 1.54 ms, 25 times
// what their bytes take (pipe 50 %, issue slots 41 %); the tensor cores take 64 and 128
// only.
//
// Single token: as the KDA decode step, the state is streamed once through
// registers; HBM bandwidth bounds it (8 dk dv bytes per head): 512
// sequences of 96 heads, 128 x 128 states, 0.94 ms, 6.9 TB/s.
#include "kda_ssm_pieces.cuh"

namespace kda {
namespace {

template <int DK, int DV>
struct ScanShape {
  static constexpr int PV = DV < 32 ? DV : 32;        // columns per block
  static constexpr int RG = DK >= 64 ? 8 : 4;         // row groups of a column
  static constexpr int NR = DK / RG;                  // rows per thread, in float4 pieces
  static constexpr int NT = PV * RG;                  // threads per block
  static constexpr int TB = 16;                       // tokens per stage
};

// STATES: the first pass over pieces.
template <int DK, int DV, typename IO, bool STATES>
__global__ void __launch_bounds__(ScanShape<DK, DV>::NT)
    ssm_fwd_simt_kernel(const SsmArgs a, const PieceArgs pa) {
  using Sh = ScanShape<DK, DV>;
  constexpr int PV = Sh::PV, RG = Sh::RG, NR = Sh::NR, NT = Sh::NT, TB = Sh::TB;
  static_assert(TB <= 32, "a warp scans a stage's decays");
  __shared__ float s_x[2][TB][PV];
  __shared__ alignas(16) float s_b[2][TB][DK], s_c[2][TB][DK];
  // per token: e^{G_t} and e^{-G_t} D_t where the stage decays mildly, else a_t and D_t; then e^{G} of the
  // stage (0 where it does not)
  __shared__ float s_e[2][TB], s_w[2][TB], s_end[2];
  const int tid = threadIdx.x, rg = tid % RG, p = tid / RG;
  const int h = blockIdx.x % a.H, col0 = blockIdx.y * PV;
  Piece pc;
  if (!find_piece<STATES>(pa, a.T, blockIdx.x / a.H, pc)) return;
  const int grp = h / (a.H / a.G);
  const int64_t t0 = pc.start, L = pc.end - t0;
  const IO* x = (const IO*)a.x + (int64_t)h * DV + col0;
  const IO* b = (const IO*)a.b + (int64_t)grp * DK;
  const IO* c = (const IO*)a.c + (int64_t)grp * DK;
  IO* out = (IO*)a.out + (int64_t)h * DV + col0 + p;
  const float rate = -decay_rate(a.A_log[h]) * 1.4426950408889634f, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  const float skip = a.D ? a.D[h] : 0.f;

  // Row j of piece k of this thread: 4 (rg + RG k) + j.
  auto row = [&](int k, int j) { return (int64_t)(4 * (rg + RG * k) + j) * DV; };
  float s[NR];
  const int64_t at0 = (int64_t)h * DK * DV + col0 + p, seq = (int64_t)a.H * DK * DV;
  float* slots = pa.state + at0;
#pragma unroll
  for (int k = 0; k < NR / 4; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v = 0.f;
      if (!STATES && pc.split) {
        if (a.init || pc.before > 0) v = slots[(pc.slot0 + pc.before) * seq + row(k, j)];
      } else if (a.init && (!STATES || pc.first)) {
        v = a.init[pc.n * seq + at0 + row(k, j)];
        if (STATES) {  // kept for the second pass
          slots[pc.slot0 * seq + row(k, j)] = v;
          v = 0.f;
        }
      }
      s[4 * k + j] = v;
    }

  constexpr int XB = (TB * PV + NT - 1) / NT, KB = (TB * DK + NT - 1) / NT;
  float rx[XB], rb[KB], rc[KB], rd = 0.f, total = 0.f;
  auto fetch = [&](int64_t at) {  // tokens [at, at + TB) to registers, zeros behind the end
#pragma unroll
    for (int i = 0; i < XB; ++i) {
      const int e = tid + i * NT, t = e / PV;
      rx[i] = (e < TB * PV && at + t < L) ? to_f32(x[(t0 + at + t) * a.ldx + e % PV]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int e = tid + i * NT, t = e / DK;
      const bool in = e < TB * DK && at + t < L;
      rb[i] = in ? to_f32(b[(t0 + at + t) * a.ldb + e % DK]) : 0.f;
      if (!STATES) rc[i] = in ? to_f32(c[(t0 + at + t) * a.ldc + e % DK]) : 0.f;
    }
    if (tid < TB && at + tid < L) rd = a.delta[(t0 + at + tid) * a.H + h];
  };
  auto stage = [&](int buf, int64_t at) {
#pragma unroll
    for (int i = 0; i < XB; ++i) {
      const int e = tid + i * NT;
      if (e < TB * PV) (&s_x[buf][0][0])[e] = rx[i];
    }
#pragma unroll
    for (int i = 0; i < KB; ++i) {
      const int e = tid + i * NT;
      if (e < TB * DK) {
        (&s_b[buf][0][0])[e] = rb[i];
        if (!STATES) (&s_c[buf][0][0])[e] = rc[i];
      }
    }
    if (tid < 32) {
      const float d = tid < TB && at + tid < L ? (a.dt_bias ? softplus_f32(rd + bias) : rd) : 0.f;
      const float g = rate * d;  // log2
      float sum = g;
#pragma unroll
      for (int o = 1; o < TB; o <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, sum, o);
        if (tid >= o) sum += u;
      }
      const float end = __shfl_sync(0xffffffffu, sum, TB - 1);
      total += end;
      const bool mild = end >= -20.f;
      if (tid < TB) {
        s_e[buf][tid] = exp2f(mild ? sum : g);
        s_w[buf][tid] = mild ? exp2f(-sum) * d : d;
      }
      if (tid == 0) s_end[buf] = mild ? exp2f(end) : 0.f;
    }
  };
  if (L > 0) {
    fetch(0);
    stage(0, 0);
  }
  __syncthreads();
  for (int64_t at = 0; at < L; at += TB) {
    const int buf = (int)(at / TB) & 1;
    if (at + TB < L) fetch(at + TB);
    const int m = (int)(L - at < TB ? L - at : TB);
    const float end = s_end[buf];
    IO* o = out + (t0 + at) * ((int64_t)a.H * DV);
    auto token = [&](int t, bool mild) {
      const float xv = s_x[buf][t][p], dx = s_w[buf][t] * xv, ev = s_e[buf][t];
      float y0 = 0.f, y1 = 0.f;
#pragma unroll
      for (int k = 0; k < NR / 4; ++k) {
        const float4 bv = *reinterpret_cast<const float4*>(&s_b[buf][t][4 * (rg + RG * k)]);
        const float bb[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) s[4 * k + j] = mild ? fmaf(bb[j], dx, s[4 * k + j]) : fmaf(ev, s[4 * k + j], bb[j] * dx);
        if (!STATES) {
          const float4 cv = *reinterpret_cast<const float4*>(&s_c[buf][t][4 * (rg + RG * k)]);
          y0 = fmaf(s[4 * k], cv.x, y0);
          y1 = fmaf(s[4 * k + 1], cv.y, y1);
          y0 = fmaf(s[4 * k + 2], cv.z, y0);
          y1 = fmaf(s[4 * k + 3], cv.w, y1);
        }
      }
      if (STATES) return;
      float y = y0 + y1;
#pragma unroll
      for (int q = RG / 2; q > 0; q >>= 1) y += __shfl_xor_sync(0xffffffffu, y, q);
      if (rg == 0 && t < m) o[(int64_t)t * a.H * DV] = from_f32<IO>(fmaf(skip, xv, mild ? y * ev : y));
    };
    // (rows behind the end have steps of zero: they change nothing)
    if (end != 0.f) {
#pragma unroll 8
      for (int t = 0; t < TB; ++t) token(t, true);
#pragma unroll
      for (int k = 0; k < NR; ++k) s[k] *= end;
    } else {
#pragma unroll 2
      for (int t = 0; t < m; ++t) token(t, false);
    }
    if (at + TB < L) stage(buf ^ 1, at + TB);
    __syncthreads();
  }
  float* dst = nullptr;
  if (STATES) {
    dst = slots + (pc.slot0 + pc.before + 1) * seq;
    if (tid == 0 && blockIdx.y == 0) pa.decay[(int64_t)(pc.slot0 + pc.before) * a.H + h] = total;
  } else if (a.fin && pc.last) {
    dst = a.fin + pc.n * seq + at0;
  }
  if (dst) {
#pragma unroll
    for (int k = 0; k < NR / 4; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[row(k, j)] = s[4 * k + j];
  }
}

template <int DK, int DV>
struct StepShape {
  static constexpr int COLQ = DV / 4;                               // float4 column groups
  static constexpr int RG = (256 / COLQ) < DK ? (256 / COLQ) : DK;  // row groups
  static constexpr int ROWS = DK / RG;                              // rows per thread
  static constexpr int NT = COLQ * RG;                              // threads per block
};

template <int DK, int DV, typename IO>
__global__ void __launch_bounds__(StepShape<DK, DV>::NT)
    ssm_step_kernel(const SsmArgs a, float* __restrict__ state) {
  using Sh = StepShape<DK, DV>;
  constexpr int COLQ = Sh::COLQ, RG = Sh::RG, ROWS = Sh::ROWS;
  __shared__ float s_b[DK], s_c[DK];
  __shared__ float4 s_y[RG][COLQ];
  const int tid = threadIdx.x, cq = tid % COLQ, rg = tid / COLQ;
  const int64_t bh = blockIdx.x;
  const int h = (int)(bh % a.H);
  const int64_t n = bh / a.H;
  float4* S = reinterpret_cast<float4*>(state + bh * DK * DV);
  // The state's loads go first; the token is staged while they are in flight.
  float4 s[ROWS];
#pragma unroll
  for (int m = 0; m < ROWS; ++m) s[m] = __ldcs(S + (rg * ROWS + m) * COLQ + cq);
  const int grp = h / (a.H / a.G);
  const IO* b = (const IO*)a.b + n * a.ldb + (int64_t)grp * DK;
  const IO* c = (const IO*)a.c + n * a.ldc + (int64_t)grp * DK;
  const IO* xp = (const IO*)a.x + n * a.ldx + (int64_t)h * DV + 4 * cq;
  for (int i = tid; i < DK; i += Sh::NT) {
    s_b[i] = to_f32(b[i]);
    s_c[i] = to_f32(c[i]);
  }
  float d = a.delta[bh];
  if (a.dt_bias) d = softplus_f32(d + a.dt_bias[h]);
  const float av = expf(-decay_rate(a.A_log[h]) * d), skip = a.D ? a.D[h] : 0.f;
  const float4 x = make_float4(to_f32(xp[0]), to_f32(xp[1]), to_f32(xp[2]), to_f32(xp[3]));
  const float4 dx = make_float4(d * x.x, d * x.y, d * x.z, d * x.w);
  __syncthreads();
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int m = 0; m < ROWS; ++m) {
    const int i = rg * ROWS + m;
    const float bi = s_b[i], ci = s_c[i];
    s[m].x = fmaf(av, s[m].x, bi * dx.x);
    s[m].y = fmaf(av, s[m].y, bi * dx.y);
    s[m].z = fmaf(av, s[m].z, bi * dx.z);
    s[m].w = fmaf(av, s[m].w, bi * dx.w);
    y.x = fmaf(s[m].x, ci, y.x);
    y.y = fmaf(s[m].y, ci, y.y);
    y.z = fmaf(s[m].z, ci, y.z);
    y.w = fmaf(s[m].w, ci, y.w);
    __stcs(S + i * COLQ + cq, s[m]);
  }
  s_y[rg][cq] = y;
  __syncthreads();
  if (rg == 0) {
#pragma unroll
    for (int r = 1; r < RG; ++r) {
      const float4 v = s_y[r][cq];
      y.x += v.x; y.y += v.y; y.z += v.z; y.w += v.w;
    }
    IO* o = (IO*)a.out + bh * DV + 4 * cq;
    o[0] = from_f32<IO>(fmaf(skip, x.x, y.x));
    o[1] = from_f32<IO>(fmaf(skip, x.y, y.y));
    o[2] = from_f32<IO>(fmaf(skip, x.z, y.z));
    o[3] = from_f32<IO>(fmaf(skip, x.w, y.w));
  }
}

PiecePlan simt_plan(int N, int64_t T, int H, int dk, int dv, bool packed) {
  // four blocks per SM at a time; pieces of at least 128 tokens
  return plan_pieces(N, T, H * (dv < 32 ? 1 : dv / 32), 4 * 148, 0.6, 2, H, dk, dv, packed);
}

struct Fwd {
  template <int DK, int DV, typename IO>
  static cudaError_t go(const SsmArgs& a, float* workspace, cudaStream_t s) {
    using Sh = ScanShape<DK, DV>;
    const PiecePlan p = simt_plan(a.N, a.T, a.H, DK, DV, a.cu != nullptr);
    PieceArgs pa;
    cudaError_t e = prepare_pieces(p, a, workspace, &pa, s);
    if (e != cudaSuccess) return e;
    const unsigned slabs = DV / Sh::PV;
    if (p.first_pass) {
      ssm_fwd_simt_kernel<DK, DV, IO, true><<<dim3((unsigned)(p.first_pass * a.H), slabs), Sh::NT, 0, s>>>(a, pa);
      if ((e = compose_pieces(p, a, pa, s)) != cudaSuccess) return e;
    }
    ssm_fwd_simt_kernel<DK, DV, IO, false><<<dim3((unsigned)(p.pieces * a.H), slabs), Sh::NT, 0, s>>>(a, pa);
    return cudaGetLastError();
  }
};
struct Step {
  template <int DK, int DV, typename IO>
  static cudaError_t go(const SsmArgs& a, float* state, cudaStream_t s) {
    ssm_step_kernel<DK, DV, IO><<<(unsigned)((int64_t)a.N * a.H), StepShape<DK, DV>::NT, 0, s>>>(a, state);
    return cudaGetLastError();
  }
};

template <typename F, int DK, int DV>
cudaError_t by_type(const SsmArgs& a, float* state, bool bf16, cudaStream_t s) {
  return bf16 ? F::template go<DK, DV, __nv_bfloat16>(a, state, s) : F::template go<DK, DV, float>(a, state, s);
}
template <typename F, int DK>
cudaError_t by_dv(const SsmArgs& a, float* state, bool bf16, cudaStream_t s) {
  switch (a.dv) {
    case 16: return by_type<F, DK, 16>(a, state, bf16, s);
    case 32: return by_type<F, DK, 32>(a, state, bf16, s);
    case 64: return by_type<F, DK, 64>(a, state, bf16, s);
    case 128: return by_type<F, DK, 128>(a, state, bf16, s);
  }
  return cudaErrorInvalidValue;
}
template <typename F>
cudaError_t by_dims(const SsmArgs& a, float* state, bool bf16, cudaStream_t s) {
  switch (a.dk) {
    case 16: return by_dv<F, 16>(a, state, bf16, s);
    case 32: return by_dv<F, 32>(a, state, bf16, s);
    case 64: return by_dv<F, 64>(a, state, bf16, s);
    case 128: return by_dv<F, 128>(a, state, bf16, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t ssm_simt_workspace(int N, int64_t T, int H, int dk, int dv, bool packed) {
  return simt_plan(N, T, H, dk, dv, packed).total;
}
cudaError_t launch_ssm_fwd_simt(const SsmArgs& a, void* workspace, bool bf16, cudaStream_t s) {
  return by_dims<Fwd>(a, static_cast<float*>(workspace), bf16, s);
}
cudaError_t launch_ssm_step(const SsmArgs& a, float* state, bool bf16, cudaStream_t s) {
  return by_dims<Step>(a, state, bf16, s);
}

}  // namespace kda
