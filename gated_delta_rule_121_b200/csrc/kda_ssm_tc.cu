// Selective state-space scan over prompts on the sm_100a tensor cores (tcgen05
// / TMEM / TMA): bf16 x, b, c with dk, dv in {64, 128}, in chunks of 64 tokens.
//
// Over a chunk, with g_t = -exp(A_log) D_t, the in-chunk sums G_t = g_1 + .. +
// g_t, their total G_C and the state S before the chunk (dk x dv):
//   M_ts = (c_t . b_s) e^{G_t - G_s} D_s               (s <= t)
//   y_t  = e^{G_t} S^T c_t + sum_s M_ts x_s + D x_t
//   S   <- e^{G_C} S + sum_s b_s (e^{G_C - G_s} D_s x_s)^T
// No exponent is positive, whatever the decays.
//
// A block walks one piece of a sequence for one tile of 128 value columns: a
// head of dv = 128, or two heads of dv = 64 that read the same b and c (one
// head and 64 idle columns where a group has an odd number of heads).  All
// four products have M = 128 value columns or 64 tokens, fp32 accumulators in
// TMEM, and run transposed, so that a TMEM lane is a value column:
//   G  [t, s] = c_t . b_s                    (M = 64; A, B from shared memory)
//   YI [p, t] = sum_n S[p, n] c_t[n]          (A: S as bf16 in TMEM)
//   YM [p, t] = sum_s x_s[p] M_ts             (A: x as it lies; B: M as bf16)
//   U  [p, n] = sum_s w_s x_s[p] b_s[n]       (A: w x in TMEM; B: b as it lies)
// Two heads share one YM accumulator: along K, head 0's x stands over a tile of
// zeros and head 1's under one, each against its own M.
//
// Rounding.  x, b, c are bf16 and exact.  w x is split into three bf16 terms by
// truncation (8 + 8 + 8 bits: exact), so that the state, which is returned and
// carried in fp32, keeps fp32 accuracy; the state itself stays in registers and
// takes each chunk's U by one fp32 multiply-add per element.  S and M enter the
// output's products as bf16 (half a step each, 2^-8 relative): y is rounded to
// bf16 itself, and the three are of one size.
//
// Roles (23 warps, one block per SM): wx (4 warps) weights x and stores its
// terms; scores (4) turn G into M; state (8) holds S; out (4) combines YI, YM
// and the skip and stores y by TMA from x's own tile; one warp each for the
// loads, the MMA issue and the chunk's scalars.  The MMAs of a chunk take
// ~1500 cycles of tensor pipe at dv = 64 (half of it U's three terms); the
// other roles' instructions per chunk stay below that, so the tensor pipe is
// the bound that the layout aims at.
//
// Pieces.  A sequence longer than the plan's piece length is cut into pieces
// that run in parallel: a first pass (states only) gives each piece's own state
// and total decay, and a block of the second pass starts from their
// composition, S_in(r + 1) = e^{G(r)} S_in(r) + S(r).
#include <cuda.h>

#include "kda_layer.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace {

constexpr int CH = 64;       // tokens per chunk
constexpr int PT = 128;      // value columns per tile
constexpr int NST = 3;       // stages of x, b, c
constexpr float LOG2E = 1.4426950408889634f;
constexpr uint64_t WAIT_NS = 2000000000ull;  // limit of every in-kernel wait

constexpr int W_WX = 0, W_SC = 4, W_OUT = 8, W_ST = 12, W_TMA = 20, W_MMA = 21, W_DEC = 22, NWARP = 23;
constexpr int NTHR = 32 * NWARP;
enum { GRP_WX = 1, GRP_SC, GRP_OUT, GRP_ST };  // named barriers

enum Bar {
  B_FULL0 = 0, B_DEC0 = B_FULL0 + NST, B_EMPTY0 = B_DEC0 + NST, B_WX = B_EMPTY0 + NST, B_U, B_UFREE, B_G, B_GFREE,
  B_SRDY, B_SFREE, B_M0, B_M1, B_Y0, B_Y1, B_YFREE, B_DRAIN, NUM_BARS
};

// Scalars of a chunk, per head: floats at these offsets.
constexpr int SC_W = 0, SC_CUM = 64, SC_D = 128, SC_ECUM = 192, SC_ER = 256, SC_ECD = 320, SC_FLOATS = 512;
// SC_W e^{G_C - G_s} D_s; SC_CUM G_t (log2); SC_D D_s; SC_ECUM e^{G_t}; SC_ER e^{G_t - R_q} with R_q = G before the
// 16-token block q of t; SC_ECD + 64 (q - 1): e^{R_q - G_s} D_s for s before block q.

template <int DK, int DV>
struct Cfg {
  static constexpr int HEADS = PT / DV;                  // heads per tile, at most
  static constexpr uint32_t KV_BYTES = CH * DK * 2;      // b or c of a chunk
  static constexpr uint32_t X_BYTES = CH * PT * 2;
  static constexpr uint32_t STAGE = X_BYTES + 2 * KV_BYTES;
  static constexpr uint32_t M_BYTES = CH * CH * 2;       // one head's scores
  static constexpr uint32_t ZERO = 2048;                 // 16 rows of zeros of 64 columns
  // shared memory: zeros, the stages, zeros (the zero tiles lie below and above x: descriptor strides are positive)
  static constexpr uint32_t SM_Z0 = 0, SM_STAGE = ZERO, SM_Z1 = SM_STAGE + NST * STAGE, SM_M = SM_Z1 + ZERO;
  static constexpr uint32_t SM_DEC = SM_M + 2 * HEADS * M_BYTES;
  static constexpr uint32_t SM_MISC = SM_DEC + NST * HEADS * SC_FLOATS * 4;
  static constexpr uint32_t BYTES = SM_MISC + 512 + 1024;
  // TMEM columns
  static constexpr uint32_t TM_WX = 0, TM_S = 96, TM_YI = TM_S + DK / 2, TM_YM = TM_YI + 64, TM_U = TM_YM + 64,
                            TM_G = TM_U + DK, TM_END = TM_G + 64;
  static constexpr uint32_t TM_COLS = 512;
  static_assert(TM_END <= TM_COLS, "TMEM");
  static_assert(BYTES <= 227 * 1024, "shared memory");
};
constexpr uint32_t MS_TMEM = 384, MS_ABORT = 388, MS_TOTAL = 392;  // in SM_MISC, behind the barriers
static_assert(NUM_BARS * 8 <= MS_TMEM, "barrier area");

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tmap), "r"(src),
               "r"(c0), "r"(c1)
               : "memory");
}
// 16 lanes x 16 columns (fp32): thread l gets rows l/4 and l/4 + 8, of each 8
// columns numbers 2 (l % 4) and the next: {r, c}, {r, c+1}, {r+8, c}, {r+8, c+1},
// then the same of the next 8 columns.  Not waited for.
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "r"(taddr));
}
// Waits for this thread's TMEM loads; ties 16 of their registers to the wait.
__device__ __forceinline__ void tmem_wait_ld(float (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}
// 16 lanes x 16 columns of 32-bit values, row l/4 (and + 8), column l % 4 of each 4.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Four 8x8 tiles of 16-bit elements, transposed on the way (lane l gives the
// address of row l % 8 of tile l / 8; it holds row l / 4, columns 2 (l % 4) and
// the next of the transposed tile).
__device__ __forceinline__ void ldsm_x4_t(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
__device__ __forceinline__ void stsm_x4_t(uint32_t saddr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void stsm_x4(uint32_t saddr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, int a_mn, int b_mn) {
  return idesc_f16_f32(M, N, a_mn, b_mn) | (1u << 7) | (1u << 10);  // A, B format 1 = bf16
}
__device__ __forceinline__ float2 bf16x2_f32(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// The upper halves of two fp32 values (their truncation to bf16), the first in the low half.
__device__ __forceinline__ uint32_t upper_halves(float2 v) {
  return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
}
__device__ __forceinline__ float2 minus_upper(float2 v) {  // exact
  return make_float2(v.x - __uint_as_float(__float_as_uint(v.x) & 0xffff0000u),
                     v.y - __uint_as_float(__float_as_uint(v.y) & 0xffff0000u));
}

// ------------------------------------------------------------------ pieces
// One piece of a sequence: tokens [start, end) of sequence n, its r-th piece
// of `pieces`.  A sequence of several pieces has `pieces` slots for states from
// slot0 on (the initial state, then the own states of all pieces but the last)
// and as many for decays.
struct Piece {
  int n, r, pieces, slot0;
  int64_t start, end;
};
struct PieceEntry {  // table entry of a packed batch; n < 0: none
  int n, r, pieces, slot0, start, end, pad[2];
};

struct TcArgs {
  SsmArgs a;
  int hpt, tiles;        // heads per tile, tiles of 128 columns
  int64_t piece_len;     // tokens per piece, a multiple of the chunk
  int per_seq;           // pieces per sequence of a batch of equal lengths
  const PieceEntry* table;
  float* piece_state;    // [slots][H][dk][dv]
  float* piece_decay;    // [slots][H]: log2 of a piece's total decay
};

__device__ __forceinline__ bool find_piece(const TcArgs& t, int index, Piece& p) {
  if (t.table) {
    const PieceEntry e = t.table[index];
    if (e.n < 0) return false;
    p.n = e.n; p.r = e.r; p.pieces = e.pieces; p.slot0 = e.slot0; p.start = e.start; p.end = e.end;
    return true;
  }
  p.n = index / t.per_seq;
  p.slot0 = p.n * t.per_seq;
  p.r = index - p.n * t.per_seq;
  p.pieces = t.per_seq;
  const int64_t s0 = (int64_t)p.n * t.a.T;
  p.start = s0 + p.r * t.piece_len;
  p.end = min(p.start + t.piece_len, s0 + t.a.T);
  return true;
}

// The pieces of a packed batch, in the sequences' order (one block; entries
// behind the last one are marked unused).  Running sums of the pieces and of
// the slots that sequences of several pieces take; offsets that are no
// offsets may claim more than there is, and what lies beyond is left out.
__global__ void __launch_bounds__(1024) ssm_piece_table_kernel(Seqs q, int64_t piece_len, int capacity, int slots,
                                                               PieceEntry* table) {
  __shared__ int2 part[1024];
  __shared__ int2 carry;
  const int tid = threadIdx.x;
  if (tid == 0) carry = make_int2(0, 0);
  __syncthreads();
  for (int n0 = 0; n0 < q.N; n0 += 1024) {
    const int n = n0 + tid;
    int64_t s = 0, e = 0;
    int cnt = 0;
    if (n < q.N) {
      s = q.begin(n);
      e = max(q.end(n), s);
      cnt = (int)max((e - s + piece_len - 1) / piece_len, (int64_t)1);
    }
    const int own = cnt > 1 ? cnt : 0;
    part[tid] = make_int2(cnt, own);
    __syncthreads();
    for (int o = 1; o < 1024; o <<= 1) {
      const int2 v = tid >= o ? part[tid - o] : make_int2(0, 0);
      __syncthreads();
      part[tid].x += v.x;
      part[tid].y += v.y;
      __syncthreads();
    }
    const int first = carry.x + part[tid].x - cnt, slot0 = carry.y + part[tid].y - own;
    for (int r = 0; r < cnt; ++r) {
      const int64_t a = s + r * piece_len;
      if (first + r < capacity)
        table[first + r] = {slot0 + own <= slots ? n : -1, r, cnt, slot0, (int)a, (int)min(a + piece_len, e), {0, 0}};
    }
    __syncthreads();
    if (tid == 1023) {
      carry.x += part[1023].x;
      carry.y += part[1023].y;
    }
    __syncthreads();
  }
  for (int i = carry.x + tid; i < capacity; i += 1024) table[i].n = -1;
}

// ------------------------------------------------------------------ roles
struct Ctx {
  uint8_t* sm;
  uint32_t sb, tmem;
  uint64_t* bars;
  volatile int* abort;
  DeviceStatus* status;
  Piece piece;
  int h0, heads, tile;   // first head of the tile, heads in it
  int nchunks;
};

// Bounded wait that also gives up once another role has.
__device__ __forceinline__ bool wait_bar(const Ctx& x, int bar, uint32_t parity) {
  uint64_t* b = &x.bars[bar];
  if (mbar_try_wait(b, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(b, parity)) {
    if (*x.abort) return false;
    if (globaltimer_ns() - t0 > WAIT_NS) {
      *x.abort = 1;
      record_error(x.status, KDA_ERR_TIMEOUT, bar);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ int valid_rows(const Ctx& x, int i) {
  const int64_t left = x.piece.end - x.piece.start - (int64_t)i * CH;
  return left < CH ? (int)left : CH;
}

template <int DK, int DV, bool STATES>
__device__ __forceinline__ void role_load(const Ctx& x, const void* tx, const void* tb, const void* tc, int group) {
  using K = Cfg<DK, DV>;
  int issued = 0;
  for (int i = 0; i < x.nchunks; ++i) {
    const int st = i % NST;
    if (i >= NST && !wait_bar(x, B_EMPTY0 + st, (i / NST - 1) & 1)) break;
    uint64_t* bar = &x.bars[B_FULL0 + st];
    const uint32_t stg = x.sb + K::SM_STAGE + st * K::STAGE;
    const int tok = (int)(x.piece.start + (int64_t)i * CH);
    const int atoms = x.heads * DV / 64;
    mbar_arrive_expect_tx(bar, atoms * 8192 + (STATES ? 1 : 2) * K::KV_BYTES);
    for (int k = 0; k < DK / 64; ++k) {
      tma_load_2d(stg + K::X_BYTES + k * 8192, tb, bar, group * DK + 64 * k, tok);
      if (!STATES) tma_load_2d(stg + K::X_BYTES + K::KV_BYTES + k * 8192, tc, bar, group * DK + 64 * k, tok);
    }
    for (int k = 0; k < atoms; ++k) tma_load_2d(stg + k * 8192, tx, bar, x.h0 * DV + 64 * k, tok);
    issued = i + 1;
  }
  // No load stays in flight behind the block.
  for (int i = issued > NST ? issued - NST : 0; i < issued; ++i) mbar_wait(&x.bars[B_FULL0 + i % NST], (i / NST) & 1, WAIT_NS);
}

template <int DK, int DV, bool STATES>
__device__ __forceinline__ void role_mma(const Ctx& x) {
  using K = Cfg<DK, DV>;
  auto stage = [&](int i) { return x.sb + K::SM_STAGE + (i % NST) * K::STAGE; };
  auto scores = [&](int i) {  // G of chunk i
    const uint32_t b = stage(i) + K::X_BYTES, c = b + K::KV_BYTES;
    const uint32_t id = idesc_bf16_f32(64, 64, 0, 0);
#pragma unroll
    for (int k = 0; k < DK / 16; ++k) {
      const uint32_t o = (k >> 2) * 8192 + (k & 3) * 32;
      umma_ss(x.tmem + K::TM_G, sdesc_sw128(c + o, 16, 1024), sdesc_sw128(b + o, 16, 1024), id, k > 0);
    }
    umma_commit(&x.bars[B_G]);
  };
  if (!STATES) {
    if (!wait_bar(x, B_FULL0, 0)) return;
    scores(0);
  }
  for (int i = 0; i < x.nchunks; ++i) {
    const uint32_t xs = stage(i), b = xs + K::X_BYTES, c = b + K::KV_BYTES;
    // U: the small terms first
    if (!wait_bar(x, B_WX, i & 1)) return;
    if (i > 0 && !wait_bar(x, B_UFREE, (i - 1) & 1)) return;
    tc_fence_after();
    {
      const uint32_t id = idesc_bf16_f32(128, DK, 0, 1);
#pragma unroll
      for (int term = 2; term >= 0; --term)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_tmem_a(x.tmem + K::TM_U, x.tmem + K::TM_WX + term * 32 + k * 8, sdesc_sw128(b + k * 2048, 8192, 1024), id,
                      term < 2 || k > 0);
      umma_commit(&x.bars[B_U]);
      if (STATES) umma_commit(&x.bars[B_EMPTY0 + i % NST]);
    }
    if (STATES) continue;
    if (i + 1 < x.nchunks) {
      if (!wait_bar(x, B_FULL0 + (i + 1) % NST, ((i + 1) / NST) & 1)) return;
      if (!wait_bar(x, B_GFREE, i & 1)) return;
      tc_fence_after();
      scores(i + 1);
    }
    if (!wait_bar(x, B_SRDY, i & 1)) return;
    if (i > 0 && !wait_bar(x, B_YFREE, (i - 1) & 1)) return;
    tc_fence_after();
    {
      const uint32_t id = idesc_bf16_f32(128, 64, 0, 0);
#pragma unroll
      for (int k = 0; k < DK / 16; ++k)
        umma_tmem_a(x.tmem + K::TM_YI, x.tmem + K::TM_S + k * 8, sdesc_sw128(c + (k >> 2) * 8192 + (k & 3) * 32, 16, 1024),
                    id, k > 0);
      umma_commit(&x.bars[B_SFREE]);
    }
    if (!wait_bar(x, B_M0 + (i & 1), (i >> 1) & 1)) return;
    tc_fence_after();
    {
      const uint32_t id = idesc_bf16_f32(128, 64, 1, 0);
      const uint32_t m = x.sb + K::SM_M + (i & 1) * K::HEADS * K::M_BYTES;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // x of head 0 and what stands below it: its other columns (dv = 128), the idle half, or zeros
        const uint32_t xk = xs + k * 2048;
        const uint32_t below = x.heads == 2 ? x.sb + K::SM_Z1 - xk : 8192u;
        umma_ss(x.tmem + K::TM_YM, sdesc_sw128(xk, below, 1024), sdesc_sw128(m + k * 32, 16, 1024), id, k > 0);
      }
      if (x.heads == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t z = x.sb + K::SM_Z0, xk = xs + 8192 + k * 2048;
          umma_ss(x.tmem + K::TM_YM, sdesc_sw128(z, xk - z, 1024), sdesc_sw128(m + K::M_BYTES + k * 32, 16, 1024), id, 1);
        }
      }
      umma_commit(&x.bars[B_Y0 + (i & 1)]);
    }
  }
}

// Decays and steps of every chunk; lane l takes tokens 2 l and 2 l + 1.
template <int DK, int DV, bool STATES>
__device__ __forceinline__ void role_decay(const Ctx& x, const TcArgs& t) {
  using K = Cfg<DK, DV>;
  const SsmArgs& a = t.a;
  const int lane = threadIdx.x & 31;
  float rate[K::HEADS], bias[K::HEADS], total[K::HEADS], raw[K::HEADS][2];
#pragma unroll
  for (int h = 0; h < K::HEADS; ++h) {
    const int hh = x.h0 + (h < x.heads ? h : 0);
    rate[h] = -expf(a.A_log[hh]) * LOG2E;
    bias[h] = a.dt_bias ? a.dt_bias[hh] : 0.f;
    total[h] = 0.f;
  }
  auto fetch = [&](int i) {
    const int v = valid_rows(x, i);
#pragma unroll
    for (int h = 0; h < K::HEADS; ++h)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        raw[h][k] = (h < x.heads && 2 * lane + k < v)
                        ? a.delta[(x.piece.start + (int64_t)i * CH + 2 * lane + k) * a.H + x.h0 + h] : 0.f;
  };
  if (x.nchunks > 0) fetch(0);
  for (int i = 0; i < x.nchunks; ++i) {
    const int st = i % NST, v = valid_rows(x, i);
    float cur[K::HEADS][2];
#pragma unroll
    for (int h = 0; h < K::HEADS; ++h) { cur[h][0] = raw[h][0]; cur[h][1] = raw[h][1]; }
    if (i + 1 < x.nchunks) fetch(i + 1);
    if (i >= NST && !__all_sync(0xffffffffu, wait_bar(x, B_EMPTY0 + st, (i / NST - 1) & 1))) return;
#pragma unroll
    for (int h = 0; h < K::HEADS; ++h) {
      float* o = reinterpret_cast<float*>(x.sm + K::SM_DEC) + (st * K::HEADS + h) * SC_FLOATS;
      float d[2], g[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        d[k] = a.dt_bias ? softplus_f32(cur[h][k] + bias[h]) : cur[h][k];
        if (2 * lane + k >= v) d[k] = 0.f;
        g[k] = rate[h] * d[k];
      }
      // sums up to each token, and from behind it to the chunk's end (each
      // summed in its own direction: a weight near one has an exponent near zero)
      float up = g[0] + g[1], down = up;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, up, s), w = __shfl_down_sync(0xffffffffu, down, s);
        if (lane >= s) up += u;
        if (lane + s < 32) down += w;
      }
      float before = __shfl_up_sync(0xffffffffu, up, 1), behind = __shfl_down_sync(0xffffffffu, down, 1);
      if (lane == 0) before = 0.f;
      if (lane == 31) behind = 0.f;
      const float c0 = before + g[0], c1 = up, r1 = behind, r0 = behind + g[1];
      const float sum = __shfl_sync(0xffffffffu, up, 31);
      total[h] += sum;
      reinterpret_cast<float2*>(o + SC_W)[lane] = make_float2(ex2(r0) * d[0], ex2(r1) * d[1]);
      if (lane == 0) reinterpret_cast<float*>(x.sm + K::SM_MISC + MS_TOTAL)[st * 2 + h] = ex2(sum);
      if (!STATES) {
        reinterpret_cast<float2*>(o + SC_CUM)[lane] = make_float2(c0, c1);
        reinterpret_cast<float2*>(o + SC_D)[lane] = make_float2(d[0], d[1]);
        reinterpret_cast<float2*>(o + SC_ECUM)[lane] = make_float2(ex2(c0), ex2(c1));
        float mine = 0.f;
#pragma unroll
        for (int q = 1; q < 4; ++q) {
          const float ref = __shfl_sync(0xffffffffu, up, 8 * q - 1);  // G before token 16 q
          if (lane < 8 * q)
            reinterpret_cast<float2*>(o + SC_ECD + 64 * (q - 1))[lane] = make_float2(ex2(ref - c0) * d[0], ex2(ref - c1) * d[1]);
          if ((lane >> 3) == q) mine = ref;
        }
        reinterpret_cast<float2*>(o + SC_ER)[lane] = make_float2(ex2(c0 - mine), ex2(c1 - mine));
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&x.bars[B_DEC0 + st]);
  }
  if (STATES && lane == 0)
    for (int h = 0; h < x.heads; ++h) t.piece_decay[(int64_t)(x.piece.slot0 + x.piece.r) * a.H + x.h0 + h] = total[h];
}

// w x, split into three bf16 terms, as the A operand of U.
template <int DK, int DV>
__device__ __forceinline__ void role_wx(const Ctx& x) {
  using K = Cfg<DK, DV>;
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3, tid = threadIdx.x - 32 * W_WX;
  const uint32_t tl = x.tmem + ((uint32_t)(wq * 32) << 16);
  bool ok = true;
  for (int i = 0; i < x.nchunks; ++i) {
    const int st = i % NST, v = valid_rows(x, i);
    ok = ok && wait_bar(x, B_DEC0 + st, (i / NST) & 1);
    ok = ok && wait_bar(x, B_FULL0 + st, (i / NST) & 1);
    ok = ok && (i == 0 || wait_bar(x, B_U, (i - 1) & 1));
    if (!named_sync_and(GRP_WX, 128, ok)) return;
    tc_fence_after();
    uint8_t* stg = x.sm + K::SM_STAGE + st * K::STAGE;
    if (v < CH) {
      // Rows behind the sequence's end hold other data: x and b become zero,
      // so that nothing of them (an infinity among it) reaches a product.
      constexpr int ATOMS = 2 + DK / 64;
      for (int e = tid; e < ATOMS * (CH - v) * 8; e += 128) {
        const int atom = e / ((CH - v) * 8), k = e - atom * (CH - v) * 8;
        *reinterpret_cast<uint4*>(stg + atom * 8192 + v * 128 + k * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      named_sync(GRP_WX, 128);
    }
    const int head = DV == 64 && wq >= 2 ? 1 : 0;
    const float* w = reinterpret_cast<const float*>(x.sm + K::SM_DEC) + (st * K::HEADS + head) * SC_FLOATS + SC_W;
    const uint32_t xa = smem_u32(stg) + (wq >> 1) * 8192;
#pragma unroll
    for (int half = 0; half < 2; ++half) {      // 16 columns of the warp's 32
      const int pc = (wq & 1) * 4 + half * 2;   // their first 8-column chunk in the atom
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {          // 32 tokens
        uint32_t hi[8], mid[8], lo[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {           // 16 tokens: tiles (columns 0-7, 8-15) x (tokens 0-7, 8-15)
          const int t0 = 32 * tb + 16 * k;
          const int row = t0 + ((lane >> 4) & 1) * 8 + (lane & 7), ch = pc + ((lane >> 3) & 1);
          uint32_t raw[4];
          ldsm_x4_t(xa + row * 128 + ((ch ^ (row & 7)) << 4), raw);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 wt = *reinterpret_cast<const float2*>(w + t0 + (j >> 1) * 8 + 2 * (lane & 3));
            float2 val = __fmul2_rn(bf16x2_f32(raw[j]), wt);
            hi[4 * k + j] = upper_halves(val);
            val = minus_upper(val);
            mid[4 * k + j] = upper_halves(val);
            val = minus_upper(val);
            lo[4 * k + j] = upper_halves(val);
          }
        }
        const uint32_t ta = tl + ((uint32_t)(half * 16) << 16) + K::TM_WX + tb * 16;
        tmem_st_16x128b_x4(ta, hi);
        tmem_st_16x128b_x4(ta + 32, mid);
        tmem_st_16x128b_x4(ta + 64, lo);
      }
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(&x.bars[B_WX]);
  }
}

// G to M: decay, step and causal mask, bf16, as the B operand of YM.  Warp q
// has tokens 16 q .. 16 q + 15; tiles above the diagonal stay zero.
template <int DK, int DV>
__device__ __forceinline__ void role_scores(const Ctx& x) {
  using K = Cfg<DK, DV>;
  const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3;
  const uint32_t tl = x.tmem + ((uint32_t)(q * 32) << 16) + K::TM_G;
  const int r0 = 16 * q + (lane >> 2), cl = 2 * (lane & 3);
  // this lane's row address in a 16x16 tile (four 8x8 matrices: rows 0-7, rows 8-15, then columns 8-15)
  const int srow = 16 * q + ((lane >> 3) & 1) * 8 + (lane & 7), sch = (lane >> 4) & 1;
  bool ok = true;
  for (int i = 0; i < x.nchunks; ++i) {
    const int st = i % NST;
    ok = ok && wait_bar(x, B_DEC0 + st, (i / NST) & 1);
    ok = ok && (i < 2 || wait_bar(x, B_Y0 + (i & 1), ((i >> 1) - 1) & 1));
    ok = ok && wait_bar(x, B_G, i & 1);
    if (!named_sync_and(GRP_SC, 128, ok)) return;
    tc_fence_after();
    float g[4][8];
    {
      float ga[16], gb[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) ga[k] = gb[k] = 0.f;
      tmem_ld_16x256b_x2(tl, ga);
      if (q >= 1) tmem_ld_16x256b_x2(tl + 16, ga + 8);
      if (q >= 2) tmem_ld_16x256b_x2(tl + 32, gb);
      if (q >= 3) tmem_ld_16x256b_x2(tl + 48, gb + 8);
      tmem_wait_ld(ga);
      tmem_wait_ld(gb);
#pragma unroll
      for (int k = 0; k < 8; ++k) { g[0][k] = ga[k]; g[1][k] = ga[8 + k]; g[2][k] = gb[k]; g[3][k] = gb[8 + k]; }
    }
    tc_fence_before();
    mbar_arrive(&x.bars[B_GFREE]);
    const uint32_t mb = x.sb + K::SM_M + (i & 1) * K::HEADS * K::M_BYTES;
#pragma unroll
    for (int h = 0; h < K::HEADS; ++h) {
      if (h >= x.heads) break;
      const float* s = reinterpret_cast<const float*>(x.sm + K::SM_DEC) + (st * K::HEADS + h) * SC_FLOATS;
      const uint32_t mh = mb + h * K::M_BYTES + srow * 128;
      const float er0 = s[SC_ER + r0], er1 = s[SC_ER + r0 + 8];
      const float c0 = s[SC_CUM + r0], c1 = s[SC_CUM + r0 + 8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > q) break;
        float m[8];
        if (j < q) {  // the whole tile lies before the rows: two factors, none above one
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 e = *reinterpret_cast<const float2*>(s + SC_ECD + 64 * (q - 1) + 16 * j + 8 * k + cl);
            m[4 * k] = g[j][4 * k] * er0 * e.x;
            m[4 * k + 1] = g[j][4 * k + 1] * er0 * e.y;
            m[4 * k + 2] = g[j][4 * k + 2] * er1 * e.x;
            m[4 * k + 3] = g[j][4 * k + 3] * er1 * e.y;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int sc = 16 * q + 8 * k + cl;
            const float2 cs = *reinterpret_cast<const float2*>(s + SC_CUM + sc), ds = *reinterpret_cast<const float2*>(s + SC_D + sc);
            m[4 * k] = sc <= r0 ? g[j][4 * k] * ex2(c0 - cs.x) * ds.x : 0.f;
            m[4 * k + 1] = sc + 1 <= r0 ? g[j][4 * k + 1] * ex2(c0 - cs.y) * ds.y : 0.f;
            m[4 * k + 2] = sc <= r0 + 8 ? g[j][4 * k + 2] * ex2(c1 - cs.x) * ds.x : 0.f;
            m[4 * k + 3] = sc + 1 <= r0 + 8 ? g[j][4 * k + 3] * ex2(c1 - cs.y) * ds.y : 0.f;
          }
        }
        const uint32_t pk[4] = {pack_bf16x2(m[0], m[1]), pack_bf16x2(m[2], m[3]), pack_bf16x2(m[4], m[5]),
                                pack_bf16x2(m[6], m[7])};
        stsm_x4(mh + (((2 * j + sch) ^ (srow & 7)) << 4), pk);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&x.bars[B_M0 + (i & 1)]);
  }
}

// S in registers: thread (lane p, half of the key channels).
template <int DK, int DV, bool STATES>
__device__ __forceinline__ void role_state(const Ctx& x, const TcArgs& t) {
  using K = Cfg<DK, DV>;
  constexpr int NC = DK / 2;
  const SsmArgs& a = t.a;
  const int w = (threadIdx.x >> 5) - W_ST, lane = threadIdx.x & 31, p = (w & 3) * 32 + lane, n0 = (w >> 2) * NC;
  const uint32_t tl = x.tmem + ((uint32_t)((w & 3) * 32) << 16);
  const int hl = DV == 64 ? p / 64 : 0;
  const bool live = hl < x.heads;
  const int head = live ? hl : 0;
  const int64_t at = ((int64_t)x.h0 + head) * DK * DV + (p & (DV - 1)) + (int64_t)n0 * DV, seq = (int64_t)a.H * DK * DV;
  float S[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) S[n] = 0.f;
  const bool split = x.piece.pieces > 1;
  float* slots = t.piece_state + at;  // slot s of this thread's elements at slots + s * seq
  if (!STATES && live && split) {
    // the state before this piece, from the pieces before it
    const int64_t s0 = x.piece.slot0;
    if (a.init) {
#pragma unroll
      for (int n = 0; n < NC; ++n) S[n] = slots[s0 * seq + (int64_t)n * DV];
    }
    for (int r = 0; r < x.piece.r; ++r) {
      const float dec = ex2(t.piece_decay[(s0 + r) * a.H + x.h0 + head]);
      const float* o = slots + (s0 + r + 1) * seq;
#pragma unroll
      for (int n = 0; n < NC; ++n) S[n] = fmaf(S[n], dec, o[(int64_t)n * DV]);
    }
  } else if (live && a.init && (!STATES || x.piece.r == 0)) {
    const float* o = a.init + x.piece.n * seq + at;
#pragma unroll
    for (int n = 0; n < NC; ++n) S[n] = o[(int64_t)n * DV];
    if (STATES) {  // kept for the second pass, whose last piece may write over the initial state
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        slots[(int64_t)x.piece.slot0 * seq + (int64_t)n * DV] = S[n];
        S[n] = 0.f;
      }
    }
  }
  auto publish = [&]() {  // S as bf16 pairs: the A operand of YI
#pragma unroll
    for (int k = 0; k < NC / 16; ++k) {
      uint32_t pk[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) pk[j] = pack_bf16x2(S[16 * k + 2 * j], S[16 * k + 2 * j + 1]);
      tmem_st8(tl + K::TM_S + (n0 >> 1) + 8 * k, pk);
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(&x.bars[B_SRDY]);
  };
  __syncwarp();
  if (!STATES && x.nchunks > 0) publish();
  bool ok = true;
  for (int i = 0; i < x.nchunks; ++i) {
    const int st = i % NST;
    ok = ok && wait_bar(x, B_DEC0 + st, (i / NST) & 1);
    ok = ok && wait_bar(x, B_U, i & 1);
    if (!named_sync_and(GRP_ST, 256, ok)) return;
    tc_fence_after();
    const float dec = reinterpret_cast<const float*>(x.sm + K::SM_MISC + MS_TOTAL)[st * 2 + head];
#pragma unroll
    for (int k = 0; k < NC / 16; ++k) {
      float u[16];
      tmem_ld16(tl + K::TM_U + n0 + 16 * k, u);
#pragma unroll
      for (int j = 0; j < 16; ++j) S[16 * k + j] = fmaf(S[16 * k + j], dec, u[j]);
    }
    tc_fence_before();
    mbar_arrive(&x.bars[B_UFREE]);
    __syncwarp();
    if (lane == 0) mbar_arrive(&x.bars[B_EMPTY0 + st]);
    if (!STATES && i + 1 < x.nchunks) {
      ok = wait_bar(x, B_SFREE, i & 1);
      __syncwarp();
      tc_fence_after();
      publish();
    }
  }
  if (!live || !ok) return;
  float* o = nullptr;
  if (STATES)
    o = slots + (int64_t)(x.piece.slot0 + x.piece.r + 1) * seq;
  else if (a.fin && x.piece.r == x.piece.pieces - 1)
    o = a.fin + x.piece.n * seq + at;
  if (o) {
#pragma unroll
    for (int n = 0; n < NC; ++n) o[(int64_t)n * DV] = S[n];
  }
}

// y = e^{G_t} YI + YM + D x, over x's own tile, then out by TMA (a chunk cut
// short by the sequence's end: row by row).
template <int DK, int DV>
__device__ __forceinline__ void role_out(const Ctx& x, const TcArgs& t, const void* to) {
  using K = Cfg<DK, DV>;
  const SsmArgs& a = t.a;
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3, tid = threadIdx.x - 32 * W_OUT;
  const uint32_t tl = x.tmem + ((uint32_t)(wq * 32) << 16);
  const int hl = DV == 64 && wq >= 2 ? 1 : 0;
  const float skip = a.D ? a.D[x.h0 + (hl < x.heads ? hl : 0)] : 0.f;
  const float2 skip2 = make_float2(skip, skip);
  const int atoms = x.heads * DV / 64;
  bool ok = true;
  for (int i = 0; i < x.nchunks; ++i) {
    const int st = i % NST, v = valid_rows(x, i);
    ok = ok && wait_bar(x, B_DEC0 + st, (i / NST) & 1);
    ok = ok && wait_bar(x, B_FULL0 + st, (i / NST) & 1);
    ok = ok && wait_bar(x, B_Y0 + (i & 1), (i >> 1) & 1);
    if (!named_sync_and(GRP_OUT, 128, ok)) break;
    tc_fence_after();
    uint8_t* stg = x.sm + K::SM_STAGE + st * K::STAGE;
    const float* ec = reinterpret_cast<const float*>(x.sm + K::SM_DEC) + (st * K::HEADS + hl) * SC_FLOATS + SC_ECUM;
    const uint32_t xa = smem_u32(stg) + (wq >> 1) * 8192;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int pc = (wq & 1) * 4 + half * 2;
      const uint32_t ta = tl + ((uint32_t)(half * 16) << 16);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {  // 16 tokens
        float yi[16], *ym = yi + 8;
        tmem_ld_16x256b_x2(ta + K::TM_YI + 16 * tb, yi);
        tmem_ld_16x256b_x2(ta + K::TM_YM + 16 * tb, ym);
        const int row = 16 * tb + ((lane >> 4) & 1) * 8 + (lane & 7), ch = pc + ((lane >> 3) & 1);
        const uint32_t xaddr = xa + row * 128 + ((ch ^ (row & 7)) << 4);
        uint32_t raw[4];
        ldsm_x4_t(xaddr, raw);
        tmem_wait_ld(yi);
        uint32_t pk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 e = *reinterpret_cast<const float2*>(ec + 16 * tb + (j >> 1) * 8 + 2 * (lane & 3));
          float2 y = __ffma2_rn(e, make_float2(yi[2 * j], yi[2 * j + 1]), make_float2(ym[2 * j], ym[2 * j + 1]));
          y = __ffma2_rn(skip2, bf16x2_f32(raw[j]), y);
          pk[j] = pack_bf16x2(y.x, y.y);
        }
        stsm_x4_t(xaddr, pk);
      }
    }
    tc_fence_before();
    mbar_arrive(&x.bars[B_YFREE]);
    fence_proxy_async_smem();
    named_sync(GRP_OUT, 128);
    const int64_t tok = x.piece.start + (int64_t)i * CH;
    if (v == CH) {
      if (tid == 0) {
        for (int k = 0; k < atoms; ++k) tma_store_2d(to, smem_u32(stg) + k * 8192, x.h0 * DV + 64 * k, (int)tok);
        bulk_commit();
        bulk_wait_read0();
        mbar_arrive(&x.bars[B_EMPTY0 + st]);
      }
    } else {  // only a piece's last chunk
      __nv_bfloat16* out = (__nv_bfloat16*)a.out + (int64_t)x.h0 * DV;
      for (int e = tid; e < atoms * v * 8; e += 128) {
        const int atom = e / (v * 8), row = (e - atom * v * 8) >> 3, c = e & 7;
        const uint4 u = *reinterpret_cast<const uint4*>(stg + atom * 8192 + row * 128 + ((c ^ (row & 7)) << 4));
        *reinterpret_cast<uint4*>(out + (tok + row) * ((int64_t)a.H * DV) + atom * 64 + c * 8) = u;
      }
    }
  }
  if (tid == 0) bulk_wait_all();
}

template <int DK, int DV, bool STATES>
__global__ void __launch_bounds__(NTHR, 1)
    ssm_tc_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tb,
                  const __grid_constant__ CUtensorMap tc, const __grid_constant__ CUtensorMap to,
                  const __grid_constant__ TcArgs t) {
  using K = Cfg<DK, DV>;
  extern __shared__ uint8_t smem_raw[];
  Ctx x;
  x.tile = blockIdx.x % t.tiles;
  if (!find_piece(t, blockIdx.x / t.tiles, x.piece)) return;
  if (STATES && x.piece.r == x.piece.pieces - 1) return;  // nothing follows it
  x.sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  x.sb = smem_u32(x.sm);
  x.bars = reinterpret_cast<uint64_t*>(x.sm + K::SM_MISC);
  x.abort = reinterpret_cast<volatile int*>(x.sm + K::SM_MISC + MS_ABORT);
  x.status = t.a.status;
  x.heads = t.hpt;
  x.h0 = x.tile * t.hpt;
  x.nchunks = (int)((x.piece.end - x.piece.start + CH - 1) / CH);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NUM_BARS; ++i) {
      int n = 1;
      if (i >= B_EMPTY0 && i < B_EMPTY0 + NST) n = 1 + 8;
      if (i == B_WX || i == B_GFREE || i == B_M0 || i == B_M1 || i == B_YFREE) n = 128;
      if (i == B_UFREE || i == B_SRDY) n = 256;
      mbar_init(&x.bars[i], n);
    }
    fence_mbar_init();
    *x.abort = 0;
    prefetch_tmap(&tx);
    prefetch_tmap(&tb);
    prefetch_tmap(&tc);
    prefetch_tmap(&to);
  }
  if (!STATES) {  // zero tiles and score tiles
    for (int e = tid; e < (int)(K::ZERO / 16); e += NTHR) {
      reinterpret_cast<uint4*>(x.sm + K::SM_Z0)[e] = make_uint4(0u, 0u, 0u, 0u);
      reinterpret_cast<uint4*>(x.sm + K::SM_Z1)[e] = make_uint4(0u, 0u, 0u, 0u);
    }
    for (int e = tid; e < (int)(2 * K::HEADS * K::M_BYTES / 16); e += NTHR)
      reinterpret_cast<uint4*>(x.sm + K::SM_M)[e] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(reinterpret_cast<uint32_t*>(x.sm + K::SM_MISC + MS_TMEM), K::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  x.tmem = *reinterpret_cast<volatile uint32_t*>(x.sm + K::SM_MISC + MS_TMEM);

  if (warp == W_TMA) {
    if (lane == 0) role_load<DK, DV, STATES>(x, &tx, &tb, &tc, x.h0 / (t.a.H / t.a.G));
  } else if (warp == W_MMA) {
    if (lane == 0) {
      if (x.nchunks > 0) role_mma<DK, DV, STATES>(x);
      umma_commit(&x.bars[B_DRAIN]);  // every product has ended before TMEM is released
      mbar_wait(&x.bars[B_DRAIN], 0, WAIT_NS);
    }
  } else if (warp == W_DEC) {
    role_decay<DK, DV, STATES>(x, t);
  } else if (warp >= W_ST) {
    role_state<DK, DV, STATES>(x, t);
  } else if (warp >= W_OUT) {
    if (!STATES) role_out<DK, DV>(x, t, &to);
  } else if (warp >= W_SC) {
    if (!STATES) role_scores<DK, DV>(x);
  } else {
    role_wx<DK, DV>(x);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(x.tmem, K::TM_COLS);
  }
}

// ------------------------------------------------------------------ host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// bf16 rows of `width` columns, `ld` elements apart; boxes of 64 columns x 64 rows, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* ptr, int64_t width, int64_t ld, int64_t rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, CH};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int SMS = 148;         // of a B200
constexpr int MIN_PIECE = 4;     // chunks in a piece, at least
constexpr int MAX_PIECES = 32;   // of a sequence of known length (a piece adds up the ones before it)

struct Plan {
  int hpt, tiles, per_seq;
  int64_t piece_len, pieces, slots;  // pieces, slots: upper bounds for packed batches
  bool split;
  size_t table, decay, state, total;  // workspace offsets
};

Plan make_plan(int N, int64_t T, int H, int G, int dk, int dv, bool packed) {
  Plan p;
  p.hpt = dv == 64 && (H / G) % 2 == 0 ? 2 : 1;
  p.tiles = H / p.hpt;
  const int64_t chunks = (T + CH - 1) / CH;  // of a sequence, or of the packed total
  const int64_t chains = (int64_t)N * p.tiles;
  if (!packed) {
    // Pieces in parallel against the states of all but the last of them a
    // second time (about half the work of a chunk): the count whose two
    // passes have the fewest chunk times, in waves of one block per SM.
    int best = 1;
    double cost = (double)((chains + SMS - 1) / SMS) * chunks;
    for (int r = 2; r <= MAX_PIECES && chunks / r >= MIN_PIECE; ++r) {
      const int64_t len = (chunks + r - 1) / r;
      const double c = (double)((chains * r + SMS - 1) / SMS) * (len + 3) + 0.5 * ((chains * (r - 1) + SMS - 1) / SMS) * (len + 3) + 6;
      if (c < cost) {
        cost = c;
        best = r;
      }
    }
    const int64_t len = (chunks + best - 1) / best;
    p.per_seq = (int)(len > 0 ? (chunks + len - 1) / len : 1);
    if (p.per_seq < 1) p.per_seq = 1;
    p.piece_len = (len > 0 ? len : 1) * CH;
    p.pieces = (int64_t)N * p.per_seq;
    p.split = p.per_seq > 1;
    p.slots = p.split ? p.pieces : 0;
  } else {
    // The lengths are on the device: pieces of twice the SMs' number in all,
    // so that one long sequence does not hold the batch up.
    int64_t len = (chunks * p.tiles + 2 * SMS - 1) / (2 * SMS);
    if (len < MIN_PIECE) len = MIN_PIECE;
    p.per_seq = 0;
    p.piece_len = len * CH;
    p.pieces = N + T / p.piece_len;
    p.split = T > p.piece_len;
    // a sequence of L > len tokens has at most L / len + 1 < 2 L / len pieces
    p.slots = p.split ? 2 * T / p.piece_len : 0;
  }
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  size_t off = 256;  // the status word
  p.table = off;
  if (packed) off += up((size_t)p.pieces * sizeof(PieceEntry));
  p.decay = off;
  off += up((size_t)p.slots * H * sizeof(float));
  p.state = off;
  off += (size_t)p.slots * H * dk * dv * sizeof(float);
  p.total = off;
  return p;
}

template <int DK, int DV>
cudaError_t launch(const TcArgs& t, const Plan& p, cudaStream_t s) {
  using K = Cfg<DK, DV>;
  const SsmArgs& a = t.a;
  const int64_t rows = a.cu ? a.T : (int64_t)a.N * a.T;
  CUtensorMap tx, tb, tc, to;
  if (!make_map(&tx, a.x, (int64_t)a.H * DV, a.ldx, rows) || !make_map(&tb, a.b, (int64_t)a.G * DK, a.ldb, rows) ||
      !make_map(&tc, a.c, (int64_t)a.G * DK, a.ldc, rows) ||
      !make_map(&to, a.out, (int64_t)a.H * DV, (int64_t)a.H * DV, rows))
    return cudaErrorInvalidValue;
  const unsigned blocks = (unsigned)(p.pieces * p.tiles);
  if (t.table) {
    ssm_piece_table_kernel<<<1, 1024, 0, s>>>(Seqs{a.cu, a.N, a.T}, p.piece_len, (int)p.pieces, (int)p.slots,
                                              const_cast<PieceEntry*>(t.table));
  }
  cudaError_t e;
  if (p.split) {
    auto* k1 = ssm_tc_kernel<DK, DV, true>;
    if ((e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::BYTES)) != cudaSuccess) return e;
    k1<<<blocks, NTHR, K::BYTES, s>>>(tx, tb, tc, to, t);
  }
  auto* k2 = ssm_tc_kernel<DK, DV, false>;
  if ((e = cudaFuncSetAttribute(k2, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::BYTES)) != cudaSuccess) return e;
  k2<<<blocks, NTHR, K::BYTES, s>>>(tx, tb, tc, to, t);
  return cudaGetLastError();
}

}  // namespace

bool ssm_tc_supported(int dk, int dv, bool bf16) { return bf16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }

size_t ssm_tc_workspace(int N, int64_t T, int H, int G, int dk, int dv, bool packed) {
  return make_plan(N, T, H, G, dk, dv, packed).total;
}

cudaError_t launch_ssm_fwd_tc(const SsmArgs& a, void* workspace, cudaStream_t s) {
  const Plan p = make_plan(a.N, a.T, a.H, a.G, a.dk, a.dv, a.cu != nullptr);
  char* ws = static_cast<char*>(workspace);
  TcArgs t;
  t.a = a;
  t.hpt = p.hpt;
  t.tiles = p.tiles;
  t.piece_len = p.piece_len;
  t.per_seq = p.per_seq;
  t.table = a.cu ? reinterpret_cast<const PieceEntry*>(ws + p.table) : nullptr;
  t.piece_decay = reinterpret_cast<float*>(ws + p.decay);
  t.piece_state = reinterpret_cast<float*>(ws + p.state);
  if (a.dk == 128) return a.dv == 128 ? launch<128, 128>(t, p, s) : launch<128, 64>(t, p, s);
  return a.dv == 128 ? launch<64, 128>(t, p, s) : launch<64, 64>(t, p, s);
}

}  // namespace kda
