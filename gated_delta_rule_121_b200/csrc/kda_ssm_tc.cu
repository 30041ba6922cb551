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
// The scores' exponents.  A difference of two sums over the whole chunk keeps only
// what the sums' size leaves of it (sums of 1e6: 6 %), so they are made from sums
// over 16 tokens: for tokens of one sixteen the difference of their sums to its
// end; else the sum from behind s to the end of its sixteen, the whole sixteens
// between, and from the start of t's sixteen to t.  A token's log decay counts as
// MIN_LOG2 where it is below that: a score across such a token is zero in fp32
// either way, for the largest D_s as well, and the sums stay within 4096, so that an
// exponent is off by 2^-10 at most: 0.07 % of the score, of which half a bf16 step
// is 0.4 %.
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
// Rounding.  x, b, c are bf16 and exact.  w x enters U in four bf16 terms that
// leave out 2^-25 of it (role_wx), so that the state, which is returned and
// carried in fp32, keeps fp32 accuracy; the state itself stays in registers and
// takes each chunk's U by one fp32 multiply-add per element.  S and M enter the
// output's products as bf16 (half a step each, 2^-8 relative): y is rounded to
// bf16 itself, and the three are of one size where the terms of a sum do not cancel;
// where they do, y is off by half a step of their magnitudes.
//
// Roles (32 warps, one block per SM): wx (4 warps) weights x and stores its
// terms; scores (8) turn G into M; state (16) holds S and combines YI, YM and
// the skip over x's own tile; one warp each for the copies, the issue of U and
// G, that of YI and YM, and the chunk's scalars.
//
// Long sequences are cut into pieces that run in parallel (kda_ssm_pieces.cuh).
//
// Measured, 64K tokens, 96 heads, dk = 128, dv = 64 (48 tiles, three pieces): 0.95
// ms on the same buffers again and again, 1.10 with other inputs in between.  A
// chunk takes 0.95 us in the first pass and 2 us in the second.  Nothing is
// saturated in the second pass (issue slots 64 % busy, tensor pipe 52 %, the
// shared-memory pipe of the roles' own accesses 42 %, DRAM 28 %): its time is what
// the roles wait for one another along a chunk's chain of products.  U's four
// terms are 60 % of the tensor work there and all of it in the first pass.  A state
// of 64 columns per thread in eight warps (fewer instructions in all) does not fit
// the registers that remain.
#include <cuda.h>

#include <algorithm>

#include "kda_ssm_pieces.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace {

constexpr int CH = PIECE_CHUNK;  // tokens per chunk
constexpr int PT = 128;          // value columns per tile
constexpr float LOG2E = 1.4426950408889634f;

// First warps of the roles.
constexpr int W_WX = 0, W_SC = 4, W_ST = 12, ST_WARPS = 16, W_MOVE = W_ST + ST_WARPS, W_MMY = W_MOVE + 1,
              W_MMU = W_MOVE + 2, W_DEC = W_MOVE + 3, NWARP = W_MOVE + 4;
constexpr int NTHR = 32 * NWARP;
constexpr int N_WX = 128, N_SC = 256, N_ST = 32 * ST_WARPS;  // threads
constexpr int GRP_WX = 1;                                    // named barrier of wx

// Hand-offs.  Per stage: XFULL x has landed, XFREE (first pass) it has been used,
// DEC the scalars are there, KFULL / KFREE the same of b and c, XREAD wx has read
// x, YOUT y stands in x's place.  Per chunk: WX half of w x is there, U it has been
// used (and with the second half U is there), UFREE U has been read, G scores' Gram
// is there, M scores are there (and G has been read), SRDY / SFREE S as bf16 is
// there / has been used, Y both parts of y are there, YFREE they have been read.
// A barrier whose waiter can fall a phase behind is doubled by the chunk's parity.
// x and the scalars share a ring of NX stages, b and c have one of NB.
constexpr int MAXST = 6;
enum Bar {
  B_XFULL = 0,
  B_XFREE = B_XFULL + MAXST,
  B_DEC = B_XFREE + MAXST,
  B_KFULL = B_DEC + MAXST,
  B_KFREE = B_KFULL + MAXST,
  B_XREAD = B_KFREE + MAXST,
  B_YOUT = B_XREAD + MAXST,
  B_WX = B_YOUT + MAXST,  // [chunk % 2][half]
  B_U = B_WX + 4,         // [chunk % 2][half]
  B_UFREE = B_U + 4,      // [chunk % 2]
  B_M = B_UFREE + 2,      // [chunk % 2]
  B_Y = B_M + 2,          // [chunk % 2]
  B_G = B_Y + 2,
  B_SRDY,
  B_SFREE,
  B_YFREE,
  B_DRAIN,
  NUM_BARS
};

// Scalars of a chunk, per head, at these 32-bit words: the steps D_s, and in their
// place DOWN_s + log2 D_s (the scores' columns); the
// weights w_s = e^{G_C - G_s} D_s as three bf16 terms (pairs of tokens, 32 words
// each); G_t; and DOWN, the sums of log decays from behind a token to the end of
// its sixteen (zero for the last one, in whose place the sixteen's total stands): both
// in log2 units.
constexpr int SC_D = 0, SC_COL = 0, SC_W = 64, SC_CUM = 160, SC_DOWN = 224;
constexpr float MIN_LOG2 = -256.f;  // of a token's decay

// In SM_MISC, behind the barriers: TMEM address, abort flag, totals e^{G_C} by slot
// and head, the log decays that each of the scalars' warps has seen, by head; the
// block's items.
constexpr uint32_t MS_TMEM = 488, MS_ABORT = 492, MS_TOTAL = 496, MS_SUM = 544, MS_ITEMS = 560;
constexpr int MAX_ITEMS = 7;  // of a block
constexpr uint32_t MISC = MS_ITEMS + MAX_ITEMS * 24;
static_assert(NUM_BARS * 8 <= MS_TMEM, "barrier area");

template <int DK, int DV, bool STATES>
struct Cfg {
  static constexpr int HEADS = PT / DV;                  // heads per tile, at most
  static constexpr int NX = STATES ? 6 : 5, NB = STATES ? 6 : 3;
  static constexpr uint32_t KV = CH * DK * 2;            // b or c of a chunk
  static constexpr uint32_t X_BYTES = CH * PT * 2, K_BYTES = STATES ? KV : 2 * KV;
  static constexpr uint32_t M_BYTES = STATES ? 0 : CH * CH * 2;  // one head's scores
  static constexpr uint32_t ZERO = STATES ? 0 : 2048;            // 16 rows of zeros of 64 columns
  static constexpr int SC_FLOATS = STATES ? 160 : 288, SC_SLOT = HEADS * SC_FLOATS * 4;
  // shared memory: zeros, x, zeros (the zero tiles lie below and above x: descriptor strides are positive)
  static constexpr uint32_t SM_Z0 = 0, SM_X = ZERO, SM_Z1 = SM_X + NX * X_BYTES, SM_K = SM_Z1 + ZERO;
  static constexpr uint32_t SM_M = SM_K + NB * K_BYTES, SM_DEC = SM_M + 2 * HEADS * M_BYTES;
  static constexpr uint32_t SM_RAW = SM_DEC + NX * SC_SLOT;  // delta of four chunks to come, per warp
  static constexpr int DECS = STATES ? 2 : 1;                // warps for the scalars
  static constexpr uint32_t RAW = 4 * HEADS * CH * 4;
  static constexpr uint32_t SM_MISC = SM_RAW + DECS * RAW;
  static constexpr uint32_t BYTES = SM_MISC + MISC + 1024;
  // TMEM columns; the first pass has room for two of w x and U, so that one is read while the next is made
  static constexpr int NU = STATES ? 2 : 1;
  static constexpr uint32_t TM_WX = 0, TM_S = 128, TM_YI = TM_S + DK / 2, TM_YM = TM_YI + 64,
                            TM_U = STATES ? 256 : TM_YM + 64, TM_G = TM_U + NU * DK, TM_END = TM_G + (STATES ? 0 : 64);
  static constexpr uint32_t TM_COLS = 512;
  static_assert(NX <= MAXST && NB <= MAXST, "stages");
  static_assert(TM_END <= TM_COLS, "TMEM");
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(tmap), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ void tma_prefetch_2d(const void* tmap, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tmap), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tmap), "r"(src),
               "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// 16 lanes x 32 columns (fp32): thread l gets rows l/4 and l/4 + 8, of each 8
// columns numbers 2 (l % 4) and the next: {r, c}, {r, c+1}, {r+8, c}, {r+8, c+1},
// then the same of the next 8 columns, and so on.
__device__ __forceinline__ void tmem_ld_16x256b_x4_wait(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
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
// 16 columns from each of two places.
__device__ __forceinline__ void tmem_ld_16x256b_x2x2_wait(uint32_t ta, uint32_t tb, float (&a)[8], float (&b)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]), "=f"(a[6]), "=f"(a[7]), "=f"(b[0]),
        "=f"(b[1]), "=f"(b[2]), "=f"(b[3]), "=f"(b[4]), "=f"(b[5]), "=f"(b[6]), "=f"(b[7])
      : "r"(ta), "r"(tb)
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
// MMAs whose descriptors differ in their low words only (address and atom
// stride, both in 16-byte units): 128-byte swizzle, 1024 bytes between groups
// of 8 rows, the sm_100 descriptor version.
constexpr uint32_t DESC_HI = (2u << 29) | (1u << 14) | (1024u >> 4);
__device__ __forceinline__ void umma_ss_lo(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"(DESC_HI)
      : "memory");
}
__device__ __forceinline__ void umma_ts_lo(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"(DESC_HI)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float2 bf16x2_f32(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// The upper halves of two fp32 values (their truncation to bf16), the first in the low half.
__device__ __forceinline__ uint32_t upper_halves(float2 v) {
  return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
}
__device__ __forceinline__ float2 below_upper(float2 v) {  // what that leaves, exactly
  return make_float2(v.x - __uint_as_float(__float_as_uint(v.x) & 0xffff0000u),
                     v.y - __uint_as_float(__float_as_uint(v.y) & 0xffff0000u));
}
// max(a, b), and what is not a number stays so.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// Packed bf16 arithmetic, rounded to nearest.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t fms_bf16x2(uint32_t a, uint32_t b, uint32_t c) {  // a b - c
  uint32_t d;
  asm("{\n\t.reg .b32 n;\n\tneg.bf16x2 n, %3;\n\tfma.rn.bf16x2 %0, %1, %2, n;\n\t}" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

struct TcArgs {
  SsmArgs a;
  PieceArgs p;
  int hpt, tiles;  // heads per tile, tiles of 128 columns
  int items;       // pieces times tiles
  int blocks, per_block;  // of the second pass, and items of a block there
  uint32_t wait_ns;       // limit of the waits
  int stop_at;            // a test's: the loads' role stands still before this chunk
};

// ------------------------------------------------------------------ roles
// Every role walks all chunks, so each block runs seven programs at once.  Their
// loops are kept rolled and short: the instruction caches hold all of them only
// then (with the roles unrolled, warps waited for instructions most of the
// time, 3.6 us a chunk).  For the same reason the waits are short and inline.
struct Ctx {
  uint8_t* sm;
  uint32_t sb, tmem, bars;   // shared-window addresses of sm and of the barriers; TMEM base
  int heads;                 // of a tile
  int items, nchunks;        // of the block
  const int4* item;          // what the items are (item_index)
};

// A block's items (a tile of a piece each): one in the first pass; in the second up
// to MAX_ITEMS, for which the block's start (launch, barriers, TMEM, the first loads)
// is paid once and the next item's loads and first products run beside the end of
// the last one (191 packed prompts of up to 200 tokens, H = 16: 94 us, with a block
// per item 132).  Every gridDim.x-th item in alternating direction, since the table of
// a packed batch has the long ones first.
__device__ __forceinline__ int item_index(int turn) {
  return turn * gridDim.x + (turn & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}
__device__ __forceinline__ int chunks_of(int tokens) { return (tokens + CH - 1) / CH; }
// In shared memory, per item: its tokens [tok, end) (none: tok = end), first head and
// sequence; and its slot0 and 8 before + flags.
constexpr int SPLIT = 1, LAST = 2, VALID = 4;
// The chunks of a block's items one after the other; next() is called before the first.
template <bool ONE>  // one item only, which has chunks
struct Walk {
  int turn = 0, tok = 0, end = 0, h0 = 0, n = -1;
  __device__ __forceinline__ bool next(const Ctx& x) {  // whether it starts an item
    tok += CH;
    if (ONE ? turn > 0 : tok < end) return false;
    tok = end = 0;
    bool found = false;
#pragma unroll 1
    while (turn < x.items && !found) {
      const int4 d = x.item[turn++];
      found = d.x < d.y;
      if (found) tok = d.x, end = d.y, h0 = d.z, n = d.w;
    }
    return found;
  }
};

// A role's wait.  It ends once the block's abort flag is raised, which it looks at
// every 256 tests.  The loads' role raises it (wait_warp): where anything of a block
// stands still, so does that role, which lives as long as the block has work, and
// it measures the time.  Behind that stands a limit of tests, for the
// case that the loads' role itself is not there any more.  The roles that only
// compute run on over whatever is there (every access stays inside its
// buffers) and do not look at the result; the ones that start copies or
// products stop.  All that is waited for are the block's own loads and products.
// Written as one block, so that a wait that finds its phase complete takes three
// instructions (and without a time hint: with one, a wait becomes a loop of sleeps
// that takes issue slots from the other roles and wakes late; with a clock in
// every wait a 64K prompt takes 2 % longer).
constexpr uint32_t MAX_TESTS = 1u << 27;  // of the phase's barrier: a test takes some 50 ns
__device__ __forceinline__ bool wait_at(uint32_t bars, uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n, f;\n\t"
      "mov.u32 n, 0;\n"
      "TEST:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\t"
      "and.b32 f, n, 255;\n\t"
      "setp.ne.u32 q, f, 0;\n\t"
      "@q bra TEST;\n\t"
      "ld.volatile.shared.u32 f, [%3];\n\t"
      "setp.lt.u32 q, n, %4;\n\t"
      "setp.eq.and.u32 q, f, 0, q;\n\t"
      "@q bra TEST;\n\t"
      "mov.u32 f, 1;\n\t"
      "st.volatile.shared.u32 [%3], f;\n"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(bars + MS_ABORT), "n"(MAX_TESTS)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_bar(const Ctx& x, int bar, uint32_t parity) {
  return wait_at(x.bars, x.bars + 8 * bar, parity);
}
__device__ __forceinline__ void arrive(const Ctx& x, int bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(x.bars + 8 * bar) : "memory");
}
__device__ __forceinline__ void commit(const Ctx& x, int bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(x.bars + 8 * bar)
               : "memory");
}
// The loads' role's waits, by wall time, and for all lanes of its warp alike.
__device__ __forceinline__ bool test_256(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 0;\n"
      "TEST:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 q, n, 256;\n\t"
      "@q bra TEST;\n"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_warp(const Ctx& x, int bar, uint32_t parity, uint32_t ns) {
  const uint32_t at = x.bars + 8 * bar;
  if (__all_sync(0xffffffffu, test_256(at, parity))) return true;
  const uint32_t t0 = globaltimer_lo();  // (turns over after 4.3 s: twice the longest limit)
  do {
    if (__all_sync(0xffffffffu, test_256(at, parity))) return true;
  } while (__all_sync(0xffffffffu, globaltimer_lo() - t0 < ns));
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(x.bars + MS_ABORT), "r"(1) : "memory");
  return false;
}
// A copy or product in flight has ended, whatever else the block gave up.
__device__ __forceinline__ void land(uint32_t bar, uint32_t parity) {
  const uint32_t t0 = globaltimer_lo();
  while (!test_256(bar, parity) && globaltimer_lo() - t0 < SSM_WAIT_NS) {}
}
// A chunk's stage in a ring of N and the parity of its use, counted along.
template <int N>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) {
      st = 0;
      ph ^= 1;
    }
  }
};

// Loads, and the stores of y out of x's tile: by TMA, or row by row where the
// sequence's end cuts the last chunk short.  A stage of x is loaded anew once
// its y has been read for the store.
template <int DK, int DV, bool STATES>
__device__ __forceinline__ void role_move(const Ctx& x, const TcArgs& t, const void* tx, const void* tb, const void* tc,
                                          const void* to, bool leader) {
  using K = Cfg<DK, DV, STATES>;
  const int atoms = x.heads * DV / 64, per_group = t.a.H / t.a.G;
  int nk = 0, nx = 0;  // chunks whose loads have been issued
  Walk<STATES> wk, wx, wo;     // chunks to load next (b and c; x), and to store
  Ring<K::NB> k;
  Ring<K::NX> s;
  auto load_k = [&]() {
    wk.next(x);
    if (leader) {
      const uint32_t bar = x.bars + 8 * (B_KFULL + k.st), dst = x.sb + K::SM_K + k.st * K::K_BYTES;
      const int col = wk.h0 / per_group * DK;
      expect_tx(bar, K::K_BYTES);
#pragma unroll
      for (int e = 0; e < DK / 64; ++e) {
        tma_load_2d(dst + e * 8192, tb, bar, col + 64 * e, wk.tok);
        if (!STATES) tma_load_2d(dst + K::KV + e * 8192, tc, bar, col + 64 * e, wk.tok);
      }
    }
    ++nk;
    k.next();
  };
  auto load_x = [&]() {
    const bool fresh = wx.next(x);
    if (leader) {
      const uint32_t bar = x.bars + 8 * (B_XFULL + s.st), dst = x.sb + K::SM_X + s.st * K::X_BYTES;
      expect_tx(bar, atoms * 8192);
      tma_load_2d(dst, tx, bar, wx.h0 * DV, wx.tok);
      if (atoms == 2) tma_load_2d(dst + 8192, tx, bar, wx.h0 * DV + 64, wx.tok);
    }
    ++nx;
    s.next();
    if (fresh && leader && nx > 1 && t.a.init) {  // the item's initial state into L2
      const float* o = t.a.init + ((int64_t)wx.n * t.a.H + wx.h0) * DK * DV;
      for (int h = 0; h < x.heads; ++h) prefetch_l2(o + h * DK * DV, DK * DV * 4);
    }
  };
#pragma unroll 1
  for (int i = -K::NX; i < x.nchunks; ++i) {  // chunk i's store; the loads run ahead
    if (i == t.stop_at && !wait_warp(x, B_DRAIN, 0, t.wait_ns)) break;
    if (leader && i >= 0 && wx.tok + 2 * CH < wx.end) {  // into L2, a chunk before its load
      for (int e = 0; e < atoms; ++e) tma_prefetch_2d(tx, wx.h0 * DV + 64 * e, wx.tok + 2 * CH);
    }
    // k, s: the stages of chunks i + NB, i + NX, which are those of chunk i
    if (i + K::NB >= 0 && i + K::NB < x.nchunks) {
      if (i >= 0 && !wait_warp(x, B_KFREE + k.st, k.ph ^ 1, t.wait_ns)) break;
      load_k();
    }
    if (!STATES && i >= 0) {
      wo.next(x);
      const int st = i % K::NX;
      if (!wait_warp(x, B_YOUT + st, (i / K::NX) & 1, t.wait_ns)) break;
      const int v = min(wo.end - wo.tok, CH), col = wo.h0 * DV;
      const uint32_t at = K::SM_X + st * K::X_BYTES;
      if (v == CH) {
        if (leader) {
          tma_store_2d(to, x.sb + at, col, wo.tok);
          if (atoms == 2) tma_store_2d(to, x.sb + at + 8192, col + 64, wo.tok);
          bulk_commit();
          if (i + K::NX < x.nchunks) bulk_wait_read0();
        }
      } else {
        __nv_bfloat16* out = (__nv_bfloat16*)t.a.out + col;
#pragma unroll 1
        for (int e = threadIdx.x & 31; e < atoms * v * 8; e += 32) {
          const int atom = e / (v * 8), r = (e - atom * v * 8) >> 3, c = e & 7;
          const uint4 u = *reinterpret_cast<const uint4*>(x.sm + at + atom * 8192 + r * 128 + ((c ^ (r & 7)) << 4));
          *reinterpret_cast<uint4*>(out + ((int64_t)wo.tok + r) * ((int64_t)t.a.H * DV) + atom * 64 + c * 8) = u;
        }
        fence_proxy_async_smem();  // read before the next load into this stage
      }
    }
    if (i + K::NX < x.nchunks) {
      if (STATES && i >= 0 && !wait_warp(x, B_XFREE + s.st, s.ph ^ 1, t.wait_ns)) break;
      __syncwarp();
      load_x();
    }
  }
  // The last chunk has been used (a chunk's y has: the loop above has waited for it).
  if (STATES && nx > 0 && nx == x.nchunks) wait_warp(x, B_XFREE + (nx - 1) % K::NX, ((nx - 1) / K::NX) & 1, t.wait_ns);
  // No copy stays in flight behind the block: the latest load of every stage, and every store.
#pragma unroll 1
  for (int i = 0; i < MAXST; ++i) {
    const int cx = nx - 1 - i, ck = nk - 1 - i;
    if (i < K::NX && cx >= 0) land(x.bars + 8 * (B_XFULL + cx % K::NX), (cx / K::NX) & 1);
    if (i < K::NB && ck >= 0) land(x.bars + 8 * (B_KFULL + ck % K::NB), (ck / K::NB) & 1);
  }
  if (leader) bulk_wait_all();
}

// Two warps issue the products, U and the next chunk's G, and YI and YM (one
// warp for all of them was the slowest role, and held YI back until the scores
// had been made).  The whole warp walks the chunks, so that addresses stay
// warp-uniform; one lane issues.
template <int DK, int DV, bool STATES>
__device__ __forceinline__ void role_mma_u(const Ctx& x, bool leader) {
  using K = Cfg<DK, DV, STATES>;
  constexpr uint32_t LBO = 8192 >> 4;  // between 64-column atoms
  const uint32_t b0 = (x.sb + K::SM_K) >> 4;
  Ring<K::NX> s, sn;  // this chunk's stages, and the next one's
  Ring<K::NB> kr, kn;
#pragma unroll 1
  for (int i = STATES ? 0 : -1; i < x.nchunks; ++i) {
    if (i >= 0) {
      if (STATES && !wait_bar(x, B_KFULL + kr.st, kr.ph)) return;
      if (i >= K::NU && !wait_bar(x, B_UFREE + ((i - K::NU) & 1), ((i - K::NU) >> 1) & 1)) return;
      const uint32_t d = x.tmem + K::TM_U + (K::NU == 2 ? (i & 1) * DK : 0);
      uint32_t bb = (b0 + (uint32_t)kr.st * (K::K_BYTES >> 4)) | (LBO << 16), ta = x.tmem + K::TM_WX + (K::NU == 2 ? (i & 1) * 128 : 0);
      // by halves of the chunk, the small terms first
#pragma unroll 1
      for (int half = 0; half < 2; ++half, bb += 256, ta += 64) {
        if (!wait_bar(x, B_WX + 2 * (i & 1) + half, (i >> 1) & 1)) return;
        tc_fence_after();
        if (leader) {
          constexpr uint32_t id = idesc_bf16_f32(128, DK, 0, 1);
#pragma unroll
          for (int term = 3; term >= 0; --term) {
            umma_ts_lo(d, ta + 16 * term, bb, id, half > 0 || term < 3);
            umma_ts_lo(d, ta + 16 * term + 8, bb + 128, id, true);
          }
          commit(x, B_U + 2 * (i & 1) + half);
        }
      }
      if (leader) {
        commit(x, B_KFREE + kr.st);
        if (STATES) commit(x, B_XFREE + s.st);
      }
      s.next();
      kr.next();
    }
    if (!STATES && i + 1 < x.nchunks) {
      // the scalars as well, so that the scores' role has one wait for all
      if (!wait_bar(x, B_KFULL + kn.st, kn.ph) || !wait_bar(x, B_DEC + sn.st, sn.ph)) return;
      if (i >= 0 && !wait_bar(x, B_M + (i & 1), (i >> 1) & 1)) return;
      tc_fence_after();
      if (leader) {
        constexpr uint32_t id = idesc_bf16_f32(64, 64, 0, 0);
        const uint32_t bk = b0 + (uint32_t)kn.st * (K::K_BYTES >> 4), ck = bk + (K::KV >> 4);
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
          const uint32_t o = (k >> 2) * LBO + (k & 3) * 2;
          umma_ss_lo(x.tmem + K::TM_G, ck + o, bk + o, id, k > 0);
        }
        commit(x, B_G);
      }
      kn.next();
      sn.next();
    }
  }
}

template <int DK, int DV>
__device__ __forceinline__ void role_mma_y(const Ctx& x, bool leader) {
  using K = Cfg<DK, DV, false>;
  constexpr uint32_t LBO = 8192 >> 4;
  const uint32_t x0 = (x.sb + K::SM_X) >> 4, c0 = (x.sb + K::SM_K + K::KV) >> 4;
  const uint32_t z0 = (x.sb + K::SM_Z0) >> 4, z1 = (x.sb + K::SM_Z1) >> 4, m0 = (x.sb + K::SM_M) >> 4;
  const uint32_t tm = x.tmem;
  const bool two = x.heads == 2;
  Ring<K::NX> s;
  Ring<K::NB> kr;
#pragma unroll 1
  for (int i = 0; i < x.nchunks; ++i, s.next(), kr.next()) {
    if (!wait_bar(x, B_KFULL + kr.st, kr.ph)) return;
    if (!wait_bar(x, B_SRDY, i & 1)) return;
    if (i > 0 && !wait_bar(x, B_YFREE, (i - 1) & 1)) return;
    tc_fence_after();
    if (leader) {
      constexpr uint32_t id = idesc_bf16_f32(128, 64, 0, 0);
      const uint32_t ck = c0 + (uint32_t)kr.st * (K::K_BYTES >> 4);
#pragma unroll
      for (int k = 0; k < DK / 16; ++k)
        umma_ts_lo(tm + K::TM_YI, tm + K::TM_S + k * 8, ck + (k >> 2) * LBO + (k & 3) * 2, id, k > 0);
      commit(x, B_SFREE);
      commit(x, B_KFREE + kr.st);
    }
    // (and x read by wx, since y goes over it once Y is there)
    if (!wait_bar(x, B_M + (i & 1), (i >> 1) & 1) || !wait_bar(x, B_XREAD + s.st, s.ph)) return;
    tc_fence_after();
    if (leader) {
      constexpr uint32_t id = idesc_bf16_f32(128, 64, 1, 0);
      const uint32_t m = m0 + (i & 1) * (K::HEADS * K::M_BYTES >> 4), xs = x0 + s.st * (K::X_BYTES >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // x of head 0 and what stands below it: its other columns (dv = 128), the idle half, or zeros
        const uint32_t xk = xs + k * 128, below = two ? z1 - xk : LBO;
        umma_ss_lo(tm + K::TM_YM, xk | (below << 16), m + k * 2, id, k > 0);
      }
      if (two) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t xk = xs + LBO + k * 128;
          umma_ss_lo(tm + K::TM_YM, z0 | ((xk - z0) << 16), m + (K::M_BYTES >> 4) + k * 2, id, 1);
        }
      }
      commit(x, B_Y + (i & 1));
    }
  }
}

// Decays and steps of every chunk.  delta comes three chunks ahead; the steps
// are made 32 at a time (neighbours in memory: element e of a chunk is head
// e % heads of token e / heads); then a half-warp takes a head, a lane 4 tokens
// (with one head in the tile the upper half-warp repeats the lower one's).  In the
// first pass two warps take every other chunk: it has little else to do, and one
// warp's chain of dependent steps would hold it up.
template <int DK, int DV, bool STATES>
__device__ __forceinline__ void role_decay(const Ctx& x, const TcArgs& t, int which) {
  using K = Cfg<DK, DV, STATES>;
  constexpr int E = 2 * K::HEADS;  // elements per lane, at most
  const SsmArgs& a = t.a;
  const int lane = threadIdx.x & 31, l = lane & 15;
  const int h = x.heads == 2 ? lane >> 4 : 0;
  const bool writes = (lane >> 4) == h;
  Walk<STATES> wf, wp;  // chunks to fetch delta of, and to make the scalars of
  float rate = 0.f, bias = 0.f;
  const bool soft = a.dt_bias != nullptr;
  float total = 0.f;
  const int sh = x.heads - 1, per = 32 >> sh, tok = lane >> sh;  // tokens per 32 elements; this lane's first
  const int64_t step = (int64_t)per * a.H;
  if (which) {
    wf.next(x);
    wp.next(x);
  }
  uint32_t dst = 0;
  const uint32_t raw0 = x.sb + K::SM_RAW + which * K::RAW + lane * 4;
  auto fetch = [&]() {
    wf.next(x);
    const float* p = a.delta + (int64_t)(wf.tok + tok) * a.H + wf.h0 + (lane & sh);
    const int left = wf.end - wf.tok - tok;  // tokens from this lane's first one on (none behind the last chunk)
#pragma unroll
    for (int k = 0; k < E; ++k, p += step) {
      if (k * per < CH) {
        const bool in = k * per < left;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(raw0 + dst + k * 128), "l"(in ? p : a.delta),
                     "r"(in ? 4u : 0u)  // 0: zeros
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (K::DECS == 2) wf.next(x);
    dst = (dst + K::HEADS * CH * 4) & (4 * K::HEADS * CH * 4 - 1);
  };
  const float* raw = reinterpret_cast<const float*>(x.sm + K::SM_RAW + which * K::RAW) + lane;
  float* put_d = reinterpret_cast<float*>(x.sm + K::SM_DEC) + (lane & sh) * K::SC_FLOATS + SC_D + tok;
  float* out = reinterpret_cast<float*>(x.sm + K::SM_DEC) + h * K::SC_FLOATS + 4 * l;
  Ring<K::NX> s;
  if (which) s.next();
  const int mine = (x.nchunks - which + K::DECS - 1) / K::DECS;  // this warp's chunks
#pragma unroll 1
  for (int m = mine > 0 ? -3 : 0; m < mine; ++m) {
    __syncwarp();  // the values before have been read
    fetch();       // three of its chunks ahead
    if (m < 0) continue;
    const int i = m * K::DECS + which;
    if (wp.next(x) || m == 0) {  // a new item
      rate = -decay_rate(a.A_log[wp.h0 + h]) * LOG2E;
      bias = soft ? a.dt_bias[wp.h0 + (lane & sh)] : 0.f;
    }
    const int v = min(wp.end - wp.tok, CH);
    asm volatile("cp.async.wait_group 3;" ::: "memory");
    __syncwarp();
    float d[E];
#pragma unroll
    for (int k = 0; k < E; ++k) d[k] = raw[(m & 3) * K::HEADS * CH + 32 * k];
    if (soft) {  // all of a lane's elements at once: one after the other they would hold the block up
#pragma unroll
      for (int k = 0; k < E; ++k) d[k] = softplus_f32(d[k] + bias);
    }
    if (i >= K::NX) wait_bar(x, (STATES ? B_XFREE : B_YOUT) + s.st, s.ph ^ 1);  // the slot has been read
    const int slot = s.st * (K::SC_SLOT / 4);
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (k * per < CH) put_d[slot + k * per] = tok + k * per < v ? d[k] : 0.f;
    __syncwarp();
    float* o = out + slot;
    const float4 d4 = *reinterpret_cast<const float4*>(o + SC_D);
    const float g0 = max_nan(rate * d4.x, MIN_LOG2), g1 = max_nan(rate * d4.y, MIN_LOG2);
    const float g2 = max_nan(rate * d4.z, MIN_LOG2), g3 = max_nan(rate * d4.w, MIN_LOG2);
    // sums up to each token, and from behind it to the chunk's end (each
    // summed in its own direction: a weight near one has an exponent near zero)
    const float c1 = g0 + g1, c2 = c1 + g2, c3 = c2 + g3, r1 = g3 + g2, r0 = r1 + g1;
    float up = c3, down = r0 + g0;
#pragma unroll
    for (int e = 1; e < 16; e <<= 1) {
      const float u = __shfl_up_sync(0xffffffffu, up, e, 16), w = __shfl_down_sync(0xffffffffu, down, e, 16);
      if (l >= e) up += u;
      if (l + e < 16) down += w;
    }
    const float sum = __shfl_sync(0xffffffffu, up, 15, 16);
    float before = __shfl_up_sync(0xffffffffu, up, 1, 16), behind = __shfl_down_sync(0xffffffffu, down, 1, 16);
    if (l == 0) before = 0.f;
    if (l == 15) behind = 0.f;
    total += sum;
    // the same to the end of the token's sixteen (four lanes)
    const bool last = (l & 3) == 3;
    float near = 0.f, sixteen = 0.f;
    if (!STATES) {
      float part = r0 + g0;
#pragma unroll
      for (int e = 1; e < 4; e <<= 1) {
        const float w = __shfl_down_sync(0xffffffffu, part, e, 4);
        if ((l & 3) + e < 4) part += w;
      }
      near = __shfl_down_sync(0xffffffffu, part, 1, 4);
      if (last) near = 0.f;
      sixteen = __shfl_sync(0xffffffffu, part, 0, 4);
    }
    if (writes) {
      float2 w01 = make_float2(ex2(r0 + behind) * d4.x, ex2(r1 + behind) * d4.y);
      float2 w23 = make_float2(ex2(g3 + behind) * d4.z, ex2(behind) * d4.w);
      uint2* w = reinterpret_cast<uint2*>(o + SC_W - 2 * l);  // o is 4 l words in: two words per lane
#pragma unroll
      for (int k = 0; k < 3; ++k) {  // by truncation: exact in three terms
        w[16 * k] = make_uint2(upper_halves(w01), upper_halves(w23));
        w01 = below_upper(w01);
        w23 = below_upper(w23);
      }
      if (!STATES) {
        *reinterpret_cast<float4*>(o + SC_CUM) = make_float4(before + g0, before + c1, before + c2, before + c3);
        const float w0 = r0 + near, w1 = r1 + near, w2 = g3 + near;
        *reinterpret_cast<float4*>(o + SC_DOWN) = make_float4(w0, w1, w2, last ? sixteen : near);
        *reinterpret_cast<float4*>(o + SC_COL) =
            make_float4(w0 + __log2f(d4.x), w1 + __log2f(d4.y), w2 + __log2f(d4.z), near + __log2f(d4.w));
      }
      if (l == 0) reinterpret_cast<float*>(x.sm + K::SM_MISC + MS_TOTAL)[s.st * 2 + h] = ex2(sum);
    }
    __syncwarp();
    if (lane == 0) arrive(x, B_DEC + s.st);
    if (K::DECS == 2) wp.next(x);
    s.next();
    if (K::DECS == 2) s.next();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (STATES && l == 0 && writes) reinterpret_cast<float*>(x.sm + K::SM_MISC + MS_SUM)[which * 2 + h] = total;
}

// w x as the A operand of U, in four bf16 terms.  With w = w1 + w2 + w3 (bf16
// each), x w1 and x w2 have at most 16 bits, so that bf16 a = x w1 rounded and
// x w1 - a by a fused multiply-add are exact together; the rest, x w3 and what
// x w2 leaves, is 2^-16 of the whole and is rounded to 8 bits of it.  Five packed
// instructions per two elements; a split of the fp32 product takes twelve.
// By halves of the chunk: a half's terms are replaced as soon as its products
// have read them.  Halves [tb0, tb1) of every chunk are this thread's: both, or in
// the first pass, which has eight warps for it, one.
template <int DK, int DV, bool STATES>
__device__ __forceinline__ void role_wx(const Ctx& x, int tb0, int tb1) {
  using K = Cfg<DK, DV, STATES>;
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3, tid = threadIdx.x - 32 * W_WX;
  const uint32_t tl = x.tmem + ((uint32_t)(wq * 32) << 16) + K::TM_WX;
  const int head = DV == 64 && wq >= 2 ? 1 : 0;
  // this lane's row in 16 tokens and its 8-column chunk (tiles: columns 0-7, 8-15, then tokens 8-15)
  const int row = ((lane >> 4) & 1) * 8 + (lane & 7), ch = (wq & 1) * 4 + ((lane >> 3) & 1);
  const uint32_t xl = x.sb + K::SM_X + (wq >> 1) * 8192 + row * 128;
  const uint32_t sw0 = (uint32_t)(ch ^ (row & 7)) << 4, sw1 = (uint32_t)((ch + 2) ^ (row & 7)) << 4;
  Walk<STATES> wv;
  Ring<K::NX> s;
  Ring<K::NB> kr;
#pragma unroll 1
  for (int i = 0; i < x.nchunks; ++i, s.next(), kr.next()) {
    wait_bar(x, B_DEC + s.st, s.ph);
    wait_bar(x, B_XFULL + s.st, s.ph);
    if (!STATES) wv.next(x);
    const int v = wv.end - wv.tok;
    if (!STATES && v < CH) {  // (the first pass's parts are whole chunks)
      // Rows behind the sequence's end hold other data: x and b become zero,
      // so that nothing of them (an infinity among it) reaches a product.
      wait_bar(x, B_KFULL + kr.st, kr.ph);
      constexpr int ATOMS = 2 + DK / 64;
#pragma unroll 1
      for (int e = tid; e < ATOMS * (CH - v) * 8; e += 128) {
        const int atom = e / ((CH - v) * 8), k = e - atom * (CH - v) * 8;
        uint8_t* at = x.sm + (atom < 2 ? K::SM_X + s.st * K::X_BYTES + atom * 8192
                                       : K::SM_K + kr.st * K::K_BYTES + (atom - 2) * 8192);
        *reinterpret_cast<uint4*>(at + v * 128 + k * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      named_sync(GRP_WX, 128);
    }
    const uint32_t* w = reinterpret_cast<const uint32_t*>(x.sm + K::SM_DEC + s.st * K::SC_SLOT) + head * K::SC_FLOATS + SC_W + (lane & 3) + 16 * tb0;
    uint32_t xa = xl + s.st * K::X_BYTES + 4096 * tb0;
#pragma unroll 1
    for (int tb = tb0; tb < tb1; ++tb, w += 16, xa += 4096) {  // 32 tokens
      uint32_t w1[4], w2[4], w3[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w1[k] = w[4 * k];
        w2[k] = w[32 + 4 * k];
        w3[k] = w[64 + 4 * k];
      }
      if (i >= K::NU) wait_bar(x, B_U + 2 * ((i - K::NU) & 1) + tb, ((i - K::NU) >> 1) & 1);
      __syncwarp();
      tc_fence_after();
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {  // 16 columns of the warp's 32
        uint32_t a1[8], e1[8], a2[8], lo[8];
        const uint32_t xe = xa + (half ? sw1 : sw0);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t raw[4];
          ldsm_x4_t(xe + k * 2048, raw);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int o = 4 * k + j, m = 2 * k + (j >> 1);
            a1[o] = mul_bf16x2(raw[j], w1[m]);
            e1[o] = fms_bf16x2(raw[j], w1[m], a1[o]);
            a2[o] = mul_bf16x2(raw[j], w2[m]);
            lo[o] = fma_bf16x2(raw[j], w3[m], fms_bf16x2(raw[j], w2[m], a2[o]));
          }
        }
        const uint32_t ta = tl + ((uint32_t)(half * 16) << 16) + tb * 64 + (K::NU == 2 ? (i & 1) * 128 : 0);
        tmem_st_16x128b_x4(ta, a1);
        tmem_st_16x128b_x4(ta + 16, e1);
        tmem_st_16x128b_x4(ta + 32, a2);
        tmem_st_16x128b_x4(ta + 48, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive(x, B_WX + 2 * (i & 1) + tb);
      if (!STATES && tb) arrive(x, B_XREAD + s.st);  // the outputs may go over x
    }
  }
}

// G to M: decay, step and causal mask, bf16, as the B operand of YM.  Warps q
// and q + 4 have tokens 16 q .. 16 q + 15, a head each (dv = 64) or 32 columns
// each; what lies above the diagonal is zero.
template <int DK, int DV>
__device__ __forceinline__ void role_scores(const Ctx& x) {
  using K = Cfg<DK, DV, false>;
  const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3, second = (threadIdx.x - 32 * W_SC) >> 7;
  const uint32_t tl = x.tmem + ((uint32_t)(q * 32) << 16) + K::TM_G;
  // this thread's rows r0, r0 + 8 and columns cl, cl + 1 (+ 8); its row address in a
  // 16x16 tile (four 8x8 matrices: rows 0-7, rows 8-15, then columns 8-15)
  const int r0 = 16 * q + (lane >> 2), cl = 2 * (lane & 3);
  const int srow = 16 * q + ((lane >> 3) & 1) * 8 + (lane & 7), sch = (lane >> 4) & 1;
  const bool by_head = x.heads == 2;
  const int sc_off = by_head ? second * K::SC_FLOATS : 0, j_first = by_head ? 0 : second, j_step = by_head ? 1 : 2;
  const uint32_t ml = x.sb + K::SM_M + srow * 128 + (by_head ? second * K::M_BYTES : 0);
  // bits of the pairs (row r0 + 8 (k % 2), columns 8 (k / 2) + cl and the next) that
  // lie on or below the diagonal, in the 32 columns that it crosses
  uint32_t keep[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int below = r0 + 8 * (k & 1) - (32 * (q >> 1) + 8 * (k >> 1) + cl);
    keep[k] = below > 0 ? 0xffffffffu : (below == 0 ? 0xffffu : 0u);
  }
  Ring<K::NX> s;
#pragma unroll 1
  for (int i = 0; i < x.nchunks; ++i, s.next()) {
    if (i >= 2) wait_bar(x, B_Y + (i & 1), ((i >> 1) - 1) & 1);  // M's buffer
    wait_bar(x, B_G, i & 1);                        // (the scalars are there before G)
    __syncwarp();
    tc_fence_after();
    const float* sc = reinterpret_cast<const float*>(x.sm + K::SM_DEC + s.st * K::SC_SLOT) + sc_off;
    const uint32_t mb = ml + (i & 1) * K::HEADS * K::M_BYTES;
    // sums from the rows to the end of their sixteen; its total, and those of the sixteens 1 and 2 before it
    const float down0 = sc[SC_DOWN + r0], down1 = lane < 28 ? sc[SC_DOWN + r0 + 8] : 0.f;
    const float all = sc[SC_DOWN + 16 * q + 15], mid2 = q == 3 ? sc[SC_DOWN + 47] : 0.f, mid1 = q >= 2 ? sc[SC_DOWN + 31] + mid2 : 0.f;
#pragma unroll 1
    for (int j = j_first; j <= q >> 1; j += j_step) {  // 32 columns at a time, so that their chains overlap
      float g[16];
      tmem_ld_16x256b_x4_wait(tl + 32 * j, g);
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // columns 32 j + 8 k + cl, and the next
        // between the column's sixteen (2 j + k / 2) and the rows' end (the rows' own, or one cut out below: nothing)
        const float from = 2 * j + (k >> 1) >= q ? 0.f : all + (j > 0 ? 0.f : k < 2 ? mid1 : mid2);
        const float2 e = *reinterpret_cast<const float2*>(sc + SC_COL + 32 * j + 8 * k + cl);
        const float2 a0 = __fadd2_rn(make_float2(from - down0, from - down0), e);
        const float2 a1 = __fadd2_rn(make_float2(from - down1, from - down1), e);
        const float2 m0 = __fmul2_rn(make_float2(g[4 * k], g[4 * k + 1]), make_float2(ex2(a0.x), ex2(a0.y)));
        const float2 m1 = __fmul2_rn(make_float2(g[4 * k + 2], g[4 * k + 3]), make_float2(ex2(a1.x), ex2(a1.y)));
        g[4 * k] = m0.x;
        g[4 * k + 1] = m0.y;
        g[4 * k + 2] = m1.x;
        g[4 * k + 3] = m1.y;
      }
      uint32_t pk[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) pk[k] = pack_bf16x2(g[2 * k], g[2 * k + 1]);
      if (j == q >> 1) {  // cut out, not multiplied: what stands above the diagonal may be anything
#pragma unroll
        for (int k = 0; k < 8; ++k) pk[k] &= keep[k];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t t4[4] = {pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]};
        stsm_x4(mb + (((4 * j + 2 * k + sch) ^ (srow & 7)) << 4), t4);
      }
    }
    tc_fence_before();
    fence_proxy_async_smem();
    arrive(x, B_M + (i & 1));  // G may be overwritten, M is there
  }
}

// S in registers: thread (lane p, a quarter of the key channels); and the
// outputs.  Sixteen warps, so that U, YI and YM are free again soon: the next
// chunk's products wait for them.
template <int DK, int DV, bool STATES>
__device__ __forceinline__ void role_state(const Ctx& x, const TcArgs& t) {
  using K = Cfg<DK, DV, STATES>;
  constexpr int NC = DK * 4 / ST_WARPS;
  const SsmArgs& a = t.a;
  const int w = (threadIdx.x >> 5) - W_ST, lane = threadIdx.x & 31, p = (w & 3) * 32 + lane, n0 = (w >> 2) * NC;
  const uint32_t tl = x.tmem + ((uint32_t)((w & 3) * 32) << 16);
  const int hl = DV == 64 ? p / 64 : 0;
  const bool live = hl < x.heads;
  const int head = live ? hl : 0, hl_sc = head * K::SC_FLOATS;
  const int64_t at0 = (p & (DV - 1)) + (int64_t)n0 * DV, seq = (int64_t)a.H * DK * DV;
  float S[NC];
  // at: this thread's elements in a sequence's states
  auto start = [&](int sequence, int slot0, int flags, int64_t at) {  // the state before an item
    const int before = flags >> 3;
#pragma unroll
    for (int n = 0; n < NC; ++n) S[n] = 0.f;
    float* slots = t.p.state + at;  // slot s of this thread's elements at slots + s * seq
    const int64_t s0 = slot0;
    const bool cut = !STATES && (flags & SPLIT);  // the first pass left it then
    if (live && (cut ? a.init || before > 0 : a.init && (!STATES || before == 0))) {
      const float* o = cut ? slots + (s0 + before) * seq : a.init + sequence * seq + at;
#pragma unroll
      for (int n = 0; n < NC; ++n) S[n] = o[(int64_t)n * DV];
      if (STATES) {  // kept for the second pass
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          slots[s0 * seq + (int64_t)n * DV] = S[n];
          S[n] = 0.f;
        }
      }
    }
  };
  auto finish = [&](int sequence, int slot0, int flags, int64_t at) {  // the state after an item
    float* o = nullptr;
    if (STATES)
      o = t.p.state + at + ((int64_t)slot0 + (flags >> 3) + 1) * seq;
    else if (a.fin && (flags & LAST))
      o = a.fin + sequence * seq + at;
    if (live && o) {
#pragma unroll
      for (int n = 0; n < NC; ++n) o[(int64_t)n * DV] = S[n];
    }
  };
  const float* totals = reinterpret_cast<const float*>(x.sm + K::SM_MISC + MS_TOTAL) + head;
  // outputs: this warp has tokens 16 part .. 16 part + 15 of value columns 32 q .. 32 q + 31
  const int q = w & 3, part = w >> 2;
  float skip = 0.f, skip_now = 0.f;  // D of the chunk before, and of this one
  const int row = 16 * part + ((lane >> 4) & 1) * 8 + (lane & 7), ch = (q & 1) * 4 + ((lane >> 3) & 1);
  const uint32_t xl = x.sb + K::SM_X + (q >> 1) * 8192 + row * 128;
  const uint32_t sw0 = (uint32_t)(ch ^ (row & 7)) << 4, sw1 = (uint32_t)((ch + 2) ^ (row & 7)) << 4;
  Ring<K::NX> s, so;  // stages of the chunk, and of the one before it
  int turn = -1, left = 0;  // this item's turn, its chunks left
#pragma unroll 1
  for (int i = 0;; ++i) {
#pragma unroll 1
    for (int begin = 0; left == 0 && turn < x.items; begin ^= 1) {  // the end of an item, and the next one's start
      if (begin && ++turn == x.items) break;
      if (turn < 0) continue;
      const int4 d = x.item[turn];
      const int2 f = reinterpret_cast<const int2*>(x.item + MAX_ITEMS)[turn];
      if (!(f.y & VALID)) continue;
      const int hh = d.z + head;
      const int64_t at = (int64_t)hh * DK * DV + at0;
      if (begin) {
        left = chunks_of(d.y - d.x);
        if (!STATES && a.D) skip_now = a.D[hh];
        start(d.w, f.x, f.y, at);
      } else {
        finish(d.w, f.x, f.y, at);
      }
    }
    const bool more = turn < x.items;  // whether there is a chunk i
    if (!STATES && more) {  // S before the chunk as bf16 pairs: the A operand of YI
      if (i > 0) wait_bar(x, B_SFREE, (i - 1) & 1);
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < NC / 16; ++k) {
        uint32_t pk[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) pk[j] = pack_bf16x2(S[16 * k + 2 * j], S[16 * k + 2 * j + 1]);
        tmem_st8(tl + K::TM_S + (n0 >> 1) + 8 * k, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive(x, B_SRDY);
    }
    if (!STATES && i > 0) {  // y of the chunk before: e^{G_t} YI + YM + D x, over x's own tile
      const int o = i - 1;
      wait_bar(x, B_Y + (o & 1), (o >> 1) & 1);
      __syncwarp();
      tc_fence_after();
      const float* ec = reinterpret_cast<const float*>(x.sm + K::SM_DEC + so.st * K::SC_SLOT) + hl_sc + SC_CUM + 16 * part + 2 * (lane & 3);
      const uint32_t xa = xl + so.st * K::X_BYTES;
      const float2 ca = *reinterpret_cast<const float2*>(ec), cb = *reinterpret_cast<const float2*>(ec + 8);
      const float2 f[2] = {make_float2(ex2(ca.x), ex2(ca.y)), make_float2(ex2(cb.x), ex2(cb.y))};
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // 16 columns of the warp's 32
        float yi[8], ym[8];
        uint32_t raw[4], pk[4];
        const uint32_t te = tl + K::TM_YI + 16 * part + ((uint32_t)(half * 16) << 16), xe = xa + (half ? sw1 : sw0);
        ldsm_x4_t(xe, raw);
        tmem_ld_16x256b_x2x2_wait(te, te + (K::TM_YM - K::TM_YI), yi, ym);
        if (half) {
          tc_fence_before();
          arrive(x, B_YFREE);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 y = __ffma2_rn(f[j >> 1], make_float2(yi[2 * j], yi[2 * j + 1]), make_float2(ym[2 * j], ym[2 * j + 1]));
          y = __ffma2_rn(make_float2(skip, skip), bf16x2_f32(raw[j]), y);
          pk[j] = pack_bf16x2(y.x, y.y);
        }
        stsm_x4_t(xe, pk);
      }
      fence_proxy_async_smem();
      arrive(x, B_YOUT + so.st);  // (and the stage's scalars have been read)
      so.next();
    }
    if (!more) break;
    skip = skip_now;
    --left;
    {  // S after the chunk
      wait_bar(x, B_U + 2 * (i & 1) + 1, (i >> 1) & 1);  // (made from this chunk's scalars)
      __syncwarp();
      tc_fence_after();
      const float dec = totals[s.st * 2];
      const float2 dec2 = make_float2(dec, dec);
#pragma unroll
      for (int k = 0; k < NC / 16; ++k) {
        float u[16];
        tmem_ld16(tl + K::TM_U + (K::NU == 2 ? (i & 1) * DK : 0) + n0 + 16 * k, u);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 v = __ffma2_rn(make_float2(S[16 * k + j], S[16 * k + j + 1]), dec2, make_float2(u[j], u[j + 1]));
          S[16 * k + j] = v.x;
          S[16 * k + j + 1] = v.y;
        }
      }
      tc_fence_before();
      arrive(x, B_UFREE + (i & 1));
      if (STATES) {
        __syncwarp();
        if (lane == 0) arrive(x, B_XFREE + s.st);
      }
      s.next();
    }
  }
}

template <int DK, int DV, bool STATES>
__global__ void __launch_bounds__(NTHR, 1)
    ssm_tc_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tb,
                  const __grid_constant__ CUtensorMap tc, const __grid_constant__ CUtensorMap to,
                  const __grid_constant__ TcArgs t) {
  using K = Cfg<DK, DV, STATES>;
  extern __shared__ uint8_t smem_raw[];
  Ctx x;
  if (STATES) start_next();
  Piece piece;
  if (STATES && !find_piece<true>(t.p, t.a.T, blockIdx.x / t.tiles, piece)) return;
  x.sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  x.sb = smem_u32(x.sm);
  x.bars = x.sb + K::SM_MISC;
  x.heads = t.hpt;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  uint8_t* misc = x.sm + K::SM_MISC;
  if (tid < NUM_BARS) {
    int n = 1;
    if (tid >= B_XFREE && tid < B_XFREE + MAXST) n = ST_WARPS + 1;  // (states only)
    if (!STATES && ((tid >= B_KFREE && tid < B_KFREE + MAXST) || tid == B_DRAIN)) n = 2;
    if ((tid >= B_WX && tid < B_WX + 4) || (tid >= B_XREAD && tid < B_XREAD + MAXST)) n = N_WX;
    if (tid == B_UFREE || tid == B_UFREE + 1 || tid == B_SRDY || tid == B_YFREE ||
        (tid >= B_YOUT && tid < B_YOUT + MAXST))
      n = N_ST;
    if (tid == B_M || tid == B_M + 1) n = N_SC;
    mbar_init(reinterpret_cast<uint64_t*>(misc) + tid, n);
    fence_mbar_init();
  }
  if (tid == 0) {
    *reinterpret_cast<volatile int*>(misc + MS_ABORT) = 0;
    prefetch_tmap(&tx);
    prefetch_tmap(&tb);
    prefetch_tmap(&tc);
    prefetch_tmap(&to);
  }
  int4* item = reinterpret_cast<int4*>(misc + MS_ITEMS);
  x.item = item;
  x.items = STATES ? 1 : t.per_block;
  if (tid >= 64 && tid < 64 + x.items) {
    const int index = item_index(tid - 64);
    int4 d = make_int4(0, 0, 0, 0);
    int2 s = make_int2(0, 0);
    if (STATES || (index < t.items && find_piece<STATES>(t.p, t.a.T, index / t.tiles, piece))) {
      d = make_int4((int)piece.start, (int)piece.end, index % t.tiles * t.hpt, piece.n);
      s = make_int2(piece.slot0, piece.before * 8 + VALID + (piece.last ? LAST : 0) + (piece.split ? SPLIT : 0));
    }
    item[tid - 64] = d;
    reinterpret_cast<int2*>(item + MAX_ITEMS)[tid - 64] = s;
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
    tmem_alloc(reinterpret_cast<uint32_t*>(misc + MS_TMEM), K::TM_COLS);
    tmem_relinquish();
  }
  if (!STATES) await_last();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  x.nchunks = 0;
  for (int k = 0; k < x.items; ++k) {
    const int4 d = x.item[k];
    x.nchunks += chunks_of(d.y - d.x);
  }
  x.tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(misc + MS_TMEM), 0);

  if (warp >= W_MOVE) {
    if (warp == W_MOVE) {
      role_move<DK, DV, STATES>(x, t, &tx, &tb, &tc, &to, elect_one());
    } else if (warp == W_DEC) {
      role_decay<DK, DV, STATES>(x, t, 0);
    } else if (STATES && warp == W_MMY) {
      role_decay<DK, DV, STATES>(x, t, STATES);
    } else {
      const bool leader = elect_one();
      if (warp == W_MMU) role_mma_u<DK, DV, STATES>(x, leader);
      else if (!STATES) role_mma_y<DK, DV>(x, leader);
      __syncwarp();
      if (leader) commit(x, B_DRAIN);  // every product has ended before TMEM is released
      land(x.bars + 8 * B_DRAIN, 0);
    }
  } else if (warp >= W_ST) {
    role_state<DK, DV, STATES>(x, t);
  } else if (warp >= W_SC) {
    if (!STATES) role_scores<DK, DV>(x);
    else if (warp < W_SC + 4) role_wx<DK, DV, STATES>(x, 1, 2);
  } else {
    role_wx<DK, DV, STATES>(x, 0, STATES ? 1 : 2);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (STATES && tid < x.heads) {
    const float* sum = reinterpret_cast<const float*>(misc + MS_SUM) + tid;
    t.p.decay[(int64_t)(piece.slot0 + piece.before) * t.a.H + blockIdx.x % t.tiles * t.hpt + tid] = sum[0] + sum[2];
  }
  if (tid == 0 && *reinterpret_cast<volatile int*>(misc + MS_ABORT) != 0) record_error(t.a.status, KDA_ERR_TIMEOUT, 1);
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

constexpr int PLACES = 148;  // blocks at a time, one per SM

// Heads per tile.
int heads_per_tile(int H, int G, int dv) { return dv == 64 && (H / G) % 2 == 0 ? 2 : 1; }

PiecePlan plan(int N, int64_t T, int H, int G, int dk, int dv, bool packed) {
  // one block per SM; a chunk of the first pass takes about 0.4 of one of the second
  return plan_pieces(N, T, H / heads_per_tile(H, G, dv), PLACES, 0.4, 4, H, dk, dv, packed);
}

template <int DK, int DV, bool STATES>
cudaError_t ready() {
  return cudaFuncSetAttribute(ssm_tc_kernel<DK, DV, STATES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)Cfg<DK, DV, STATES>::BYTES);
}

template <int DK, int DV>
cudaError_t launch(const TcArgs& t, const PiecePlan& p, cudaStream_t s) {
  const SsmArgs& a = t.a;
  const int64_t rows = a.cu ? a.T : (int64_t)a.N * a.T;
  CUtensorMap tx, tb, tc, to;
  if (!make_map(&tx, a.x, (int64_t)a.H * DV, a.ldx, rows) || !make_map(&tb, a.b, (int64_t)a.G * DK, a.ldb, rows) ||
      !make_map(&tc, a.c, (int64_t)a.G * DK, a.ldc, rows) ||
      !make_map(&to, a.out, (int64_t)a.H * DV, (int64_t)a.H * DV, rows))
    return cudaErrorInvalidValue;
  cudaError_t e;
  if (p.first_pass) {
    if ((e = ready<DK, DV, true>()) != cudaSuccess) return e;
    ssm_tc_kernel<DK, DV, true><<<(unsigned)(p.first_pass * t.tiles), NTHR, Cfg<DK, DV, true>::BYTES, s>>>(tx, tb, tc, to, t);
    if ((e = compose_pieces(p, a, t.p, s)) != cudaSuccess) return e;
  }
  if ((e = ready<DK, DV, false>()) != cudaSuccess) return e;
  constexpr int bytes = Cfg<DK, DV, false>::BYTES;
  if (p.first_pass) return launch_overlapped(ssm_tc_kernel<DK, DV, false>, t.blocks, NTHR, bytes, s, tx, tb, tc, to, t);
  ssm_tc_kernel<DK, DV, false><<<(unsigned)t.blocks, NTHR, bytes, s>>>(tx, tb, tc, to, t);
  return cudaGetLastError();
}

}  // namespace

bool ssm_tc_supported(int dk, int dv, bool bf16) { return bf16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }

size_t ssm_tc_workspace(int N, int64_t T, int H, int G, int dk, int dv, bool packed) {
  return plan(N, T, H, G, dk, dv, packed).total;
}

cudaError_t launch_ssm_fwd_tc(const SsmArgs& a, void* workspace, cudaStream_t s, uint64_t wait_ns, int stop_at) {
  const PiecePlan p = plan(a.N, a.T, a.H, a.G, a.dk, a.dv, a.cu != nullptr);
  TcArgs t;
  t.a = a;
  t.wait_ns = (uint32_t)std::min<uint64_t>(wait_ns, SSM_WAIT_NS);
  t.stop_at = stop_at;
  t.hpt = heads_per_tile(a.H, a.G, a.dv);
  t.tiles = a.H / t.hpt;
  t.items = (int)(p.pieces * t.tiles);
  // as many blocks as the device holds, or a multiple of that where they would have
  // too many items; all with the same number of items where that is known here
  t.blocks = std::min(t.items, (t.items + PLACES * MAX_ITEMS - 1) / (PLACES * MAX_ITEMS) * PLACES);
  t.per_block = (t.items + t.blocks - 1) / t.blocks;
  if (!a.cu) t.blocks = (t.items + t.per_block - 1) / t.per_block;
  cudaError_t e = prepare_pieces(p, a, workspace, &t.p, s);
  if (e != cudaSuccess) return e;
  if (a.dk == 128) return a.dv == 128 ? launch<128, 128>(t, p, s) : launch<128, 64>(t, p, s);
  return a.dv == 128 ? launch<64, 128>(t, p, s) : launch<64, 64>(t, p, s);
}

}  // namespace kda
