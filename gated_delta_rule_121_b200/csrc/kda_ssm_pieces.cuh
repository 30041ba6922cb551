// Pieces of long sequences in the selective scan.  The state after a piece is
// e^{G} S_in + S_own, with G the piece's total log decay and S_own its state from
// zero, so a sequence can be cut into pieces that run in parallel: a first pass
// (states only, up to the last piece's start) gives S_own and G of parts of
// pieces; a running composition turns them into the state at each part's end; the
// second pass starts a piece from it.  The first pass also keeps the initial state,
// since the last piece of the second may write the final state over it while others
// still start.
#pragma once
#include "kda_layer.cuh"

namespace kda {

constexpr int PIECE_CHUNK = 64;  // pieces are whole chunks of this many tokens

// Tokens [start, end) of sequence n: a piece, or in the first pass a part of one.
// A sequence of several pieces has slots from slot0 on, for states (the initial
// one, then those at the parts' ends) and for the parts' total decays; `before` counts the parts
// before this one.
struct Piece {
  int n, slot0, before;
  bool first, last, split;  // of its sequence; whether the sequence has several
  int64_t start, end;
};
struct PieceEntry {  // table entry of a packed batch (parts are whole pieces there); n < 0: none
  int n, r, pieces, slot0, start, end, pad[2];
};
struct PieceArgs {
  int64_t len, part;        // tokens per piece, and per part
  int per_seq, parts;       // of a batch of equal lengths: pieces per sequence, parts per piece
  const PieceEntry* table;  // packed batches
  float* state;             // [slots][H][dk][dv]
  float* decay;             // [slots][H]: log2 of a part's total decay
};

template <bool FIRST_PASS>
__device__ __forceinline__ bool find_piece(const PieceArgs& a, int64_t T, int index, Piece& p) {
  if (a.table) {
    const PieceEntry e = a.table[index];
    if (e.n < 0 || (FIRST_PASS && e.r == e.pieces - 1)) return false;  // (nothing follows a last piece)
    p.n = e.n; p.slot0 = e.slot0; p.before = e.r; p.start = e.start; p.end = e.end;
    p.first = e.r == 0;
    p.last = e.r == e.pieces - 1;
    p.split = e.pieces > 1;
    return true;
  }
  const int per = FIRST_PASS ? (a.per_seq - 1) * a.parts : a.per_seq;
  p.n = index / per;
  const int r = index - p.n * per;
  p.slot0 = p.n * a.per_seq * a.parts;
  p.before = FIRST_PASS ? r : r * a.parts;
  p.first = r == 0;
  p.last = !FIRST_PASS && r == per - 1;
  p.split = a.per_seq > 1;
  const int64_t s0 = (int64_t)p.n * T;
  p.start = s0 + r * (FIRST_PASS ? a.part : a.len);
  p.end = FIRST_PASS ? p.start + a.part : min(p.start + a.len, s0 + T);
  return true;
}

struct PiecePlan {
  int per_seq, parts;
  int64_t len, part, slots;           // tokens per piece and part; slots and the blocks: upper bounds for packed batches
  int64_t pieces, first_pass;         // pieces in all, and parts of the first pass (0: there is none)
  size_t table, decay, state, total;  // workspace offsets, the status word first; they grow with N and T
};
// `blocks` blocks per piece; `places` blocks at a time on the device; `first` the
// cost of a chunk of the first pass against one of the second; parts of at
// least `least` chunks.
PiecePlan plan_pieces(int N, int64_t T, int blocks, int places, double first, int least, int H, int dk, int dv, bool packed);
// The pieces' part of a launch's arguments, and for packed batches their table.
cudaError_t prepare_pieces(const PiecePlan& p, const SsmArgs& a, void* workspace, PieceArgs* out, cudaStream_t s);
// On the tensor-core path the launches from the first pass on overlap: a kernel lets
// the next one's blocks start as soon as all of its own have (start_next), and that one
// waits for the kernel before it to end, with all its writes, before it touches what
// they share (await_last).  A launch, a block's barriers and TMEM are ready by then.
// (The CUDA-core path's passes neither let a kernel start early nor start early.)
__device__ __forceinline__ void start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void await_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), unsigned blocks, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Between the passes: the parts' own states become the states at their ends.
cudaError_t compose_pieces(const PiecePlan& p, const SsmArgs& a, const PieceArgs& pa, cudaStream_t s);

}  // namespace kda
