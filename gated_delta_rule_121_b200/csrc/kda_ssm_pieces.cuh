// Pieces of long sequences in the selective scan.  The state after a piece is
// e^{G} S_in + S_own, with G the piece's total log decay and S_own its state from
// zero, so a sequence can be cut into pieces that run in parallel: a first pass
// (states only, of every piece but a sequence's last) gives S_own and G, and a
// block of the second pass composes its incoming state from the pieces before
// it.  The first pass also keeps the initial state, since the last piece of the
// second may write the final state over it while others still start.
#pragma once
#include "kda_layer.cuh"

namespace kda {

constexpr int PIECE_CHUNK = 64;  // pieces are whole chunks of this many tokens

// Tokens [start, end) of sequence n, its r-th piece of `pieces`.  A sequence of
// several pieces has `pieces` slots from slot0 on, for states (the initial one,
// then those of all pieces but the last) and for total decays.
struct Piece {
  int n, r, pieces, slot0;
  int64_t start, end;
};
struct PieceEntry {  // table entry of a packed batch; n < 0: none
  int n, r, pieces, slot0, start, end, pad[2];
};
struct PieceArgs {
  int64_t len;              // tokens per piece
  int per_seq;              // pieces per sequence of a batch of equal lengths
  const PieceEntry* table;  // packed batches
  float* state;             // [slots][H][dk][dv]
  float* decay;             // [slots][H]: log2 of a piece's total decay
};

__device__ __forceinline__ bool find_piece(const PieceArgs& a, int64_t T, int index, Piece& p) {
  if (a.table) {
    const PieceEntry e = a.table[index];
    if (e.n < 0) return false;
    p.n = e.n; p.r = e.r; p.pieces = e.pieces; p.slot0 = e.slot0; p.start = e.start; p.end = e.end;
    return true;
  }
  p.n = index / a.per_seq;
  p.slot0 = p.n * a.per_seq;
  p.r = index - p.n * a.per_seq;
  p.pieces = a.per_seq;
  const int64_t s0 = (int64_t)p.n * T;
  p.start = s0 + p.r * a.len;
  p.end = min(p.start + a.len, s0 + T);
  return true;
}

struct PiecePlan {
  int per_seq;
  int64_t len, pieces, slots;         // pieces, slots: upper bounds for packed batches
  bool split;                         // whether there is a first pass
  size_t table, decay, state, total;  // workspace offsets, the status word first
};
// `blocks` blocks per piece; `places` blocks at a time on the device; `first` the
// cost of a chunk of the first pass against one of the second; pieces of at
// least `least` chunks.
PiecePlan plan_pieces(int N, int64_t T, int blocks, int places, double first, int least, int H, int dk, int dv, bool packed);
// The pieces' part of a launch's arguments, and for packed batches their table.
cudaError_t prepare_pieces(const PiecePlan& p, const SsmArgs& a, void* workspace, PieceArgs* out, cudaStream_t s);

}  // namespace kda
