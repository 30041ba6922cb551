// Cutting sequences into pieces (kda_ssm_pieces.cuh): the host's plan, and the
// table of a packed batch, whose lengths are on the device.
#include "kda_ssm_pieces.cuh"

#include <algorithm>

namespace kda {
namespace {

constexpr int MAX_PARTS = 64;   // of a sequence of known length
// And of all sequences of a batch, in numbers of blocks that the device holds at a
// time: it bounds the workspace (155 MB for the largest states) for any length, so
// that the bound grows with the length.  By the cost model below no batch loses more
// than 2.5 % by it, and only some of more than 24K tokens a sequence do.
constexpr int MAX_WAVES = 16;

// The pieces of a packed batch (one block): first the ones that others follow,
// which are whole, then the last ones by length, the longest first, so that blocks
// that take every so-manyth piece get about the same work; entries behind the last
// one are marked unused.  Pieces of one length class, and the sequences' slots, come
// in any order: no result depends on it.  Offsets that are no offsets may claim
// more than there is, and what lies beyond is left out.
// Pieces are twice as long where one sequence holds more than half of the tokens: it
// fills the device with them then.
constexpr int CLASSES = 64;  // of lengths
__global__ void __launch_bounds__(1024) ssm_piece_table_kernel(Seqs q, int64_t len, int capacity, int slots,
                                                               PieceEntry* table) {
  __shared__ int place[CLASSES + 1];  // sizes of the classes, then the next free places; 0: pieces that others follow
  __shared__ int used, total, longs;  // slots, pieces; sequences of more than half of the tokens
  const int tid = threadIdx.x;
  if (tid <= CLASSES) place[tid] = 0;
  if (tid == 0) used = longs = 0;
  __syncthreads();
  for (int n = tid; n < q.N; n += 1024)
    if (2 * (q.end(n) - q.begin(n)) > q.T) atomicAdd(&longs, 1);
  __syncthreads();
  if (longs) len *= 2;
  auto pieces = [&](int n, int64_t& s, int64_t& e, int& cls) {  // and the class of the last one
    s = q.begin(n);
    e = max(q.end(n), s);
    const int cnt = (int)max((e - s + len - 1) / len, (int64_t)1);
    cls = CLASSES - (int)((e - s - (cnt - 1) * len) * (CLASSES - 1) / len);
    return cnt;
  };
  int64_t s, e;
  int cls;
  for (int n = tid; n < q.N; n += 1024) {
    const int cnt = pieces(n, s, e, cls);
    if (cnt > 1) atomicAdd(&place[0], cnt - 1);
    atomicAdd(&place[cls], 1);
  }
  __syncthreads();
  if (tid == 0) {
    int at = 0;
    for (int c = 0; c <= CLASSES; ++c) {
      const int size = place[c];
      place[c] = at;
      at += size;
    }
    total = at;
  }
  __syncthreads();
  for (int n = tid; n < q.N; n += 1024) {
    const int cnt = pieces(n, s, e, cls);
    const int slot0 = cnt > 1 ? atomicAdd(&used, cnt) : 0, first = cnt > 1 ? atomicAdd(&place[0], cnt - 1) : 0;
    const int last = atomicAdd(&place[cls], 1), own = cnt > 1 && slot0 + cnt > slots ? -1 : n;
    for (int r = 0; r < cnt; ++r) {
      const int64_t a = s + r * len;
      const int i = r < cnt - 1 ? first + r : last;
      if (i < capacity) table[i] = {own, r, cnt, slot0, (int)a, (int)min(a + len, e), {0, 0}};
    }
  }
  for (int i = total + tid; i < capacity; i += 1024) table[i].n = -1;
}

// One sequence's states after each of its parts, in place: S_r = e^{G_r} S_{r-1} + own
// state of part r.  (Each piece adding up all parts before it read the states again
// and again: 32 us of a block's 88 for 37 pieces.)  A thread has four elements and
// loads four parts at once; bound by the latency of that chain, ~4 us for 37 parts.
constexpr int CT = 128;
__global__ void __launch_bounds__(CT) ssm_compose_kernel(PieceArgs p, bool init, int H, int size, int blocks) {
  start_next();
  await_last();
  const int entry = blockIdx.x / blocks, elem = ((blockIdx.x - entry * blocks) * CT + threadIdx.x) * 4;
  int64_t slot0 = (int64_t)entry * p.per_seq * p.parts;
  int parts = (p.per_seq - 1) * p.parts;
  if (p.table) {
    const PieceEntry e = p.table[entry];
    if (e.n < 0 || e.r > 0) return;
    slot0 = e.slot0;
    parts = e.pieces - 1;
  }
  const int seq = H * size;
  if (elem >= seq) return;
  float4* o = reinterpret_cast<float4*>(p.state + slot0 * seq + elem);
  const float* decay = p.decay + slot0 * H + elem / size;
  const int64_t step = seq / 4;
  float4 S = init ? *o : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int r = 0; r < parts; r += 4) {
    float4 own[4];
    float dec[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (r + k >= parts) break;
      own[k] = o[(r + k + 1) * step];
      dec[k] = exp2f(decay[(int64_t)(r + k) * H]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (r + k >= parts) break;
      S.x = fmaf(S.x, dec[k], own[k].x);
      S.y = fmaf(S.y, dec[k], own[k].y);
      S.z = fmaf(S.z, dec[k], own[k].z);
      S.w = fmaf(S.w, dec[k], own[k].w);
      o[(r + k + 1) * step] = S;
    }
  }
}

}  // namespace

PiecePlan plan_pieces(int N, int64_t T, int blocks, int places, double first, int least, int H, int dk, int dv,
                      bool packed) {
  PiecePlan p;
  int64_t room;  // slots and pieces beyond the sequences that any shorter or smaller batch may need
  const int64_t chunks = (T + PIECE_CHUNK - 1) / PIECE_CHUNK;  // of a sequence, or of the packed total
  if (!packed) {
    // Pieces per sequence and parts per piece with the fewest chunk times in the
    // two passes, in waves of blocks; 3 chunk times for a block's start and 6 for
    // what comes between the passes.  (Tensor cores, in the second pass's chunks of 2
    // us: a block's start is 6 to 7 us, the composition 4 to 12 for 4 to 32 parts, a chunk
    // of the first pass 0.95.  CUDA cores, fp32, 64 x 32: a chunk takes 14 us, one of the
    // first pass 8; starts and composition are the smaller there, and cuts a little
    // coarser than they could be.)
    const int64_t chains = (int64_t)N * blocks, shortest = chunks / least;
    room = shortest < 2 ? 0 : std::min(N * std::min<int64_t>(MAX_PARTS, shortest), (int64_t)MAX_WAVES * places / blocks);
    auto waves = [&](int64_t n) { return (double)((n + places - 1) / places); };
    int64_t part = chunks > 0 ? chunks : 1;
    int parts = 1;
    double cost = waves(chains) * chunks;
    for (int r = 2; r <= MAX_PARTS; ++r)
      for (int q = 1; q <= 4 && r * q <= MAX_PARTS && chunks / (r * q) >= least && (int64_t)N * r * q <= room; ++q) {
        const int64_t len = (chunks + r * q - 1) / (r * q);
        const double c = waves(chains * r) * (len * q + 3) + first * waves(chains * (r - 1) * q) * (len + 3) + 6;
        if (c < cost) {
          cost = c;
          part = len;
          parts = q;
        }
      }
    p.parts = parts;
    p.part = part * PIECE_CHUNK;
    p.len = p.part * parts;
    p.per_seq = (int)((chunks + part * parts - 1) / (part * parts));
    if (p.per_seq < 1) p.per_seq = 1;
    p.pieces = (int64_t)N * p.per_seq;
    p.first_pass = (int64_t)N * (p.per_seq - 1) * parts;
    p.slots = p.first_pass > 0 ? p.pieces * parts : 0;
  } else {
    // The lengths are on the device: pieces for twice the device's places in
    // all, so that a long sequence does not hold the batch up.
    int64_t len = (chunks * blocks + 2 * places - 1) / (2 * places);
    if (len < least) len = least;
    p.per_seq = p.parts = 1;
    p.len = p.part = len * PIECE_CHUNK;
    p.pieces = N + T / p.len;
    p.first_pass = T > p.len ? T / p.len : 0;  // the pieces that others follow are whole
    // a sequence of L > len tokens has at most L / len + 1 < 2 L / len pieces
    p.slots = p.first_pass ? 2 * T / p.len : 0;
    room = std::min<int64_t>(2 * T / (least * PIECE_CHUNK), 4 * (int64_t)places / blocks);
  }
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  size_t off = 256;  // the status word
  p.table = off;
  if (packed) off += up((size_t)(N + room / 2 + 1) * sizeof(PieceEntry));
  p.decay = off;
  off += up((size_t)room * H * sizeof(float));
  p.state = off;
  off += (size_t)room * H * dk * dv * sizeof(float);
  p.total = off;
  return p;
}

cudaError_t prepare_pieces(const PiecePlan& p, const SsmArgs& a, void* workspace, PieceArgs* out, cudaStream_t s) {
  char* ws = static_cast<char*>(workspace);
  out->len = p.len;
  out->part = p.part;
  out->per_seq = p.per_seq;
  out->parts = p.parts;
  out->table = nullptr;
  out->decay = reinterpret_cast<float*>(ws + p.decay);
  out->state = reinterpret_cast<float*>(ws + p.state);
  if (!a.cu) return cudaSuccess;
  PieceEntry* table = reinterpret_cast<PieceEntry*>(ws + p.table);
  out->table = table;
  ssm_piece_table_kernel<<<1, 1024, 0, s>>>(Seqs{a.cu, a.N, a.T}, p.len, (int)p.pieces, (int)p.slots, table);
  return cudaGetLastError();
}

cudaError_t compose_pieces(const PiecePlan& p, const SsmArgs& a, const PieceArgs& pa, cudaStream_t s) {
  const int size = a.dk * a.dv, blocks = (a.H * size + 4 * CT - 1) / (4 * CT);
  const int64_t entries = a.cu ? p.first_pass : a.N;  // packed: a sequence's first piece is among the ones that others follow
  return launch_overlapped(ssm_compose_kernel, (unsigned)(entries * blocks), CT, 0, s, pa, a.init != nullptr, a.H, size,
                           blocks);
}

}  // namespace kda
