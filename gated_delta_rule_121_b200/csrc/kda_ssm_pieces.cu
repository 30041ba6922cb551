// Cutting sequences into pieces (kda_ssm_pieces.cuh): the host's plan, and the
// table of a packed batch, whose lengths are on the device.
#include "kda_ssm_pieces.cuh"

namespace kda {
namespace {

constexpr int MAX_PARTS = 64;  // of a sequence of known length (a piece adds up the ones before it)

// The pieces of a packed batch, in the sequences' order (one block; entries
// behind the last one are marked unused).  Running sums of the pieces and of
// the slots that sequences of several pieces take; offsets that are no
// offsets may claim more than there is, and what lies beyond is left out.
// Pieces are twice as long where one sequence holds more than half of the tokens:
// its pieces alone fill the device then, and a piece adds up the states of all
// before it (65536 tokens, H = 8, one sequence of 62K: 152 us against 224;
// 32768 tokens in sequences of up to 10000, H = 48: 358 us against 332 for the
// short pieces).
__global__ void __launch_bounds__(1024) ssm_piece_table_kernel(Seqs q, int64_t len, int capacity, int slots,
                                                               PieceEntry* table) {
  __shared__ int2 part[1024];
  __shared__ int2 carry;
  __shared__ int longs;  // sequences of more than half of the tokens
  const int tid = threadIdx.x;
  if (tid == 0) {
    carry = make_int2(0, 0);
    longs = 0;
  }
  __syncthreads();
  for (int n = tid; n < q.N; n += 1024)
    if (2 * (q.end(n) - q.begin(n)) > q.T) atomicAdd(&longs, 1);
  __syncthreads();
  if (longs) len *= 2;
  for (int n0 = 0; n0 < q.N; n0 += 1024) {
    const int n = n0 + tid;
    int64_t s = 0, e = 0;
    int cnt = 0;
    if (n < q.N) {
      s = q.begin(n);
      e = max(q.end(n), s);
      cnt = (int)max((e - s + len - 1) / len, (int64_t)1);
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
      const int64_t a = s + r * len;
      if (first + r < capacity)
        table[first + r] = {slot0 + own <= slots ? n : -1, r, cnt, slot0, (int)a, (int)min(a + len, e), {0, 0}};
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

}  // namespace

PiecePlan plan_pieces(int N, int64_t T, int blocks, int places, double first, int least, int H, int dk, int dv,
                      bool packed) {
  PiecePlan p;
  const int64_t chunks = (T + PIECE_CHUNK - 1) / PIECE_CHUNK;  // of a sequence, or of the packed total
  if (!packed) {
    // Pieces per sequence and parts per piece with the fewest chunk times in the
    // two passes, in waves of blocks; 3 chunk times for a block's start and 6 for
    // the second launch.
    const int64_t chains = (int64_t)N * blocks;
    auto waves = [&](int64_t n) { return (double)((n + places - 1) / places); };
    int64_t part = chunks > 0 ? chunks : 1;
    int parts = 1;
    double cost = waves(chains) * chunks;
    for (int r = 2; r <= MAX_PARTS; ++r)
      for (int q = 1; q <= 4 && r * q <= MAX_PARTS && chunks / (r * q) >= least; ++q) {
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
    p.first_pass = T > p.len ? p.pieces : 0;
    // a sequence of L > len tokens has at most L / len + 1 < 2 L / len pieces
    p.slots = p.first_pass ? 2 * T / p.len : 0;
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

}  // namespace kda
