// kv.h — declarations shared by the paged key/value cache's translation units (not part of the ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace moe {

// The batch and the cache as the kernels see them.
struct KvBatch {
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* pages;
  long long pages_stride;
  int pages_cols;
  int n_seqs;
  int n_tokens;
  int max_new;
};

struct KvCache {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int n_pages;
  int kv_heads;
  int page_log2;
  int head_dim;
  int e4m3;
};

struct KvRows {
  const uint16_t* ptr;
  long long token_stride;
  long long head_stride;
};

// Up to 256 (token, query head) rows of one sequence and kv head, and the tiles of 128 keys they see.
struct KvRowTile {
  int seq;
  int row0;   // first token row
  int nt;     // tokens
  int p0;     // position of the first (below 0: it sees nothing)
  int front;  // tiles of the sinks, before the window's
  int skip;   // tiles between the two
  int count;  // tiles in all
  int unused;
};

// A pair's share of the work: units [begin, end), and the item it begins in.
struct KvShare {
  long long begin, end;
  int entry, part, u0;  // the row tile, the kv head (and half of V's width) and the unit of the item
  int unused;
};

// An item that shares cut into pieces, to be joined.
struct KvJoin {
  int row0, nt;     // its tokens; nt 0: nothing to join
  int part;
  int first, count; // the pairs that have pieces of it
  int first_place;  // where the first one's is
  int unused[2];
};

// The row tiles of a call, in the workspace.
struct KvChunkList {
  int* first_tile;        // [max_seqs] of each sequence
  KvRowTile* tiles;
  long long* first_unit;  // [row tiles] shares of the work are counted in units, see kv_chunk.cu
  int* n_tiles;
  int max_tiles;          // the list's room
  KvShare* shares;        // [kChunkMaxPairs]
  KvJoin* joins;          // [kChunkMaxPairs], by the share that begins inside the item
};

struct KvAttn {
  KvBatch b;
  KvCache c;
  KvRows q;
  int group;    // query heads per kv head
  int q_heads;
  float scale;
  int window;   // 0: none
  int sinks;
  uint16_t* out;
  float* lse;   // or NULL
  unsigned int* status;
  int* counters;    // [max_seqs * kv_heads] pieces finished of each item, zero between calls
  int* counters_in; // [2 * kDecodeMaxCtas] the same, of groups of an item's pieces
  float* partial;   // pieces of items that several CTAs share
  KvChunkList list;      // the same for chunks of tokens
  int item_cost;         // what an item costs beside its key tiles, in key tiles (chunks of tokens)
  float* chunk_partial;
};

// The single-token kernel: CTAs (two to an SM), and the floats of a piece: eight heads' outputs, then
// their running maxima and sums.
constexpr int kDecodeMaxCtas = 304;
constexpr int kDecodeHeads = 8;
__host__ __device__ constexpr long long decode_piece_floats(int head_dim) {
  return static_cast<long long>(kDecodeHeads) * head_dim + 2 * kDecodeHeads;
}

// The kernel for chunks: pairs of CTAs (one to an SM), tokens of a row tile, and the floats of a piece:
// 256 rows of 256 (or 128) outputs, then their maxima and sums.
constexpr int kChunkMaxPairs = 76;
constexpr long long kChunkPieceFloats = 256 * 258;
inline int chunk_tokens(int group) { return 256 / group; }

bool encode_row_chunks(CUtensorMap* map, const void* ptr, uint64_t rows, uint64_t row_bytes, uint32_t box_rows,
                       uint32_t box_chunks, uint32_t chunk_bytes = 128, bool swizzle = true);

cudaError_t launch_kv_write(const KvBatch& b, const KvCache& c, const KvRows& k, const KvRows& v, unsigned int* status,
                            cudaStream_t s);
cudaError_t launch_kv_read(const KvBatch& b, const KvCache& c, uint16_t* k_out, uint16_t* v_out, unsigned int* status,
                           cudaStream_t s);
cudaError_t kv_decode_setup();
cudaError_t launch_kv_decode(const KvAttn& a, int ctas, cudaStream_t s);
cudaError_t kv_chunk_setup(int* pairs);
cudaError_t launch_kv_chunk(const KvAttn& a, int pairs, cudaStream_t s);

#ifdef __CUDACC__
// What a batch says of one sequence, with every value brought into range.
struct KvSeq {
  int row0;    // first token row
  int n;       // new tokens
  int len;     // tokens in the cache
};

__device__ __forceinline__ KvSeq kv_sequence(const KvBatch& b, const KvCache& c, int seq, unsigned int* status) {
  const int r0 = b.cu_q[seq], r1 = b.cu_q[seq + 1], len = b.kv_len[seq];
  KvSeq s;
  s.row0 = min(max(r0, 0), b.n_tokens);
  s.n = min(max(r1 - s.row0, 0), min(b.n_tokens - s.row0, b.max_new));
  const long long room = static_cast<long long>(b.pages_cols) << c.page_log2;
  s.len = static_cast<int>(min(static_cast<long long>(max(len, 0)), min(room, 0x7fffff00LL)));
  if (s.row0 != r0 || s.row0 + s.n != r1 || s.len != len || (seq == 0 && r0 != 0)) atomicOr(status, 0x10u);
  return s;
}

// Rows of no sequence: those before the first one's and those from the last one's end on.
struct KvNoRows {
  int before, after;
};

__device__ __forceinline__ KvNoRows kv_no_rows(const KvBatch& b) {
  if (b.n_seqs == 0) return {0, 0};
  return {min(max(b.cu_q[0], 0), b.n_tokens), min(max(b.cu_q[b.n_seqs], 0), b.n_tokens)};
}

// The positions one token sees: [0, sinks) and [lo, p], p < 0 for none.
struct KvSpan {
  int p;
  int lo;
  int sinks;  // at most lo
};

__device__ __forceinline__ KvSpan kv_span(int p, int window, int sinks) {
  KvSpan s;
  s.p = p;
  s.lo = window > 0 ? max(0, p - window + 1) : 0;
  s.sinks = min(sinks, s.lo);
  return s;
}

// The page that holds page `i` of sequence `seq`, or -1 (and the status bit) if its id is no page.
__device__ __forceinline__ int kv_page(const KvBatch& b, const KvCache& c, int seq, int i, unsigned int* status) {
  const int page = b.pages[seq * b.pages_stride + i];
  if (static_cast<unsigned>(page) < static_cast<unsigned>(c.n_pages)) return page;
  atomicOr(status, 0x10u);
  return -1;
}
#endif

}  // namespace moe
