// kv_moves.cu — trees of drafted tokens in the form the attention reads, and tokens that move within the cache: a
// tree's accepted path, and the page under way of beams that follow their parents.
//
// What moves is little (a few tokens of each sequence, a fraction of a page of each beam) and is read and written once,
// all layers' in a launch, so the launch and the chain of small loads before the first row (lengths, path, page
// ids, rows) bound it; only many beams' pages in many layers come near HBM's rate. In a graph, the path of one tree in one
// layer takes 1.8 us and a user's beams 2.2; from Python the calls take 10 and 7. The pages under way of 16 users' 5 beams in
// 6 layers, of which two in five move (50 MB read and written): 12.2 us, 4.1 TB/s.
#include "internal.h"
#include "kv.h"
#include "ptx.cuh"

namespace moe {

namespace {

// ------------------------------------------------------------------ trees

constexpr int kNodes = 256;
constexpr int kWords = kNodes / 32;

// A sequence's tree per CTA, a thread per node, which walks up to the root over parents in shared memory.
__global__ void __launch_bounds__(kNodes) kv_tree_masks_kernel(const KvBatch b, const KvCache c, const int32_t* parents, uint32_t* masks,
                                                         int32_t* depth, unsigned int* status) {
  __shared__ int parent[kNodes];
  pdl_wait();
  pdl_launch_dependents();
  const int i = threadIdx.x;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  if (static_cast<int>(blockIdx.x) >= b.n_seqs) {  // the last CTA: rows of no sequence
    const KvNoRows none = kv_no_rows(b);
    for (int r = i; r < b.n_tokens; r += kNodes) {
      if (r >= none.before && r < none.after) continue;
      reinterpret_cast<uint4*>(masks)[2LL * r] = reinterpret_cast<uint4*>(masks)[2LL * r + 1] = zero;
      depth[r] = 0;
    }
    return;
  }
  const KvSeq s = kv_sequence(b, c, blockIdx.x, status);
  int p = -1;
  if (i < s.n) {
    p = parents[s.row0 + i];
    if (p < -1 || p >= i) {
      atomicOr(status, kStatusBadIndex);
      p = -1;
    }
  }
  parent[i] = p;
  __syncthreads();
  if (i >= s.n) return;
  uint32_t w[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) w[k] = 0u;
  int steps = 0;
  for (int j = i; j >= 0; j = parent[j], ++steps) {
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      if (j >> 5 == k) w[k] |= 1u << (j & 31);
  }
  uint4* to = reinterpret_cast<uint4*>(masks) + 2LL * (s.row0 + i);
  to[0] = make_uint4(w[0], w[1], w[2], w[3]);
  to[1] = make_uint4(w[4], w[5], w[6], w[7]);
  depth[s.row0 + i] = steps - 1;
}

// ------------------------------------------------------------------ moves

// The bytes of a row (a head's keys or values of a token), and where it lies.
struct Plane {
  uint8_t* rows;
  float* scales;  // or NULL
};

__device__ __forceinline__ Plane plane_of(const KvLayers& l, int z) {
  const KvLayer& a = l.layer[z >> 1];
  return z & 1 ? Plane{a.v, a.v_scale} : Plane{a.k, a.k_scale};
}

constexpr int kKeepThreads = 128;
constexpr int kKeepVecs = 4;
constexpr int kKeepPath = kNodes;

// A sequence, kv head and plane (a layer's keys or values) per CTA. The path ascends and node i of it lies at or
// after slot i, so taken in order, kKeepVecs vectors to a thread, all read before any is written, no row is
// written before it has been read.
__global__ void __launch_bounds__(kKeepThreads)
    kv_keep_kernel(const KvBatch b, const KvCache c, const __grid_constant__ KvLayers l, const int32_t* nodes, long long nodes_stride,
                   int nodes_cols, const int32_t* counts, int32_t* new_len, unsigned int* status) {
  __shared__ int from[kKeepPath], to[kKeepPath];  // cache rows of head 0 and slot, -1: nothing to move
  __shared__ int first_bad;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, seq = blockIdx.x, head = blockIdx.y;
  const KvSeq s = kv_sequence(b, c, seq, status);
  const int old = s.len - s.n;
  const int asked = counts[seq];
  int count = old < 0 ? 0 : min(min(max(asked, 0), nodes_cols), s.n);
  if (tid == 0) first_bad = count;
  __syncthreads();
  const int32_t* path = nodes + seq * nodes_stride;
  for (int i = tid; i < count; i += kKeepThreads) {
    const int at = path[i];
    const bool ok = at >= i && at < s.n && (i == 0 || path[i - 1] < at);
    if (!ok) atomicMin(&first_bad, i);
  }
  __syncthreads();
  const bool bad = first_bad < count || old < 0 || count != asked;
  count = first_bad;
  if (tid == 0 && bad) atomicOr(status, kStatusBadIndex);
  if (new_len && tid == 0 && head == 0 && blockIdx.z == 0) new_len[seq] = old < 0 ? s.len : old + count;
  for (int i = tid; i < count; i += kKeepThreads) {
    const int src = old + path[i], dst = old + i;
    int f = -1, t = -1;
    if (src != dst) {
      const int sp = kv_page(b, c, seq, src >> c.page_log2, status), dp = kv_page(b, c, seq, dst >> c.page_log2, status);
      if (sp >= 0 && dp >= 0) {
        const int mask = (1 << c.page_log2) - 1;
        f = ((sp * c.kv_heads + head) << c.page_log2) + (src & mask);
        t = ((dp * c.kv_heads + head) << c.page_log2) + (dst & mask);
      }
    }
    from[i] = f;
    to[i] = t;
  }
  __syncthreads();
  const Plane p = plane_of(l, blockIdx.z);
  const int vecs_log2 = 31 - __clz(c.head_dim * (c.e4m3 ? 1 : 2) / 16);  // vectors of a row: 8 to 64
  uint4* rows = reinterpret_cast<uint4*>(p.rows);
  const int items = count << vecs_log2;
  for (int base = 0; base < items; base += kKeepThreads * kKeepVecs) {
    uint4 x[kKeepVecs];
    float sc[kKeepVecs];
#pragma unroll
    for (int j = 0; j < kKeepVecs; ++j) {
      const int item = base + j * kKeepThreads + tid, i = item >> vecs_log2, v = item & ((1 << vecs_log2) - 1);
      if (item >= items || from[i] < 0) continue;
      x[j] = rows[(static_cast<long long>(from[i]) << vecs_log2) + v];
      if (v == 0 && p.scales) sc[j] = p.scales[from[i]];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kKeepVecs; ++j) {
      const int item = base + j * kKeepThreads + tid, i = item >> vecs_log2, v = item & ((1 << vecs_log2) - 1);
      if (item >= items || from[i] < 0) continue;
      rows[(static_cast<long long>(to[i]) << vecs_log2) + v] = x[j];
      if (v == 0 && p.scales) p.scales[to[i]] = sc[j];
    }
    __syncthreads();
  }
}

constexpr int kReorderThreads = 128;
// Blocks in all, each with as many vectors as it takes. A page is seldom nearly full: 18 users' 2 beams of 6 to 31 tokens on
// pages of 128, 6 layers, take 33 us with a block for each vector that there could be, 12 with these (14 with a quarter, 16
// with four times as many).
constexpr int kReorderCtas = 16 * 152;
constexpr int kReorderRegs = 8;  // beams whose vectors a thread holds in registers (8 beams: 24.6 us, in shared memory 26.6)

// Blocks of a user and plane, then (of the first plane) one for the user's table. A thread takes one vector of one
// slot and head, of all the user's beams: it reads what any beam takes from another, then writes, so no other
// thread has a part in its values. More than kReorderRegs beams' vectors go through shared memory of its own.
template <bool REGS>
__global__ void __launch_bounds__(kReorderThreads)
    kv_reorder_kernel(const KvCache c, const __grid_constant__ KvLayers l, int32_t* pages, long long pages_stride, int pages_cols,
                      const int32_t* lengths, const int32_t* parents, int beams, int move_blocks, int first_group,
                      unsigned int* status) {
  extern __shared__ uint4 held[];  // [beams][kReorderThreads]
  __shared__ int source[64], page[64];  // [beams] the parent if it is another, else -1; the page under way
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, user = blockIdx.x;
  const bool table = static_cast<int>(blockIdx.y) == move_blocks;
  if (table && (blockIdx.z != 0 || !first_group)) return;
  const long long room = static_cast<long long>(pages_cols) << c.page_log2;
  const int given = lengths[user];
  const int length = static_cast<int>(min(static_cast<long long>(max(given, 0)), min(room, 0x7fffff00LL)));
  const int whole = length >> c.page_log2, rest = length & ((1 << c.page_log2) - 1);
  const int vecs_log2 = 31 - __clz(c.head_dim * (c.e4m3 ? 1 : 2) / 16);
  const int items = table ? whole : (rest * c.kv_heads) << vecs_log2;
  if (!table && static_cast<int>(blockIdx.y) * kReorderThreads >= items) return;
  const long long row0 = static_cast<long long>(user) * beams;
  if (tid < beams) {
    int of = parents[row0 + tid];
    bool bad = given != length;
    if (static_cast<unsigned>(of) >= static_cast<unsigned>(beams)) {
      of = tid;
      bad = true;
    }
    int at = -1;
    if (!table) {
      at = pages[(row0 + tid) * pages_stride + whole];
      if (static_cast<unsigned>(at) >= static_cast<unsigned>(c.n_pages)) {
        at = -1;
        bad = true;
      }
    }
    if (bad) atomicOr(status, kStatusBadIndex);
    page[tid] = at;
    source[tid] = of == tid ? -1 : of;
  }
  __syncthreads();
  if (table) {
    for (int i = tid; i < whole; i += kReorderThreads) {
      int32_t* at = pages + row0 * pages_stride + i;
      int* mine = reinterpret_cast<int*>(held) + tid;
      for (int k = 0; k < beams; ++k)
        if (source[k] >= 0) mine[k * kReorderThreads] = at[source[k] * pages_stride];
      for (int k = 0; k < beams; ++k)
        if (source[k] >= 0) at[k * pages_stride] = mine[k * kReorderThreads];
    }
    return;
  }
  const Plane p = plane_of(l, blockIdx.z);
  uint4* rows = reinterpret_cast<uint4*>(p.rows);
  auto moves = [&](int k) { return source[k] >= 0 && page[k] >= 0 && page[source[k]] >= 0; };
  for (int item = blockIdx.y * kReorderThreads + tid; item < items; item += move_blocks * kReorderThreads) {
    const int v = item & ((1 << vecs_log2) - 1), row = item >> vecs_log2;  // (a head's slots lie next to each other)
    const int head = row / rest, slot = row - head * rest;
    auto place = [&](int k) { return (static_cast<long long>(page[k] * c.kv_heads + head) << c.page_log2) + slot; };
    const bool scaled = v == 0 && p.scales;
    if constexpr (REGS) {
      uint4 x[kReorderRegs];
      float sc[kReorderRegs];
#pragma unroll
      for (int k = 0; k < kReorderRegs; ++k) {
        if (k >= beams || !moves(k)) continue;
        const long long from = place(source[k]);
        x[k] = rows[(from << vecs_log2) + v];
        if (scaled) sc[k] = p.scales[from];
      }
#pragma unroll
      for (int k = 0; k < kReorderRegs; ++k) {
        if (k >= beams || !moves(k)) continue;
        const long long to = place(k);
        rows[(to << vecs_log2) + v] = x[k];
        if (scaled) p.scales[to] = sc[k];
      }
    } else {
      uint4* mine = held + tid;
      for (int k = 0; k < beams; ++k)
        if (moves(k))
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(mine + k * kReorderThreads)),
                       "l"(rows + (place(source[k]) << vecs_log2) + v)
                       : "memory");
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (int k = 0; k < beams; ++k)
        if (moves(k)) rows[(place(k) << vecs_log2) + v] = mine[k * kReorderThreads];
      if (!scaled) continue;
      for (int k = 0; k < beams; ++k)
        if (moves(k)) mine[k * kReorderThreads].x = __float_as_uint(p.scales[place(source[k])]);
      for (int k = 0; k < beams; ++k)
        if (moves(k)) p.scales[place(k)] = __uint_as_float(mine[k * kReorderThreads].x);
    }
  }
}

}  // namespace

cudaError_t kv_moves_setup() {
  return cudaFuncSetAttribute(kv_reorder_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * kReorderThreads * 16);
}

cudaError_t launch_kv_tree(const KvBatch& b, const KvCache& c, const int32_t* parents, uint32_t* masks, int32_t* depth,
                           unsigned int* status, cudaStream_t s) {
  return launch_pdl(kv_tree_masks_kernel, dim3(b.n_seqs + 1), dim3(kNodes), 0, s, b, c, parents, masks, depth, status);
}

cudaError_t launch_kv_keep(const KvBatch& b, const KvCache& c, const KvLayers& l, int n_layers, const int32_t* nodes,
                           long long nodes_stride, int nodes_cols, const int32_t* counts, int32_t* new_len, unsigned int* status,
                           cudaStream_t s) {
  return launch_pdl(kv_keep_kernel, dim3(b.n_seqs, c.kv_heads, 2 * n_layers), dim3(kKeepThreads), 0, s, b, c, l, nodes,
                    nodes_stride, nodes_cols, counts, new_len, status);
}

cudaError_t launch_kv_reorder(const KvCache& c, const KvLayers& l, int n_layers, int32_t* pages, long long pages_stride,
                              int pages_cols, const int32_t* lengths, const int32_t* parents, int users, int beams,
                              bool first_group, unsigned int* status, cudaStream_t s) {
  const int vecs = c.head_dim * (c.e4m3 ? 1 : 2) / 16;
  const int most = (((1 << c.page_log2) - 1) * c.kv_heads * vecs + kReorderThreads - 1) / kReorderThreads;
  const int planes = 2 * n_layers, share = planes > 0 ? (kReorderCtas + users * planes - 1) / (users * planes) : 0;
  const int move_blocks = share < most ? share : most;
  const dim3 grid(users, move_blocks + 1, n_layers > 0 ? 2 * n_layers : 1);
  const size_t smem = static_cast<size_t>(beams) * kReorderThreads * (beams <= kReorderRegs ? 4 : 16);
  const int first = first_group ? 1 : 0;
  return beams <= kReorderRegs ? launch_pdl(kv_reorder_kernel<true>, grid, dim3(kReorderThreads), smem, s, c, l, pages, pages_stride,
                                            pages_cols, lengths, parents, beams, move_blocks, first, status)
                               : launch_pdl(kv_reorder_kernel<false>, grid, dim3(kReorderThreads), smem, s, c, l, pages,
                                            pages_stride, pages_cols, lengths, parents, beams, move_blocks, first, status);
}

}  // namespace moe
