// The caches of beams follow their parents (tria_reorder): in every layer,
// sequence s takes the rows that sequence parent[s] had, in place.
//
// Row r of a segment of s lies r rows behind the segment's first one, and so
// does row r of the parent's: 16 bytes of a row depend on the same 16 bytes of
// the other sequences of the group alone. A thread takes such a piece for the
// whole group - loads those of all parents, then stores - and the copy needs
// no second buffer and no order between threads. Sequences that are their own
// parent are not touched. Segments' blocks of rows are contiguous in every
// plane, so a piece's place is the same distance from each sequence's block.
//
// Groups with more moves than a thread holds pieces (kBatch) go in batches, in
// an order in which nobody is overwritten before its rows have been read:
// first the places that nobody reads, until only rings are left
// (a survivor that stays in its place is read and never written, so that
// in-place selections need a single round). Rings then keep one piece aside.
//
// Bound by memory: bytes read once a distinct parent and written once a moved
// sequence. All layers are one launch, whose CTAs stride over blocks of
// rows (layer, group, KV head, rows): how many there are is known on the
// device alone, where n_live is.
//
// 36 layers, 4 groups of 8 beams, 401 rows of 8 KV heads x 128 dims: 249 us in fp16,
// 5.5 TB/s of those bytes; one group of 32 beams, 1003 rows, q8_0 keys and q4_0
// values 277 us, 4.2 TB/s: five planes with loads of their own, two of them and the
// positions in pieces of four bytes. One layer of four beams takes 8 us, nearly all of it
// the start and the end of a kernel.
#include <string.h>

#include <algorithm>

#include "attend_internal.cuh"

namespace tria {

namespace {

constexpr int kReorderThreads = 256, kBatch = 4;
constexpr int kMaxLayers = 128, kMaxBeams = TRIA_MAX_BEAMS;
constexpr int kMaxUnits = 2048;       // (layer, group) pairs of a launch
// Rows of a block at most: 16 KB of keys, so that a batch of four moves fills the
// threads' loads twice (128-byte rows, 32 beams x 1003 rows x 36 layers: 276 us with
// 128 of them, 290 with 64; 256-byte rows: 258 and 249)
constexpr int kBlockBytes = 16384, kLeastMaxBlock = 64, kMostMaxBlock = 256;

struct ReorderLayer {
  uint8_t *k, *ks, *v, *vs;
  int32_t *pos, *n_live;
};

struct ReorderArgs {
  const int32_t* parent;
  Ctrl* ctrl;
  int32_t n_layers, n_groups, n_seqs, n_kv;
  int32_t k_rb, v_rb, ks_rb, vs_rb;   // bytes of a row of each plane (0: none)
  int32_t words;                      // every row of the scales starts on 4 bytes, in every layer
  int32_t max_block;
  int32_t cap[kMaxSeqs];
  int64_t row0[kMaxSeqs];
  int32_t seq0[kMaxSeqs + 1];
  ReorderLayer layer[kMaxLayers];
};

// A move: dst, src (sequences); of a ring, the first one keeps what it
// overwrites aside and the last one takes that.
constexpr uint32_t kKeep = 1u << 16, kTake = 1u << 17;
__device__ __forceinline__ int dst_of(uint32_t op) { return op & 0xFF; }
__device__ __forceinline__ int src_of(uint32_t op) { return (op >> 8) & 0xFF; }

// What a block's moves copy: first rows of the sources and the destinations in
// a plane, rows (none behind the last move).
struct Moves {
  int64_t from[kMaxBeams + kBatch], to[kMaxBeams + kBatch];
  int rows[kMaxBeams + kBatch];
};

// Rows of a plane by the M moves from `at` on, a piece of T at a time, P pieces of
// each move in flight, everything of a piece read before anything is written. (A
// piece is the same thread's in every batch.)
template <int M, typename T>
__device__ __forceinline__ void copy_plane(uint8_t* plane, int rb, const Moves& B, int at) {
  constexpr int P = 8 / M;
  const int per = rb / (int)sizeof(T);
  int n = 0;
  const T* from[M];
  T* to[M];
  int most[M];
#pragma unroll
  for (int j = 0; j < M; ++j) {
    from[j] = reinterpret_cast<const T*>(plane + B.from[at + j] * rb);
    to[j] = reinterpret_cast<T*>(plane + B.to[at + j] * rb);
    most[j] = B.rows[at + j] * per;
    n = max(n, most[j]);
  }
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += P * kReorderThreads) {
    T x[M][P];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < M; ++j)
        if (i + p * kReorderThreads < most[j]) x[j][p] = from[j][i + p * kReorderThreads];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < M; ++j)
        if (i + p * kReorderThreads < most[j]) to[j][i + p * kReorderThreads] = x[j][p];
  }
}

// A batch's moves of one block, plane by plane.
template <int M>
__device__ __forceinline__ void copy_moves(const ReorderArgs& A, const ReorderLayer& L, const Moves& B, int at) {
#pragma unroll 1
  for (int x = 0; x < 2; ++x) {
    copy_plane<M, uint4>(x ? L.v : L.k, x ? A.v_rb : A.k_rb, B, at);
    const int rb = x ? A.vs_rb : A.ks_rb;
    if (rb && A.words) copy_plane<M, uint32_t>(x ? L.vs : L.ks, rb, B, at);
    else if (rb) copy_plane<M, uint16_t>(x ? L.vs : L.ks, rb, B, at);
  }
  copy_plane<M, uint32_t>(reinterpret_cast<uint8_t*>(L.pos), 4, B, at);
}

// More moves than a batch, rings among them: move by move, piece by piece.
template <typename T>
__device__ __forceinline__ void copy_rings(const ReorderArgs& A, uint8_t* plane, int rb, const int32_t* n_live, const uint32_t* ops, int m,
                                           int g, int r0, int most) {
  const int per = rb / (int)sizeof(T);
#pragma unroll 1
  for (int i = threadIdx.x; i < most * per; i += kReorderThreads) {
    const int row = r0 + i / per;
    T aside{};
#pragma unroll 1
    for (int j = 0; j < m; ++j) {
      const uint32_t op = ops[j];
      const int s = src_of(op), d = dst_of(op);
      const T* from = reinterpret_cast<const T*>(plane + (A.row0[s] + (int64_t)g * A.cap[s] + r0) * rb) + i;
      T* to = reinterpret_cast<T*>(plane + (A.row0[d] + (int64_t)g * A.cap[d] + r0) * rb) + i;
      const bool live = row < *((volatile const int32_t*)(n_live + s));
      T x = aside;
      if (live && !(op & kTake)) x = *from;
      if ((op & kKeep) && row < *((volatile const int32_t*)(n_live + d))) aside = *to;
      if (live) *to = x;
    }
  }
}

// Moves of a group in an order that overwrites nothing unread, by a warp (lane:
// sequence of the group); -1 when a parent is outside the group. *ring: rings
// are among them that a batch may cut.
__device__ __forceinline__ int order_moves(const ReorderArgs& A, int group, uint32_t* ops, bool* ring) {
  const int lane = threadIdx.x & 31, first = A.seq0[group], size = A.seq0[group + 1] - first;
  const int64_t at = lane < size ? (int64_t)A.parent[first + lane] - first : lane;
  *ring = false;
  if (__any_sync(0xffffffffu, lane < size && (at < 0 || at >= size))) return -1;
  const int p = (int)at;
  uint32_t left = __ballot_sync(0xffffffffu, lane < size && p != lane);
  int n = 0;
  while (left) {
    const bool mine = (left >> lane) & 1u;
    const uint32_t read = __reduce_or_sync(0xffffffffu, mine ? 1u << p : 0u);
    const uint32_t ready = left & ~read;
    if (ready) {
      if ((ready >> lane) & 1u) ops[n + __popc(ready & ((1u << lane) - 1u))] = (uint32_t)(first + lane) | (uint32_t)(first + p) << 8;
      n += __popc(ready);
      left &= ~ready;
      continue;
    }
    // every place left is read by one other: rings
    const int head = __ffs(left) - 1;
    int x = head;
    do {
      const int from = __shfl_sync(0xffffffffu, p, x);
      if (lane == 0)
        ops[n] = (uint32_t)(first + x) | (uint32_t)(first + from) << 8 | (x == head ? kKeep : 0u) | (from == head ? kTake : 0u);
      ++n;
      left &= ~(1u << x);
      x = from;
    } while (x != head);
    *ring = true;
  }
  *ring = *ring && n > kBatch;
  return n;
}

__global__ void __launch_bounds__(kReorderThreads, 2) k_reorder(const __grid_constant__ ReorderArgs A) {
  __shared__ uint32_t s_op[kMaxSeqs];                      // a group's moves from its first sequence on
  __shared__ int s_n[kMaxSeqs];                            // how many (-1: a parent outside the group)
  __shared__ uint8_t s_ring[kMaxSeqs];
  __shared__ int s_first[kMaxUnits + 1], s_rows[kMaxUnits];
  __shared__ int s_scan[40];
  __shared__ Moves s_moves[2];                             // of this block and the one before
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int group = warp; group < A.n_groups; group += kReorderThreads / 32) {
    bool ring;
    const int n = order_moves(A, group, s_op + A.seq0[group], &ring);
    if (lane == 0) {
      s_n[group] = n;
      s_ring[group] = ring;
      if (n < 0 && blockIdx.x == 0) report(A.ctrl, TRIA_ERR_DEVICE_ARG, (uint32_t)A.seq0[group]);
    }
  }
  __syncthreads();

  // ---- rows of each unit (layer, group): of the longest parent that moves
  const int units = A.n_layers * A.n_groups, per = (units + kReorderThreads - 1) / kReorderThreads;
  auto unit_rows = [&](int u, uint32_t* error) {           // -1: the unit is left as it is
    const int layer = u / A.n_groups, group = u - layer * A.n_groups, first = A.seq0[group];
    const int32_t* n_live = A.layer[layer].n_live;
    *error = 0;
    if (s_n[group] < 0) return -1;
    if (s_n[group] == 0) return 0;
#pragma unroll 8
    for (int s = first; s < A.seq0[group + 1]; ++s) {
      const int n = *((volatile const int32_t*)(n_live + s));
      if (n < 0 || n > A.cap[s]) *error = TRIA_ERR_DEVICE_ARG;
    }
    if (*error) return -1;
    int most = 0;
    for (int j = 0; j < s_n[group]; ++j) {
      const uint32_t op = s_op[first + j];
      const int n = *((volatile const int32_t*)(n_live + src_of(op)));
      if (n > A.cap[dst_of(op)]) *error = TRIA_ERR_CAPACITY;
      most = max(most, n);
    }
    return *error ? -1 : most;
  };
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int u = (int)threadIdx.x * per + i;
    if (u >= units) break;
    uint32_t error;
    const int rows = unit_rows(u, &error);
    if (error && blockIdx.x == 0) report(A.ctrl, error, (uint32_t)A.seq0[u % A.n_groups]);
    s_rows[u] = rows;
    sum += (max(rows, 0) + 7) / 8;
  }
  int all;
  block_exclusive_scan(sum, &all, s_scan);
  // blocks small enough that every CTA has some, large enough that a plane's piece is no single load
  const int block = (int)min((int64_t)A.max_block, max((int64_t)8, (int64_t)all * A.n_kv * 2 / (int64_t)gridDim.x & ~(int64_t)7));
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int u = (int)threadIdx.x * per + i;
    if (u < units) mine += A.n_kv * ((max(s_rows[u], 0) + block - 1) / block);
  }
  int total, before = block_exclusive_scan(mine, &total, s_scan);
  for (int i = 0; i < per; ++i) {
    const int u = (int)threadIdx.x * per + i;
    if (u >= units) break;
    s_first[u] = before;
    before += A.n_kv * ((max(s_rows[u], 0) + block - 1) / block);
  }
  if (threadIdx.x == 0) s_first[units] = total;
  if (threadIdx.x < 2 * kBatch) {
    Moves& B = s_moves[threadIdx.x / kBatch];
    B.from[kMaxBeams + threadIdx.x % kBatch] = B.to[kMaxBeams + threadIdx.x % kBatch] = 0;
    B.rows[kMaxBeams + threadIdx.x % kBatch] = 0;
  }
  __syncthreads();

  int turn = 0;
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int u = 0, hi = units - 1;                             // the last unit that starts at or before it
    while (u < hi) {
      const int mid = (u + hi + 1) >> 1;
      if (s_first[mid] <= item) u = mid; else hi = mid - 1;
    }
    const int layer = u / A.n_groups, group = u - layer * A.n_groups;
    const int blocks = (s_rows[u] + block - 1) / block, x = item - s_first[u], g = x / blocks, r0 = (x - g * blocks) * block;
    const ReorderLayer& L = A.layer[layer];
    const uint32_t* ops = s_op + A.seq0[group];
    const int n = s_n[group];
    if (s_ring[group]) {
      const int most = min(block, s_rows[u] - r0);
      copy_rings<uint4>(A, L.k, A.k_rb, L.n_live, ops, n, g, r0, most);
      copy_rings<uint4>(A, L.v, A.v_rb, L.n_live, ops, n, g, r0, most);
      if (A.ks_rb) copy_rings<uint16_t>(A, L.ks, A.ks_rb, L.n_live, ops, n, g, r0, most);
      if (A.vs_rb) copy_rings<uint16_t>(A, L.vs, A.vs_rb, L.n_live, ops, n, g, r0, most);
      copy_rings<uint32_t>(A, reinterpret_cast<uint8_t*>(L.pos), 4, L.n_live, ops, n, g, r0, most);
      continue;
    }
    Moves& B = s_moves[turn ^= 1];
    if (warp == 0) {
      const uint32_t op = ops[min(lane, n - 1)];
      const int s = src_of(op), d = dst_of(op);
      B.from[lane] = A.row0[s] + (int64_t)g * A.cap[s] + r0;
      B.to[lane] = A.row0[d] + (int64_t)g * A.cap[d] + r0;
      B.rows[lane] = lane < n ? max(0, min(block, *((volatile const int32_t*)(L.n_live + s)) - r0)) : 0;
    }
    __syncthreads();
#pragma unroll 1
    for (int at = 0; at < n; at += kBatch) {
      if (n - at <= 2) copy_moves<2>(A, L, B, at);
      else copy_moves<4>(A, L, B, at);
    }
  }

  // ---- the last CTA to finish sets n_live, which nobody reads any more
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(&A.ctrl->reorder_ticket, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  for (int u = threadIdx.x; u < units; u += kReorderThreads) {
    if (s_rows[u] < 0) continue;
    const int layer = u / A.n_groups, group = u - layer * A.n_groups, first = A.seq0[group], n = s_n[group];
    int32_t* n_live = A.layer[layer].n_live;
    int now[kMaxBeams];                                    // (its place is local memory)
#pragma unroll 8
    for (int j = 0; j < n; ++j) now[j] = *((volatile const int32_t*)(n_live + src_of(s_op[first + j])));
#pragma unroll 1
    for (int j = 0; j < n; ++j) n_live[dst_of(s_op[first + j])] = now[j];
  }
  if (threadIdx.x == 0) atomicExch(&A.ctrl->reorder_ticket, 0u);
}

}  // namespace

}  // namespace tria

using namespace tria;

namespace {

tria_status check_groups(const int32_t* seq0, int n_groups, int n_seqs) {
  if (!seq0 || n_groups < 1 || n_groups > kMaxSeqs || seq0[0] != 0 || seq0[n_groups] != n_seqs) return TRIA_ERR_INVALID_ARG;
  for (int i = 0; i < n_groups; ++i)
    if (seq0[i + 1] < seq0[i]) return TRIA_ERR_INVALID_ARG;
  for (int i = 0; i < n_groups; ++i)
    if (seq0[i + 1] - seq0[i] > TRIA_MAX_BEAMS) return TRIA_ERR_UNSUPPORTED;
  return TRIA_OK;
}

tria_status check_reorder(const tria_layer_cache* caches, int n_layers, const int32_t* seq0, int n_groups) {
  if (!caches || n_layers < 1) return TRIA_ERR_INVALID_ARG;
  if (n_layers > kMaxLayers) return TRIA_ERR_UNSUPPORTED;
  const tria_layer_cache& c0 = caches[0];
  const void* planes[6 * kMaxLayers];
  int n_planes = 0;
  tria_status r;
  for (int i = 0; i < n_layers; ++i) {
    const tria_layer_cache& c = caches[i];
    if ((r = check_cache(&c, 2)) != TRIA_OK) return r;     // (bits are moved: scales may start on any value)
    if (c.n_seqs != c0.n_seqs || c.n_kv_heads != c0.n_kv_heads || c.head_dim != c0.head_dim || c.k_type != c0.k_type ||
        c.v_type != c0.v_type)
      return TRIA_ERR_INVALID_ARG;
    for (int s = 0; s < c0.n_seqs; ++s)
      if (c.seq_row0[s] != c0.seq_row0[s] || c.capacity[s] != c0.capacity[s]) return TRIA_ERR_INVALID_ARG;
    for (const void* x : {(const void*)c.k, (const void*)c.v, (const void*)c.k_scale, (const void*)c.v_scale, (const void*)c.pos,
                          (const void*)c.n_live})
      if (x) planes[n_planes++] = x;
  }
  std::sort(planes, planes + n_planes);                    // no plane may be moved twice
  if (std::adjacent_find(planes, planes + n_planes) != planes + n_planes) return TRIA_ERR_INVALID_ARG;
  return check_groups(seq0, n_groups, c0.n_seqs);
}

int row_bytes(int type, int hd) { return type == TRIA_F32 ? 4 * hd : (type == TRIA_F16 ? 2 * hd : (type == TRIA_Q8_0 ? hd : hd / 2)); }

}  // namespace

extern "C" size_t tria_reorder_workspace_size(const tria_layer_cache* caches, int32_t n_layers, const int32_t* seq0, int32_t n_groups) {
  return check_reorder(caches, n_layers, seq0, n_groups) == TRIA_OK ? sizeof(Ctrl) : 0;
}

extern "C" tria_status tria_reorder(const tria_layer_cache* caches, int32_t n_layers, const int32_t* seq0, int32_t n_groups,
                                    const int32_t* parent, void* ws, size_t ws_bytes, void* stream) {
  tria_status r;
  if ((r = check_reorder(caches, n_layers, seq0, n_groups)) != TRIA_OK) return r;
  if (!parent || (uintptr_t)parent % 4 != 0) return TRIA_ERR_INVALID_ARG;
  if (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < sizeof(Ctrl)) return TRIA_ERR_WORKSPACE;
  const tria_layer_cache& c = caches[0];
  ReorderArgs A;
  memset(&A, 0, sizeof(A));
  A.parent = parent;
  A.ctrl = (Ctrl*)ws;
  A.n_groups = n_groups;
  A.n_seqs = c.n_seqs;
  A.n_kv = c.n_kv_heads;
  A.k_rb = row_bytes(c.k_type, c.head_dim);
  A.v_rb = row_bytes(c.v_type, c.head_dim);
  A.max_block = std::min(std::max(kBlockBytes / A.k_rb, kLeastMaxBlock), kMostMaxBlock) & ~7;
  A.ks_rb = c.k_scale ? c.head_dim / 16 : 0;
  A.vs_rb = c.v_scale ? c.head_dim / 16 : 0;
  uintptr_t ends = A.ks_rb | A.vs_rb;
  for (int i = 0; i < n_layers; ++i) ends |= (uintptr_t)caches[i].k_scale | (uintptr_t)caches[i].v_scale;
  A.words = ends % 4 == 0;
  int64_t rows = 0;
  for (int s = 0; s < c.n_seqs; ++s) {
    A.cap[s] = c.capacity[s];
    A.row0[s] = c.seq_row0[s];
    rows = std::max<int64_t>(rows, c.capacity[s]);
  }
  memcpy(A.seq0, seq0, sizeof(int32_t) * (n_groups + 1));
  const cudaStream_t st = (cudaStream_t)stream;
  const int at_once = std::min(kMaxLayers, kMaxUnits / n_groups);
  for (int l0 = 0; l0 < n_layers; l0 += at_once) {
    A.n_layers = std::min(at_once, n_layers - l0);
    for (int i = 0; i < A.n_layers; ++i) {
      const tria_layer_cache& x = caches[l0 + i];
      A.layer[i] = {(uint8_t*)x.k, (uint8_t*)x.k_scale, (uint8_t*)x.v, (uint8_t*)x.v_scale, x.pos, x.n_live};
    }
    // blocks of 8 rows at least
    const int64_t blocks = (int64_t)A.n_layers * n_groups * A.n_kv * ((rows + 7) / 8);
    const int grid = (int)std::min<int64_t>(std::max<int64_t>(blocks, 1), 2 * (int64_t)sm_count());
    k_reorder<<<grid, kReorderThreads, 0, st>>>(A);
    if (cudaGetLastError() != cudaSuccess) return TRIA_ERR_CUDA;
  }
  return TRIA_OK;
}
