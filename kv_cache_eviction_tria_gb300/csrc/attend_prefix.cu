// Attention of several continuations of one prompt (tria_attend_prefix): new
// tokens over the rows of a shared prefix, read for all sequences that continue it
// together, and over each sequence's own rows.
//
//   out = (o1 e^(l1 - m) + o2 e^(l2 - m)) / (e^(l1 - m) + e^(l2 - m)),
//   lse = m + ln(e^(l1 - m) + e^(l2 - m)),   m = max(l1, l2)
//
// of the two attentions' outputs o and log-sum-exps l, both in fp32. The own rows are
// tria_attend's; the prefix, too, or k_attend_group's, whose join then takes the own
// rows in. That join and k_attend_group start while the kernel before them ends.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "attend_internal.cuh"

namespace tria {

namespace {

constexpr int kJoinThreads = 256;

struct JoinArgs {
  const float *o1, *l1, *o2, *l2;    // [tokens][heads][hd], [tokens][heads]
  void* out;
  float* lse;
  int64_t out_stride;
  const int32_t *live1, *live2;
  int32_t n_tokens, nq, hd, type, n_seqs, n_prefixes;
  int32_t tok0[kMaxSeqs + 1], seq0[kMaxSeqs + 1], cap1[kMaxSeqs], cap2[kMaxSeqs];
};

__device__ __forceinline__ int last_at(const int32_t* first, int n, int x) {   // the last i < n with first[i] <= x
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A thread joins four dims of a token's head.
__global__ void __launch_bounds__(kJoinThreads) k_join_prefix(const __grid_constant__ JoinArgs A) {
  const int per = A.hd / 4;
  const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  if (i >= (int64_t)A.n_tokens * A.nq * per) return;
  const int64_t x = i / per;
  const int d = (int)(i - x * per) * 4, tok = (int)(x / A.nq), head = (int)(x - (int64_t)tok * A.nq);
  const int s = last_at(A.tok0, A.n_seqs, tok), p = last_at(A.seq0, A.n_prefixes, s);
  const int n1 = A.live1[p], n2 = A.live2[s];
  if (n1 < 0 || n1 > A.cap1[p] || n2 < 0 || n2 > A.cap2[s]) return;
  const float l1 = A.l1[x], l2 = A.l2[x], m = fmaxf(l1, l2), base = m == -INFINITY ? 0.f : m;
  const float w1 = expf(l1 - base), w2 = expf(l2 - base), sum = w1 + w2;
  const float f1 = sum > 0.f || sum != sum ? w1 / sum : 0.f, f2 = sum > 0.f || sum != sum ? w2 / sum : 0.f;
  const float4 a = *reinterpret_cast<const float4*>(A.o1 + i * 4), b = *reinterpret_cast<const float4*>(A.o2 + i * 4);
  const float v[4] = {fmaf(a.x, f1, b.x * f2), fmaf(a.y, f1, b.y * f2), fmaf(a.z, f1, b.z * f2), fmaf(a.w, f1, b.w * f2)};
  const int64_t to = (int64_t)tok * A.out_stride + (int64_t)head * A.hd + d;
  for (int k = 0; k < 4; ++k) act_store(A.out, A.type, to + k, v[k]);
  if (d == 0 && A.lse) A.lse[x] = sum == 0.f ? -INFINITY : m + logf(sum);
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Tokens of each prefix's sequences.
void prefix_tokens(const int32_t* seq0, int n_prefixes, const int32_t* tok0, int32_t* out) {
  for (int p = 0; p <= n_prefixes; ++p) out[p] = tok0[seq0[p]];
}

// Whether the prefixes are a matter for k_attend_group, which cuts their rows over
// the GPU. The others are k_attend's: of up to 16 columns (token x query head of a KV
// head's group) the step kernel, of more the prompt kernel. `rows` are those that a CTA
// would get, by the capacities, 128 columns at a time. Measured as whole calls, in us, of 8 KV
// heads x 128 dims:
//   up to 16 columns: fp16 planes always (4 columns: 777 rows 19.3 against 27.5 by the step
//   kernel, 65536 rows 66 against 72; 16 columns 64 against 79). Of quantised ones the step
//   kernel widens nothing and is faster in the long run (q8_0, 4 columns: 8192 rows 32 against 34,
//   65536 rows 84 against 62): up to kGroupShort rows.
//   up to kGroupFew columns (of quantised planes kGroupFewQ) always: 256 columns of 32768
//   fp16 rows 81 against 104, 512 of q8_0 160 against 213.
//   up to kGroupCols while a CTA gets kGroupLong rows at most: 512 columns of fp16, 16384
//   rows 64 against 77, 32768 rows 117 against 107; 1024 of q8_0, 4096 rows 70 against 78.
// Other shapes take the same limits. Of 168 calls (8 KV heads x 64, 128 and 256 dims, 4 x 256;
// 4 to 1024 columns of 777 to 65536 rows; fp16, q8_0 and q4_0) 152 take the faster side. The worst of
// the others: 16 columns of 32768 q8_0 rows x 256 dims (4 heads 93 against 57, 8 heads 122 against
// 85), 1024 columns of 16384 such rows of 8 heads (405 against 296), 512 columns of 32768 fp16
// rows x 64 dims (104 against 84).
// One choice for a call: with a prefix of more columns beside it, a long quantised one of few
// takes k_attend_group's roundings too.
constexpr int kGroupFew = 256, kGroupFewQ = 512, kGroupCols = 1024, kGroupShort = 512, kGroupLong = 4096;

bool by_group(const tria_layer_cache* c, int64_t most, int64_t units, int64_t rows) {
  if (!tensor_types(c, TRIA_F16) || most == 0 || units > kMaxSegments) return false;
  for (int p = 0; p < c->n_seqs; ++p)                      // (a row of a TMA tile has a signed 32-bit coordinate)
    if (c->seq_row0[p] + (int64_t)c->n_kv_heads * c->capacity[p] >= ((int64_t)1 << 31)) return false;
  const bool quantised = c->k_type != TRIA_F16 || c->v_type != TRIA_F16;
  if (most <= kStepCols) return !quantised || rows <= kGroupShort;
  return most <= (quantised ? kGroupFewQ : kGroupFew) || (most <= kGroupCols && rows <= kGroupLong);
}

struct PrefixLayout {
  AttendLayout shared, own;
  bool group;           // the prefix by k_attend_group
  int units;            // of it
  size_t span, table, part, o1, l1, o2, l2, total;
};

// The layout covers every type of queries, as attend_layout. The two caches'
// kernels run one after the other and share their space, but for what the join reads.
PrefixLayout prefix_layout(const tria_layer_cache* prefix, const tria_layer_cache* cache, const int32_t* seq0, int nq, const int32_t* tok0) {
  PrefixLayout L{};
  int32_t tp[kMaxSeqs + 1];
  prefix_tokens(seq0, prefix->n_seqs, tok0, tp);
  const int G = nq / cache->n_kv_heads, hd = cache->head_dim;
  int64_t units = 0, most = 0, rows_of_units = 0;
  for (int p = 0; p < prefix->n_seqs; ++p) {
    const int64_t cols = (int64_t)(tp[p + 1] - tp[p]) * G;
    most = std::max(most, cols);
    units += (cols + 127) / 128 * cache->n_kv_heads;
    rows_of_units += (cols + 127) / 128 * cache->n_kv_heads * prefix->capacity[p];
  }
  L.own = attend_layout(cache, G, tok0);
  L.group = by_group(prefix, most, units, rows_of_units / L.own.sms);
  L.units = (int)units;
  // fp32 queries take the other kernels whatever the columns, with a layout that has no room for fp16 copies
  L.shared = attend_layout(prefix, G, tp);
  const size_t shared = L.group ? L.shared.wide_k : L.shared.total;
  const size_t rows = (size_t)tok0[cache->n_seqs] * nq, values = up256(rows * hd * sizeof(float));
  L.span = up256(std::max(shared, L.own.total));
  L.table = up256(L.span + (L.group ? 2 * sizeof(int32_t) * (size_t)prefix->n_seqs * prefix->n_kv_heads : 0));
  L.part = up256(L.table + (L.group ? sizeof(int32_t) * (size_t)(kMaxSegments + 1) : 0));
  L.o1 = up256(L.part + (L.group ? sizeof(float) * group_part_values(hd) * (L.units + (size_t)L.own.sms) : 0));
  L.o2 = L.o1 + values;
  L.l1 = L.o2 + values;
  L.l2 = L.l1 + up256(rows * sizeof(float));
  L.total = L.l2 + up256(rows * sizeof(float));
  return L;
}

tria_status check_prefix(const tria_layer_cache* prefix, const tria_layer_cache* cache, const int32_t* seq0, int nq, const int32_t* tok0) {
  tria_status r;
  if ((r = check_cache(prefix)) != TRIA_OK) return r;
  if ((r = check_attend_shape(cache, nq, tok0)) != TRIA_OK) return r;
  if (!seq0 || prefix->n_kv_heads != cache->n_kv_heads || prefix->head_dim != cache->head_dim) return TRIA_ERR_INVALID_ARG;
  if (seq0[0] != 0 || seq0[prefix->n_seqs] != cache->n_seqs) return TRIA_ERR_INVALID_ARG;
  for (int p = 0; p < prefix->n_seqs; ++p)
    if (seq0[p + 1] < seq0[p]) return TRIA_ERR_INVALID_ARG;
  return TRIA_OK;
}

}  // namespace

}  // namespace tria

using namespace tria;

extern "C" size_t tria_attend_prefix_workspace_size(const tria_layer_cache* prefix, const tria_layer_cache* cache, const int32_t* seq0,
                                                    int32_t n_q_heads, const int32_t* tok0) {
  if (check_prefix(prefix, cache, seq0, n_q_heads, tok0) != TRIA_OK) return 0;
  return prefix_layout(prefix, cache, seq0, n_q_heads, tok0).total;
}

extern "C" tria_status tria_attend_prefix(const tria_layer_cache* prefix, const tria_layer_cache* cache, const int32_t* seq0,
                                          const tria_attention* a, void* ws, size_t ws_bytes, void* stream) {
  tria_status r;
  if (!a) return TRIA_ERR_INVALID_ARG;
  if ((r = check_prefix(prefix, cache, seq0, a->n_q_heads, a->tok0)) != TRIA_OK) return r;
  const int n_tokens = a->tok0[cache->n_seqs], hd = cache->head_dim, G = a->n_q_heads / cache->n_kv_heads;
  if ((r = check_attention(a, n_tokens, hd)) != TRIA_OK) return r;
  const PrefixLayout L = prefix_layout(prefix, cache, seq0, a->n_q_heads, a->tok0);
  if (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < L.total) return TRIA_ERR_WORKSPACE;
  if (n_tokens == 0) return TRIA_OK;
  int32_t tp[kMaxSeqs + 1];
  prefix_tokens(seq0, prefix->n_seqs, a->tok0, tp);
  if ((r = check_attend_rows(prefix, G, tp, a->type)) != TRIA_OK || (r = check_attend_rows(cache, G, a->tok0, a->type)) != TRIA_OK) return r;
  const cudaStream_t st = (cudaStream_t)stream;
  uint8_t* at = (uint8_t*)ws;
  float *o1 = (float*)(at + L.o1), *l1 = (float*)(at + L.l1), *o2 = (float*)(at + L.o2), *l2 = (float*)(at + L.l2);
  AttendArgs A;
  auto own_rows = [&] {
    AttendArgs B;
    fill_attend(B, cache, a);
    B.out = o2;
    B.lse = l2;
    B.out_stride = (int64_t)a->n_q_heads * hd;
    B.out_type = TRIA_F32;
    B.sink = 0;
    return run_attend(B, cache, a->tok0, a->round_keys != 0, L.own, ws, st) == cudaSuccess;
  };
  fill_attend(A, prefix, a);
  if (L.group && tensor_types(prefix, a->type)) {
    A.ctrl = (Ctrl*)ws;
    A.table = (int32_t*)(at + L.table);
    A.part = (float*)(at + L.part);
    for (int p = 0, unit = 0; p < prefix->n_seqs; ++p) {
      A.seq[p] = {prefix->seq_row0[p], 0, prefix->capacity[p], tp[p], tp[p + 1] - tp[p], unit};
      unit += (A.seq[p].t * G + 127) / 128 * A.n_kv;
    }
    A.units = L.units;
    if (A.window > 0) {
      int32_t* span = (int32_t*)(at + L.span);
      if (launch_attend_span(A, span, st) != cudaSuccess) return TRIA_ERR_CUDA;
      A.span = span;
    }
    const int grid = L.own.sms;
    // (the own rows' kernel first: the prefix's may start before it has ended, and needs what came before)
    if (!own_rows() || launch_attend_group(A, a->round_keys != 0, grid, st) != cudaSuccess) return TRIA_ERR_CUDA;
    GroupOwn own;
    own.n_seqs = cache->n_seqs;
    memcpy(own.tok0, a->tok0, sizeof(int32_t) * cache->n_seqs);
    memcpy(own.cap, cache->capacity, sizeof(int32_t) * cache->n_seqs);
    return launch_join_group(A, o2, l2, cache->n_live, own, grid, st) == cudaSuccess ? TRIA_OK : TRIA_ERR_CUDA;
  }
  A.out = o1;
  A.lse = l1;
  A.out_stride = (int64_t)a->n_q_heads * hd;
  A.out_type = TRIA_F32;
  if (!own_rows()) return TRIA_ERR_CUDA;
  if (run_attend(A, prefix, tp, a->round_keys != 0, L.shared, ws, st) != cudaSuccess) return TRIA_ERR_CUDA;
  JoinArgs J;
  memset(&J, 0, sizeof(J));
  J.o1 = o1;
  J.o2 = o2;
  J.l1 = l1;
  J.l2 = l2;
  J.out = a->out;
  J.lse = a->lse;
  J.out_stride = a->out_stride;
  J.live1 = prefix->n_live;
  J.live2 = cache->n_live;
  J.n_tokens = n_tokens;
  J.nq = a->n_q_heads;
  J.hd = hd;
  J.type = a->type;
  J.n_seqs = cache->n_seqs;
  J.n_prefixes = prefix->n_seqs;
  memcpy(J.tok0, a->tok0, sizeof(int32_t) * (cache->n_seqs + 1));
  memcpy(J.seq0, seq0, sizeof(int32_t) * (prefix->n_seqs + 1));
  memcpy(J.cap1, prefix->capacity, sizeof(int32_t) * prefix->n_seqs);
  memcpy(J.cap2, cache->capacity, sizeof(int32_t) * cache->n_seqs);
  const int64_t threads = (int64_t)n_tokens * a->n_q_heads * (hd / 4);
  k_join_prefix<<<(unsigned)((threads + kJoinThreads - 1) / kJoinThreads), kJoinThreads, 0, st>>>(J);
  return cudaGetLastError() == cudaSuccess ? TRIA_OK : TRIA_ERR_CUDA;
}
