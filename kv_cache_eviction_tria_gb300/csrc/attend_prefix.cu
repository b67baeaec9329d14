// Attention of several continuations of one prompt (tria_attend_prefix): new
// tokens over the rows of a shared prefix, read once for all sequences that
// continue it, and over each sequence's own rows.
//
//   out = (o1 e^(l1 - m) + o2 e^(l2 - m)) / (e^(l1 - m) + e^(l2 - m)),
//   lse = m + ln(e^(l1 - m) + e^(l2 - m)),   m = max(l1, l2)
//
// of the two attentions' outputs o and log-sum-exps l, both in fp32.
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

struct PrefixLayout {
  AttendLayout shared, own;
  size_t o1, l1, o2, l2, total;
};

// Tokens of each prefix's sequences.
void prefix_tokens(const int32_t* seq0, int n_prefixes, const int32_t* tok0, int32_t* out) {
  for (int p = 0; p <= n_prefixes; ++p) out[p] = tok0[seq0[p]];
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

PrefixLayout prefix_layout(const tria_layer_cache* prefix, const tria_layer_cache* cache, const int32_t* seq0, int nq, const int32_t* tok0) {
  PrefixLayout L;
  int32_t tp[kMaxSeqs + 1];
  prefix_tokens(seq0, prefix->n_seqs, tok0, tp);
  const int G = nq / cache->n_kv_heads;
  L.shared = attend_layout(prefix, G, tp);
  L.own = attend_layout(cache, G, tok0);
  const size_t rows = (size_t)tok0[cache->n_seqs] * nq, values = up256(rows * cache->head_dim * sizeof(float));
  L.o1 = up256(std::max(L.shared.total, L.own.total));     // (the two run one after the other)
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
  AttendArgs A;
  for (int own = 0; own < 2; ++own) {
    const tria_layer_cache* c = own ? cache : prefix;
    fill_attend(A, c, a);
    A.out = at + (own ? L.o2 : L.o1);
    A.lse = (float*)(at + (own ? L.l2 : L.l1));
    A.out_stride = (int64_t)a->n_q_heads * hd;
    A.out_type = TRIA_F32;
    if (own) A.sink = 0;
    if (run_attend(A, c, own ? a->tok0 : tp, a->round_keys != 0, own ? L.own : L.shared, ws, st) != cudaSuccess) return TRIA_ERR_CUDA;
  }
  JoinArgs J;
  memset(&J, 0, sizeof(J));
  J.o1 = (const float*)(at + L.o1);
  J.o2 = (const float*)(at + L.o2);
  J.l1 = (const float*)(at + L.l1);
  J.l2 = (const float*)(at + L.l2);
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
