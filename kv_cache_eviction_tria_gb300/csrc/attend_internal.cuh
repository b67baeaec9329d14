// Declarations shared by the operators around the cache: rotation and append
// (rope.cu) and attention (attend*.cu).
#pragma once

#include <cuda_bf16.h>

#include <atomic>
#include <new>

#include "attend_plan.h"
#include "tria_internal.cuh"

// Opaque rotation handle of the C ABI.
struct tria_rope {
  int32_t head_dim, nonrot_dim, layout;
  double mscale;
  unsigned long long* turns;   // [rot / 2] device: frac(w_f / 2 pi) * 2^64
};

namespace tria {

inline bool act_ok(int type) { return type == TRIA_F32 || type == TRIA_F16 || type == TRIA_BF16; }

// Token offsets of the sequences of a call: tok0[0] = 0, not descending.
inline tria_status check_tokens(const int32_t* tok0, int n_seqs) {
  if (tok0[0] != 0) return TRIA_ERR_INVALID_ARG;
  for (int s = 0; s < n_seqs; ++s)
    if (tok0[s + 1] < tok0[s]) return TRIA_ERR_INVALID_ARG;
  return TRIA_OK;
}

// SMs of the current device (without a device, of a whole GB300). Asked once a
// device: calls that take microseconds need it each time.
inline int sm_count() {
  static std::atomic<int> known[16];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 152;
  if (dev < 16 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
  if (dev < 16) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// One attention call, passed by value.
struct AttendSeq {
  int64_t row0;
  int64_t wide0;      // first of its rows in the widened planes
  int32_t cap;
  int32_t tok0;       // first token of the sequence in q / out / pos
  int32_t t;          // its tokens
  int32_t unit0;      // units (see the kernels) of the sequences before it
};

struct AttendArgs {
  const void* q;
  void* out;
  float* lse;
  const int32_t* pos;
  int64_t q_stride, out_stride;
  const uint8_t* k;
  const uint8_t* ks;
  const uint8_t* v;
  const uint8_t* vs;
  const int32_t* cpos;
  const int32_t* n_live;
  Ctrl* ctrl;
  uint32_t* count;     // arrivals per unit, zero between calls
  float* part;         // partial results of split units
  int32_t* table;      // first tile of each unit, and the number of tiles (attend_group.cu)
  uint16_t* wide_k;    // fp16 copies of quantised planes (prompts; NULL: none)
  uint16_t* wide_kl;   // what fp16 leaves of the keys (NULL: not taken into account)
  uint16_t* wide_v;
  int64_t wide_rows;   // of each of them (widened_rows)
  const int32_t* span; // decode steps with a window: [sequence][KV head] {first, past the last} row that a token sees
  int32_t n_seqs, n_kv, G, hd, nq;
  int32_t type, k_type, v_type;
  int32_t out_type;    // type, or F32 where results are joined with others
  int32_t window, sink;
  int32_t units;       // units of one KV head over all sequences
  int32_t split;       // parts a unit is cut into
  float scale;         // logits are scale * q . k
  AttendSeq seq[kMaxSeqs];
};

// The kernels of a call run one after the other and share the arrival counters
// and the space of the partial results. The layout covers every type of
// queries. The counters lie at kCountersAt, whatever the shape: a decode step counts
// segments, the fp32 kernel the units that it splits, at most kMaxSegments both.
struct AttendLayout {
  size_t count, span, part, wide_k, wide_kl, wide_v, total;
  int split, prompt_split, sms;
};

// attend.cu: checks of a call, its layout and its kernels over one cache
tria_status check_attend_shape(const tria_layer_cache* c, int n_q_heads, const int32_t* tok0);
tria_status check_attention(const tria_attention* a, int n_tokens, int hd);
tria_status check_attend_rows(const tria_layer_cache* c, int G, const int32_t* tok0, int type);
AttendLayout attend_layout(const tria_layer_cache* c, int G, const int32_t* tok0);
bool tensor_types(const tria_layer_cache* c, int type);   // whether the tensor-core kernels take them
void fill_attend(AttendArgs& A, const tria_layer_cache* cache, const tria_attention* a);
cudaError_t run_attend(AttendArgs& A, const tria_layer_cache* cache, const int32_t* tok0, bool round_keys, const AttendLayout& L, void* ws,
                       cudaStream_t st);
cudaError_t launch_attend_plain(const AttendArgs& A, cudaStream_t st);
cudaError_t launch_attend_span(const AttendArgs& A, int32_t* span, cudaStream_t st);
// attend_step_*.cu: up to 16 columns (tokens x group) a sequence, one CTA per worker
cudaError_t launch_attend_step_f16_f16(const AttendArgs& A, int cols, int workers, cudaStream_t st);
cudaError_t launch_attend_step_f16_q8(const AttendArgs& A, int cols, int workers, cudaStream_t st);
cudaError_t launch_attend_step_f16_q4(const AttendArgs& A, int cols, int workers, cudaStream_t st);
cudaError_t launch_attend_step_q8_f16(const AttendArgs& A, int cols, int workers, cudaStream_t st);
cudaError_t launch_attend_step_q8_q8(const AttendArgs& A, int cols, int workers, cudaStream_t st);
cudaError_t launch_attend_step_q8_q4(const AttendArgs& A, int cols, int workers, cudaStream_t st);
cudaError_t launch_attend_step_q4_f16(const AttendArgs& A, int cols, int workers, cudaStream_t st);
cudaError_t launch_attend_step_q4_q8(const AttendArgs& A, int cols, int workers, cudaStream_t st);
cudaError_t launch_attend_step_q4_q4(const AttendArgs& A, int cols, int workers, cudaStream_t st);
// attend_prompt.cu: tiles of prompt_dims(hd) dims, units of prompt_cols(hd) columns
inline int prompt_dims(int hd) { return hd <= 64 ? 64 : (hd <= 128 ? 128 : 256); }
inline int prompt_cols(int hd) { return hd > 128 ? 128 : 256; }
cudaError_t launch_attend_prompt(const AttendArgs& A, cudaStream_t st);

// attend_group.cu: units of 128 columns of a prefix and KV head (A.units of all of
// them), a part of group_part_values(hd) values a unit and CTA; the own rows'
// sequences for the join
struct GroupOwn {
  int32_t n_seqs;
  int32_t tok0[kMaxSeqs], cap[kMaxSeqs];
};
size_t group_part_values(int hd);
cudaError_t launch_attend_group(const AttendArgs& A, bool round_keys, int grid, cudaStream_t st);
cudaError_t launch_join_group(const AttendArgs& A, const float* o2, const float* l2, const int32_t* own_live, const GroupOwn& own, int grid,
                              cudaStream_t st);

__device__ __forceinline__ float act_load(const void* p, int type, int64_t i) {
  if (type == TRIA_F32) return reinterpret_cast<const float*>(p)[i];
  if (type == TRIA_F16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ void act_store(void* p, int type, int64_t i, float x) {
  if (type == TRIA_F32)
    reinterpret_cast<float*>(p)[i] = x;
  else if (type == TRIA_F16)
    reinterpret_cast<__half*>(p)[i] = __float2half_rn(x);
  else
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
}

// rows [0, n) with pos <= p (positions ascend with the rows)
__device__ __forceinline__ int rows_upto(const int32_t* pos, int n, int64_t p) {
  if (n == 0 || pos[n - 1] <= p) return n;
  int lo = 0, hi = n - 1;            // pos[hi] > p
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pos[mid] <= p) lo = mid + 1; else hi = mid;
  }
  return lo;
}

}  // namespace tria
