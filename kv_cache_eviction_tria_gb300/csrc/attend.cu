// Attention over the cache (tria_attend): argument checks, the split of the
// sequences between the kernels, and the fp32 kernel.
//
//   out(t, h) = sum_r softmax_r(scale q(t, h) . K_r) V_r   over the rows r of
//   KV head h / G that token t sees: r < n_live, pos_r <= p_t and, with a
//   window, p_t - pos_r < window or r < sink.
//
// Positions ascend with the rows, so a token sees a prefix (the sink) and one
// run of rows; only those are read.
//
// A sequence takes one of three kernels. Up to 16 columns (token x query head
// of a KV head's group), as many as the small products have, are a decode step:
// a stream over the rows, bound by memory (attend_step.cuh). More are a prompt:
// products of 128-row tiles on the fifth-generation tensor cores
// (attend_prompt.cu). 4 tokens x 4 heads take 216 us as a step and 242 us as a
// prompt over 8 sequences of 32768 fp16 rows, 54 and 90 us over one of them, 25 and
// 27 us over 777 rows. Over q4_0 rows, which a prompt widens to fp16 first, they take
// 126 and 795 us (567 us with round_keys), 42 and 194 us over one sequence: there a
// step of more columns would win by far, but it is not built.
//
// The fp32 kernel (k_attend_plain) takes fp32 queries or fp32 planes of the
// cache, where results are held to fp32 accuracy, and the head_dims that the
// other two are not built for. A CTA handles a unit of up to 8 columns or one
// part of its rows; each warp walks batches of 4 rows with its own running
// maximum and sum. Dims lie over the lanes, so that a row is read once, in one
// piece, and queries and sums stay in registers; the 32 products of a batch
// (rows x columns) are summed over the lanes by 31 exchanges that leave each
// lane with one logit. The next keys are asked for while a batch is computed.
// About 75 instructions a row bind it: 8 sequences, 206246 fp32 rows (head_dim
// 128, 4 query heads per KV head) take 500 us, 3.4 TB/s; 1024 tokens over their
// own rows 488 us, 18 TFLOP/s. (With tiles in shared memory and a lane per row,
// nine reads of shared memory to eight FMAs, they took 6260 and 2707 us.)
#include <math.h>
#include <string.h>

#include <algorithm>

#include "attend_internal.cuh"

namespace tria {

namespace {

constexpr int kCols = 8;
constexpr int kPlainWarps = 4, kRows = 4;   // rows of a warp at once: rows x columns = lanes
static_assert(kRows * kCols == 32, "a logit per lane");

// Dim e (of 32-wide block j, this lane's) of rows base + off[r] of a plane, as
// fp32; the rows' blocks of 32 dims are read by a warp at a time.
template <int N>
__device__ __forceinline__ void load_rows(const uint8_t* data, const uint8_t* scale, int type, int64_t base, const int* off, int lane,
                                          float (*x)[N]) {
  constexpr int hd = 32 * N;
  if (type == TRIA_F32) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int j = 0; j < N; ++j) x[r][j] = __ldg(reinterpret_cast<const float*>(data) + (base + off[r]) * hd + 32 * j + lane);
  } else if (type == TRIA_F16) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int j = 0; j < N; ++j)
        x[r][j] = __half2float(__ushort_as_half(__ldg(reinterpret_cast<const uint16_t*>(data) + (base + off[r]) * hd + 32 * j + lane)));
  } else {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float d = __half2float(__ushort_as_half(__ldg(reinterpret_cast<const uint16_t*>(scale) + (base + off[r]) * N + j)));
        int c;
        if (type == TRIA_Q8_0) {
          c = __ldg(reinterpret_cast<const int8_t*>(data) + (base + off[r]) * hd + 32 * j + lane);
        } else {
          const int b = __ldg(data + (base + off[r]) * (hd / 2) + 16 * j + (lane & 15));
          c = (lane < 16 ? b & 15 : b >> 4) - 8;
        }
        x[r][j] = (float)c * d;
      }
  }
}

template <int N>
__global__ void __launch_bounds__(kPlainWarps * 32) k_attend_plain(const __grid_constant__ AttendArgs A) {
  constexpr int hd = 32 * N;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float s_o[kCols * hd];
  __shared__ __align__(16) float s_w[kPlainWarps][32];
  __shared__ float s_m[kPlainWarps][kCols], s_l[kPlainWarps][kCols];
  __shared__ int s_last;

  const int part = blockIdx.x % A.split, y = blockIdx.x / A.split;
  const int g = y % A.n_kv, unit = y / A.n_kv;
  int lo_s = 0, hi_s = A.n_seqs - 1;
  while (lo_s < hi_s) {
    const int mid = (lo_s + hi_s + 1) >> 1;
    if (A.seq[mid].unit0 <= unit) lo_s = mid; else hi_s = mid - 1;
  }
  const AttendSeq& S = A.seq[lo_s];
  const int c0 = (unit - S.unit0) * kCols, ncol = min(kCols, S.t * A.G - c0);
  const int n = *((volatile const int32_t*)(A.n_live + lo_s));
  if (n < 0 || n > S.cap) {
    if (threadIdx.x == 0) report(A.ctrl, TRIA_ERR_DEVICE_ARG, (uint32_t)lo_s);
    return;
  }
  const int64_t row0 = S.row0 + (int64_t)g * S.cap;
  const int32_t* rpos = A.cpos + row0;
  int pmin = INT32_MAX, pmax = INT32_MIN;
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    if (c < ncol) {
      const int p = A.pos[S.tok0 + (c0 + c) / A.G];
      pmin = min(pmin, p);
      pmax = max(pmax, p);
    }
  const int hi = rows_upto(rpos, n, pmax);
  const int lo = A.window > 0 ? rows_upto(rpos, hi, (int64_t)pmin - A.window) : 0;
  const int sr = min(A.sink, lo);
  const int R = sr + hi - lo;
  const int v0 = (int)((int64_t)part * R / A.split), v1 = (int)((int64_t)(part + 1) * R / A.split);

  float q[kCols][N], o[kCols][N];
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    const int col = c0 + min(c, ncol - 1);
    const int64_t at = (int64_t)(S.tok0 + col / A.G) * A.q_stride + (int64_t)(g * A.G + col % A.G) * hd + lane;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      q[c][j] = act_load(A.q, A.type, at + 32 * j) * A.scale;
      o[c][j] = 0.f;
    }
  }
  // this lane's logit of a batch: row lane / 8, column lane % 8 (columns past
  // the last one repeat it, and are not written)
  const int my_p = A.pos[S.tok0 + (c0 + min(lane & 7, ncol - 1)) / A.G];
  float M = -INFINITY, l = 0.f;
  auto row_of = [&](int v) { return v < sr ? v : lo + v - sr; };
  auto rows_at = [&](int v, int* off) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) off[r] = row_of(min(v + r, v1 - 1));
  };
  float k[kRows][N];
  int off[kRows], v = v0 + warp * kRows;
  if (v < v1) {
    rows_at(v, off);
    load_rows<N>(A.k, A.ks, A.k_type, row0, off, lane, k);
  }
  for (; v < v1; v += kPlainWarps * kRows) {
    const int my = row_of(min(v + (lane >> 3), v1 - 1)), p = rpos[my];
    float x[kRows][N];
    load_rows<N>(A.v, A.vs, A.v_type, row0, off, lane, x);
    // products of this lane's dims, then their sums: a lane ends with the one of its number
    float s[kRows * kCols];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        s[r * kCols + c] = q[c][0] * k[r][0];
#pragma unroll
        for (int j = 1; j < N; ++j) s[r * kCols + c] = fmaf(q[c][j], k[r][j], s[r * kCols + c]);
      }
    if (v + kPlainWarps * kRows < v1) {                    // the next keys are on their way meanwhile
      rows_at(v + kPlainWarps * kRows, off);
      load_rows<N>(A.k, A.ks, A.k_type, row0, off, lane, k);
    }
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) {
      const bool up = (lane & w) != 0;
#pragma unroll
      for (int i = 0; i < w; ++i) {
        const float give = up ? s[i] : s[i + w], keep = up ? s[i + w] : s[i];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
      }
    }
    const bool see = v + (lane >> 3) < v1 && p <= my_p && (A.window <= 0 || (int64_t)my_p - p < A.window || my < A.sink);
    const float xc = see ? s[0] : -INFINITY;
    float top = fmaxf(xc, __shfl_xor_sync(0xffffffffu, xc, 8));
    top = fmaxf(M, fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)));
    const float base = top == -INFINITY ? 0.f : top;
    if (__any_sync(0xffffffffu, top > M)) {
      const float a = expf(M - base);
      l *= a;
      M = top;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const float ac = __shfl_sync(0xffffffffu, a, c);
#pragma unroll
        for (int j = 0; j < N; ++j) o[c][j] *= ac;
      }
    }
    const float w = see ? expf(xc - base) : 0.f;
    l += w;
    s_w[warp][lane] = w;
    const bool all = __all_sync(0xffffffffu, see);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 w4 = *reinterpret_cast<const float4*>(&s_w[warp][r * kCols + 4 * h]);
        const float wc[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (all || wc[c] != 0.f) {                       // a hidden row's values never count, whatever they are
#pragma unroll
            for (int j = 0; j < N; ++j) o[4 * h + c][j] = fmaf(wc[c], x[r][j], o[4 * h + c][j]);
          }
      }
    __syncwarp();
  }
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  // the warps' results, merged in warp order
  if (lane < kCols) {
    s_m[warp][lane] = M;
    s_l[warp][lane] = l;
  }
  __syncthreads();
  float mt[kCols], lt[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    mt[c] = s_m[0][c];
#pragma unroll
    for (int w = 1; w < kPlainWarps; ++w) mt[c] = fmaxf(mt[c], s_m[w][c]);
    const float base = mt[c] == -INFINITY ? 0.f : mt[c];
    lt[c] = 0.f;
#pragma unroll
    for (int w = 0; w < kPlainWarps; ++w) lt[c] += s_l[w][c] * expf(s_m[w][c] - base);
  }
  for (int w = 0; w < kPlainWarps; ++w) {
    if (warp == w) {
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const float a = expf(s_m[w][c] - (mt[c] == -INFINITY ? 0.f : mt[c]));
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float* d = s_o + c * hd + j * 32 + lane;
          *d = (w ? *d : 0.f) + o[c][j] * a;
        }
      }
    }
    __syncthreads();
  }
  auto write = [&](int c, int e, float val, float top, float sum) {
    const int col = c0 + c, tok = S.tok0 + col / A.G, head = g * A.G + col % A.G;
    act_store(A.out, A.type, (int64_t)tok * A.out_stride + (int64_t)head * hd + e, sum > 0.f || sum != sum ? val / sum : 0.f);
    if (e == 0 && A.lse) A.lse[(int64_t)tok * A.nq + head] = top + logf(sum);
  };
  if (A.split == 1) {
    for (int i = threadIdx.x; i < ncol * hd; i += blockDim.x) {
      const int c = i / hd;
      float top = mt[0], sum = lt[0];
#pragma unroll
      for (int k = 1; k < kCols; ++k)
        if (c == k) {
          top = mt[k];
          sum = lt[k];
        }
      write(c, i - c * hd, s_o[i], top, sum);
    }
    return;
  }
  // a part of the unit: the last of its CTAs to arrive merges the parts in order
  const int pstride = kCols * (hd + 2);
  float* slot = A.part + ((int64_t)y * A.split + part) * pstride;
  for (int i = threadIdx.x; i < kCols * hd; i += blockDim.x) slot[2 * kCols + i] = s_o[i];
  if (threadIdx.x == 0) {
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      slot[c] = mt[c];
      slot[kCols + c] = lt[c];
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(&A.count[y], 1u) == (uint32_t)A.split - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  const float* parts = A.part + (int64_t)y * A.split * pstride;
  for (int i = threadIdx.x; i < ncol * hd; i += blockDim.x) {
    const int c = i / hd;
    float top = -INFINITY, sum = 0.f, val = 0.f;
    for (int k = 0; k < A.split; ++k) top = fmaxf(top, __ldcg(parts + k * pstride + c));
    const float base = top == -INFINITY ? 0.f : top;
    for (int k = 0; k < A.split; ++k) {
      const float a = expf(__ldcg(parts + k * pstride + c) - base);
      sum = fmaf(__ldcg(parts + k * pstride + kCols + c), a, sum);
      val = fmaf(__ldcg(parts + k * pstride + 2 * kCols + i), a, val);
    }
    write(c, i - c * hd, val, top, sum);
  }
  if (threadIdx.x == 0) A.count[y] = 0u;
}

// Rows besides the sink that some token of a sequence sees in each segment: a
// warp per segment searches the positions in 32 parts (three rounds for 4096
// candidates), since every CTA of the attention needs the count of every one.
__global__ void __launch_bounds__(128) k_attend_span(const __grid_constant__ AttendArgs A, int32_t* span) {
  const int u = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (u >= A.n_seqs * A.n_kv) return;
  const int s = u / A.n_kv, g = u - s * A.n_kv;
  const AttendSeq& S = A.seq[s];
  const int n = *((volatile const int32_t*)(A.n_live + s));
  if (S.t == 0 || n < 0 || n > S.cap) return;
  const int32_t* rpos = A.cpos + S.row0 + (int64_t)g * S.cap;
  int pl = INT32_MAX, ph = INT32_MIN;
  for (int i = lane; i < S.t; i += 32) {
    const int p = A.pos[S.tok0 + i];
    pl = min(pl, p);
    ph = max(ph, p);
  }
  const int last = n > 0 ? rpos[n - 1] : 0;
  pl = __reduce_min_sync(0xffffffffu, pl);
  ph = __reduce_max_sync(0xffffffffu, ph);
  auto upto = [&](int lo, int hi, int64_t p) {   // rows with a position <= p, between lo and hi of them
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32;
      const int r = min(hi, lo + (lane + 1) * step) - 1;   // last row of this lane's share
      const int k = __popc(__ballot_sync(0xffffffffu, rpos[r] <= p));
      lo = min(hi, lo + k * step);
      if (k < 32) hi = min(hi, lo + step - 1);
    }
    return lo;
  };
  const int hi = n == 0 || last <= ph ? n : upto(0, n, ph);
  // positions ascend strictly, so at most window + (ph - pl) rows lie in reach
  const int lo = upto((int)max((int64_t)0, hi - (A.window + (int64_t)ph - pl)), hi, (int64_t)pl - A.window);
  if (lane == 0) {
    span[2 * u] = lo;
    span[2 * u + 1] = hi;
  }
}

}  // namespace

cudaError_t launch_attend_plain(const AttendArgs& A, cudaStream_t st) {
  const int64_t grid = (int64_t)A.units * A.n_kv * A.split;
  if (grid == 0) return cudaSuccess;
  using Fn = void (*)(AttendArgs);
  static constexpr Fn fn[TRIA_MAX_HEAD_DIM / 32] = {k_attend_plain<1>, k_attend_plain<2>, k_attend_plain<3>, k_attend_plain<4>,
                                                    k_attend_plain<5>, k_attend_plain<6>, k_attend_plain<7>, k_attend_plain<8>};
  fn[A.hd / 32 - 1]<<<(unsigned)grid, kPlainWarps * 32, 0, st>>>(A);
  return cudaGetLastError();
}

cudaError_t launch_attend_span(const AttendArgs& A, int32_t* span, cudaStream_t st) {
  k_attend_span<<<(A.n_seqs * A.n_kv + 3) / 4, 128, 0, st>>>(A, span);
  return cudaGetLastError();
}

}  // namespace tria

using namespace tria;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Which kernel a sequence of t tokens takes.
enum { kPathNone, kPathPlain, kPathStep, kPathPrompt };

bool tensor_types(const tria_layer_cache* c, int type) {
  return type != TRIA_F32 && c->k_type != TRIA_F32 && c->v_type != TRIA_F32 &&
         c->head_dim >= 64;
}

// (The prompt kernel's tiles are 64 dims wide at least, narrower planes would
// be mostly padding.) The decode kernel is built for these head_dims; few tokens of other ones take
// the fp32 kernel.
bool step_dims(int hd) { return hd == 64 || hd == 96 || hd == 128 || hd == 256; }

int path_of(bool tensor, int hd, int t, int G) {
  if (t == 0) return kPathNone;
  if (!tensor) return kPathPlain;
  if (prompt_cols_reached(t, G)) return kPathPrompt;
  return step_dims(hd) ? kPathStep : kPathPlain;
}

// The kernels of a call run one after the other and share the arrival counters
// and the space of the partial results. The layout covers every type of
// queries. The counters, which have to be zero between calls, take the same
// place for every shape, so that a workspace may serve calls of different
// shapes: a decode step counts segments, the fp32 kernel the units that it
// splits, at most kMaxSegments both.
struct AttendLayout {
  size_t count, span, part, wide_k, wide_kl, wide_v, total;
  int split, prompt_split, sms;
};

// Parts of a unit of a prompt: as many as make the last wave of CTAs (one per
// SM) full, each part costing a share of a fixed start and of the merge; none
// under 512 rows of the capacity.
int prompt_split(int64_t units, int cap_max, int sms) {
  if (units == 0) return 1;
  int best = 1;
  double least = 1e30;
  for (int k = 1; k <= 16 && (k == 1 || (int64_t)k * 512 <= cap_max); ++k) {
    if (k > 1 && units * k > 2 * sms) break;
    const double t = (double)((units * k + sms - 1) / sms) / k + 0.02 * k;
    if (t < least - 1e-9) {
      least = t;
      best = k;
    }
  }
  return best;
}

AttendLayout attend_layout(const tria_layer_cache* c, int G, const int32_t* tok0) {
  AttendLayout L{};
  int64_t units = 0, prompts = 0;
  int cap_max = 0, cols = 0;
  for (int s = 0; s < c->n_seqs; ++s) {
    const int64_t x = (int64_t)(tok0[s + 1] - tok0[s]) * G;
    units += (x + kCols - 1) / kCols;
    if (x <= kStepCols) cols = std::max(cols, (int)x);
    else prompts += (x + prompt_cols(c->head_dim) - 1) / prompt_cols(c->head_dim);
    cap_max = std::max(cap_max, c->capacity[s]);
  }
  L.sms = sm_count();
  L.split = plain_split(units * c->n_kv_heads, cap_max, L.sms, kMaxSegments);
  L.count = up256(sizeof(Ctrl));
  L.span = up256(L.count + sizeof(uint32_t) * (size_t)kMaxSegments);
  L.part = up256(L.span + 2 * sizeof(int32_t) * (size_t)c->n_seqs * c->n_kv_heads);
  const size_t plain = L.split > 1 ? (size_t)(units * c->n_kv_heads) * L.split * kCols * (c->head_dim + 2) : 0;
  // a part a warp (at most 12 a CTA) and two a CTA
  const size_t step = (size_t)L.sms * 14 * (cols <= 8 ? 8 : 16) * (c->head_dim + 2);
  L.prompt_split = prompt_split(prompts * c->n_kv_heads, cap_max, L.sms);
  const size_t prompt = L.prompt_split > 1
      ? (size_t)(prompts * c->n_kv_heads) * L.prompt_split * prompt_cols(c->head_dim) * (prompt_dims(c->head_dim) + 2) : 0;
  L.wide_k = up256(L.part + sizeof(float) * std::max(std::max(plain, step), prompt));
  const int64_t wide = widened_rows(c->n_seqs, c->n_kv_heads, G, c->capacity, tok0, nullptr);
  const size_t plane = up256((size_t)wide * c->head_dim * 2);
  const bool tensor = tensor_types(c, TRIA_F16);
  const size_t keys = tensor && c->k_type != TRIA_F16 ? plane : 0;
  L.wide_kl = L.wide_k + keys;
  L.wide_v = L.wide_kl + keys;
  L.total = L.wide_v + (tensor && c->v_type != TRIA_F16 ? plane : 0);
  return L;
}

cudaError_t launch_step(const AttendArgs& A, int cols, int workers, cudaStream_t st) {
  using Fn = cudaError_t (*)(const AttendArgs&, int, int, cudaStream_t);
  static constexpr Fn fn[3][3] = {
      {launch_attend_step_f16_f16, launch_attend_step_f16_q8, launch_attend_step_f16_q4},
      {launch_attend_step_q8_f16, launch_attend_step_q8_q8, launch_attend_step_q8_q4},
      {launch_attend_step_q4_f16, launch_attend_step_q4_q8, launch_attend_step_q4_q4}};
  static_assert(TRIA_F16 == 1 && TRIA_Q8_0 == 2 && TRIA_Q4_0 == 3, "table order");
  return fn[A.k_type - 1][A.v_type - 1](A, cols, workers, st);
}

tria_status check_attend_shape(const tria_layer_cache* c, int n_q_heads, const int32_t* tok0) {
  tria_status r;
  if ((r = check_cache(c)) != TRIA_OK) return r;
  if (!tok0 || n_q_heads < 1) return TRIA_ERR_INVALID_ARG;
  if (n_q_heads % c->n_kv_heads != 0 || n_q_heads / c->n_kv_heads > TRIA_MAX_GROUP) return TRIA_ERR_UNSUPPORTED;
  if ((r = check_tokens(tok0, c->n_seqs)) != TRIA_OK) return r;
  // columns (token x head) are counted in 32 bits
  return (int64_t)tok0[c->n_seqs] * n_q_heads < ((int64_t)1 << 31) ? TRIA_OK : TRIA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" size_t tria_attend_workspace_size(const tria_layer_cache* cache, int32_t n_q_heads, const int32_t* tok0) {
  if (check_attend_shape(cache, n_q_heads, tok0) != TRIA_OK) return 0;
  return attend_layout(cache, n_q_heads / cache->n_kv_heads, tok0).total;
}

extern "C" tria_status tria_attend(const tria_layer_cache* cache, const tria_attention* a, void* ws, size_t ws_bytes,
                                   void* stream) {
  tria_status r;
  if (!a) return TRIA_ERR_INVALID_ARG;
  if ((r = check_attend_shape(cache, a->n_q_heads, a->tok0)) != TRIA_OK) return r;
  if (!act_ok(a->type)) return TRIA_ERR_UNSUPPORTED;
  if (a->window < 0 || a->sink < 0 || !(a->scale >= 0.0) || !isfinite((float)a->scale)) return TRIA_ERR_INVALID_ARG;
  if (a->round_keys != 0 && a->round_keys != 1) return TRIA_ERR_INVALID_ARG;
  const int hd = cache->head_dim, nq = a->n_q_heads, n_tokens = a->tok0[cache->n_seqs];
  const int size = a->type == TRIA_F32 ? 4 : 2;
  if (n_tokens > 0) {
    if (!a->q || !a->out || !a->pos || !aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->pos, 4) ||
        (a->lse && !aligned(a->lse, 4)))
      return TRIA_ERR_INVALID_ARG;
    if (a->q_stride < (int64_t)nq * hd || a->out_stride < (int64_t)nq * hd || (a->q_stride * size) % 16 != 0 ||
        (a->out_stride * size) % 16 != 0)
      return TRIA_ERR_INVALID_ARG;
  }
  const int G = nq / cache->n_kv_heads;
  const AttendLayout L = attend_layout(cache, G, a->tok0);
  if (!ws || !aligned(ws, 256) || ws_bytes < L.total) return TRIA_ERR_WORKSPACE;
  if (n_tokens == 0) return TRIA_OK;
  AttendArgs A;
  memset(&A, 0, sizeof(A));
  A.q = a->q;
  A.out = a->out;
  A.lse = a->lse;
  A.pos = a->pos;
  A.q_stride = a->q_stride;
  A.out_stride = a->out_stride;
  A.k = (const uint8_t*)cache->k;
  A.ks = (const uint8_t*)cache->k_scale;
  A.v = (const uint8_t*)cache->v;
  A.vs = (const uint8_t*)cache->v_scale;
  A.cpos = cache->pos;
  A.n_live = cache->n_live;
  A.ctrl = (Ctrl*)ws;
  A.count = (uint32_t*)((uint8_t*)ws + L.count);
  A.part = (float*)((uint8_t*)ws + L.part);
  A.n_seqs = cache->n_seqs;
  A.n_kv = cache->n_kv_heads;
  A.G = G;
  A.hd = hd;
  A.nq = nq;
  A.type = a->type;
  A.k_type = cache->k_type;
  A.v_type = cache->v_type;
  A.window = a->window;
  A.sink = a->sink;
  A.scale = (float)(a->scale != 0.0 ? a->scale : 1.0 / sqrt((double)hd));
  const bool tensor = tensor_types(cache, a->type);
  int units = 0, cols = 0;
  bool plain = false, step = false, prompt = false;
  for (int s = 0; s < cache->n_seqs; ++s) {
    A.seq[s].row0 = cache->seq_row0[s];
    A.seq[s].cap = cache->capacity[s];
    A.seq[s].tok0 = a->tok0[s];
    const int t = a->tok0[s + 1] - a->tok0[s], path = path_of(tensor, hd, t, G);
    plain = plain || path == kPathPlain;
    prompt = prompt || path == kPathPrompt;
    if (path == kPathStep) {
      step = true;
      cols = std::max(cols, t * G);
    }
  }
  if (prompt)   // a row of a TMA tile has a signed 32-bit coordinate
    for (int s = 0; s < cache->n_seqs; ++s)
      if (cache->seq_row0[s] + (int64_t)cache->n_kv_heads * cache->capacity[s] >= ((int64_t)1 << 31)) return TRIA_ERR_UNSUPPORTED;
  // each kernel sees the sequences it takes, the others without tokens
  auto take = [&](int path) {
    const int per = path == kPathPrompt ? prompt_cols(hd) : kCols;
    units = 0;
    for (int s = 0; s < cache->n_seqs; ++s) {
      const int t = a->tok0[s + 1] - a->tok0[s];
      A.seq[s].t = path_of(tensor, hd, t, G) == path ? t : 0;
      A.seq[s].unit0 = units;
      units += (A.seq[s].t * G + per - 1) / per;
    }
    A.units = units;
  };
  const cudaStream_t st = (cudaStream_t)stream;
  if (step) {
    take(kPathStep);
    if (A.window > 0) {
      int32_t* span = (int32_t*)((uint8_t*)ws + L.span);
      if (launch_attend_span(A, span, st) != cudaSuccess) return TRIA_ERR_CUDA;
      A.span = span;
    }
    if (launch_step(A, cols, L.sms, st) != cudaSuccess) return TRIA_ERR_CUDA;
  }
  if (prompt) {
    take(kPathPrompt);
    A.split = L.prompt_split;
    int64_t first[kMaxSeqs];
    A.wide_rows = widened_rows(cache->n_seqs, cache->n_kv_heads, G, cache->capacity, a->tok0, first);
    for (int s = 0; s < cache->n_seqs; ++s) A.seq[s].wide0 = first[s];
    if (cache->k_type != TRIA_F16) {
      A.wide_k = (uint16_t*)((uint8_t*)ws + L.wide_k);
      if (!a->round_keys) A.wide_kl = (uint16_t*)((uint8_t*)ws + L.wide_kl);
    }
    if (cache->v_type != TRIA_F16) A.wide_v = (uint16_t*)((uint8_t*)ws + L.wide_v);
    if (launch_attend_prompt(A, st) != cudaSuccess) return TRIA_ERR_CUDA;
  }
  if (plain) {
    take(kPathPlain);
    A.split = L.split;
    if (launch_attend_plain(A, st) != cudaSuccess) return TRIA_ERR_CUDA;
  }
  return TRIA_OK;
}
