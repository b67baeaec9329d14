// The best continuations of groups of beams (tria_beam_select): one step of
// beam search, from the logits to the chosen (beam, token) pairs.
//
//   v(b, t) = total_b + x_bt - ln sum_u exp(x_bu), the n_out largest of a group
//
// One pass over the logits: a CTA takes a part of a beam's row in pieces that
// its registers hold, and from it the largest logit, the sum of exponentials
// relative to it and the part's n_out best tokens (within a beam the order is the
// logits', so they are found before the sum is known; where v in 64 bits does not tell two
// of a beam's logits apart, they still do). The last CTA of a
// group to arrive adds the sums up and chooses among the parts' lists; the CTAs
// write 8 + 8 n_out bytes each, against 16 KB or more read.
//
// Choosing k of many: of 32 or 128 runs of threads' values (at least k), the
// k-th largest of their best values is a bound that k values reach. The few
// that do (about runs ln(runs / (runs - k)) of random ones) go to a list in
// shared memory and are ranked by counting, with their index (the smaller one
// first), so that no two are equal and the result does not depend on the order
// of arrival. Where more reach the bound than the list holds, it is taken
// again with the indices (ties: a masked vocabulary), and where that leaves too
// many (large values on few threads) the best are taken one after the other.
// A part's later pieces are held against the first one's bound, without meeting
// the other threads. The parts' lists are sorted, so the last CTA bounds their first
// entries and reads on in the few lists that reach that.
//
// Sums: exponentials (of differences from the largest logit, 4 units of 2^-24)
// and their sums in fp32, the logarithm and v in fp64. A thread has the same
// tokens of a row whatever its alignment, so equal rows have equal sums, bit by
// bit, and equal candidates of two beams stay equal.
//
// 128 beams of 151936 bf16 logits, 8 chosen of 8: 25 us, 39 MB (512 CTAs, five pieces each); 108
// beams of 50021 fp32 logits, 64 chosen of up to 32: 33 us; 4 beams of 32000 fp16 logits: 10 us. Neither memory
// (0.17 of its rate) nor instructions (0.4 of the issue slots) are the bound but the steps that
// wait for one another: a piece's loads, its largest value, the bound, the list, the ranking,
// then the last CTA's merge; a kernel's start and end are half of the smallest call.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "attend_internal.cuh"

namespace tria {

namespace {

constexpr int kSelThreads = 256, kHeld = 32;               // logits of a thread
constexpr int kMaxOut = TRIA_MAX_CHOICES, kMaxBeams = TRIA_MAX_BEAMS;
constexpr int kList = 1024;                                // candidates ranked by counting
constexpr float kLog2e = 1.4426950408889634f;
// a continuation among equal values: beam, then logit, then token
constexpr int kTokenBits = 19, kBeamAt = kTokenBits + 32;
static_assert(TRIA_MAX_VOCAB <= 1 << kTokenBits && kMaxBeams <= 1 << (64 - kBeamAt), "a continuation's place has 64 bits");

struct BeamArgs {
  const void* logits;
  int64_t stride;
  const float* total;
  const int32_t* ended;
  float* total_out;
  int32_t* parent_out;
  int32_t* token_out;
  int32_t* ended_out;
  uint32_t* count;      // [groups] arrivals, zero between calls
  float2* part;         // [beams][parts] {largest logit, sum of 2^((x - it) log2 e): NaN where a logit is NaN or +inf}
  uint2* best;          // [beams][parts][n_out] {ordered logit (0: none), token}, best first
  int32_t vocab, n_out, n_groups, end_token, in_place;
  int32_t held, per, parts;   // logits of a thread at a time, how many times, CTAs of a row
  int32_t vec;          // rows start on 16-byte boundaries
  int32_t seq0[kMaxSeqs + 1];
};

// floats by size, -0 as 0 (no NaN): larger keys are larger floats, none is 0
__device__ __forceinline__ uint32_t order32(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_order32(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k); }
__device__ __forceinline__ uint64_t order64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double from_order64(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? k ^ 0x8000000000000000ull : ~k));
}

__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Candidate: key (0: none) and place among equal ones; before(a, b): a is the better one.
struct Cand {
  uint64_t key;
  uint64_t at;
};
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) { return a.key > b.key || (a.key == b.key && a.at < b.at); }
__device__ __forceinline__ Cand from_lane(const Cand& x, int o) {      // of the lane whose number differs in bit o
  return {__shfl_xor_sync(0xffffffffu, x.key, o), __shfl_xor_sync(0xffffffffu, x.at, o)};
}

struct Choose {
  Cand run[128];
  Cand list[kList];
  Cand out[kMaxOut];
  Cand warp_best[kSelThreads / 32];
  __align__(16) float top[128];       // of runs of threads, as values alone
  __align__(16) uint32_t least[4];
  uint16_t some[kList];       // lists that reach the bound
  Cand bound;
  int n, n_some;
};

// The want-th largest of the runs' largest values (-inf where there are fewer),
// `top` being this thread's: at least `want` values of the threads reach it.
__device__ __forceinline__ float find_least(Choose& C, int want, float top) {
  const int tid = threadIdx.x, lane = tid & 31, runs = want <= 16 ? 32 : 128;
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  if (runs == 32) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
    if ((tid & 7) == 0) C.top[tid >> 3] = top;
  } else if ((tid & 1) == 0) {
    C.top[tid >> 1] = top;
  }
  __syncthreads();
  // the smallest value that fewer than `want` others exceed: of 32 runs every warp
  // finds it for itself, of 128 the first four warps share them
  if (runs == 32 || tid < runs) {
    const float v = C.top[runs == 32 ? lane : tid];
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < runs; j += 4) {
      const float4 y = *reinterpret_cast<const float4*>(C.top + j);
      above += (y.x > v) + (y.y > v) + (y.z > v) + (y.w > v);
    }
    const uint32_t least = __reduce_min_sync(0xffffffffu, above < want ? order32(v) : 0xFFFFFFFFu);
    if (runs == 32) return from_order32(least);
    if (lane == 0) C.least[tid >> 5] = least;
  }
  __syncthreads();
  const uint4 y = *reinterpret_cast<const uint4*>(C.least);
  return from_order32(min(min(y.x, y.y), min(y.z, y.w)));
}

// The candidates in C.list (n <= kList, the same in all threads), best first,
// into C.out. Many are first held against a bound of their own: counting takes
// as long as there are candidates. worth(): values that keep the order.
template <typename Worth>
__device__ __forceinline__ int rank_list(Choose& C, int n, int want, Worth worth) {
  const int tid = threadIdx.x;
  if (n > 2 * want && n > 64) {
    Cand mine[kList / kSelThreads];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kList / kSelThreads; ++k)
      if (k * kSelThreads + tid < n) {
        mine[k] = C.list[k * kSelThreads + tid];
        top = fmaxf(top, worth(mine[k]));
      }
    const float least = find_least(C, want, top);          // (meets the others: every candidate has been read)
    if (tid == 0) C.n = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kList / kSelThreads; ++k)
      if (k * kSelThreads + tid < n && worth(mine[k]) >= least) C.list[atomicAdd(&C.n, 1)] = mine[k];
    __syncthreads();
    n = C.n;
  }
  for (int i = tid; i < n; i += kSelThreads) {
    const Cand x = C.list[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += before(C.list[j], x);
    if (rank < want) C.out[rank] = x;
  }
  __syncthreads();
  return min(n, want);
}

// Into C.bound: the want-th best of the runs' best candidates (runs without one
// rank by their number), `mine` being this thread's.
__device__ __forceinline__ void find_bound(Choose& C, int want, Cand mine) {
  const int tid = threadIdx.x, runs = want <= 16 ? 32 : 128, of = kSelThreads / runs;   // of: threads of a run
  for (int o = 1; o < of; o <<= 1) {
    const Cand y = from_lane(mine, o);
    if (before(y, mine)) mine = y;
  }
  if (tid % of == 0) C.run[tid / of] = mine;
  __syncthreads();
  if (tid < runs) {
    const Cand x = C.run[tid];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < runs; ++j) {
      const Cand y = C.run[j];
      rank += before(y, x) || (y.key == x.key && y.at == x.at && j < tid);
    }
    if (rank == want - 1) C.bound = x;
  }
  __syncthreads();
}

// The best `want` of the candidates that each(f) shows to f, thread by thread
// and the same ones at every call, into C.out, best first; returns how many
// there are (fewer when there are no more). `mine`: this thread's best one. All
// threads of the CTA take part; any order, any ties.
template <typename Each, typename Worth>
__device__ __forceinline__ int choose(Choose& C, int want, Cand mine, Each each, Worth worth) {
  const int tid = threadIdx.x, lane = tid & 31;
  __syncthreads();
  if (tid == 0) C.n = 0;
  find_bound(C, want, mine);
  const Cand bound = C.bound;
  each([&](uint64_t key, uint64_t at) {
    const Cand x = {key, at};
    if (key == 0 || before(bound, x)) return;
    const int i = atomicAdd(&C.n, 1);
    if (i < kList) C.list[i] = x;
  });
  __syncthreads();
  const int n = C.n;
  if (n <= kList) return rank_list(C, n, want, worth);
  Cand last = {~0ull, 0};                                  // every candidate comes after it
  for (int k = 0; k < want; ++k) {
    Cand top = {0, ~0ull};
    each([&](uint64_t key, uint64_t at) {
      const Cand x = {key, at};
      if (key != 0 && before(last, x) && before(x, top)) top = x;
    });
    for (int o = 1; o < 32; o <<= 1) {
      const Cand y = from_lane(top, o);
      if (before(y, top)) top = y;
    }
    if (lane == 0) C.warp_best[tid >> 5] = top;
    __syncthreads();
    top = C.warp_best[0];
    for (int w = 1; w < kSelThreads / 32; ++w)
      if (before(C.warp_best[w], top)) top = C.warp_best[w];
    if (tid == 0) C.out[k] = top;
    __syncthreads();
    if (top.key == 0) return k;
    last = top;
  }
  return want;
}

template <typename T>
__device__ __forceinline__ float to_float(T x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __half>) return __half2float(x);
  else return __bfloat162float(x);
}

template <typename T>
__global__ void __launch_bounds__(kSelThreads, 4) k_beam_select(const __grid_constant__ BeamArgs A) {
  constexpr int N = 16 / sizeof(T), V = kHeld / N;         // values of a load, loads of a thread
  __shared__ Choose C;
  __shared__ double s_base[kMaxBeams];
  __shared__ float s_top[kSelThreads / 32], s_sum[kSelThreads / 32];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int beam = blockIdx.x / A.parts, part = blockIdx.x - beam * A.parts;
  const int held = A.held, piece = held * kSelThreads;     // tokens of a thread and of the CTA at a time
  const int from = part * A.per * piece, end = min(from + A.per * piece, A.vocab);
  const bool over = A.ended && A.ended[beam] != 0;
  const T* row = reinterpret_cast<const T*>(A.logits) + (int64_t)beam * A.stride;
  const bool ends = over && A.end_token >= from && A.end_token < end;   // its one continuation lies in the part
  if (tid == 0) {
    C.n = ends;
    if (ends) C.list[0] = {order32(0.f), (uint32_t)A.end_token};
  }
  // ---- the part, piece by piece: the warps' largest logits, the threads' sums relative to them, and the logits
  // that reach the first piece's bound
  float wtop = -INFINITY, sum = 0.f, least = 0.f;
#pragma unroll 1
  for (int first = over ? end : from; first < end; first += piece) {
    // value e of load j of a thread is token first + (j * 256 + tid) * N + e
    float x[kHeld];
    auto token = [&](int i) { return first + ((i / N) * kSelThreads + tid) * N + i % N; };
    if (A.vec && first + piece <= end) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (j * N < held) w = __ldcs(reinterpret_cast<const uint4*>(row + token(j * N)));
        const T* y = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int e = 0; e < N; ++e) x[j * N + e] = j * N < held ? to_float(y[e]) : -INFINITY;
      }
    } else {                                               // a row's last piece, or rows that start anywhere
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        x[i] = -INFINITY;
        if (i < held && token(i) < end) x[i] = to_float(row[token(i)]);
      }
    }
    float most[4];                                         // of eight values each
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      most[k] = x[8 * k];
#pragma unroll
      for (int i = 1; i < 8; ++i) most[k] = fmaxf(most[k], x[8 * k + i]);
    }
    const float top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
    float now = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
    if (now > wtop) {
      sum *= exp2_ftz((wtop - now) * kLog2e);
      wtop = now;
    }
    // (a NaN or +inf makes the sum NaN, nothing else does)
    const float base = wtop == -INFINITY ? 0.f : wtop;
    float2 sums = make_float2(sum, 0.f);
#pragma unroll
    for (int i = 0; i < kHeld; i += 2) {
      float2 e = __fmul2_rn(__fadd2_rn(make_float2(x[i], x[i + 1]), make_float2(-base, -base)), make_float2(kLog2e, kLog2e));
      e.x = exp2_ftz(e.x);
      e.y = exp2_ftz(e.y);
      sums = __fadd2_rn(sums, e);
    }
    sum = sums.x + sums.y;
    if (first == from) least = find_least(C, A.n_out, top);
    if (top >= least && top > -INFINITY) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (most[k] >= least) {
#pragma unroll
          for (int i = 8 * k; i < 8 * k + 8; ++i)
            if (x[i] >= least && x[i] > -INFINITY) {
              const int place = atomicAdd(&C.n, 1);
              if (place < kList) C.list[place] = {order32(x[i]), (uint32_t)token(i)};
            }
        }
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    s_top[warp] = ends ? 0.f : wtop;
    s_sum[warp] = ends ? 1.f : sum;                        // (of a beam that is over, anything but NaN)
  }
  __syncthreads();
  const int want = min(A.n_out, end - from);
  auto logit = [](const Cand& y) { return from_order32((uint32_t)y.key); };
  int n = C.n;
  if (n <= kList) {
    n = rank_list(C, n, A.n_out, logit);
    if (n < want) {
      // the others are -inf, the first ones of them: among so many tokens there are enough
      const int t = from + tid;
      const bool none = tid < want + n && t < end && (over ? t != A.end_token : to_float(row[t]) == -INFINITY);
      const uint32_t those = __ballot_sync(0xffffffffu, none);
      if (lane == 0 && warp < 4) C.least[warp] = __popc(those);   // (want + n < 128)
      __syncthreads();
      int place = n + __popc(those & ((1u << lane) - 1u));
      for (int w = 0; w < min(warp, 3); ++w) place += C.least[w];
      if (none && place < want) C.out[place] = {order32(-INFINITY), (uint32_t)t};
      n = want;
      __syncthreads();
    }
  } else {                                                 // ties, or large values on few threads
    auto each = [&](auto f) {
#pragma unroll 1
      for (int t = from + tid; t < end; t += kSelThreads) f(order32(to_float(row[t])), (uint32_t)t);
    };
    Cand mine = {0, 0};
    each([&](uint64_t key, uint64_t at) {
      const Cand y = {key, at};
      if (before(y, mine)) mine = y;
    });
    n = choose(C, A.n_out, mine, each, logit);
  }
  uint2* best = A.best + (int64_t)blockIdx.x * A.n_out;
  for (int i = tid; i < A.n_out; i += kSelThreads) best[i] = i < n ? make_uint2((uint32_t)C.out[i].key, (uint32_t)C.out[i].at) : make_uint2(0, 0);
  if (warp == 0) {
    const float t = lane < kSelThreads / 32 ? s_top[lane] : -INFINITY;
    float all = t;
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
    float s = lane >= kSelThreads / 32 ? 0.f : (t > -INFINITY ? s_sum[lane] * exp2_ftz((t - all) * kLog2e) : s_sum[lane]);
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) A.part[blockIdx.x] = make_float2(all, s);
  }
  // ---- the last CTA of the group chooses among the parts' lists
  int group = 0, hi = A.n_groups - 1;
  while (group < hi) {
    const int mid = (group + hi + 1) >> 1;
    if (A.seq0[mid] <= beam) group = mid; else hi = mid - 1;
  }
  const int b0 = A.seq0[group], beams = A.seq0[group + 1] - b0, lists = beams * A.parts;
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(&A.count[group], 1u) == (uint32_t)lists - 1;
    __threadfence();
    C.n = C.n_some = 0;
  }
  __syncthreads();
  if (!s_last) return;
  {
    // eight lanes a beam
    const int b = tid >> 3;
    const float2* p = A.part + (int64_t)(b0 + min(b, beams - 1)) * A.parts;
    float t = -INFINITY, s = 0.f;
    for (int i = tid & 7; i < A.parts; i += 8) {
      const float2 y = __ldcg(p + i);
      const float m = fmaxf(t, y.x), mb = m == -INFINITY ? 0.f : m;
      s = s * exp2_ftz((t - mb) * kLog2e) + y.y * exp2_ftz((y.x - mb) * kLog2e);
      t = m;
    }
    float all = t;
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
    s *= exp2_ftz((t - (all == -INFINITY ? 0.f : all)) * kLog2e);
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((tid & 7) == 0 && b < beams) {
      const float tot = A.total[b0 + b];
      const bool gone = A.ended && A.ended[b0 + b] != 0;
      // -inf: every continuation is worth that
      s_base[b] = s != s || all == -INFINITY || !(fabsf(tot) < INFINITY) ? -INFINITY
                  : gone ? (double)tot : (double)tot - ((double)all + log((double)s));
    }
  }
  __syncthreads();
  auto entry = [&](int l, int r) -> Cand {                 // place r of list l
    const int b = l / A.parts;
    const double base_v = s_base[b];
    uint2 e = __ldcg(A.best + ((int64_t)b0 * A.parts + l) * A.n_out + r);
    double v = -INFINITY;
    if (base_v == -INFINITY) e = make_uint2(l == b * A.parts && r < A.vocab, (uint32_t)r);   // its first tokens
    else v = base_v + (double)from_order32(e.x);
    return {e.x ? order64(v) : 0ull, (uint64_t)b << kBeamAt | (uint64_t)~e.x << kTokenBits | e.y};
  };
  // lists are sorted: those whose first candidate reaches the bound of the first ones, and of these the
  // candidates that do (values rounded to fp32, which keeps their order)
  int step = 1;                                            // few lists lie on threads far from one another
  while (step * 2 * lists <= kSelThreads) step *= 2;
  const bool on = tid % step == 0;
  auto worth = [](const Cand& y) { return y.key ? (float)from_order64(y.key) : -INFINITY; };
  float mine = -INFINITY, head = -INFINITY;                // of this thread's lists, and of the first of them
  if (on)
    for (int l = tid / step; l < lists; l += kSelThreads / step) {
      const float y = worth(entry(l, 0));
      if (l == tid / step) head = y;
      mine = fmaxf(mine, y);
    }
  const float reach = find_least(C, A.n_out, mine);
  if (on && mine >= reach)
    for (int l = tid / step; l < lists; l += kSelThreads / step) {
      if ((l == tid / step ? head : worth(entry(l, 0))) < reach) continue;
      const int i = atomicAdd(&C.n_some, 1);
      if (i < kList) C.some[i] = (uint16_t)l;
    }
  __syncthreads();
  const int n_some = C.n_some;
  if (n_some <= kList)                                     // eight threads a list, eight entries at a time
    for (int i = tid >> 3; i < n_some; i += kSelThreads / 8)
      for (int r = tid & 7; r < A.n_out; r += 8) {
        const Cand y = entry(C.some[i], r);
        if (y.key == 0 || worth(y) < reach) break;
        const int place = atomicAdd(&C.n, 1);
        if (place < kList) C.list[place] = y;
      }
  __syncthreads();
  int got = C.n;
  if (n_some <= kList && got <= kList) {
    got = rank_list(C, got, A.n_out, worth);
  } else {
    auto each = [&](auto f) {
      for (int c = tid; c < lists * A.n_out; c += kSelThreads) {
        const Cand y = entry(c % lists, c / lists);
        f(y.key, y.at);
      }
    };
    Cand own = {0, ~0ull};
    each([&](uint64_t key, uint64_t place) {
      const Cand y = {key, place};
      if (before(y, own)) own = y;
    });
    got = choose(C, A.n_out, own, each, worth);
  }
  // ---- out: best first, or every parent's best one in the parent's place
  int to = -1, parent = 0, tok = 0, done = 0;
  float val = 0.f;
  if (tid < got) {
    const Cand y = C.out[tid];
    parent = (int)(y.at >> kBeamAt);
    tok = (int)(y.at & ((1u << kTokenBits) - 1));
    val = (float)from_order64(y.key);
    to = tid;
    done = tok == A.end_token || (A.ended && A.ended[b0 + parent] != 0);
  }
  if (A.in_place && warp == 0) {                           // (n_out is the group's beams: a lane each)
    const uint32_t same = __match_any_sync(0xffffffffu, to >= 0 ? parent : -1 - lane);
    const bool stays = to >= 0 && (same & ((1u << lane) - 1u)) == 0;
    const uint32_t taken = __reduce_or_sync(0xffffffffu, stays ? 1u << parent : 0u);
    const uint32_t others = __ballot_sync(0xffffffffu, to >= 0 && !stays);
    if (stays) to = parent;
    else if (to >= 0) to = __fns(~taken, 0, __popc(others & ((1u << lane) - 1u)) + 1);
  }
  __syncthreads();                                         // total and ended, which may be the outputs, have been read
  if (to >= 0) {
    const int64_t o = (int64_t)group * A.n_out + to;
    A.total_out[o] = val;
    A.parent_out[o] = b0 + parent;
    A.token_out[o] = tok;
    if (A.ended_out) A.ended_out[o] = done;
  }
  if (tid == 0) A.count[group] = 0u;
}

}  // namespace

}  // namespace tria

using namespace tria;

namespace {

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

tria_status check_beams(const int32_t* seq0, int n_groups, int vocab, int n_out) {
  if (!seq0 || n_groups < 1 || seq0[0] != 0 || vocab < 1 || n_out < 1) return TRIA_ERR_INVALID_ARG;
  if (n_groups > kMaxSeqs || vocab > TRIA_MAX_VOCAB || n_out > TRIA_MAX_CHOICES) return TRIA_ERR_UNSUPPORTED;
  for (int i = 0; i < n_groups; ++i) {
    const int64_t n = (int64_t)seq0[i + 1] - seq0[i];
    if (n < 1 || n_out > n * vocab) return TRIA_ERR_INVALID_ARG;
    if (n > TRIA_MAX_BEAMS || seq0[i + 1] > kMaxSeqs) return TRIA_ERR_UNSUPPORTED;
  }
  return TRIA_OK;
}

struct BeamLayout {
  size_t count, part, best, total;
  int held, per, parts;
};

// Logits of a thread at a time: the most that still give every SM a CTA, so
// that a small call is spread over the GPU. Pieces of a CTA: as few as keep the
// CTAs of a large one resident at once (four an SM).
BeamLayout beam_layout(const int32_t* seq0, int n_groups, int vocab, int n_out) {
  BeamLayout L{};
  const int beams = seq0[n_groups], sms = sm_count();
  auto pieces = [&] { return (vocab + L.held * kSelThreads - 1) / (L.held * kSelThreads); };
  for (L.held = kHeld; L.held > 8 && (int64_t)beams * pieces() < sms;) L.held /= 2;
  for (L.per = 1; L.per < pieces() && (int64_t)beams * ((pieces() + L.per - 1) / L.per) > 4 * (int64_t)sms;) ++L.per;
  L.parts = (pieces() + L.per - 1) / L.per;
  L.count = kCountersAt;
  L.part = kScratchAt;
  L.best = up256(L.part + sizeof(float2) * (size_t)beams * L.parts);
  L.total = up256(L.best + sizeof(uint2) * (size_t)beams * L.parts * n_out);
  return L;
}

}  // namespace

extern "C" size_t tria_beam_select_workspace_size(const int32_t* seq0, int32_t n_groups, int32_t vocab, int32_t n_out) {
  return check_beams(seq0, n_groups, vocab, n_out) == TRIA_OK ? beam_layout(seq0, n_groups, vocab, n_out).total : 0;
}

extern "C" tria_status tria_beam_select(const tria_beams* b, void* ws, size_t ws_bytes, void* stream) {
  tria_status r;
  if (!b) return TRIA_ERR_INVALID_ARG;
  if ((r = check_beams(b->seq0, b->n_groups, b->vocab, b->n_out)) != TRIA_OK) return r;
  if (!act_ok(b->type)) return TRIA_ERR_UNSUPPORTED;
  const int size = b->type == TRIA_F32 ? 4 : 2;
  auto off = [](const void* p, int a) { return (uintptr_t)p % a != 0; };
  if (!b->logits || !b->total || !b->total_out || !b->parent_out || !b->token_out || b->stride < b->vocab || off(b->logits, size) ||
      off(b->total, 4) || off(b->ended, 4) || off(b->total_out, 4) || off(b->parent_out, 4) || off(b->token_out, 4) || off(b->ended_out, 4))
    return TRIA_ERR_INVALID_ARG;
  if (b->end_token < -1 || b->end_token >= b->vocab || (b->ended && b->end_token < 0) || (b->in_place != 0 && b->in_place != 1))
    return TRIA_ERR_INVALID_ARG;
  bool square = true;                                      // every group has n_out beams
  for (int i = 0; i < b->n_groups; ++i) square = square && b->seq0[i + 1] - b->seq0[i] == b->n_out;
  if (!square && (b->in_place || b->total_out == b->total || (b->ended_out && b->ended_out == b->ended))) return TRIA_ERR_INVALID_ARG;
  const BeamLayout L = beam_layout(b->seq0, b->n_groups, b->vocab, b->n_out);
  if (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < L.total) return TRIA_ERR_WORKSPACE;
  BeamArgs A;
  memset(&A, 0, sizeof(A));
  A.logits = b->logits;
  A.stride = b->stride;
  A.total = b->total;
  A.ended = b->ended;
  A.total_out = b->total_out;
  A.parent_out = b->parent_out;
  A.token_out = b->token_out;
  A.ended_out = b->ended_out;
  A.count = (uint32_t*)((uint8_t*)ws + L.count);
  A.part = (float2*)((uint8_t*)ws + L.part);
  A.best = (uint2*)((uint8_t*)ws + L.best);
  A.vocab = b->vocab;
  A.n_out = b->n_out;
  A.n_groups = b->n_groups;
  A.held = L.held;
  A.per = L.per;
  A.parts = L.parts;
  A.end_token = b->end_token;
  A.in_place = b->in_place;
  A.vec = (uintptr_t)b->logits % 16 == 0 && (b->stride * size) % 16 == 0;
  memcpy(A.seq0, b->seq0, sizeof(int32_t) * (b->n_groups + 1));
  const int grid = b->seq0[b->n_groups] * L.parts;
  const cudaStream_t st = (cudaStream_t)stream;
  if (b->type == TRIA_F32) k_beam_select<float><<<grid, kSelThreads, 0, st>>>(A);
  else if (b->type == TRIA_F16) k_beam_select<__half><<<grid, kSelThreads, 0, st>>>(A);
  else k_beam_select<__nv_bfloat16><<<grid, kSelThreads, 0, st>>>(A);
  return cudaGetLastError() == cudaSuccess ? TRIA_OK : TRIA_ERR_CUDA;
}
