// Rotary positions with the per-head norm of queries and keys in the same
// pass, alone (tria_rotate) or written into the cache in its own format
// (tria_append_qkv).
//
// A head x of head_dim values, rot = head_dim - nonrot_dim of them rotated:
//   y = x / sqrt(mean(x^2) + eps) * norm                  (when a norm is given)
//   (a, b) -> m (a cos t - b sin t, a sin t + b cos t),   t = w_f * position
// for pair f < rot/2 at (f, f + rot/2) or (2f, 2f + 1); m and w_f come from
// the long-context scaling. Phases are taken as in the scorer: w_f / 2 pi as a
// 64-bit fraction of a turn, so that position x turn mod 2^64 is the exact
// fractional turn at any position and no floating-point range reduction is
// needed.
//
// Layout: a lane owns 8 pairs of a head (16 values), head_dim / 16 lanes make
// a head and a warp takes 32 / (lanes per head, rounded up to a power of two)
// heads at once, so that both members of a pair sit in one lane and the norm
// is a shuffle reduction. A warp keeps its lanes' sines and cosines over the
// heads of a token that it handles: they cost about as much as a group. Heads
// come through shared memory: with loads into registers the bytes in flight
// (16 KB an SM) held the kernel at 2.9 TB/s. Warps take equal, contiguous shares
// of all tokens' groups of heads (whole tokens dealt out in turn left many idle
// at the end), and while a warp rotates, the next heads are on their way into
// its second stage: 8191 tokens of 40 heads x 128 bf16 values take 39.4 us (4.3
// TB/s; 46.8 with one stage and tokens in turn). With the cache's formats behind
// them, one stage of twice the size is better: 22487 tokens' queries, keys and
// values (32 + 8 + 8 heads; q8_0 keys, q4_0 values) take 156.5 us (3.8 TB/s), 171
// with two stages, whose smaller pieces cost more instructions than they hide.
// Keys on their way into the cache go through shared memory once more, because
// their quantisation blocks (32 consecutive dims) do not line up with the
// pairs. Prompts are bound by the instructions of 16 warps a SM (half of the
// issue slots; with 20 to 24 warps and fewer registers each they were slower),
// single tokens by latency (4 to 6 us a call).
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "attend_internal.cuh"

namespace tria {

namespace {

constexpr int kRopeWarps = 16;      // one CTA per SM
constexpr int kRopeSmem = 226 * 1024;
constexpr int rope_stages(bool cache) { return cache ? 1 : 2; }
constexpr int kPartDirect = 0, kPartKey = 1, kPartValue = 2;

struct RopePart {
  const void* x;
  void* out;             // direct: rotated heads; key / value: the held values (may be NULL)
  const float* norm;
  int64_t x_stride, out_stride;   // values between tokens
  int32_t heads;
  int32_t groups;        // warps' worth of heads per token
  int32_t kind;
};

struct RopeArgs {
  RopePart part[3];
  int32_t n_parts, n_tokens, groups;   // groups: of all parts, per token
  int32_t per_warp, stage;             // groups a warp handles at once; bytes of a stage of them
  int32_t hd, rot, layout, lanes;      // lanes: per head, a power of two
  float eps, mscale, inv_hd;
  const unsigned long long* turns;
  const int32_t* pos;
  // cache (append only)
  uint8_t* k;
  uint8_t* ks;
  uint8_t* v;
  uint8_t* vs;
  int32_t* cpos;
  int32_t* n_live;
  const int32_t* n_before;
  Ctrl* ctrl;
  int32_t n_seqs, k_type, v_type;
  int64_t row0[kMaxSeqs];
  int32_t cap[kMaxSeqs];
  int32_t tok0[kMaxSeqs + 1];
};

// eight values as fp32
__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __half* p, float* x) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float* x) {
  uint4 u;
  __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = u;
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float* x) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = u;
}

// Four codes as the bytes of a word, from floats to which kMagic = 1.5 x 2^23
// has been added: rounding to integers happened in that sum, and the integer
// lies in the low mantissa bits.
constexpr float kMagic = 12582912.f;
__device__ __forceinline__ uint32_t bytes_of(const float* m) {
  const uint32_t lo = __byte_perm(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// Codes of 16 values: round(x / d) away from zero (q8_0) and min(15, floor(x / d
// + 8.5)) (q4_0) of the correctly rounded fp32 quotient, as kMagic + code. x
// times the reciprocal is within 2^-22 of the quotient relative to it (at most
// 128), so only within 2^-14 of a border between codes can the two differ, and
// only then are the divisions made.
__device__ __forceinline__ void codes_q8(const float* x, float d, float* m) {
  const float inv = __frcp_rn(d);
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float q = x[i] * inv;
    m[i] = q + kMagic;
    far = fmaxf(far, fabsf(q - (m[i] - kMagic)));
  }
  if (far <= 0.5f - 0x1p-14f && d >= 0x1p-120f) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) m[i] = (d > 0.f ? fminf(fmaxf(roundf(__fdiv_rn(x[i], d)), -127.f), 127.f) : 0.f) + kMagic;
}
__device__ __forceinline__ void codes_q4(const float* x, float d, float* m) {
  const float inv = __frcp_rn(d);
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float q = __fadd_rn(__fmul_rn(x[i], inv), 8.5f) - 0.5f;   // floor(q + 0.5) is q rounded, but for borders
    m[i] = q + kMagic;
    far = fmaxf(far, fabsf(q - (m[i] - kMagic)));
    m[i] = fminf(m[i], kMagic + 15.f);
  }
  if (far <= 0.5f - 0x1p-14f && fabsf(d) >= 0x1p-120f) return;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    m[i] = (d != 0.f ? fminf(fmaxf(floorf(__fadd_rn(__fdiv_rn(x[i], d), 8.5f)), 0.f), 15.f) : 8.f) + kMagic;
}

// The larger / smaller value, NaN when either is one (a block that holds a NaN
// or an infinity gets a NaN for its scale and reads as NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// cos and sin of 2 pi x / 2^32: the quadrant off the top bits, Taylor's series
// on what is left (|r| <= pi / 4: 5e-10 and 2e-9 off).
__device__ __forceinline__ void turn_cos_sin(uint32_t x, float& c, float& s) {
  const uint32_t quad = (x + 0x20000000u) >> 30;
  const float r = (float)(int)(x - (quad << 30)) * 1.46291807926715968e-9f;   // 2 pi / 2^32
  const float z = r * r;
  float ps = fmaf(z, 2.7557319224e-6f, -1.9841269841e-4f);
  ps = fmaf(z, ps, 8.3333333333e-3f);
  ps = fmaf(z, ps, -1.6666666667e-1f);
  const float sr = fmaf(r * z, ps, r);
  float pc = fmaf(z, -2.7557319224e-7f, 2.4801587302e-5f);
  pc = fmaf(z, pc, -1.3888888889e-3f);
  pc = fmaf(z, pc, 4.1666666667e-2f);
  pc = fmaf(z, pc, -0.5f);
  const float cr = fmaf(z, pc, 1.f);
  const float a = (quad & 1u) ? sr : cr, b = (quad & 1u) ? cr : sr;
  c = (quad == 1u || quad == 2u) ? -a : a;
  s = (quad & 2u) ? -b : b;
}

// 16 consecutive values (dims e0 .. e0 + 15) of a head into cache row `row` of
// a plane; the lane next to it (lane ^ 1) holds the other half of the 32-wide
// block. x becomes the values that the plane now stands for. All lanes of the
// warp call it (`on`: this lane has values to store).
__device__ __forceinline__ void hold16(float* x, int type, uint8_t* data, uint8_t* scale, int64_t row, int hd, int e0,
                                       bool on) {
  if (type == TRIA_F32) {
    if (on) {
      float* d = reinterpret_cast<float*>(data) + row * hd + e0;
      store8<float>(d, x);
      store8<float>(d + 8, x + 8);
    }
    return;
  }
  if (type == TRIA_F16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __half2float(__float2half_rn(x[i]));
    if (on) {
      __half* d = reinterpret_cast<__half*>(data) + row * hd + e0;
      store8<__half>(d, x);
      store8<__half>(d + 8, x + 8);
    }
    return;
  }
  __half* sc = reinterpret_cast<__half*>(scale) + row * (hd / 32) + e0 / 32;
  if (type == TRIA_Q8_0) {
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) am = max_nan(am, fabsf(x[i]));
    am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, 1));
    const float d = __fdiv_rn(am, 127.f) + (am - am);   // (an infinity's scale is a NaN too: 0 x inf has no value)
    const __half dh = __float2half_rn(d);
    const float ds = __half2float(dh);
    float m[16];
    codes_q8(x, d, m);
    const uint32_t w[4] = {bytes_of(m), bytes_of(m + 4), bytes_of(m + 8), bytes_of(m + 12)};
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = (m[i] - kMagic) * ds;
    if (on) {
      *reinterpret_cast<uint4*>(data + row * hd + e0) = make_uint4(w[0], w[1], w[2], w[3]);
      if (!(e0 & 16)) *sc = dh;
    }
    return;
  }
  // q4_0: scale = m / -8 with m the first value of largest modulus
  const bool upper = (e0 & 16) != 0;
  float hi = x[0], lo = x[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    hi = max_nan(hi, x[i]);
    lo = min_nan(lo, x[i]);
  }
  float big = hi > -lo ? hi : lo;
  if (hi == -lo)                                // both signs: the first one of the lane's values
#pragma unroll 1
    for (int i = 15; i >= 0; --i) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (k == i && fabsf(x[k]) == hi) big = x[k];
    }
  const float other = __shfl_xor_sync(0xffffffffu, big, 1);
  const float first = upper ? other : big, second = upper ? big : other;
  big = fabsf(second) > fabsf(first) || second != second ? second : first;
  const float d = big * -0.125f + (big - big);          // (an infinity's is a NaN, as in q8_0)
  const __half dh = __float2half_rn(d + 0.f);   // an all-zero block's scale is +0
  const float ds = __half2float(dh);
  float m[16];
  codes_q4(x, d, m);
  const uint32_t w[4] = {bytes_of(m), bytes_of(m + 4), bytes_of(m + 8), bytes_of(m + 12)};
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = (m[i] - kMagic - 8.f) * ds;
  // byte j of a block: code j low, code j + 16 high; the lower lane writes bytes 0..7
  const uint32_t r0 = __shfl_xor_sync(0xffffffffu, upper ? w[0] : w[2], 1);
  const uint32_t r1 = __shfl_xor_sync(0xffffffffu, upper ? w[1] : w[3], 1);
  uint2 o;
  o.x = upper ? (r0 | (w[2] << 4)) : (w[0] | (r0 << 4));
  o.y = upper ? (r1 | (w[3] << 4)) : (w[1] | (r1 << 4));
  if (on) {
    *reinterpret_cast<uint2*>(data + row * (hd / 2) + (e0 / 32) * 16 + (upper ? 8 : 0)) = o;
    if (!upper) *sc = dh;
  }
}

__device__ __forceinline__ uint32_t qkv_error(int n, int t, int cap) {
  if (n < 0 || n > cap) return TRIA_ERR_DEVICE_ARG;
  if ((int64_t)n + t > cap) return TRIA_ERR_CAPACITY;
  return 0u;
}

// A lane's eight pairs: first and second members, two pairs to a register pair
// (packed fp32 arithmetic).
struct Pairs {
  float2 f[4], s[4];
};
template <int LAYOUT, typename T>
__device__ __forceinline__ void load_pairs(const T* head, int ea, int eb, Pairs& v) {
  float a[8], b[8];
  load8(head + ea, a);
  load8(head + eb, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (LAYOUT == TRIA_ROPE_HALF) {
      v.f[i] = make_float2(a[2 * i], a[2 * i + 1]);
      v.s[i] = make_float2(b[2 * i], b[2 * i + 1]);
    } else {
      const float* x = (i < 2 ? a : b) + (i & 1) * 4;
      v.f[i] = make_float2(x[0], x[2]);
      v.s[i] = make_float2(x[1], x[3]);
    }
  }
}

template <typename T, bool kCache, int LAYOUT>
__global__ void __launch_bounds__(kRopeWarps * 32, 1) k_rope(const __grid_constant__ RopeArgs A) {
  // per warp: a stage of heads; kCache: [heads of a group][head_dim + 4] floats
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hpw = 32 / A.lanes;                   // heads a warp takes at once
  const int sub = lane / A.lanes, p = lane % A.lanes;
  const bool on_dim = 16 * p < A.hd;
  const int half = A.rot / 2, f0 = 8 * p;
  const bool rotary = f0 < half;
  constexpr bool kInter = LAYOUT != TRIA_ROPE_HALF;
  const bool to_half = LAYOUT == TRIA_ROPE_INTERLEAVED_TO_HALF && rotary;
  // this lane's two runs of eight values: the first members of its pairs at
  // ea, the second ones at eb (consecutive where the pairs are interleaved)
  const int ea = kInter ? 16 * p : (rotary ? f0 : f0 + half);
  const int eb = kInter ? 16 * p + 8 : ea + (rotary ? half : (A.hd - A.rot) / 2);
  const int oa = to_half ? f0 : ea, ob = to_half ? f0 + half : eb;
  const int head_bytes = A.hd * (int)sizeof(T), group_bytes = hpw * head_bytes;
  constexpr int kStages = rope_stages(kCache);
  uint8_t* stages = smem + warp * kStages * A.stage;
  float* key_buf = reinterpret_cast<float*>(smem + kRopeWarps * kStages * A.stage) + (warp * hpw + sub) * (A.hd + 4);
  // a warp's share of the groups of all tokens (their number fits: checked by the host)
  const uint32_t total = (uint32_t)A.n_tokens * (uint32_t)A.groups;
  const uint32_t id = blockIdx.x * kRopeWarps + warp, n_warps = gridDim.x * kRopeWarps;
  uint32_t at = (uint32_t)((uint64_t)total * id / n_warps);
  const uint32_t end = (uint32_t)((uint64_t)total * (id + 1) / n_warps);

  // starts the copies of groups g0 .. g1 of a token's heads into a stage, group after group
  auto fetch = [&](uint8_t* dst, int tok, int g0, int g1) {
    int base = 0;
#pragma unroll 1
    for (int pi = 0; pi < A.n_parts; ++pi) {
      const RopePart& Q = A.part[pi];
      const int ga = max(g0 - base, 0), ge = min(g1 - base, Q.groups);
      base += Q.groups;
      if (ga >= ge) continue;
      const int bytes = (min(ge * hpw, Q.heads) - ga * hpw) * head_bytes;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(Q.x) + ((int64_t)tok * Q.x_stride + (int64_t)ga * hpw * A.hd) * (int)sizeof(T);
      for (int i = lane * 16; i < bytes; i += 512) cp_async16(dst + i, src + i);
      dst += (ge - ga) * group_bytes;
    }
  };
  // the groups at hand (of one token, at most a stage's); the next ones are on their way meanwhile
  int tok = 0, g0 = 0, g1 = 0, last_tok = -1, position = 0, seq = 0, row = 0, turn = 0;
  bool row_ok = false;
  float2 cs[4], sn[4], ns[4];                     // cosines, sines and their negatives of the pairs
  while (g1 > 0 || at < end) {
    int n_tok = 0, n_g0 = 0, n_g1 = 0;
    if (at < end) {
      n_tok = (int)(at / (uint32_t)A.groups);
      n_g0 = (int)(at - (uint32_t)n_tok * (uint32_t)A.groups);
      n_g1 = min(min(A.groups, n_g0 + A.per_warp), n_g0 + (int)(end - at));
      at += (uint32_t)(n_g1 - n_g0);
      fetch(stages + turn * A.stage, n_tok, n_g0, n_g1);
    }
    cp_async_commit();
    if constexpr (kStages == 1) {
      tok = n_tok;
      g0 = n_g0;
      g1 = n_g1;
    } else {
      turn ^= 1;
    }
    if (g1 > 0) {
      if (tok != last_tok) {
        last_tok = tok;
        position = A.pos[tok];
        if constexpr (kCache) {
          int lo = 0, hi = A.n_seqs - 1;              // the last sequence whose first token is <= tok
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (A.tok0[mid] <= tok) lo = mid; else hi = mid - 1;
          }
          seq = lo;
          const int t = A.tok0[seq + 1] - A.tok0[seq];
          const int n = A.n_before ? A.n_before[seq] : *((volatile const int32_t*)(A.n_live + seq));
          row_ok = qkv_error(n, t, A.cap[seq]) == 0u;
          row = n + (tok - A.tok0[seq]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cs[i] = make_float2(1.f, 1.f);
          sn[i] = make_float2(0.f, 0.f);
          if (rotary) {
            const unsigned long long x = (unsigned long long)(long long)position;
            turn_cos_sin((uint32_t)((x * A.turns[f0 + 2 * i]) >> 32), cs[i].x, sn[i].x);
            turn_cos_sin((uint32_t)((x * A.turns[f0 + 2 * i + 1]) >> 32), cs[i].y, sn[i].y);
            cs[i] = make_float2(cs[i].x * A.mscale, cs[i].y * A.mscale);
            sn[i] = make_float2(sn[i].x * A.mscale, sn[i].y * A.mscale);
          }
          ns[i] = make_float2(-sn[i].x, -sn[i].y);
        }
      }
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* in = stages + turn * A.stage + sub * head_bytes;
      int base = 0;
#pragma unroll 1
      for (int pi = 0; pi < A.n_parts; ++pi) {
        const RopePart& Q = A.part[pi];
        const int ga = max(g0 - base, 0), ge = min(g1 - base, Q.groups);
        base += Q.groups;
        if (ga >= ge) continue;
        int head = ga * hpw + sub;
        T* out = reinterpret_cast<T*>(Q.out) + (int64_t)tok * Q.out_stride + (int64_t)head * A.hd;
        if (kCache && Q.kind == kPartValue) {
#pragma unroll 1
          for (int gi = ga; gi < ge; ++gi, head += hpw, in += group_bytes, out += hpw * A.hd) {
            const bool on = on_dim && head < Q.heads;
            // (a lane past head_dim holds zeros; a whole head past the last one, junk
            // that goes nowhere)
            float a[16] = {};
            if (on_dim) {
              load8(reinterpret_cast<const T*>(in) + 16 * p, a);
              load8(reinterpret_cast<const T*>(in) + 16 * p + 8, a + 8);
            }
            const int64_t r = A.row0[seq] + (int64_t)head * A.cap[seq] + row;
            hold16(a, A.v_type, A.v, A.vs, r, A.hd, 16 * p, on && row_ok);
            if (on && row_ok && Q.out) {
              store8<T>(out + 16 * p, a);
              store8<T>(out + 16 * p + 8, a + 8);
            }
          }
          continue;
        }
        Pairs w;
        if (Q.norm && on_dim) load_pairs<LAYOUT>(Q.norm, ea, eb, w);
#pragma unroll 1
        for (int gi = ga; gi < ge; ++gi, head += hpw, in += group_bytes, out += hpw * A.hd) {
          const bool on = on_dim && head < Q.heads;
          Pairs a = {};
          if (on_dim) load_pairs<LAYOUT>(reinterpret_cast<const T*>(in), ea, eb, a);
          if (Q.norm) {
            float2 sq = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) sq = __ffma2_rn(a.s[i], a.s[i], __ffma2_rn(a.f[i], a.f[i], sq));
            float ss = sq.x + sq.y;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1)
              if (o < A.lanes) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(ss * A.inv_hd + A.eps);
            const float2 r2 = make_float2(r, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a.f[i] = __fmul2_rn(__fmul2_rn(a.f[i], r2), w.f[i]);
              a.s[i] = __fmul2_rn(__fmul2_rn(a.s[i], r2), w.s[i]);
            }
          }
          if (rotary) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 x = __ffma2_rn(a.f[i], cs[i], __fmul2_rn(a.s[i], ns[i]));
              a.s[i] = __ffma2_rn(a.f[i], sn[i], __fmul2_rn(a.s[i], cs[i]));
              a.f[i] = x;
            }
          }
          float b[16];                              // first members, then second ones (or pairs)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (LAYOUT == TRIA_ROPE_INTERLEAVED || (LAYOUT == TRIA_ROPE_INTERLEAVED_TO_HALF && !rotary)) {
              b[4 * i] = a.f[i].x;
              b[4 * i + 1] = a.s[i].x;
              b[4 * i + 2] = a.f[i].y;
              b[4 * i + 3] = a.s[i].y;
            } else {
              b[2 * i] = a.f[i].x;
              b[2 * i + 1] = a.f[i].y;
              b[8 + 2 * i] = a.s[i].x;
              b[8 + 2 * i + 1] = a.s[i].y;
            }
          }
          if (!kCache || Q.kind == kPartDirect) {
            if (on) {
              store8<T>(out + oa, b);
              store8<T>(out + ob, b + 8);
            }
            continue;
          }
          if constexpr (kCache) {
            // a key on its way into the cache: to consecutive dims through shared memory
            __syncwarp();
            if (on) {
              store8<float>(key_buf + oa, b);
              store8<float>(key_buf + ob, b + 8);
            }
            __syncwarp();
            if (on) {
              load8(key_buf + 16 * p, b);
              load8(key_buf + 16 * p + 8, b + 8);
            }
            const int64_t r = A.row0[seq] + (int64_t)head * A.cap[seq] + row;
            hold16(b, A.k_type, A.k, A.ks, r, A.hd, 16 * p, on && row_ok);
            if (on && row_ok) {
              if (p == 0) A.cpos[r] = position;
              if (Q.out) {
                store8<T>(out + 16 * p, b);
                store8<T>(out + 16 * p + 8, b + 8);
              }
            }
          }
        }
      }
      __syncwarp();                               // the stage is free
    }
    if constexpr (kStages == 1) {
      g1 = 0;
    } else {
      tok = n_tok;
      g0 = n_g0;
      g1 = n_g1;
    }
  }
  if constexpr (kCache) {
    // n_live changes once nothing reads it any more: at once when the rows
    // before the call are the caller's, else by the last CTA to finish
    __shared__ int s_mine;
    __syncthreads();
    if (threadIdx.x == 0) {
      s_mine = blockIdx.x == 0;
      if (!A.n_before) {
        __threadfence();
        s_mine = atomicAdd(&A.ctrl->append_ticket, 1u) == gridDim.x - 1;
        __threadfence();
        if (s_mine) atomicExch(&A.ctrl->append_ticket, 0u);
      }
    }
    __syncthreads();
    if (!s_mine) return;
    for (int s = threadIdx.x; s < A.n_seqs; s += blockDim.x) {
      const int t = A.tok0[s + 1] - A.tok0[s];
      const int n = A.n_before ? A.n_before[s] : *((volatile const int32_t*)(A.n_live + s));
      const uint32_t e = qkv_error(n, t, A.cap[s]);
      if (e)
        report(A.ctrl, e, (uint32_t)s);
      else
        A.n_live[s] = n + t;
    }
  }
}

int ceil_pow2(int x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

template <typename T, bool kCache, int LAYOUT>
cudaError_t launch_rope_tl(const RopeArgs& A, cudaStream_t st) {
  const int grid = rope_grid(A.n_tokens, A.groups, kRopeWarps, sm_count());
  const int smem = kRopeWarps * (rope_stages(kCache) * A.stage + (kCache ? (32 / A.lanes) * (A.hd + 4) * (int)sizeof(float) : 0));
  auto kern = k_rope<T, kCache, LAYOUT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kRopeWarps * 32, smem, st>>>(A);
  return cudaGetLastError();
}

template <typename T, bool kCache>
cudaError_t launch_rope_t(const RopeArgs& A, cudaStream_t st) {
  if (A.layout == TRIA_ROPE_HALF) return launch_rope_tl<T, kCache, TRIA_ROPE_HALF>(A, st);
  if (A.layout == TRIA_ROPE_INTERLEAVED) return launch_rope_tl<T, kCache, TRIA_ROPE_INTERLEAVED>(A, st);
  return launch_rope_tl<T, kCache, TRIA_ROPE_INTERLEAVED_TO_HALF>(A, st);
}

template <bool kCache>
cudaError_t launch_rope(const RopeArgs& A, int type, cudaStream_t st) {
  if (type == TRIA_F32) return launch_rope_t<float, kCache>(A, st);
  if (type == TRIA_F16) return launch_rope_t<__half, kCache>(A, st);
  return launch_rope_t<__nv_bfloat16, kCache>(A, st);
}

// Work of a warp at once: as many groups of a token as a stage holds, which
// share the sines and cosines. (A single token takes one short step in as many
// warps as it has groups.)
void finish_args(RopeArgs& A, const tria_rope* rope, int type, bool cache) {
  A.hd = rope->head_dim;
  A.rot = rope->head_dim - rope->nonrot_dim;
  A.layout = rope->layout;
  A.turns = rope->turns;
  A.mscale = (float)rope->mscale;
  A.inv_hd = 1.f / (float)A.hd;
  A.lanes = ceil_pow2(A.hd / 16);
  const int hpw = 32 / A.lanes, group_bytes = hpw * A.hd * (type == TRIA_F32 ? 4 : 2);
  A.groups = 0;
  for (int i = 0; i < A.n_parts; ++i) {
    A.part[i].groups = (A.part[i].heads + hpw - 1) / hpw;
    A.groups += A.part[i].groups;
  }
  // a warp's stages and, behind those of an append, the keys' buffer fill its share of shared
  // memory (a rotation leaves the buffer's room free)
  const int room = (kRopeSmem / kRopeWarps - hpw * (A.hd + 4) * (int)sizeof(float)) & ~15;
  A.per_warp = std::min(room / rope_stages(cache) / group_bytes, A.groups);
  A.stage = A.per_warp * group_bytes;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// units of work are counted in 32 bits
bool rope_fits(int64_t tokens, int64_t heads) { return tokens * (heads + 3) < ((int64_t)1 << 31); }

int act_size(int type) { return type == TRIA_F32 ? 4 : 2; }

tria_status check_heads(const void* x, int64_t stride, int heads, int hd, int type) {
  if (!x || !aligned(x, 16) || heads < 1) return TRIA_ERR_INVALID_ARG;
  if (stride < (int64_t)heads * hd || (stride * act_size(type)) % 16 != 0) return TRIA_ERR_INVALID_ARG;
  return TRIA_OK;
}

tria_status check_rope_desc(const tria_rope_desc* d) {
  if (!d) return TRIA_ERR_INVALID_ARG;
  const int hd = d->head_dim, nr = d->nonrot_dim;
  if (hd <= 0 || hd > TRIA_MAX_HEAD_DIM || hd % 32 != 0) return TRIA_ERR_UNSUPPORTED;
  if (nr < 0 || nr >= hd) return TRIA_ERR_INVALID_ARG;
  if ((hd - nr) % 16 != 0) return TRIA_ERR_UNSUPPORTED;
  if (d->layout < TRIA_ROPE_HALF || d->layout > TRIA_ROPE_INTERLEAVED_TO_HALF) return TRIA_ERR_INVALID_ARG;
  if (d->scaling < TRIA_ROPE_PLAIN || d->scaling > TRIA_ROPE_BANDS) return TRIA_ERR_INVALID_ARG;
  if (d->omega) {
    if (d->scaling != TRIA_ROPE_PLAIN) return TRIA_ERR_INVALID_ARG;
  } else if (!(d->theta > 1.0) || !isfinite(d->theta)) {
    return TRIA_ERR_INVALID_ARG;
  }
  if (d->scaling != TRIA_ROPE_PLAIN && (!(d->factor >= 1.0) || !isfinite(d->factor))) return TRIA_ERR_INVALID_ARG;
  if ((d->scaling == TRIA_ROPE_YARN || d->scaling == TRIA_ROPE_BANDS) && d->orig_ctx < 1) return TRIA_ERR_INVALID_ARG;
  if (!(d->mscale >= 0.0) || !isfinite(d->mscale)) return TRIA_ERR_INVALID_ARG;
  const double hi = d->high == 0.0 ? (d->scaling == TRIA_ROPE_YARN ? 32.0 : 4.0) : d->high;
  const double lo = d->low == 0.0 ? 1.0 : d->low;
  if ((d->scaling == TRIA_ROPE_YARN || d->scaling == TRIA_ROPE_BANDS) && !(lo > 0.0 && hi > lo && isfinite(hi)))
    return TRIA_ERR_INVALID_ARG;
  if (d->omega)
    for (int f = 0; f < (hd - nr) / 2; ++f)
      if (!isfinite(d->omega[f])) return TRIA_ERR_INVALID_ARG;
  return TRIA_OK;
}

void frequencies(const tria_rope_desc* d, double* w, double* mscale) {
  const int rot = d->head_dim - d->nonrot_dim, n = rot / 2;
  *mscale = d->mscale != 0.0 ? d->mscale : (d->scaling == TRIA_ROPE_YARN ? 0.1 * log(d->factor) + 1.0 : 1.0);
  if (d->omega) {
    for (int f = 0; f < n; ++f) w[f] = d->omega[f];
    return;
  }
  double theta = d->theta;
  if (d->scaling == TRIA_ROPE_NTK && rot > 2) theta *= pow(d->factor, (double)rot / (rot - 2));
  const double two_pi = 2.0 * 3.14159265358979323846;
  const double low = d->low == 0.0 ? 1.0 : d->low;
  const double high = d->high == 0.0 ? (d->scaling == TRIA_ROPE_YARN ? 32.0 : 4.0) : d->high;
  // pair index (real-valued) that turns `turns` times over the original context
  auto pair_of = [&](double turns) { return rot * log((double)d->orig_ctx / (turns * two_pi)) / (2.0 * log(theta)); };
  double lo = 0.0, hi = 0.0;
  if (d->scaling == TRIA_ROPE_YARN) {
    lo = std::max(floor(pair_of(high)), 0.0);
    hi = std::min(ceil(pair_of(low)), (double)(rot - 1));
  }
  for (int f = 0; f < n; ++f) {
    const double base = pow(theta, -2.0 * f / rot);
    double keep = 1.0;      // share of the unscaled frequency
    switch (d->scaling) {
      case TRIA_ROPE_LINEAR: keep = 0.0; break;
      case TRIA_ROPE_YARN: keep = 1.0 - std::min(std::max((f - lo) / std::max(hi - lo, 0.001), 0.0), 1.0); break;
      case TRIA_ROPE_BANDS:
        keep = std::min(std::max(((double)d->orig_ctx * base / two_pi - low) / (high - low), 0.0), 1.0);
        break;
      default: break;
    }
    const bool scaled = d->scaling != TRIA_ROPE_PLAIN && d->scaling != TRIA_ROPE_NTK;
    w[f] = scaled ? base / d->factor * (1.0 - keep) + base * keep : base;
  }
}

}  // namespace

}  // namespace tria

using namespace tria;

extern "C" tria_status tria_rope_frequencies(const tria_rope_desc* desc, double* omega_out, double* mscale_out) {
  const tria_status r = check_rope_desc(desc);
  if (r != TRIA_OK) return r;
  if (!omega_out || !mscale_out) return TRIA_ERR_INVALID_ARG;
  frequencies(desc, omega_out, mscale_out);
  return TRIA_OK;
}

extern "C" tria_status tria_load_rope(const tria_rope_desc* desc, tria_rope** out) {
  if (!out) return TRIA_ERR_INVALID_ARG;
  *out = nullptr;
  const tria_status r = check_rope_desc(desc);
  if (r != TRIA_OK) return r;
  const int n = (desc->head_dim - desc->nonrot_dim) / 2;
  double w[TRIA_MAX_HEAD_DIM / 2];
  unsigned long long turns[TRIA_MAX_HEAD_DIM / 2];
  double mscale;
  frequencies(desc, w, &mscale);
  for (int f = 0; f < n; ++f) {
    double t = w[f] / (2.0 * 3.14159265358979323846);
    t -= floor(t);
    const double scaled = ldexp(t, 64);
    turns[f] = scaled >= 18446744073709551615.0 ? 0ull : (unsigned long long)scaled;
  }
  tria_rope* h = new (std::nothrow) tria_rope;
  if (!h) return TRIA_ERR_CUDA;
  h->head_dim = desc->head_dim;
  h->nonrot_dim = desc->nonrot_dim;
  h->layout = desc->layout;
  h->mscale = mscale;
  h->turns = nullptr;
  if (cudaMalloc((void**)&h->turns, sizeof(unsigned long long) * n) != cudaSuccess ||
      cudaMemcpy(h->turns, turns, sizeof(unsigned long long) * n, cudaMemcpyHostToDevice) != cudaSuccess) {
    if (h->turns) cudaFree(h->turns);
    delete h;
    return TRIA_ERR_CUDA;
  }
  *out = h;
  return TRIA_OK;
}

extern "C" void tria_free_rope(tria_rope* rope) {
  if (!rope) return;
  cudaFree(rope->turns);
  delete rope;
}

extern "C" tria_status tria_rotate(const tria_rope* rope, tria_dtype type, const tria_heads* parts, int32_t n_parts,
                                   int32_t n_tokens, const int32_t* pos, double eps, void* stream) {
  if (!rope || !parts || n_parts < 1 || n_parts > 2 || n_tokens < 0 || !(eps >= 0.0)) return TRIA_ERR_INVALID_ARG;
  if (!act_ok(type)) return TRIA_ERR_UNSUPPORTED;
  if (n_tokens == 0) return TRIA_OK;
  if (!pos || !aligned(pos, 4)) return TRIA_ERR_INVALID_ARG;
  if (!rope_fits(n_tokens, (int64_t)parts[0].n_heads + (n_parts > 1 ? parts[1].n_heads : 0))) return TRIA_ERR_UNSUPPORTED;
  RopeArgs A;
  memset(&A, 0, sizeof(A));
  for (int i = 0; i < n_parts; ++i) {
    const tria_heads& h = parts[i];
    tria_status r;
    if ((r = check_heads(h.x, h.x_stride, h.n_heads, rope->head_dim, type)) != TRIA_OK) return r;
    if ((r = check_heads(h.out, h.out_stride, h.n_heads, rope->head_dim, type)) != TRIA_OK) return r;
    if (h.out == h.x && h.out_stride != h.x_stride && n_tokens > 1) return TRIA_ERR_INVALID_ARG;
    if (h.norm && !aligned(h.norm, 16)) return TRIA_ERR_INVALID_ARG;
    A.part[i] = RopePart{h.x, h.out, h.norm, h.x_stride, h.out_stride, h.n_heads, 0, kPartDirect};
  }
  A.n_parts = n_parts;
  A.n_tokens = n_tokens;
  A.eps = (float)eps;
  A.pos = pos;
  finish_args(A, rope, type, false);
  return launch_rope<false>(A, type, (cudaStream_t)stream) == cudaSuccess ? TRIA_OK : TRIA_ERR_CUDA;
}

extern "C" tria_status tria_append_qkv(const tria_rope* rope, const tria_layer_cache* cache, const tria_qkv* a,
                                       void* ws, size_t ws_bytes, void* stream) {
  tria_status r;
  if (!rope || !a) return TRIA_ERR_INVALID_ARG;
  if ((r = check_cache(cache)) != TRIA_OK) return r;
  if (rope->head_dim != cache->head_dim) return TRIA_ERR_INVALID_ARG;
  if (!act_ok(a->type)) return TRIA_ERR_UNSUPPORTED;
  if (!a->tok0 || a->n_q_heads < 0 || !(a->eps >= 0.0)) return TRIA_ERR_INVALID_ARG;
  if ((r = check_tokens(a->tok0, cache->n_seqs)) != TRIA_OK) return r;
  if (!ws || !aligned(ws, 256) || ws_bytes < sizeof(Ctrl)) return TRIA_ERR_WORKSPACE;
  const int n_tokens = a->tok0[cache->n_seqs];
  const int32_t* n_before = a->n_before == cache->n_live ? nullptr : a->n_before;
  if (n_before && !aligned(n_before, 4)) return TRIA_ERR_INVALID_ARG;
  if (n_tokens == 0 && !n_before) return TRIA_OK;
  if (!rope_fits(n_tokens, (int64_t)a->n_q_heads + 2 * cache->n_kv_heads)) return TRIA_ERR_UNSUPPORTED;
  const int hd = cache->head_dim;
  RopeArgs A;
  memset(&A, 0, sizeof(A));
  if (n_tokens > 0) {
    if (!a->pos || !aligned(a->pos, 4)) return TRIA_ERR_INVALID_ARG;
    if ((r = check_heads(a->k, a->k_stride, cache->n_kv_heads, hd, a->type)) != TRIA_OK) return r;
    if ((r = check_heads(a->v, a->v_stride, cache->n_kv_heads, hd, a->type)) != TRIA_OK) return r;
    if (a->n_q_heads > 0) {
      if ((r = check_heads(a->q, a->q_stride, a->n_q_heads, hd, a->type)) != TRIA_OK) return r;
      if ((r = check_heads(a->q_out, a->q_out_stride, a->n_q_heads, hd, a->type)) != TRIA_OK) return r;
      if (a->q_out == a->q && a->q_out_stride != a->q_stride && n_tokens > 1) return TRIA_ERR_INVALID_ARG;
    }
    if ((a->q_norm && !aligned(a->q_norm, 16)) || (a->k_norm && !aligned(a->k_norm, 16))) return TRIA_ERR_INVALID_ARG;
    if ((a->k_held && !aligned(a->k_held, 16)) || (a->v_held && !aligned(a->v_held, 16))) return TRIA_ERR_INVALID_ARG;
  }
  const int kv = cache->n_kv_heads;
  if (a->n_q_heads > 0)
    A.part[A.n_parts++] = RopePart{a->q, a->q_out, a->q_norm, a->q_stride, a->q_out_stride, a->n_q_heads, 0, kPartDirect};
  const int64_t held = (int64_t)kv * hd;
  A.part[A.n_parts++] = RopePart{a->k, a->k_held, a->k_norm, a->k_stride, held, kv, 0, kPartKey};
  A.part[A.n_parts++] = RopePart{a->v, a->v_held, nullptr, a->v_stride, held, kv, 0, kPartValue};
  A.n_tokens = n_tokens;
  A.eps = (float)a->eps;
  A.pos = a->pos;
  A.k = (uint8_t*)cache->k;
  A.ks = (uint8_t*)cache->k_scale;
  A.v = (uint8_t*)cache->v;
  A.vs = (uint8_t*)cache->v_scale;
  A.cpos = cache->pos;
  A.n_live = cache->n_live;
  A.n_before = n_before;
  A.ctrl = (Ctrl*)ws;
  A.n_seqs = cache->n_seqs;
  A.k_type = cache->k_type;
  A.v_type = cache->v_type;
  for (int s = 0; s < cache->n_seqs; ++s) {
    A.row0[s] = cache->seq_row0[s];
    A.cap[s] = cache->capacity[s];
  }
  for (int s = 0; s <= cache->n_seqs; ++s) A.tok0[s] = a->tok0[s];
  finish_args(A, rope, a->type, true);
  return launch_rope<true>(A, a->type, (cudaStream_t)stream) == cudaSuccess ? TRIA_OK : TRIA_ERR_CUDA;
}
