// Attention of a few new tokens over the cache (decode steps): a stream over
// the visible rows, with the query columns of a KV head (token x head, up to 8
// or 16) as one side of tensor-core products.
//
//   S = Q K^T    m16n8k16, M = columns, N = 8 rows, K = 16 dims
//   O^T = V^T P  m16n8k16, M = 16 dims, N = 8 columns, K = 16 rows
//
// S leaves a thread with rows 2t, 2t + 1 of column gid, which is the B fragment
// of the second product, so weights never leave their registers. fp16 rows are
// read with ldmatrix; 8- and 4-bit codes become fp16 exactly by bit
// insertion (1024 + code, minus the offset), with the dims of a step in the
// order in which the codes lie in a word (the queries are loaded in the same
// order). Key scales multiply the fp32 sum of each 32-wide block; value scales
// multiply the fp32 weight before its one rounding to fp16, so that an
// 8- or 4-bit cache costs no rounding that an fp16 one does not have.
//
// Weights are kept relative to M = max logit + E - 14, E the exponent of the
// largest value scale so far: weight x scale then reaches up to 2^14 in fp16
// whatever the size of the values, and the common factor cancels in O / l.
//
// The tiles of all units (sequence x KV head) are one list, cut into equal
// runs, one per warp, neighbouring ones in a CTA: the live rows are known on
// the device alone, and ragged batches stay balanced. A warp streams its run
// through a ring of cp.async stages (padded rows: no bank conflicts) from unit
// to unit without stopping: a block that met at every unit's end ran 64
// sequences of 1000 rows at 3.1 TB/s. A unit inside a run is written by its
// warp; parts of a unit go to the workspace and are merged in order, those of
// a CTA's warps when all have finished, those of several CTAs by the last one
// to arrive.
//
// fp16 rows are bound by memory: 8 sequences, 206246 rows of 8 KV heads x 128
// dims, 4 query heads each, 150 us (5.6 TB/s); 534879 rows of 4 heads x 256
// dims 372 us (5.9 TB/s). 4-bit rows are bound by the instructions that turn
// codes into fragments (about 900 a tile of 32 rows, at 0.6 of the issue
// slots): 412488 rows 142 us, 3.35 TB/s, 2.9 rows per ns against 1.4 of fp16.
// Codes used as subnormals, with the offsets in the sums, are fewer
// instructions but took 185 us: the products wait on one another.
#pragma once

#include <type_traits>

#include "attend_internal.cuh"

namespace tria {

constexpr int kStepSmem = 212 * 1024;   // stages; the unit tables need 13 KB more

// TR: rows of a tile; SB: bytes of a stage
template <int KT, int VT, int HD, int NT>
struct StepShape {
  static constexpr bool kKq = KT != TRIA_F16, kVq = VT != TRIA_F16;
  static constexpr int kRb = KT == TRIA_F16 ? 2 * HD : (KT == TRIA_Q8_0 ? HD : HD / 2);
  static constexpr int vRb = VT == TRIA_F16 ? 2 * HD : (VT == TRIA_Q8_0 ? HD : HD / 2);
  static constexpr int kStride = kRb + 16, vStride = vRb + 16;
  static constexpr int scRb = HD / 16;                     // block scales of a row
  static constexpr int TR = (KT == TRIA_Q4_0 && VT == TRIA_Q4_0) ? 32 : 16;
  static constexpr int oV = TR * kStride, oKs = oV + TR * vStride, oVs = oKs + (kKq ? TR * scRb : 0),
                       oPos = oVs + (kVq ? TR * scRb : 0);
  static constexpr int SB = (oPos + TR * 4 + 15) & ~15;
  static constexpr int kStages = 3;
  static constexpr int fit = kStepSmem / (SB * kStages);
  static constexpr int kWarps = fit >= 12 ? 12 : (fit >= 8 ? 8 : 4);
  static constexpr int kArea = SB * kStages;
  static constexpr int kOut = (HD * 8 * NT + 16 * NT) * 4;  // a warp's part of a unit, in its stages
  static_assert(kArea >= kOut, "a warp's part fits its stages");
  static_assert(kArea * kWarps <= kStepSmem, "stages fit shared memory");
};

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// (plain loads, so that constant offsets go into the instruction)
__device__ __forceinline__ uint32_t get32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint32_t get16(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// Block scales of two neighbouring rows (NB halves each, side by side).
template <int NB>
__device__ __forceinline__ void load_scales(const uint8_t* p, float* a, float* b) {
  if constexpr (NB == 3) {                                 // (not a vector's size)
    const __half* x = reinterpret_cast<const __half*>(p);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      a[i] = __half2float(x[i]);
      b[i] = __half2float(x[NB + i]);
    }
    return;
  }
  __half2 h[NB];
  if constexpr (NB == 2) {
    *reinterpret_cast<uint2*>(h) = *reinterpret_cast<const uint2*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < NB / 4; ++i) reinterpret_cast<uint4*>(h)[i] = reinterpret_cast<const uint4*>(p)[i];
  }
#pragma unroll
  for (int i = 0; i < NB / 2; ++i) {
    const float2 x = __half22float2(h[i]), y = __half22float2(h[NB / 2 + i]);
    a[2 * i] = x.x;
    a[2 * i + 1] = x.y;
    b[2 * i] = y.x;
    b[2 * i + 1] = y.y;
  }
}

// Codes of a word (q8_0: bytes 0 / 2 and 1 / 3; q4_0: the low halves of bytes
// 0 / 2 and 1 / 3, then the high halves) as fp16 pairs, exactly: 0x6400 | u is
// 1024 + u, and 1024 + 16 u for a code in the high half of a byte.
// The constants sit in registers that the compiler cannot see through: as
// immediates, of which an instruction takes one, every masked insertion became
// two.
struct Magic {
  uint32_t q8, one, low, inv, high;
  __device__ __forceinline__ Magic() {
    asm volatile("mov.b32 %0, 0x64806480;" : "=r"(q8));
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(one));
    asm volatile("mov.b32 %0, 0x64086408;" : "=r"(low));
    asm volatile("mov.b32 %0, 0x2C002C00;" : "=r"(inv));
    asm volatile("mov.b32 %0, 0xD480D480;" : "=r"(high));
  }
};
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t mask, uint32_t b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(mask), "r"(b));
  return d;
}
__device__ __forceinline__ void q8_pairs(const Magic& m, uint32_t w, uint32_t* h) {
  h[0] = h2_sub(and_xor(w, 0x00FF00FFu, m.q8), m.q8);                   // - 1152
  h[1] = h2_sub(and_xor(w >> 8, 0x00FF00FFu, m.q8), m.q8);
}
__device__ __forceinline__ void q4_pairs(const Magic& m, uint32_t w, uint32_t* h) {
  const uint32_t u = w >> 8;
  h[0] = h2_sub(and_or(w, 0x000F000Fu, m.one), m.low);                  // - 1032
  h[1] = h2_sub(and_or(u, 0x000F000Fu, m.one), m.low);
  h[2] = h2_fma(and_or(w, 0x00F000F0u, m.one), m.inv, m.high);          // / 16 - 72
  h[3] = h2_fma(and_or(u, 0x00F000F0u, m.one), m.inv, m.high);
}

template <int KT, int VT, int HD, int NT>
__global__ void __launch_bounds__(StepShape<KT, VT, HD, NT>::kWarps * 32, 1)
    k_attend_step(const __grid_constant__ AttendArgs A) {
  using H = StepShape<KT, VT, HD, NT>;
  constexpr int TR = H::TR, NB = HD / 32, NG = TR / 8;     // blocks of a row, 8-row groups of a tile
  constexpr int kWarps = H::kWarps, kStages = H::kStages, kCol = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_first[kMaxSegments + 1];                // first tile of each unit
  __shared__ int s_lo[kMaxSegments], s_hi[kMaxSegments];   // its rows besides the sink
  __shared__ int s_scan[40];
  __shared__ int s_flag[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, t4 = lane & 3;
  // (a kernel that does not need this one's results, see k_attend_group, may take SMs as they fall free)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the tile list: every unit has a tile at least (a token without rows
  // still gets its zeros), but those of sequences that take no part
  const int n_units = A.n_seqs * A.n_kv;
  constexpr int kPer = (kMaxSegments + kWarps * 32 - 1) / (kWarps * 32);   // units of a thread, consecutive
  {
    int cnt[kPer], local = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      cnt[i] = 0;
      const int u = (int)threadIdx.x * kPer + i;
      if (u >= n_units) continue;
      const int s = u / A.n_kv;
      if (A.seq[s].t == 0) continue;
      const int n = __ldg(A.n_live + s);
      if (n < 0 || n > A.seq[s].cap) {
        if (blockIdx.x == 0 && u == s * A.n_kv) report(A.ctrl, TRIA_ERR_DEVICE_ARG, (uint32_t)s);
        continue;
      }
      int lo = 0, hi = n;
      if (A.window > 0) {
        lo = A.span[2 * u];
        hi = A.span[2 * u + 1];
      }
      s_lo[u] = lo;
      s_hi[u] = hi;
      cnt[i] = max(1, (min(A.sink, lo) + TR - 1) / TR + (hi - lo + TR - 1) / TR);
      local += cnt[i];
    }
    int tot;
    int before = block_exclusive_scan(local, &tot, s_scan);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int u = (int)threadIdx.x * kPer + i;
      if (u < n_units) s_first[u] = before;
      before += cnt[i];
    }
    if (threadIdx.x == 0) s_first[n_units] = tot;
    __syncthreads();
  }
  const int64_t total = s_first[n_units];
  if (total == 0) return;
  const int64_t workers = min((int64_t)gridDim.x, (total + kWarps - 1) / kWarps);
  if ((int64_t)blockIdx.x >= workers) return;
  auto start_of = [&](int64_t i) { return i * total / workers; };
  const int64_t begin = start_of(blockIdx.x), end = start_of(blockIdx.x + 1);
  auto warp_start = [&](int64_t w) { return begin + (end - begin) * w / kWarps; };
  const int64_t wb = warp_start(warp), we = warp_start(warp + 1);   // this warp's run
  auto unit_of = [&](int64_t tile) {                       // the last unit that starts at or before it
    int u = 0, hi_u = n_units - 1;
    while (u < hi_u) {
      const int mid = (u + hi_u + 1) >> 1;
      if (s_first[mid] <= tile) u = mid; else hi_u = mid - 1;
    }
    return u;
  };
  constexpr int kSlot = kCol * (HD + 2);                   // a part: M, l per column, O [column][dim]

  const Magic mg;
  uint8_t* area = smem + warp * H::kArea;

  // a tile's rows in its segment (rows <= 0: none)
  auto tile_row = [&](int unit, int64_t tile, int& rows) {
    const int j = (int)(tile - s_first[unit]), lo = s_lo[unit];
    const int sr = min(A.sink, lo), nt_sink = (sr + TR - 1) / TR;
    if (j < nt_sink) {
      rows = min(TR, sr - j * TR);
      return j * TR;
    }
    const int r = lo + (j - nt_sink) * TR;
    rows = min(TR, s_hi[unit] - r);
    return r;
  };
  auto row_base = [&](int unit) {
    const int s = unit / A.n_kv;
    return A.seq[s].row0 + (int64_t)(unit - s * A.n_kv) * A.seq[s].cap;
  };
  int p_unit = wb < we ? unit_of(wb) : 0;                  // of the tile to fetch next
  int64_t p_row0 = row_base(p_unit);
  auto issue = [&](int64_t tile, int st) {
    if (tile >= s_first[p_unit + 1]) {
      do ++p_unit;
      while (tile >= s_first[p_unit + 1]);
      p_row0 = row_base(p_unit);
    }
    int rows;
    const int r = tile_row(p_unit, tile, rows);
    if (rows <= 0) return;
    uint8_t* d = area + st * H::SB;
    const uint8_t* ks = A.k + (p_row0 + r) * H::kRb;
    const uint8_t* vsrc = A.v + (p_row0 + r) * H::vRb;
    constexpr int kc = H::kRb / 16, vc = H::vRb / 16;      // 16-byte pieces of a row
#pragma unroll
    for (int i = 0; i < (TR * kc + 31) / 32; ++i) {
      const int x = i * 32 + lane, rr = x / kc, c = x - rr * kc;
      if (rr < rows) cp_async16(d + rr * H::kStride + c * 16, ks + rr * H::kRb + c * 16);
    }
#pragma unroll
    for (int i = 0; i < (TR * vc + 31) / 32; ++i) {
      const int x = i * 32 + lane, rr = x / vc, c = x - rr * vc;
      if (rr < rows) cp_async16(d + H::oV + rr * H::vStride + c * 16, vsrc + rr * H::vRb + c * 16);
    }
    auto copy_scales = [&](uint8_t* dst, const uint8_t* src) {
      if constexpr (H::scRb == 16) cp_async16(dst, src);
      else if constexpr (H::scRb == 8) cp_async8(dst, src);
      else if constexpr (H::scRb == 4) cp_async4(dst, src);
      else                                                 // six bytes: no asynchronous copy's size
#pragma unroll
        for (int i = 0; i < NB; ++i)
          reinterpret_cast<uint16_t*>(dst)[i] = __ldg(reinterpret_cast<const uint16_t*>(src) + i);
    };
    if (lane < rows) {
      if constexpr (H::kKq) copy_scales(d + H::oKs + lane * H::scRb, A.ks + (p_row0 + r + lane) * H::scRb);
      if constexpr (H::kVq) copy_scales(d + H::oVs + lane * H::scRb, A.vs + (p_row0 + r + lane) * H::scRb);
      cp_async4(d + H::oPos + lane * 4, A.cpos + p_row0 + r + lane);
    }
  };
  // the first tiles are on their way before anything else is asked for
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (wb + i < we) issue(wb + i, i);
    cp_async_commit();
  }

  int st = 0;
  int64_t at = wb;
  for (int unit = p_unit < n_units && wb < we ? unit_of(wb) : n_units; at < we; ++unit) {
    if (s_first[unit + 1] <= at) continue;                 // (a unit without tiles)
    const int s = unit / A.n_kv, g = unit - s * A.n_kv;
    const AttendSeq& S = A.seq[s];
    const int ncol = S.t * A.G;
    // ---- queries: A fragments, columns gid and gid + 8; qf: their exponent
    uint32_t qa[NB * 2][2 * NT];                           // [step][column half * 2 ... k low, k high]
    float qf[NT];
    int pq[NT];
    uint32_t raw[NT][NB][4];                               // pairs of fp16 or bf16, on their way before the positions
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      const int col = gid + 8 * h;
      const bool on = col < ncol;
      const int tok = S.tok0 + (on ? col / A.G : 0);
      const int64_t qoff = (int64_t)tok * A.q_stride + (int64_t)(g * A.G + (on ? col % A.G : 0)) * HD;
      const uint16_t* qp = reinterpret_cast<const uint16_t*>(A.q) + qoff;
      pq[h] = on ? A.pos[tok] : INT32_MIN;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        // dims of the thread: fp16 keys 2t, 2t+1, 8+2t, 9+2t (+16); codes 4t .. 4t+3 (+16)
        if constexpr (H::kKq) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint2 v = on ? *reinterpret_cast<const uint2*>(qp + 32 * b + 16 * k + 4 * t4) : make_uint2(0, 0);
            raw[h][b][2 * k] = v.x;
            raw[h][b][2 * k + 1] = v.y;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            raw[h][b][k] = on ? *reinterpret_cast<const uint32_t*>(qp + 32 * b + 8 * k + 2 * t4) : 0u;
        }
      }
    }
    int pmin = INT32_MAX, pmax = INT32_MIN;
    for (int i = 0; i < S.t; ++i) {
      const int p = A.pos[S.tok0 + i];
      pmin = min(pmin, p);
      pmax = max(pmax, p);
    }

#pragma unroll
    for (int h = 0; h < NT; ++h) {
      float x[NB][8];
      float am = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w = raw[h][b][k];
          const float2 f = A.type == TRIA_F16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
                                              : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
          x[b][2 * k] = f.x;
          x[b][2 * k + 1] = f.y;
          am = fmaxf(am, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      qf[h] = A.scale * 1.4426950408889634f;
      float f = 1.f;
      if (A.type != TRIA_F16) {
        // bf16's range into fp16's: times a power of two, undone in the logits
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        const int ex = (int)((__float_as_uint(am) >> 23) & 255u) - 127;
        if (ex > -120 && ex < 120) {
          f = __uint_as_float((uint32_t)(127 - ex) << 23);
          qf[h] *= __uint_as_float((uint32_t)(127 + ex) << 23);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float* y = &x[b][4 * k];
          if constexpr (H::kKq) {
            qa[2 * b + k][2 * h] = pack_h2(y[0] * f, y[2] * f);
            qa[2 * b + k][2 * h + 1] = pack_h2(y[1] * f, y[3] * f);
          } else {
            qa[2 * b + k][2 * h] = pack_h2(y[0] * f, y[1] * f);
            qa[2 * b + k][2 * h + 1] = pack_h2(y[2] * f, y[3] * f);
          }
        }
    }
    auto qfrag = [&](int st, uint32_t* a) {
      a[0] = qa[st][0];
      a[2] = qa[st][1];
      a[1] = NT == 2 ? qa[st][2 * NT - 2] : 0u;
      a[3] = NT == 2 ? qa[st][2 * NT - 1] : 0u;
    };

    float M[NT], l[NT];
    float o[HD / 16][NT][4];
    int E = H::kVq ? -24 : 0;                              // exponent of the largest value scale so far
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      M[h] = -INFINITY;
      l[h] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < HD / 16; ++i)
#pragma unroll
      for (int h = 0; h < NT; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][h][c] = 0.f;

    auto tile = [&](auto masked_c, const uint8_t* tile_p, int r, int rows) {
      constexpr bool kMasked = decltype(masked_c)::value;
      const uint32_t base = smem_u32(tile_p);
      // this thread's words: keys of rows gid, values of rows 2t, 2t + 1, 2t + 8, 2t + 9
      const uint8_t* kp = tile_p + gid * H::kStride + t4 * 4;
      const uint8_t* vp = tile_p + H::oV + 2 * t4 * H::vStride + gid * (VT == TRIA_Q8_0 ? 4 : 2);
      // logits
      float sc[NG][2 * NT];
#pragma unroll
      for (int gq = 0; gq < NG; ++gq) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (!H::kKq) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t kf[4], a[4];
            ldsm4(kf, base + (gq * 8 + (lane & 7)) * H::kStride + b * 64 + (lane >> 3) * 16);
            qfrag(2 * b, a);
            mma16816(acc, a, kf[0], kf[1]);
            qfrag(2 * b + 1, a);
            mma16816(acc, a, kf[2], kf[3]);
          }
        } else {
          // scales of rows 2t, 2t + 1
          float ks0[NB], ks1[NB];
          load_scales<NB>(tile_p + H::oKs + (gq * 8 + 2 * t4) * H::scRb, ks0, ks1);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t h[4], a[4];
            if constexpr (KT == TRIA_Q8_0) {
              q8_pairs(mg, get32(kp + gq * 8 * H::kStride + b * 32), h);
              q8_pairs(mg, get32(kp + gq * 8 * H::kStride + b * 32 + 16), h + 2);
            } else {
              q4_pairs(mg, get32(kp + gq * 8 * H::kStride + b * 16), h);
            }
            qfrag(2 * b, a);
            mma16816(c, a, h[0], h[1]);
            qfrag(2 * b + 1, a);
            mma16816(c, a, h[2], h[3]);
            const float s0 = ks0[b], s1 = ks1[b];
            acc[0] = fmaf(c[0], s0, acc[0]);
            acc[1] = fmaf(c[1], s1, acc[1]);
            if constexpr (NT == 2) {
              acc[2] = fmaf(c[2], s0, acc[2]);
              acc[3] = fmaf(c[3], s1, acc[3]);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          sc[gq][2 * h] = acc[2 * h] * qf[h];
          sc[gq][2 * h + 1] = acc[2 * h + 1] * qf[h];
        }
      }
      const int32_t* tp = reinterpret_cast<const int32_t*>(tile_p + H::oPos);
      auto sees = [&](int row, int p) {                    // row of the tile, position of the query
        if (row >= rows) return false;
        const int q = tp[row];
        return q <= p && (A.window <= 0 || (int64_t)p - q < A.window || r + row < A.sink);
      };
      if constexpr (kMasked) {
#pragma unroll
        for (int gq = 0; gq < NG; ++gq)
#pragma unroll
          for (int h = 0; h < NT; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (!sees(gq * 8 + 2 * t4 + c, pq[h])) sc[gq][2 * h + c] = -INFINITY;
      }
      // largest value scale
      int En = E;
      if constexpr (H::kVq) {
        float big = 0.f;
        const __half2* vss = reinterpret_cast<const __half2*>(tile_p + H::oVs);
        // all scales of the tile, spread over the lanes: TR * NB / 2 pairs (with an
        // odd number of blocks, some pairs belong to two rows)
#pragma unroll
        for (int i = 0; i < (TR * NB / 2 + 31) / 32; ++i) {
          const int x = i * 32 + lane;
          bool on = x < TR * NB / 2, on2 = on;
          if constexpr (kMasked) {                         // rows that some token sees
            auto some = [&](int row) {
              return row < rows && tp[row] <= pmax && (A.window <= 0 || (int64_t)pmin - tp[row] < A.window || r + row < A.sink);
            };
            on = on && some(2 * x / NB);
            on2 = NB % 2 == 0 ? on : on2 && some((2 * x + 1) / NB);
          }
          if (on || on2) {
            const float2 f = __half22float2(__habs2(vss[x]));
            if (on && f.x <= 65504.f) big = fmaxf(big, f.x);
            if (on2 && f.y <= 65504.f) big = fmaxf(big, f.y);
          }
        }
        // the exponent above the largest one (its bits order like integers)
        const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
        En = max(E, min((int)(bits >> 23) - 126, 17));
      }
      // running reference
      float Mn[NT];
      bool grow = En != E;
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        float top = -INFINITY;
#pragma unroll
        for (int gq = 0; gq < NG; ++gq) top = fmaxf(top, fmaxf(sc[gq][2 * h], sc[gq][2 * h + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        Mn[h] = fmaxf(M[h] + (float)(En - E), top + (float)(En - 14));
        grow = grow || Mn[h] > M[h];
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int h = 0; h < NT; ++h) {
          const float a = M[h] == -INFINITY ? 0.f : exp2_approx(M[h] - Mn[h]);
          l[h] *= a;
          M[h] = Mn[h];
          // the accumulator's columns are 2t, 2t + 1
          const float a0 = __shfl_sync(0xffffffffu, a, 8 * t4), a1 = __shfl_sync(0xffffffffu, a, 8 * t4 + 4);
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) {
            o[i][h][0] *= a0;
            o[i][h][1] *= a1;
            o[i][h][2] *= a0;
            o[i][h][3] *= a1;
          }
        }
        E = En;
      }
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        const float mb = M[h] == -INFINITY ? 0.f : M[h];
#pragma unroll
        for (int gq = 0; gq < NG; ++gq)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float w = exp2_approx(sc[gq][2 * h + c] - mb);
            sc[gq][2 * h + c] = w;
            l[h] += w;
          }
      }
      // weighted sum
      if constexpr (!H::kVq) {
#pragma unroll
        for (int k = 0; k < TR / 16; ++k) {
          uint32_t pb[NT][2];
#pragma unroll
          for (int h = 0; h < NT; ++h) {
            pb[h][0] = pack_h2(sc[2 * k][2 * h], sc[2 * k][2 * h + 1]);
            pb[h][1] = pack_h2(sc[2 * k + 1][2 * h], sc[2 * k + 1][2 * h + 1]);
          }
          const uint32_t va = base + H::oV + (k * 16 + (lane & 7) + ((lane >> 4) << 3)) * H::vStride + ((lane >> 3) & 1) * 16;
          if constexpr (!kMasked) {
#pragma unroll
            for (int i = 0; i < HD / 16; ++i) {
              uint32_t vf[4];
              ldsm4t(vf, va + i * 32);
#pragma unroll
              for (int h = 0; h < NT; ++h) mma16816(o[i][h], vf, pb[h][0], pb[h][1]);
            }
          } else {
            // token by token, rows that it does not see as zeros
            for (int tk = 0; tk < S.t; ++tk) {
              const int p = A.pos[S.tok0 + tk], rr = k * 16 + 2 * t4;
              const uint32_t m0 = (sees(rr, p) ? 0xFFFFu : 0u) | (sees(rr + 1, p) ? 0xFFFF0000u : 0u);
              const uint32_t m1 = (sees(rr + 8, p) ? 0xFFFFu : 0u) | (sees(rr + 9, p) ? 0xFFFF0000u : 0u);
#pragma unroll
              for (int i = 0; i < HD / 16; ++i) {
                uint32_t vf[4];
                ldsm4t(vf, va + i * 32);
                vf[0] &= m0;
                vf[1] &= m0;
                vf[2] &= m1;
                vf[3] &= m1;
#pragma unroll
                for (int h = 0; h < NT; ++h) {
                  // junk that this token sees stays out of the other columns
                  float c[4] = {0.f, 0.f, 0.f, 0.f};
                  mma16816(c, vf, pb[h][0], pb[h][1]);
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    if ((2 * t4 + (x & 1) + 8 * h) / A.G == tk) o[i][h][x] += c[x];
                }
              }
            }
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < TR / 16; ++k) {
          float vs0[NB], vs1[NB], vs2[NB], vs3[NB];        // of rows 2t, 2t + 1, 2t + 8, 2t + 9
          load_scales<NB>(tile_p + H::oVs + (k * 16 + 2 * t4) * H::scRb, vs0, vs1);
          load_scales<NB>(tile_p + H::oVs + (k * 16 + 8 + 2 * t4) * H::scRb, vs2, vs3);
          const uint8_t* vr = vp + k * 16 * H::vStride;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t pb[NT][2];
            const float s[4] = {vs0[b], vs1[b], vs2[b], vs3[b]};
#pragma unroll
            for (int h = 0; h < NT; ++h) {
              float x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float w = sc[2 * k + (i >> 1)][2 * h + (i & 1)];
                x[i] = kMasked && w == 0.f ? 0.f : w * s[i];   // a hidden row's scale never counts
              }
              pb[h][0] = pack_h2(x[0], x[1]);
              pb[h][1] = pack_h2(x[2], x[3]);
            }
            uint32_t f0[4], f1[4];                         // rows 2t, 2t+1 and 2t+8, 2t+9 of four dims
            if constexpr (VT == TRIA_Q8_0) {
              const uint8_t* w = vr + b * 32;
              const uint32_t w0 = get32(w), w1 = get32(w + H::vStride), w2 = get32(w + 8 * H::vStride), w3 = get32(w + 9 * H::vStride);
              q8_pairs(mg, __byte_perm(w0, w1, 0x5410), f0);
              q8_pairs(mg, __byte_perm(w0, w1, 0x7632), f0 + 2);
              q8_pairs(mg, __byte_perm(w2, w3, 0x5410), f1);
              q8_pairs(mg, __byte_perm(w2, w3, 0x7632), f1 + 2);
            } else {
              const uint8_t* w = vr + b * 16;
              q4_pairs(mg, __byte_perm(get16(w), get16(w + H::vStride), 0x5410), f0);
              q4_pairs(mg, __byte_perm(get16(w + 8 * H::vStride), get16(w + 9 * H::vStride), 0x5410), f1);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t vf[4] = {f0[2 * i], f0[2 * i + 1], f1[2 * i], f1[2 * i + 1]};
#pragma unroll
              for (int h = 0; h < NT; ++h) mma16816(o[2 * b + i][h], vf, pb[h][0], pb[h][1]);
            }
          }
        }
      }
    };

    const int64_t last_tile = min(we, (int64_t)s_first[unit + 1]);
    for (; at < last_tile; ++at) {
      if (at + kStages - 1 < we) issue(at + kStages - 1, st == 0 ? kStages - 1 : st - 1);
      cp_async_commit();
      cp_async_wait<kStages - 1>();
      __syncwarp();
      int rows;
      const int r = tile_row(unit, at, rows);
      const uint8_t* tile_p = area + st * H::SB;
      if (rows > 0) {
        const int32_t* tp = reinterpret_cast<const int32_t*>(tile_p + H::oPos);
        const int first = tp[0], last = tp[rows - 1];
        const bool skip = first > pmax || (A.window > 0 && (int64_t)pmin - last >= A.window && r >= A.sink);
        const bool masked = rows < TR || last > pmin ||
                            (A.window > 0 && (int64_t)pmax - first >= A.window && r + rows > A.sink);
        if (!skip) {
          if (masked) tile(std::true_type{}, tile_p, r, rows);
          else tile(std::false_type{}, tile_p, r, rows);
        }
      }
      __syncwarp();
      st = st + 1 == kStages ? 0 : st + 1;
    }

    // ---- the unit's result, or this run's part of it
#pragma unroll
    for (int h = 0; h < NT; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    auto dim_of = [&](int i, int c) {                      // the dim of an accumulator's row
      if constexpr (VT == TRIA_F16) return 16 * i + gid + 8 * (c >> 1);
      else if constexpr (VT == TRIA_Q8_0) return 32 * (i >> 1) + 4 * gid + 2 * (i & 1) + (c >> 1);
      else return 32 * (i >> 1) + 16 * (i & 1) + 2 * gid + (c >> 1);
    };
    const bool early = s_first[unit] < wb;                 // it began in an earlier run
    if (!early && s_first[unit + 1] <= we) {
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        const int col = gid + 8 * h;
        if (A.lse && t4 == 0 && col < ncol)
          A.lse[(int64_t)(S.tok0 + col / A.G) * A.nq + g * A.G + col % A.G] =
              l[h] == 0.f ? -INFINITY : (M[h] + log2f(l[h])) * 0.6931471805599453f;
        const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];
#pragma unroll
        for (int e = 0; e < 2; ++e) {                      // columns 2t, 2t + 1
          const float f = __shfl_sync(0xffffffffu, inv, 8 * t4 + 4 * e);
          const int c2 = 2 * t4 + e + 8 * h;
          if (c2 >= ncol) continue;
          const int64_t to = (int64_t)(S.tok0 + c2 / A.G) * A.out_stride + (int64_t)(g * A.G + c2 % A.G) * HD;
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) {
            act_store(A.out, A.out_type, to + dim_of(i, 0), o[i][h][e] * f);
            act_store(A.out, A.out_type, to + dim_of(i, 2), o[i][h][2 + e] * f);
          }
        }
      }
    } else {
      // the run's last unit: into its stages, which nothing uses any more
      float* slot = at == we ? reinterpret_cast<float*>(area) : A.part + (int64_t)(blockIdx.x * kWarps + warp) * kSlot;
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        if (t4 == 0) {
          slot[gid + 8 * h] = M[h];
          slot[kCol + gid + 8 * h] = l[h];
        }
#pragma unroll
        for (int i = 0; i < HD / 16; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) slot[2 * kCol + (2 * t4 + (c & 1) + 8 * h) * HD + dim_of(i, c)] = o[i][h][c];
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // ---- units that several runs share; a thread merges four dims of a column
  auto add = [&](float4& v, float f, const float4& x) {
    v.x = fmaf(x.x, f, v.x);
    v.y = fmaf(x.y, f, v.y);
    v.z = fmaf(x.z, f, v.z);
    v.w = fmaf(x.w, f, v.w);
  };
  float* cta_parts = A.part + (int64_t)gridDim.x * kWarps * kSlot;
  const int len = (int)(end - begin);
  auto write = [&](int unit, int col, int d, const float4& val, float top, float sum) {
    const int s = unit / A.n_kv, head = (unit - s * A.n_kv) * A.G + col % A.G;
    const int64_t tok = A.seq[s].tok0 + col / A.G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (d == 0 && A.lse) A.lse[tok * A.nq + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    if (A.out_type == TRIA_F32) {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(A.out) + tok * A.out_stride + (int64_t)head * HD + d) =
          make_float4(val.x * inv, val.y * inv, val.z * inv, val.w * inv);
      return;
    }
    uint32_t w[2];
    if (A.out_type == TRIA_F16) {
      w[0] = pack_h2(val.x * inv, val.y * inv);
      w[1] = pack_h2(val.z * inv, val.w * inv);
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(val.x * inv, val.y * inv), b = __floats2bfloat162_rn(val.z * inv, val.w * inv);
      w[0] = *reinterpret_cast<const uint32_t*>(&a);
      w[1] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(A.out) + tok * A.out_stride + (int64_t)head * HD + d) = make_uint2(w[0], w[1]);
  };
  int open[2] = {-1, -1};                                  // units that reach into other CTAs: the first, the last
  for (int unit = unit_of(begin); unit < n_units && s_first[unit] < end; ++unit) {
    const int64_t u0 = s_first[unit], u1 = s_first[unit + 1];
    if (u1 <= begin || u0 == u1) continue;
    const bool inside = u0 >= begin && u1 <= end;
    const int x0 = (int)(max(u0, begin) - begin), x1 = (int)(min(u1, end) - 1 - begin);
    const int w0 = ((x0 + 1) * kWarps - 1) / len, w1 = ((x1 + 1) * kWarps - 1) / len;
    if (inside && w0 == w1) continue;                      // written by its warp
    // the runs that have tiles of it, and those of them whose last unit it is
    // (their parts lie in their stages)
    uint32_t have = 0, staged = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int e = len * (w + 1) / kWarps;
      if (w < w0 || w > w1 || e == len * w / kWarps) continue;
      have |= 1u << w;
      if (e <= (int)(u1 - begin)) staged |= 1u << w;
    }
    const int which = u0 < begin ? 0 : 1;
    if (!inside) open[which] = unit;
    float* mine = cta_parts + ((int64_t)blockIdx.x * 2 + which) * kSlot;
    for (int i = threadIdx.x; i < A.seq[unit / A.n_kv].t * A.G * (HD / 4); i += kWarps * 32) {
      const int col = i / (HD / 4), d = 4 * (i - col * (HD / 4));
      auto part = [&](int w) {
        return (staged >> w) & 1u ? reinterpret_cast<const float*>(smem + w * H::kArea)
                                  : A.part + (int64_t)(blockIdx.x * kWarps + w) * kSlot;
      };
      // (loads without branches, in the place of a part that is not there one that is:
      // they are in flight together)
      float m[kWarps], l[kWarps];
      float4 v[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* x = part((have >> w) & 1u ? w : w0);
        m[w] = x[col];
        l[w] = x[kCol + col];
        v[w] = *reinterpret_cast<const float4*>(x + 2 * kCol + col * HD + d);
      }
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (!((have >> w) & 1u)) m[w] = -INFINITY;
        top = fmaxf(top, m[w]);
      }
      const float tb = top == -INFINITY ? 0.f : top;
      float4 val = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if ((have >> w) & 1u) {                            // (a NaN in another's part stays there)
          const float f = exp2_approx(m[w] - tb);
          sum = fmaf(l[w], f, sum);
          add(val, f, v[w]);
        }
      if (inside) {
        write(unit, col, d, val, top, sum);
      } else {
        *reinterpret_cast<float4*>(mine + 2 * kCol + col * HD + d) = val;
        if (d == 0) {
          mine[col] = top;
          mine[kCol + col] = sum;
        }
      }
    }
  }
  __threadfence();
  __syncthreads();
  // the CTAs of a unit: those whose runs meet its tiles
  auto cta_of = [&](int64_t tile) { return (int)(((tile + 1) * workers - 1) / total); };
  if (threadIdx.x < 2) {
    const int unit = threadIdx.x == 0 ? open[0] : open[1];
    s_flag[threadIdx.x] = 0;
    if (unit >= 0) {
      const int others = cta_of(s_first[unit + 1] - 1) - cta_of(s_first[unit]);
      s_flag[threadIdx.x] = atomicAdd(A.count + unit, 1u) == (uint32_t)others;
      __threadfence();
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (!s_flag[which]) continue;
    const int unit = which == 0 ? open[0] : open[1];
    const int c0 = cta_of(s_first[unit]), c1 = cta_of(s_first[unit + 1] - 1);
    for (int i = threadIdx.x; i < A.seq[unit / A.n_kv].t * A.G * (HD / 4); i += kWarps * 32) {
      const int col = i / (HD / 4), d = 4 * (i - col * (HD / 4));
      float top = -INFINITY, sum = 0.f;
      float4 val = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = c0; c <= c1; c += 8) {                  // eight parts' loads at a time
        float m[8], l8[8];
        float4 v8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int ck = min(c + k, c1);
          const float* x = cta_parts + ((int64_t)ck * 2 + (ck > c0 ? 0 : 1)) * kSlot;   // only the first does not start inside
          m[k] = __ldcg(x + col);
          l8[k] = __ldcg(x + kCol + col);
          v8[k] = __ldcg(reinterpret_cast<const float4*>(x + 2 * kCol + col * HD + d));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k > c1) m[k] = -INFINITY;
        float mn = top;
#pragma unroll
        for (int k = 0; k < 8; ++k) mn = fmaxf(mn, m[k]);
        const float tb = mn == -INFINITY ? 0.f : mn, f0 = exp2_approx(top - tb);
        sum *= f0;
        val = make_float4(val.x * f0, val.y * f0, val.z * f0, val.w * f0);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k <= c1) {
            const float f = exp2_approx(m[k] - tb);
            sum = fmaf(l8[k], f, sum);
            add(val, f, v8[k]);
          }
        top = mn;
      }
      write(unit, col, d, val, top, sum);
    }
    if (threadIdx.x == 0) A.count[unit] = 0u;
  }
}

template <int KT, int VT, int HD, int NT>
cudaError_t launch_attend_step_t(const AttendArgs& A, int workers, cudaStream_t st) {
  using H = StepShape<KT, VT, HD, NT>;
  auto kern = k_attend_step<KT, VT, HD, NT>;
  const int smem = H::kArea * H::kWarps;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<workers, H::kWarps * 32, smem, st>>>(A);
  return cudaGetLastError();
}

template <int KT, int VT>
cudaError_t launch_attend_step_kv(const AttendArgs& A, int cols, int workers, cudaStream_t st) {
  const bool one = cols <= 8;
  switch (A.hd) {
    case 64: return one ? launch_attend_step_t<KT, VT, 64, 1>(A, workers, st) : launch_attend_step_t<KT, VT, 64, 2>(A, workers, st);
    case 96: return one ? launch_attend_step_t<KT, VT, 96, 1>(A, workers, st) : launch_attend_step_t<KT, VT, 96, 2>(A, workers, st);
    case 128: return one ? launch_attend_step_t<KT, VT, 128, 1>(A, workers, st) : launch_attend_step_t<KT, VT, 128, 2>(A, workers, st);
    case 256: return one ? launch_attend_step_t<KT, VT, 256, 1>(A, workers, st) : launch_attend_step_t<KT, VT, 256, 2>(A, workers, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace tria
