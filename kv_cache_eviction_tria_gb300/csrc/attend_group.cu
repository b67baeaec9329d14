// Attention of many sequences' new tokens over one shared prefix, on the
// fifth-generation tensor cores: a decode step, or a few tokens each.
//
//   S = Q K^T (128 x BN, fp32 in TMEM), P = 2^(scale S - M) (fp16, written over
//   S in TMEM), O += P V (128 x head_dim, fp32 in TMEM), l = sum of P
//
// Up to 128 columns of a prefix and KV head are one unit. A step has few columns
// and many rows, so the rows are what is cut: the tiles of all units (BN
// rows each) are one list, cut into equal runs, one per CTA, neighbouring units'
// tiles of the same rows near one another in time. The live rows are known on
// the device alone, and ragged prefixes stay balanced. A CTA streams its
// run from unit to unit; each unit it meets leaves a part (M, l, O) in the
// workspace, in the place unit + CTA, which no two parts share. The parts are
// joined with the sequences' own rows by a kernel of their own.
//
// Queries lie in TMEM, so that the products read one operand from shared
// memory and leave half of its rate for filling the tiles. fp16 planes come by
// TMA. Codes come by bulk copies as they lie, and a warpgroup for keys and one for
// values widen them tile by tile on their way into the swizzled ones (each row once
// for 128 columns: the prompt kernel, whose units meet every row again and again,
// widens the planes in memory instead): values rounded once, keys as the rounded
// value and the remainder, which takes a product of its own (kLow).
//
// Two warpgroups take the tiles' softmax in turn, a thread per column of the
// unit. Scores are made two or three tiles ahead of the sums, in four buffers, so that
// neither the warpgroups nor the products wait for a tile that is being widened. Both
// warpgroups' weights add to one O, so the reference M is handed on from tile
// to tile through shared memory, before the weights are made. (With tiles of
// 128 rows the ring held too few of them: a tile's sums waited for the next
// tile's keys, and those for the sums' place, 2.4 us in turn.)
//
// Masks, junk in hidden rows, the lazy reference M and the bounded waits are those of
// the prompt kernel.
//
// 32768 fp16 rows of 8 KV heads x 128 dims, 128 columns: 33 us, 134 MB. Memory
// bounds the tiles (5.6 TB/s from the first queries to the last tile); 6 us before them go
// into the kernel's start, the tile list and the queries, while the ring fills. 512
// columns take 91 us, bound by the softmax and its hand-overs (1.42 us per 128 rows and
// 128 columns). 65536 q8_0 rows, 256 columns: 120 us, 1.95 us per 128 rows and 128 columns;
// q4_0 2.3. There the warpgroup that widens keys sets the pace: 1000 of a tile's 2240
// cycles are its conversions, the rest waits, fences and meetings. Roles at work side by
// side are bound by the supply of instructions, not by a unit: the SM's instruction cache
// gives 0.70 of the requests it can, 0.04 of them from further away, for 0.54 of
// the issue slots, and what lets more roles run at once makes each of them
// slower. With a quarter of the keys widened by the values' warpgroup the same rows took
// 155 us, with both warpgroups widening keys and values of tiles in turn 150, and with keys that need not
// wait for sums (two rings, scores three tiles ahead) 127.
#include <string.h>

#include <algorithm>

#include "attend_tc.cuh"

namespace tria {

namespace {

constexpr int kScSlots = 8, kScAhead = 4;   // tiles whose scales are held, and of these on their way

template <int HD, bool kQuant>
struct GroupShape {
  static constexpr int BN = HD == 256 ? 32 : 64;           // rows of a tile
  static constexpr int kStage = BN * HD * 2;
  static constexpr int kStages = kQuant ? 8 : 12;
  static constexpr int kRaw = BN * HD;                     // bytes of a plane's q8_0 codes
  static constexpr int kRawSlots = kQuant ? 4 : 0;         // of q8_0 codes; of 4-bit ones twice as many
  static constexpr int kRawArea = kRawSlots * kRaw;        // of a plane
  static constexpr int kPosTiles = 8;                      // more tiles than the ring holds values of
  static constexpr int kScTile = BN * HD / 16;             // bytes of a tile's block scales, of a plane
  static constexpr int oRing = 0, oRaw = kStages * kStage, oPos = oRaw + 2 * kRawArea, oScale = oPos + kPosTiles * BN * 4;
  static constexpr int oRef = oScale + (kQuant ? 2 * kScSlots * kScTile : 0);   // [warpgroup][row], then [parity][warpgroup][row]
  static constexpr int oBar = oRef + 6 * 128 * 4;
  static constexpr int kSmem = oBar + 1024;
  // TMEM columns: score buffers, outputs, queries
  static constexpr int cS = 0, cO = 4 * BN, cQ = cO + HD;
  static_assert(cQ + HD / 2 <= 512, "TMEM");
  static_assert(kSmem + (3 * kMaxSegments + 256) * 4 <= 227 * 1024, "shared memory");
};

constexpr int kGroupBars = 2 * 12 + 4 + 4 + 4 + 4 + 4 * 8;
struct GroupShared {
  uint32_t junk[12][4];                                    // rows of a value tile that held junk, by stage
  int32_t lo[8], hi[8], c_lo[4], c_hi[4];                  // positions, a warp each
  uint32_t tmem, abort;
};
static_assert(kGroupBars * 8 + sizeof(GroupShared) <= 1024, "barriers and shared state");

// two warpgroups of softmax, one that widens keys, one that widens or looks through
// values, one whose first warp issues the products and whose next ones start copies
constexpr int kGroupThreads = 640, kGroupIssue = 16, kGroupLoadK = 17, kGroupLoadV = 18, kConv = 128, kGroupRegs = 96;
// registers of a thread in each, cut from what the block starts with
constexpr int kGroupSoft = 128, kGroupConv = 80, kGroupOther = 64;
static_assert(2 * kGroupSoft + 2 * kGroupConv + kGroupOther == 5 * kGroupRegs, "register shares");

// Shared memory by its 32-bit addresses (through selected pointers, accesses
// became generic ones).
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t* v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// The rows of a tile of codes (rb bytes each) as fp16 tiles, by kConv threads; a
// thread has the same 16 dims of every kConv / (HD / 16)-th row. hi_t: code x
// scale, rounded; lo_t (kLow): what fp16 leaves of it, which fp16 holds exactly (a
// scale is a multiple of 2^-24 and a code whole, so 8 bits at most are left,
// all above 2^-24). kClean: rows from `rows` on become zeros, and so do pieces with
// junk, whose rows are marked. No branches, and short enough for four or five
// roles to stay in the instruction cache side by side: what bounds a warp here is
// the latency of its instructions (told apart at run time, types and planes
// cost a third more; 16 rows unrolled, twice as much).
template <int HD, int BN, bool kQ8, bool kLow, bool kClean>
__device__ __forceinline__ void widen_tile(uint32_t codes, int rb, uint32_t scale, int nb, uint32_t hi_t, uint32_t lo_t, int hd, int rows,
                                           uint32_t* marks, int tid) {
  constexpr int per = HD / 16, step = kConv / per, N = BN / step;   // threads of a row, rows of a thread
  static_assert(step % 8 == 0 && BN % step == 0, "a thread's rows have one place in the swizzle");
  // eight lanes store to two rows' four pieces of a 64-dim block: no bank conflicts
  const int c = (tid & 3) | (((tid >> 3) & (per / 4 - 1)) << 2), r0 = ((tid >> 2) & 1) | ((tid / (2 * per)) << 1);
  const bool there = 16 * c < hd;
  // q4_0: the low halves of a block's 16 bytes, or the high ones
  const uint32_t from = codes + r0 * rb + (there ? (kQ8 ? c * 16 : (c / 2) * 16) : 0);
  const uint32_t sc_at = scale + (there ? (r0 * nb + c / 2) * 2 : 0), sel = there ? 0x1010u : 0x4444u;
  const int up = (c & 1) * 4;
  const uint32_t at0 = (c >> 2) * (BN * 128) + swz(r0, (2 * c) & 7), at1 = at0 ^ 16;   // two neighbouring pieces
  constexpr uint32_t bias = kQ8 ? 0x64806480u : 0x64086408u;
  uint4 w[N];
  uint32_t sc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = lds128(from + i * step * rb);
    sc[i] = lds16(sc_at + i * step * nb * 2);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t s2 = __byte_perm(sc[i], 0u, sel);
    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    uint32_t v[8], hi[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // 0x64, byte: 1024 + it, exactly; less the bias, the code
      const uint32_t y = kQ8 ? x[k / 2] ^ 0x80808080u : (x[k / 2] >> up) & 0x0F0F0F0Fu;
      const uint32_t b = __byte_perm(y, 0x64646464u, k & 1 ? 0x4342 : 0x4140);
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(v[k]) : "r"(b), "r"(bias));
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(hi[k]) : "r"(v[k]), "r"(s2));
    }
    if constexpr (kLow) {
      uint32_t lo[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) asm("{\n .reg .b32 n;\n neg.f16x2 n, %3;\n fma.rn.f16x2 %0, %1, %2, n;\n}\n" : "=r"(lo[k]) : "r"(v[k]), "r"(s2), "r"(hi[k]));
      sts128(lo_t + at0 + i * step * 128, lo);
      sts128(lo_t + at1 + i * step * 128, lo + 4);
    }
    if constexpr (kClean) {
      const int rr = r0 + i * step;
      bool junk = false;
#pragma unroll
      for (int k = 0; k < 8; ++k) junk = junk || junk_h2(hi[k]);
      if (rr < rows && junk) atomicOr(&marks[rr >> 5], 1u << (rr & 31));
      if (rr >= rows || junk)
#pragma unroll
        for (int k = 0; k < 8; ++k) hi[k] = 0;
    }
    sts128(hi_t + at0 + i * step * 128, hi);
    sts128(hi_t + at1 + i * step * 128, hi + 4);
  }
}

// Starts the copy of a tile's block scales (nb halves a row, consecutive) by
// kConv threads. With an odd number of blocks a row may begin between two
// words, which no asynchronous copy takes: they are waited for.
__device__ __forceinline__ void copy_scales(uint16_t* to, const uint16_t* from, int n, bool words, int tid) {
  if (words) {
    if (2 * tid < n) cp_async4(to + 2 * tid, from + 2 * tid);
  } else {
    for (int i = tid; i < n; i += kConv) to[i] = __ldg(from + i);
  }
}

template <int HD, bool kQuant, bool kLow>
__global__ void __launch_bounds__(kGroupThreads, 1) k_attend_group(const __grid_constant__ AttendArgs A,
                                                                   const __grid_constant__ CUtensorMap map_k,
                                                                   const __grid_constant__ CUtensorMap map_v) {
  using H = GroupShape<HD, kQuant>;
  // ring entries of tile j: keys P j, their remainders P j + 1 (kLow), values P j + P - 1
  constexpr int P = kLow ? 3 : 2, BN = H::BN, ST = H::kStages;
  // tiles that scores are ahead of sums: less than there are buffers, and the keys' stages must not be those of
  // values whose sums come after them
  constexpr int kAhead = kLow ? 2 : 3;
  static_assert(P * kAhead + P - 2 < ST, "stages");
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int s_first[kMaxSegments + 1], s_lo[kMaxSegments], s_hi[kMaxSegments];   // of units: first tile, rows
  __shared__ int s_scan[40];
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + H::oBar);
  // full: a tile is in the ring; empty: its products are done; s: scores; p: weights; o: a tile's
  // sums (all three by score buffer); f: the unit's last sums; q: queries; x: every product; v: values that are looked
  // through before their tile is full; rf, re: codes (of keys, of values) are there, are used
  uint64_t *b_full = bar, *b_empty = bar + 12, *b_s = bar + 24, *b_p = b_s + 4, *b_o = b_p + 4, *b_f = b_o + 4, *b_q = b_f + 1,
           *b_x = b_q + 1, *b_v = b_x + 1, *b_rfk = b_v + 1, *b_rek = b_rfk + 8, *b_rfv = b_rek + 8, *b_rev = b_rfv + 8;
  int32_t* s_pos = reinterpret_cast<int32_t*>(smem + H::oPos);
  float* s_ref = reinterpret_cast<float*>(smem + H::oRef);
  GroupShared& X = *reinterpret_cast<GroupShared*>(smem + H::oBar + kGroupBars * 8);
  volatile uint32_t* s_abort = &X.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
  const bool kq = kQuant && A.k_type != TRIA_F16, vq = kQuant && A.v_type != TRIA_F16;

  // ---- the tile list
  auto seq_of = [&](int unit) {
    int s = 0, hi_s = A.n_seqs - 1;
#pragma unroll 1
    while (s < hi_s) {
      const int mid = (s + hi_s + 1) >> 1;
      if (A.seq[mid].unit0 <= unit) s = mid; else hi_s = mid - 1;
    }
    return s;
  };
  auto tiles_of = [&](int s) { return (A.seq[s].t * A.G + 127) / 128; };   // column tiles
  {
    constexpr int kPer = (kMaxSegments + kGroupThreads - 1) / kGroupThreads;
    int cnt[kPer], local = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      cnt[i] = 0;
      const int u = (int)threadIdx.x * kPer + i;
      if (u >= A.units) continue;
      const int s = seq_of(u), ct = tiles_of(s), g = (u - A.seq[s].unit0) / ct;
      const int n = *((volatile const int32_t*)(A.n_live + s));
      int lo = 0, hi = n;
      if (n < 0 || n > A.seq[s].cap) {
        if (blockIdx.x == 0 && u == A.seq[s].unit0) report(A.ctrl, TRIA_ERR_DEVICE_ARG, (uint32_t)s);
        hi = 0;
      } else if (A.window > 0) {
        lo = A.span[2 * (s * A.n_kv + g)];
        hi = A.span[2 * (s * A.n_kv + g) + 1];
      }
      s_lo[u] = lo;
      s_hi[u] = hi;
      cnt[i] = (min(A.sink, lo) + BN - 1) / BN + (hi - lo + BN - 1) / BN;
      local += cnt[i];
    }
    int tot;
    int before = block_exclusive_scan(local, &tot, s_scan);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int u = (int)threadIdx.x * kPer + i;
      if (u < A.units) {
        s_first[u] = before;
        if (blockIdx.x == 0) A.table[u] = before;
      }
      before += cnt[i];
    }
    if (threadIdx.x == 0) {
      s_first[A.units] = tot;
      if (blockIdx.x == 0) A.table[A.units] = tot;
    }
  }
  // The kernel starts while the one before it, over the sequences' own rows,
  // still runs on other SMs, and needs none of its results; but who waits for
  // this one to end has to find that one ended.
  auto leave = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
  if (smem_u32(smem) & 1023u) {                            // the swizzled tiles need it
    if (threadIdx.x == 0) report(A.ctrl, TRIA_ERR_CUDA, 0u);
    return leave();
  }
  if (threadIdx.x == 0) {
    X.abort = 0;
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mbar_init(&b_s[i], 1);
      mbar_init(&b_p[i], 128);
      mbar_init(&b_o[i], 1);
    }
    mbar_init(b_f, 1);
    mbar_init(b_q, 256);
    mbar_init(b_x, 1);
    mbar_init(b_v, 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mbar_init(&b_rfk[i], 1);
      mbar_init(&b_rek[i], 1);
      mbar_init(&b_rfv[i], 1);
      mbar_init(&b_rev[i], 1);
    }
    fence_mbar_init();
  }
  __syncthreads();
  const int total = s_first[A.units], workers = min((int)gridDim.x, total);
  if ((int)blockIdx.x >= workers) return leave();
  if (warp == kGroupIssue) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&X.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = X.tmem;
  asm volatile("griddepcontrol.launch_dependents;");       // (the join waits for this kernel's end; every SM has its CTA)
  // runs of `each` tiles, the first `more` of one more
  const int each = total / workers, more = total - each * workers, b = blockIdx.x;
  const int begin = b * each + min(b, more), end = begin + each + (b < more);
  auto unit_at = [&](int tile) {                           // the last unit that starts at or before it
    int u = 0, hi_u = A.units - 1;
#pragma unroll 1
    while (u < hi_u) {
      const int mid = (u + hi_u + 1) >> 1;
      if (s_first[mid] <= tile) u = mid; else hi_u = mid - 1;
    }
    return u;
  };
  const int unit_a = unit_at(begin);
  struct Unit {
    int s, g, c0, ncol, t0, t1;                            // sequence, KV head, columns, this run's tiles of it
    int lo, hi, sr, nt_sink;                               // rows besides the sink; the sink's rows and tiles
    int64_t row0;
  };
  auto unit_of = [&](int u) {
    Unit U;
    U.s = seq_of(u);
    const AttendSeq& S = A.seq[U.s];
    const int ct = tiles_of(U.s), x = u - S.unit0;
    U.g = x / ct;
    U.c0 = (x - U.g * ct) * 128;
    U.ncol = min(128, S.t * A.G - U.c0);
    U.lo = s_lo[u];
    U.hi = s_hi[u];
    U.sr = min(A.sink, U.lo);
    U.nt_sink = (U.sr + BN - 1) / BN;
    U.t0 = max(begin, s_first[u]) - s_first[u];            // (counted from the unit's first one)
    U.t1 = min(end, s_first[u + 1]) - s_first[u];
    U.row0 = S.row0 + (int64_t)U.g * S.cap;
    return U;
  };
  auto tile_row = [&](const Unit& U, int t, int& rows) {   // first row in the segment
    const bool sink = t < U.nt_sink;
    const int r = sink ? t * BN : U.lo + (t - U.nt_sink) * BN;
    rows = min(BN, (sink ? U.sr : U.hi) - r);
    return r;
  };
  // bounded waits, as in the prompt kernel: after one gave up nobody waits any more, no
  // results are written, and every role runs its loops to the end
  auto wait = [&](uint64_t* b, uint32_t parity) {
#pragma unroll 1
    for (int it = 0; it < kWaitLimit; ++it)
      if (mbar_try_wait(b, parity) || *s_abort) return;
    *s_abort = 1;
  };
  auto wait_warp = [&](uint64_t* b, uint32_t parity) {     // one answer for all lanes, see mbar_wait_warp
#pragma unroll 1
    for (int it = 0; it < kWaitLimit; ++it) {
      if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
      if (__any_sync(0xffffffffu, *s_abort != 0)) return false;
    }
    *s_abort = 1;
    return false;
  };
  auto stage = [&](int e) { return smem + H::oRing + (e % ST) * H::kStage; };
  auto free_stage = [&](int e) {
    if (e >= ST) wait(&b_empty[e % ST], ((e / ST) - 1) & 1);
  };
  const int tiles = end - begin;
  // codes as they lie: 2^slots tiles
  const int slots_k = A.k_type == TRIA_Q4_0 ? 3 : 2, slots_v = A.v_type == TRIA_Q4_0 ? 3 : 2;   // (logarithms)
  auto raw_k = [&](int j) { return smem + H::oRaw + (j & ((1 << slots_k) - 1)) * (H::kRawArea >> slots_k); };
  auto raw_v = [&](int j) { return smem + H::oRaw + H::kRawArea + (j & ((1 << slots_v) - 1)) * (H::kRawArea >> slots_v); };
  const int k_rb = A.k_type == TRIA_Q8_0 ? A.hd : A.hd / 2, v_rb = A.v_type == TRIA_Q8_0 ? A.hd : A.hd / 2;

  if (wg >= 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGroupOther));
  if (warp == kGroupIssue) {
    // ---- products (results of waits and addresses are the same in all lanes and kept in
    // such a form, see the prompt kernel)
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dk = tile_desc(smem_u32(smem + H::oRing), 16), dv = tile_desc(smem_u32(smem + H::oRing), BN * 128);
    auto scores = [&](int buf, int st, int sl) {
      const uint64_t b = dk + (uint64_t)(st * (H::kStage / 16));
      const uint32_t d = tm + H::cS + buf * BN, a = tm + H::cQ;
#pragma unroll
      for (int k = 0; k < HD / 16; ++k)
        tc_mma_ts(d, a + k * 8, b + (uint64_t)((k >> 2) * (BN * 8) + (k & 3) * 2), mma_desc(BN, false), k > 0);
      if constexpr (kLow) {
        const uint64_t bl = dk + (uint64_t)(sl * (H::kStage / 16));
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
          tc_mma_ts(d, a + k * 8, bl + (uint64_t)((k >> 2) * (BN * 8) + (k & 3) * 2), mma_desc(BN, false), 1);
      }
      tc_commit(&b_s[buf]);
      tc_commit(&b_empty[st]);
      if (kLow) tc_commit(&b_empty[sl]);
    };
    auto sums = [&](int buf, int st, bool add) {
      const uint64_t b = dv + (uint64_t)(st * (H::kStage / 16));
      const uint32_t d = tm + H::cO, a = tm + H::cS + buf * BN;
#pragma unroll
      for (int k = 0; k < BN / 16; ++k) tc_mma_ts(d, a + k * 8, b + (uint64_t)(k * 128), mma_desc(HD, true), add || k > 0);
      tc_commit(&b_o[buf]);
      tc_commit(&b_empty[st]);
    };
    bool ok = true;
    int j = 0, nu = 0;
#pragma unroll 1
    for (int u = unit_a; ok && j < tiles; ++u) {
      const int nt = min(end, s_first[u + 1]) - max(begin, s_first[u]);
      if (nt <= 0) continue;
      ok = wait_warp(b_q, nu & 1);
      // round i: the sums of tile j + i, then the scores of the tile kAhead further on, in the buffer that those of the
      // tile before have left
#pragma unroll 1
      for (int i = -kAhead; ok && i < nt; ++i) {
        if (i >= 0) {
          const int t = j + i, e = P * t + P - 1;
          ok = wait_warp(&b_full[e % ST], (e / ST) & 1) && wait_warp(&b_p[t & 3], (t >> 2) & 1);
          tc_fence_after();
          if (ok && elect_one()) {
            sums(t & 3, e % ST, i > 0);
            if (i + 1 == nt) tc_commit(b_f);
          }
          __syncwarp();
        }
        if (i + kAhead < nt) {
          const int t = j + i + kAhead, e = P * t;
          ok = ok && wait_warp(&b_full[e % ST], (e / ST) & 1) && (!kLow || wait_warp(&b_full[(e + 1) % ST], ((e + 1) / ST) & 1));
          tc_fence_after();
          if (ok && elect_one()) scores(t & 3, e % ST, (e + 1) % ST);
          __syncwarp();
        }
      }
      j += nt;
      ++nu;
    }
    // nothing may be running when the accumulators are given back
    if (elect_one()) tc_commit(b_x);
#pragma unroll 1
    for (int it = 0; it < kWaitLimit && !mbar_try_wait(b_x, 0); ++it) {
    }
  } else if (warp == kGroupLoadK || warp == kGroupLoadV) {
    // ---- key tiles of fp16 planes, codes of quantised ones (value tiles of fp16 planes are fetched by those who look
    // through them)
    const bool keys = warp == kGroupLoadK, codes = keys ? kq : vq;
    if (lane == 0 && (keys || codes)) {
      const uint8_t* plane = keys ? A.k : A.v;
      const int rb = keys ? k_rb : v_rb, slots = keys ? slots_k : slots_v;
      uint64_t *full = keys ? b_rfk : b_rfv, *empty = keys ? b_rek : b_rev;
      int j = 0;
#pragma unroll 1
      for (int u = unit_a; j < tiles; ++u) {
        if (min(end, s_first[u + 1]) <= max(begin, s_first[u])) continue;
        const Unit U = unit_of(u);
#pragma unroll 1
        for (int t = U.t0; t < U.t1; ++t, ++j) {
          int rows;
          const int r = tile_row(U, t, rows);
          if (!codes) {
            // hidden keys, and those past the last row, only reach logits that the mask replaces
            const int e = P * j;
            free_stage(e);
            if (!*s_abort) copy_tile<HD, BN>(stage(e), &map_k, U.row0 + r, &b_full[e % ST]);
          } else {
            const int x = j & ((1 << slots) - 1);
            if (j >> slots) wait(&empty[x], ((j >> slots) - 1) & 1);
            if (*s_abort) continue;
            mbar_arrive_expect_tx(&full[x], rows * rb);
            bulk_g2s(keys ? raw_k(j) : raw_v(j), plane + (U.row0 + r) * rb, rows * rb, &full[x]);
          }
        }
      }
      if (*s_abort) {                                      // waits, bounded, for copies still on their way
        for (int e = max(0, P * tiles - ST); e < P * tiles; ++e)
#pragma unroll 1
          for (int it = 0; it < 1024 && !codes && e % P == 0 && !mbar_try_wait(&b_full[e % ST], (e / ST) & 1); ++it) {
          }
#pragma unroll 1
        for (int i = max(0, tiles - (1 << slots)); i < tiles; ++i)
#pragma unroll 1
          for (int it = 0; it < 1024 && codes && !mbar_try_wait(&full[i & ((1 << slots) - 1)], (i >> slots) & 1); ++it) {
          }
      }
    }
  } else if (wg < 4 && wg >= 2) {
    // ---- codes into tiles, keys by one warpgroup and values by the other, which also keeps positions and looks through
    // values that some token does not see
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGroupConv));
    const int tid = threadIdx.x & 127, nb = A.hd / 32;
    const bool values = wg == 3, codes = values ? vq : kq;
    const uint16_t* scales = reinterpret_cast<const uint16_t*>(values ? A.vs : A.ks);
    const int rb = values ? v_rb : k_rb, slots = values ? slots_v : slots_k, entry = values ? P - 1 : 0;
    const bool q8 = (values ? A.v_type : A.k_type) == TRIA_Q8_0;
    uint64_t *raw_full = values ? b_rfv : b_rfk, *raw_empty = values ? b_rev : b_rek;
    auto meet = [&] { asm volatile("bar.sync %0, 128;" ::"r"(values ? 6 : 3) : "memory"); };
    auto scale = [&](int i) {
      return reinterpret_cast<uint16_t*>(smem + H::oScale + ((values ? kScSlots : 0) + (i & (kScSlots - 1))) * H::kScTile);
    };
    int j = 0, looked = 0;
#pragma unroll 1
    for (int u = unit_a; j < tiles && (values || codes); ++u) {
      if (min(end, s_first[u + 1]) <= max(begin, s_first[u])) continue;
      const Unit U = unit_of(u);
      const AttendSeq& S = A.seq[U.s];
      const int32_t* rpos = A.cpos + U.row0;
      const int j0 = j;
      auto fetch_scales = [&](int t) {
        int rows = 0;
        const int r = t < U.t1 ? tile_row(U, t, rows) : 0;
        copy_scales(scale(j0 + t - U.t0), scales + (U.row0 + r) * nb, rows * nb, nb % 2 == 0, tid);
        cp_async_commit();
      };
      int next_pos = INT32_MAX, pmin = 0, pmax = 0;        // position of this thread's row of the tile to come
      bool need_pos = values;                              // (until it is known)
      auto fetch_pos = [&](int t) {
        int rows = 0;
        const int r = t < U.t1 ? tile_row(U, t, rows) : 0;
        next_pos = need_pos && tid < rows ? rpos[r + tid] : INT32_MAX;
      };
      if (codes)
#pragma unroll 1
        for (int t = U.t0; t < U.t0 + kScAhead; ++t) fetch_scales(t);
      if (values) {
        // the tokens' positions, and whether they hide rows
        fetch_pos(U.t0);
        const int tok_a = U.c0 / A.G, tok_b = (U.c0 + U.ncol - 1) / A.G;
        int pl = INT32_MAX, ph = INT32_MIN;
        if (tok_a + tid <= tok_b) pl = ph = A.pos[S.tok0 + tok_a + tid];   // (128 columns at most)
        const int newest = s_hi[u] > 0 ? rpos[s_hi[u] - 1] : INT32_MIN;
        pl = __reduce_min_sync(0xffffffffu, pl);
        ph = __reduce_max_sync(0xffffffffu, ph);
        if (lane == 0) {
          X.c_lo[warp & 3] = pl;
          X.c_hi[warp & 3] = ph;
        }
        meet();
        pmin = min(min(X.c_lo[0], X.c_lo[1]), min(X.c_lo[2], X.c_lo[3]));
        pmax = max(max(X.c_hi[0], X.c_hi[1]), max(X.c_hi[2], X.c_hi[3]));
        need_pos = A.window > 0 || newest > pmin;
      }
#pragma unroll 1
      for (int t = U.t0; t < U.t1; ++t, ++j) {
        int rows;
        const int r = tile_row(U, t, rows), e = P * j + entry;
        // a warp for each thing to wait for (each costs 200 cycles even when it is there), then they meet
        const int which = warp & 3;
        if (which == 0) free_stage(e);
        else if (kLow && which == 1 && !values) free_stage(e + 1);
        else if (which == 2 && codes) wait(&raw_full[j & ((1 << slots) - 1)], (j >> slots) & 1);
        if (codes) {
          fetch_scales(t + kScAhead);
          cp_async_wait<kScAhead>();
        }
        int32_t* tp = s_pos + (j % H::kPosTiles) * BN;
        if (values) {
          // positions and marks go with the value tile, which stays until the weights are used
          if (need_pos) {
            meet();                                        // (their place is free when the tile's is)
            if (tid < BN) tp[tid] = next_pos;
            fetch_pos(t + 1);
          }
          if (which == 0 && lane < 4) X.junk[e % ST][lane] = 0;
        }
        meet();
        const bool all = !values || (rows == BN && (!need_pos || (tp[BN - 1] <= pmin && (A.window <= 0 || (int64_t)pmax - tp[0] < A.window ||
                                                                                         r + BN <= A.sink))));   // seen whole by every token
        if (codes) {
          const uint32_t hi_t = smem_u32(stage(e)), sc = smem_u32(scale(j));
          uint32_t* marks = X.junk[e % ST];
          if (!values) {
            const uint32_t lo_t = smem_u32(stage(e + 1)), from = smem_u32(raw_k(j));
            if (q8) widen_tile<HD, BN, true, kLow, false>(from, rb, sc, nb, hi_t, lo_t, A.hd, rows, marks, tid);
            else widen_tile<HD, BN, false, kLow, false>(from, rb, sc, nb, hi_t, lo_t, A.hd, rows, marks, tid);
          } else {
            const uint32_t from = smem_u32(raw_v(j));
            if (q8 && all) widen_tile<HD, BN, true, false, false>(from, rb, sc, nb, hi_t, 0u, A.hd, rows, marks, tid);
            else if (q8) widen_tile<HD, BN, true, false, true>(from, rb, sc, nb, hi_t, 0u, A.hd, rows, marks, tid);
            else if (all) widen_tile<HD, BN, false, false, false>(from, rb, sc, nb, hi_t, 0u, A.hd, rows, marks, tid);
            else widen_tile<HD, BN, false, false, true>(from, rb, sc, nb, hi_t, 0u, A.hd, rows, marks, tid);
          }
        } else {
          if (tid == 0 && !*s_abort) copy_tile<HD, BN>(stage(e), &map_v, U.row0 + r, all ? &b_full[e % ST] : b_v);
          if (all) continue;
          wait(b_v, looked & 1);
          __syncwarp();
          ++looked;
          clean_tile<HD, BN, kConv>(stage(e), rows, X.junk[e % ST], tid);
        }
        fence_proxy_async_smem();
        meet();
        if (tid == 0) {
          mbar_arrive(&b_full[e % ST]);
          if (kLow && !values) mbar_arrive(&b_full[(e + 1) % ST]);
          if (codes) mbar_arrive(&raw_empty[j & ((1 << slots) - 1)]);
        }
      }
    }
    if (*s_abort && tid == 0 && values && !vq)             // value copies still on their way
#pragma unroll 1
      for (int e = max(0, P * tiles - ST); e < P * tiles; ++e)
#pragma unroll 1
        for (int it = 0; it < 1024 && e % P == P - 1 && !mbar_try_wait(&b_full[e % ST], (e / ST) & 1); ++it) {
        }
  } else if (wg < 2) {
    // ---- softmax: a thread per column of the unit; the warpgroups take tiles in turn
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGroupSoft));
    const int m = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // Barrier 4 + w: warpgroup w has handed its reference on (and does so again only
    // after the other one has).
    auto handed = [&] {                                    // waits for the other's
      __syncwarp();
      if (wg == 0) asm volatile("bar.sync 5, 256;" ::: "memory");
      else asm volatile("bar.sync 4, 256;" ::: "memory");
      return s_ref[(wg ^ 1) * 128 + m];
    };
    auto hand = [&](float x) {
      s_ref[wg * 128 + m] = x;
      __syncwarp();
      if (wg == 0) asm volatile("bar.arrive 4, 256;" ::: "memory");
      else asm volatile("bar.arrive 5, 256;" ::: "memory");
    };
    int turn = 0;
    auto swap = [&](float x) {                             // the other's value of this row
      float* at = s_ref + 256 + (turn & 1) * 256;
      at[wg * 128 + m] = x;
      __syncwarp();
      asm volatile("bar.sync 7, 256;" ::: "memory");
      ++turn;
      return at[(wg ^ 1) * 128 + m];
    };
    int j = 0, nu = 0;
#pragma unroll 1
    for (int u = unit_a; j < tiles; ++u) {
      if (min(end, s_first[u + 1]) <= max(begin, s_first[u])) continue;
      const Unit U = unit_of(u);
      const AttendSeq& S = A.seq[U.s];
      const int32_t* rpos = A.cpos + U.row0;
      const bool on = m < U.ncol;
      const int col = U.c0 + (on ? m : 0), tl = col / A.G, head = U.g * A.G + col - tl * A.G;
      const int64_t tok = S.tok0 + tl;
      const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(A.q) + tok * A.q_stride + (int64_t)head * A.hd);
      // ---- queries: half of the row's dims, as fp16 (bf16 ones times a power of two, undone in the logits)
      constexpr int kPieces = HD / 16;                     // 16-byte pieces of half a row
      uint4 v[kPieces];
#pragma unroll
      for (int c = 0; c < kPieces; ++c) v[c] = on && 8 * (wg * kPieces + c) < A.hd ? src[wg * kPieces + c] : make_uint4(0, 0, 0, 0);
      const int p = on ? A.pos[tok] : INT32_MIN;
      const int newest = s_hi[u] > 0 ? rpos[s_hi[u] - 1] : INT32_MIN;
      {
        const int pl = __reduce_min_sync(0xffffffffu, on ? p : INT32_MAX), ph = __reduce_max_sync(0xffffffffu, p);
        if (lane == 0) {
          X.lo[warp] = pl;
          X.hi[warp] = ph;
        }
      }
      float sl = A.scale * 1.4426950408889634f, f = 1.f;
      uint32_t am = 0;
      if (A.type == TRIA_BF16) {
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) am = max(am, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
        }
      }
      am = max(am, __float_as_uint(swap(__uint_as_float(am))));   // (also makes the positions known)
      if (A.type == TRIA_BF16) {
        const int ex = (int)(am >> 7) - 127;
        if (ex > -120 && ex < 120) {
          f = __uint_as_float((uint32_t)(127 - ex) << 23);
          sl *= __uint_as_float((uint32_t)(127 + ex) << 23);
        }
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          uint32_t* w = &v[c].x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half2 h = __floats2half2_rn(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
      }
      sl = fmaxf(sl, 0x1p-126f);                           // (times -inf stays -inf)
      // (of the other warpgroup's warps, which have the same rows: what it wrote before the swap)
      const int o4 = 4 * (wg ^ 1);
      const int pmin = min(min(X.lo[o4], X.lo[o4 + 1]), min(X.lo[o4 + 2], X.lo[o4 + 3]));
      const int pmax = max(max(X.hi[o4], X.hi[o4 + 1]), max(X.hi[o4 + 2], X.hi[o4 + 3]));
      const bool need_pos = A.window > 0 || newest > pmin;
#pragma unroll
      for (int c = 0; c < kPieces; c += 4) {
        const uint32_t w[16] = {v[c].x,     v[c].y,     v[c].z,     v[c].w,     v[c + 1].x, v[c + 1].y, v[c + 1].z, v[c + 1].w,
                                v[c + 2].x, v[c + 2].y, v[c + 2].z, v[c + 2].w, v[c + 3].x, v[c + 3].y, v[c + 3].z, v[c + 3].w};
        tc_st16(lane_base + H::cQ + wg * (HD / 4) + c * 4, w);
      }
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(b_q);
      // rows at or before it are outside the window
      const int pold = A.window > 0 ? (int)max((int64_t)INT32_MIN, (int64_t)p - A.window) : INT32_MIN;
      const uint32_t to = lane_base + H::cO;
      float M = -INFINITY, l = 0.f;
      bool poison = false;
#pragma unroll 1
      for (int t = U.t0; t < U.t1; ++t, ++j) {
        if ((j & 1) != wg) continue;
        wait(&b_s[j & 3], (j >> 2) & 1);
        __syncwarp();
        tc_fence_after();
        const uint32_t ts = lane_base + H::cS + (j & 3) * BN;
        uint32_t x[BN];
#pragma unroll
        for (int c = 0; c < BN; c += 32) tc_ld32(x + c, ts + c);
        int rows;
        const int r = tile_row(U, t, rows);
        bool masked = rows < BN;
        const int ev = P * j + P - 1;
        if (need_pos || masked) {
          wait(&b_full[ev % ST], (ev / ST) & 1);           // positions and marks are there
          __syncwarp();
        }
        const int32_t* tp = s_pos + (j % H::kPosTiles) * BN;
        if (need_pos)
          masked = masked || tp[BN - 1] > pmin || (A.window > 0 && (int64_t)pmax - tp[0] >= A.window && r + BN > A.sink);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < BN; c += 32) tc_pin(x + c);
        if (masked) {
          // the row's token sees rows [cl, ch) of the tile and, of the first rows, [0, cf)
          int cl = 0, ch = rows, cf = 0;
          if (need_pos) {
            auto upto = [&](int pos) {                     // rows with a position <= pos
              int a = 0, b = rows;
#pragma unroll 1
              while (a < b) {
                const int mid = (a + b) >> 1;
                if (tp[mid] <= pos) a = mid + 1; else b = mid;
              }
              return a;
            };
            ch = upto(p);
            if (A.window > 0) {
              cl = min(ch, upto(pold));
              cf = min(ch, max(0, A.sink - r));
            }
          }
          auto below = [](int n) { return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u); };   // bits of rows < n
#pragma unroll
          for (int c0 = 0; c0 < BN; c0 += 32) {
            const uint32_t seen = (below(ch - c0) & ~below(cl - c0)) | below(cf - c0);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((seen >> c) & 1u)) x[c0 + c] = 0xFF800000u;   // -inf
            if (X.junk[ev % ST][c0 >> 5] & seen) poison = true;   // (a tile's marks are words of 32 rows)
          }
        }
        float tops[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) tops[k] = __uint_as_float(x[k]);
#pragma unroll
        for (int c = 4; c < BN - 4; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) tops[k] = fmaxf(fmaxf(tops[k], __uint_as_float(x[c + k])), __uint_as_float(x[c + 4 + k]));
#pragma unroll
        for (int k = 0; k < 4; ++k) tops[k] = fmaxf(tops[k], __uint_as_float(x[BN - 4 + k]));
        float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        top = top * sl - kShift;
        const bool first = t == U.t0;
        const float before = first ? -INFINITY : handed();   // M after the tile before
        const bool move = (top > before + kLazy || before == -INFINITY) && top > -INFINITY;
        const float now = move ? top : before;
        if (t + 1 < U.t1) hand(now);
        if (now > M) {                                     // (since this warpgroup's last tile)
          l *= exp2_fast(M - now);
          M = now;
        }
        if (!first && __any_sync(0xffffffffu, move)) {
          // the sums of the tile before, and of the one before that, may be running (with one barrier for all
          // of them, a parity could not tell either from sums done two tiles earlier)
          wait(&b_o[(j - 1) & 3], ((j - 1) >> 2) & 1);
          __syncwarp();
          tc_fence_after();
          const float a = move ? exp2_fast(before - now) : 1.f;
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
            uint32_t o[16];
            tc_ld16(o, to + c);
            tc_wait_ld();
            tc_pin16(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
            tc_st16(to + c, o);
          }
        }
        const float mb = M == -INFINITY ? 0.f : M;
        const float2 sl2 = make_float2(sl, sl), mb2 = make_float2(-mb, -mb);
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < BN; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 e = __ffma2_rn(make_float2(__uint_as_float(x[c + 2 * k]), __uint_as_float(x[c + 2 * k + 1])), sl2, mb2);
            e.x = exp2_fast(e.x);
            e.y = exp2_fast(e.y);
            ls[k & 1] = __fadd2_rn(ls[k & 1], e);
            const __half2 y = __floats2half2_rn(e.x, e.y);
            w[k] = *reinterpret_cast<const uint32_t*>(&y);
          }
          tc_st16(ts + c / 2, w);
        }
        l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&b_p[j & 3]);
      }
      // ---- the unit's part: each warpgroup writes half of the dims
      const float M2 = swap(M), top = fmaxf(M, M2);        // (the last tile's is the larger one)
      l = M == -INFINITY ? l : l * exp2_fast(M - top);
      l += swap(l);
      poison = swap(poison ? 1.f : 0.f) != 0.f || poison;
      wait(b_f, nu & 1);
      __syncwarp();
      tc_fence_after();
      float* slot = A.part + (int64_t)(u + (int)blockIdx.x) * 128 * (HD + 2) + m;
      const bool write = __all_sync(0xffffffffu, *s_abort == 0);
      if (write && wg == 0 && on) {
        slot[0] = top;
        slot[128] = l;
      }
#pragma unroll 1
      for (int c = wg * (HD / 2); c < (wg + 1) * (HD / 2); c += 32) {
        uint32_t o[32];
        tc_ld32(o, to + c);
        tc_wait_ld();
        tc_pin(o);
        if (write && on)
#pragma unroll
          for (int k = 0; k < 32; ++k) slot[(int64_t)(2 + c + k) * 128] = poison ? __uint_as_float(0x7FC00000u) : __uint_as_float(o[k]);
      }
      tc_fence_before();
      ++nu;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && *s_abort) report(A.ctrl, TRIA_ERR_TIMEOUT, 0u);
  if (warp == kGroupIssue) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  leave();
}

// Joins the parts of a unit with its tokens' own rows (o2, l2). A thread takes
// kJoinDims dims of a column and every Q-th part, whose loads are all in flight; the
// Q threads of a column meet in shared memory, in order. `wide` is the width in
// columns of a block's row of threads, a power of two from 32 to 128, no wider than
// the units need, and Q the most that lets the grid start at once.
constexpr int kJoinDims = 8, kJoinLoads = 5, kJoinBlocks = 5;   // (blocks of 128 threads per SM, by registers)

template <int HD, int Q>
__global__ void __launch_bounds__(128 * Q, kJoinBlocks / Q) k_join_group(const __grid_constant__ AttendArgs A, const float* o2, const float* l2,
                                                                         const int32_t* own_live, const __grid_constant__ GroupOwn own,
                                                                         int grid, int wide) {
  __shared__ float s_m[Q][128], s_l[Q][128], s_v[Q][kJoinDims][128];
  const int u = blockIdx.x, th = threadIdx.x & 127, part = threadIdx.x >> 7, c = th & (wide - 1);
  const int d0 = ((int)blockIdx.y * 128 + th) / wide * kJoinDims;
  int s = 0, hi_s = A.n_seqs - 1;
#pragma unroll 1
  while (s < hi_s) {
    const int mid = (s + hi_s + 1) >> 1;
    if (A.seq[mid].unit0 <= u) s = mid; else hi_s = mid - 1;
  }
  const AttendSeq& S = A.seq[s];
  const int ct = (S.t * A.G + 127) / 128, x = u - S.unit0, g = x / ct, col = (x - g * ct) * 128 + c;
  const bool on = col < S.t * A.G;
  const int tok = S.tok0 + (on ? col / A.G : 0), head = g * A.G + (on ? col % A.G : 0);
  const int64_t at = (int64_t)tok * A.nq + head;
  asm volatile("griddepcontrol.wait;" ::: "memory");       // (started while the parts are made)
  const int total = A.table[A.units], t0 = A.table[u], t1 = A.table[u + 1];
  // the sequence's own rows join the first parts
  float m = -INFINITY, l = 0.f, v[kJoinDims];
#pragma unroll
  for (int e = 0; e < kJoinDims; ++e) v[e] = 0.f;
  if (part == 0 && on) {
    const float4* o = reinterpret_cast<const float4*>(o2 + at * A.hd + d0);
#pragma unroll
    for (int e = 0; e < kJoinDims / 4; ++e) {
      const float4 y = o[e];
      v[4 * e] = y.x;
      v[4 * e + 1] = y.y;
      v[4 * e + 2] = y.z;
      v[4 * e + 3] = y.w;
    }
    m = l2[at] * 1.4426950408889634f;
    l = m == -INFINITY ? 0.f : 1.f;
  }
  int c0 = 0, parts = 0;
  if (t1 > t0) {
    const int workers = min(grid, total), each = total / workers, more = total - each * workers;
    auto cta_of = [&](int tile) { return tile < more * (each + 1) ? tile / (each + 1) : more + (tile - more * (each + 1)) / each; };
    c0 = cta_of(t0);
    parts = cta_of(t1 - 1) - c0 + 1;
  }
  constexpr int64_t kSlot = 128 * (HD + 2);
  const float* p = A.part + (int64_t)(u + c0) * kSlot + c;
  if (on)
    for (int k0 = part; k0 < parts; k0 += Q * kJoinLoads) {
      float pm[kJoinLoads], pl[kJoinLoads], pv[kJoinLoads][kJoinDims];
#pragma unroll
      for (int k = 0; k < kJoinLoads; ++k) {
        const float* y = p + min(k0 + k * Q, parts - 1) * kSlot;   // (in the place of a part that is not there one that is)
        pm[k] = y[0];
        pl[k] = y[128];
#pragma unroll
        for (int e = 0; e < kJoinDims; ++e) pv[k][e] = y[(2 + d0 + e) * 128];
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kJoinLoads; ++k)
        if (k0 + k * Q < parts) top = fmaxf(top, pm[k]);
      const float tb = top == -INFINITY ? 0.f : top, f0 = exp2f(m - tb);
      l *= f0;
#pragma unroll
      for (int e = 0; e < kJoinDims; ++e) v[e] *= f0;
#pragma unroll
      for (int k = 0; k < kJoinLoads; ++k)
        if (k0 + k * Q < parts) {
          const float f = exp2f(pm[k] - tb);
          l = fmaf(pl[k], f, l);
#pragma unroll
          for (int e = 0; e < kJoinDims; ++e) v[e] = fmaf(pv[k][e], f, v[e]);
        }
      m = top;
    }
  s_m[part][th] = m;
  s_l[part][th] = l;
#pragma unroll
  for (int e = 0; e < kJoinDims; ++e) s_v[part][e][th] = v[e];
  __syncthreads();
  if (part != 0 || !on) return;
  int q = 0, hi_q = own.n_seqs - 1;                        // the token's sequence
  while (q < hi_q) {
    const int mid = (q + hi_q + 1) >> 1;
    if (own.tok0[mid] <= tok) q = mid; else hi_q = mid - 1;
  }
  const int n1 = *((volatile const int32_t*)(A.n_live + s)), n2 = *((volatile const int32_t*)(own_live + q));
  if (n1 < 0 || n1 > S.cap || n2 < 0 || n2 > own.cap[q]) return;
  float top = m;
#pragma unroll
  for (int k = 1; k < Q; ++k) top = fmaxf(top, s_m[k][th]);
  const float tb = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < kJoinDims; ++e) v[e] = 0.f;
#pragma unroll
  for (int k = 0; k < Q; ++k) {
    const float f = exp2f(s_m[k][th] - tb);
    sum = fmaf(s_l[k][th], f, sum);
#pragma unroll
    for (int e = 0; e < kJoinDims; ++e) v[e] = fmaf(s_v[k][e][th], f, v[e]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t w[kJoinDims / 2];
#pragma unroll
  for (int e = 0; e < kJoinDims / 2; ++e) w[e] = pack_out(A.type, v[2 * e] * inv, v[2 * e + 1] * inv);
  *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(A.out) + (int64_t)tok * A.out_stride + (int64_t)head * A.hd + d0) =
      make_uint4(w[0], w[1], w[2], w[3]);
  if (d0 == 0 && A.lse) A.lse[at] = sum == 0.f ? -INFINITY : (tb + log2f(sum)) * 0.6931471805599453f;
}

template <int HD, bool kQuant, bool kLow>
cudaError_t launch_group_t(const AttendArgs& A, int grid, cudaStream_t st) {
  using H = GroupShape<HD, kQuant>;
  auto kern = k_attend_group<HD, kQuant, kLow>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, H::kSmem);
  if (e != cudaSuccess) return e;
  // the warpgroups' register shares are cut from what the block starts with
  cudaFuncAttributes attr;
  const cudaError_t e2 = cudaFuncGetAttributes(&attr, kern);
  if (e2 != cudaSuccess) return e2;
  if (attr.numRegs != kGroupRegs) return cudaErrorInvalidConfiguration;
  CUtensorMap mk, mv;
  memset(&mk, 0, sizeof(mk));
  memset(&mv, 0, sizeof(mv));
  int64_t rows = 0;
  for (int s = 0; s < A.n_seqs; ++s) rows = std::max(rows, A.seq[s].row0 + (int64_t)A.n_kv * A.seq[s].cap);
  if (A.k_type == TRIA_F16 && !plane_map_f16(&mk, A.k, A.hd, rows, H::BN)) return cudaErrorInvalidValue;
  if (A.v_type == TRIA_F16 && !plane_map_f16(&mv, A.v, A.hd, rows, H::BN)) return cudaErrorInvalidValue;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kGroupThreads);
  cfg.dynamicSmemBytes = H::kSmem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, A, mk, mv);
}

template <int HD>
cudaError_t launch_group_hd(const AttendArgs& A, bool low, int grid, cudaStream_t st) {
  if (A.k_type == TRIA_F16 && A.v_type == TRIA_F16) return launch_group_t<HD, false, false>(A, grid, st);
  return low ? launch_group_t<HD, true, true>(A, grid, st) : launch_group_t<HD, true, false>(A, grid, st);
}

template <int HD, int Q>
cudaError_t launch_join_t(const AttendArgs& A, const float* o2, const float* l2, const int32_t* own_live, const GroupOwn& own, int grid, int wide,
                          cudaStream_t st) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(A.units, A.hd / kJoinDims * wide / 128);
  cfg.blockDim = dim3(128 * Q);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_join_group<HD, Q>, A, o2, l2, own_live, own, grid, wide);
}

template <int HD>
cudaError_t launch_join_hd(const AttendArgs& A, const float* o2, const float* l2, const int32_t* own_live, const GroupOwn& own, int grid,
                           cudaStream_t st) {
  int cols = 0;
  for (int s = 0; s < A.n_seqs; ++s) cols = std::max(cols, A.seq[s].t * A.G);
  const int wide = cols <= 32 ? 32 : (cols <= 64 ? 64 : 128);
  const int64_t blocks = (int64_t)A.units * (A.hd / kJoinDims) * wide / 128, room = (int64_t)kJoinBlocks * grid;
  if (4 * blocks <= room) return launch_join_t<HD, 4>(A, o2, l2, own_live, own, grid, wide, st);
  if (2 * blocks <= room) return launch_join_t<HD, 2>(A, o2, l2, own_live, own, grid, wide, st);
  return launch_join_t<HD, 1>(A, o2, l2, own_live, own, grid, wide, st);
}

}  // namespace

size_t group_part_values(int hd) { return 128 * (size_t)(prompt_dims(hd) + 2); }

cudaError_t launch_attend_group(const AttendArgs& A, bool round_keys, int grid, cudaStream_t st) {
  if (A.units == 0) return cudaSuccess;
  const bool low = A.k_type != TRIA_F16 && !round_keys;
  switch (prompt_dims(A.hd)) {
    case 64: return launch_group_hd<64>(A, low, grid, st);
    case 128: return launch_group_hd<128>(A, low, grid, st);
    default: return launch_group_hd<256>(A, low, grid, st);
  }
}

cudaError_t launch_join_group(const AttendArgs& A, const float* o2, const float* l2, const int32_t* own_live, const GroupOwn& own, int grid,
                              cudaStream_t st) {
  if (A.units == 0) return cudaSuccess;
  switch (prompt_dims(A.hd)) {
    case 64: return launch_join_hd<64>(A, o2, l2, own_live, own, grid, st);
    case 128: return launch_join_hd<128>(A, o2, l2, own_live, own, grid, st);
    default: return launch_join_hd<256>(A, o2, l2, own_live, own, grid, st);
  }
}

}  // namespace tria
