// Attention of many sequences' new tokens over one shared prefix, on the
// fifth-generation tensor cores: a decode step of 17 columns (token x query
// head of a KV head's group) or more.
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
// TMA. Codes come by bulk copies as they lie, and four warps widen them tile by
// tile on their way into the swizzled ones (each row once for all columns:
// the prompt kernel, whose units meet every row again and again, widens the planes
// in memory instead): values rounded once, keys as the rounded value and the
// remainder, which takes a product of its own (kLow). Two warpgroups share a
// tile's softmax by columns and agree on its maximum through shared memory.
//
// Masks, junk in hidden rows, the lazy reference M and the bounded waits are those of
// the prompt kernel.
#include <string.h>

#include <algorithm>

#include "attend_tc.cuh"

namespace tria {

namespace {

template <int HD, bool kQuant>
struct GroupShape {
  static constexpr int BN = HD == 256 ? 64 : 128;          // rows of a tile
  static constexpr int kStage = BN * HD * 2;
  static constexpr int kStages = (HD == 64 ? 2 : 1) * (kQuant ? 4 : 6);
  static constexpr int kRaw = BN * HD;                     // bytes of a plane's q8_0 codes
  static constexpr int kRawArea = kQuant ? 4 * kRaw : 0;   // two tiles of both planes, or four of 4-bit codes
  static constexpr int kRawSlots = 4;
  static constexpr int kPosTiles = 8;                      // more tiles than the ring holds values of
  static constexpr int kScRow = HD / 16;                   // bytes of a row's block scales
  static constexpr int oRing = 0, oRaw = kStages * kStage, oPos = oRaw + kRawArea, oScale = oPos + kPosTiles * BN * 4;
  static constexpr int oTops = oScale + (kQuant ? 2 * BN * kScRow : 0);   // [parity][warpgroup][row]
  static constexpr int oBar = oTops + 4 * 128 * 4;
  static constexpr int kSmem = oBar + 1024;
  // TMEM columns: score buffers, outputs, queries
  static constexpr int cS(int buf) { return buf * BN; }
  static constexpr int cO = 2 * BN, cQ = cO + HD;
  static_assert(cQ + HD / 2 <= 512, "TMEM");
  static_assert(kSmem + (3 * kMaxSegments + 64) * 4 <= 227 * 1024, "shared memory");
};

constexpr int kGroupBars = 2 * 12 + 2 + 2 + 5 + 2 * 4;
struct GroupShared {
  uint32_t junk[12][4];                                    // rows of a value tile that held junk, by stage
  int32_t lo[8], hi[8], c_lo[8], c_hi[8];                  // positions, a warp each
  uint32_t tmem, abort;
};
static_assert(kGroupBars * 8 + sizeof(GroupShared) <= 1024, "barriers and shared state");

// two warpgroups of softmax, two that fill tiles, one whose first warp issues the
// products and whose second one starts the copies
constexpr int kGroupThreads = 640, kGroupIssue = 16, kGroupLoad = 17, kConv = 256, kGroupRegs = 96;
// registers of a thread in each, cut from what the block starts with
constexpr int kGroupSoft = 120, kGroupConv = 88, kGroupOther = 64;
static_assert(2 * kGroupSoft + 2 * kGroupConv + kGroupOther == 5 * kGroupRegs, "register shares");

// Eight values of a quantised row: w their codes (q8_0: eight bytes; q4_0: eight
// bytes of which the low halves count), h their scale. hi: code x scale as fp16,
// lo: what fp16 leaves of it, which fp16 holds exactly (a scale is a multiple of
// 2^-24 and a code whole, so 8 bits at most are left, all above 2^-24).
template <bool kQ8, bool kLow>
__device__ __forceinline__ void widen8(uint2 w, uint32_t h, uint32_t* hi, uint32_t* lo) {
  const uint32_t sc = __byte_perm(h, h, 0x1010);
  constexpr uint32_t bias = kQ8 ? 0x64806480u : 0x64086408u;
  if (kQ8) {
    w.x ^= 0x80808080u;                                    // 0x64, code + 128: 1152 + code
    w.y ^= 0x80808080u;
  }
  const uint32_t b[4] = {__byte_perm(w.x, 0x64646464u, 0x4140), __byte_perm(w.x, 0x64646464u, 0x4342),
                         __byte_perm(w.y, 0x64646464u, 0x4140), __byte_perm(w.y, 0x64646464u, 0x4342)};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t c;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(b[k]), "r"(bias));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(hi[k]) : "r"(c), "r"(sc));
    if constexpr (kLow) asm("{\n .reg .b32 n;\n neg.f16x2 n, %3;\n fma.rn.f16x2 %0, %1, %2, n;\n}\n" : "=r"(lo[k]) : "r"(c), "r"(sc), "r"(hi[k]));
  }
}

// The rows of a tile of codes (rb bytes each) as fp16 tiles, by kConv threads; a
// thread has the same eight dims of every kConv / (HD / 8)-th row. Rows from `rows` on
// are zeros with kClean, which also replaces rows with junk and marks them.
template <int HD, int BN, bool kQ8, bool kLow, bool kClean>
__device__ __forceinline__ void widen_tile(const uint8_t* codes, int rb, const uint16_t* scale, uint8_t* hi_t, uint8_t* lo_t, int hd, int rows,
                                           uint32_t* marks, int tid) {
  constexpr int per = HD / 8, step = kConv / per, NB = HD / 32;
  static_assert(step % 8 == 0 && BN % step == 0, "a thread's rows have one place in the swizzle");
  const int c = tid % per, r0 = tid / per;
  const uint32_t to = (c >> 3) * (BN * 128) + swz(r0, c & 7);
  const uint8_t* from = codes + r0 * rb + (kQ8 ? c * 8 : (c / 4) * 16 + (c & 1) * 8);
  const bool there = 8 * c < hd;
#pragma unroll
  for (int i = 0; i < BN / step; ++i) {
    uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
    if (there && (!kClean || r0 + i * step < rows)) {
      uint2 w = *reinterpret_cast<const uint2*>(from + i * step * rb);
      if constexpr (!kQ8) {
        const int up = (c & 2) * 2;
        w.x = (w.x >> up) & 0x0F0F0F0Fu;
        w.y = (w.y >> up) & 0x0F0F0F0Fu;
      }
      widen8<kQ8, kLow>(w, scale[(r0 + i * step) * NB + c / 4], hi, lo);
      if (kClean && (junk_h2(hi[0]) || junk_h2(hi[1]) || junk_h2(hi[2]) || junk_h2(hi[3]))) {
        const int rr = r0 + i * step;
        hi[0] = hi[1] = hi[2] = hi[3] = 0;
        atomicOr(&marks[rr >> 5], 1u << (rr & 31));
      }
    }
    *reinterpret_cast<uint4*>(hi_t + to + i * step * 128) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if constexpr (kLow) *reinterpret_cast<uint4*>(lo_t + to + i * step * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

template <int HD, bool kQuant, bool kLow>
__global__ void __launch_bounds__(kGroupThreads, 1) k_attend_group(const __grid_constant__ AttendArgs A,
                                                                   const __grid_constant__ CUtensorMap map_k,
                                                                   const __grid_constant__ CUtensorMap map_v) {
  using H = GroupShape<HD, kQuant>;
  // ring entries of tile j: keys P j, their remainders P j + 1 (kLow), values P j + P - 1
  constexpr int P = kLow ? 3 : 2, BN = H::BN, ST = H::kStages, HALF = BN / 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int s_first[kMaxSegments + 1], s_lo[kMaxSegments], s_hi[kMaxSegments];   // of units: first tile, rows
  __shared__ int s_scan[40];
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + H::oBar);
  // full: a tile is in the ring; empty: its products are done; s: scores; p: weights;
  // o: a tile's sums; f: the unit's last sums; q: queries; x: every product; v: values that are looked
  // through before their tile is full; rf, re: codes are there, are used
  uint64_t *b_full = bar, *b_empty = bar + 12, *b_s = bar + 24, *b_p = b_s + 2, *b_o = b_p + 2, *b_f = b_o + 1, *b_q = b_f + 1,
           *b_x = b_q + 1, *b_v = b_x + 1, *b_rf = b_v + 1, *b_re = b_rf + H::kRawSlots;
  int32_t* s_pos = reinterpret_cast<int32_t*>(smem + H::oPos);
  float* s_tops = reinterpret_cast<float*>(smem + H::oTops);
  GroupShared& X = *reinterpret_cast<GroupShared*>(smem + H::oBar + kGroupBars * 8);
  volatile uint32_t* s_abort = &X.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
  const bool kq = kQuant && A.k_type != TRIA_F16, vq = kQuant && A.v_type != TRIA_F16;

  // ---- the tile list
  auto seq_of = [&](int unit) {
    int s = 0, hi_s = A.n_seqs - 1;
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b_s[i], 1);
      mbar_init(&b_p[i], 256);
    }
    mbar_init(b_o, 1);
    mbar_init(b_f, 1);
    mbar_init(b_q, 256);
    mbar_init(b_x, 1);
    mbar_init(b_v, 1);
#pragma unroll
    for (int i = 0; i < H::kRawSlots; ++i) {
      mbar_init(&b_rf[i], 1);
      mbar_init(&b_re[i], 1);
    }
    fence_mbar_init();
  }
  __syncthreads();
  const int64_t total = s_first[A.units];
  const int64_t workers = min((int64_t)gridDim.x, total);
  if ((int64_t)blockIdx.x >= workers) return leave();
  if (warp == kGroupIssue) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&X.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = X.tmem;
  const int begin = (int)(blockIdx.x * total / workers), end = (int)((blockIdx.x + 1) * total / workers);
  auto unit_at = [&](int tile) {                           // the last unit that starts at or before it
    int u = 0, hi_u = A.units - 1;
    while (u < hi_u) {
      const int mid = (u + hi_u + 1) >> 1;
      if (s_first[mid] <= tile) u = mid; else hi_u = mid - 1;
    }
    return u;
  };
  const int unit_a = unit_at(begin);
  struct Unit {
    int s, g, c0, ncol, t0, t1;                            // sequence, KV head, columns, this run's tiles of it
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
    U.t0 = max(begin, s_first[u]);
    U.t1 = min(end, s_first[u + 1]);
    U.row0 = S.row0 + (int64_t)U.g * S.cap;
    return U;
  };
  auto tile_row = [&](int u, int tile, int& rows) {        // first row in the segment
    const int j = tile - s_first[u], lo = s_lo[u];
    const int sr = min(A.sink, lo), nt_sink = (sr + BN - 1) / BN;
    if (j < nt_sink) {
      rows = min(BN, sr - j * BN);
      return j * BN;
    }
    const int r = lo + (j - nt_sink) * BN;
    rows = min(BN, s_hi[u] - r);
    return r;
  };
  // bounded waits, as in the prompt kernel: after one gave up nobody waits any more, no
  // results are written, and every role runs its loops to the end
  auto wait = [&](uint64_t* b, uint32_t parity) {
    for (int it = 0; it < kWaitLimit; ++it)
      if (mbar_try_wait(b, parity) || *s_abort) return;
    *s_abort = 1;
  };
  auto wait_warp = [&](uint64_t* b, uint32_t parity) {
    const int r = mbar_wait_warp(b, parity, s_abort, kWaitLimit);
    if (r == 0) *s_abort = 1;
    return r > 0;
  };
  auto stage = [&](int e) { return smem + H::oRing + (e % ST) * H::kStage; };
  auto free_stage = [&](int e) {
    if (e >= ST) wait(&b_empty[e % ST], ((e / ST) - 1) & 1);
  };
  const int tiles = end - begin;
  const int slots = kQuant && (!kq || A.k_type == TRIA_Q4_0) && (!vq || A.v_type == TRIA_Q4_0) ? 4 : 2;
  const int raw_v = H::kRawArea / slots / 2;               // a slot: codes of keys, then of values
  auto raw = [&](int j) { return smem + H::oRaw + (j % slots) * (2 * raw_v); };
  const int k_rb = A.k_type == TRIA_Q8_0 ? A.hd : A.hd / 2, v_rb = A.v_type == TRIA_Q8_0 ? A.hd : A.hd / 2;

  if (wg >= 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGroupOther));
  if (warp == kGroupIssue) {
    // ---- products (results of waits and addresses are the same in all lanes and kept in
    // such a form, see the prompt kernel)
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dk = tile_desc(smem_u32(smem + H::oRing), 16), dv = tile_desc(smem_u32(smem + H::oRing), BN * 128);
    auto scores = [&](int j, int st, int sl) {
      const uint64_t b = dk + (uint64_t)(st * (H::kStage / 16));
      const uint32_t d = tm + H::cS(j & 1), a = tm + H::cQ;
#pragma unroll
      for (int k = 0; k < HD / 16; ++k)
        tc_mma_ts(d, a + k * 8, b + (uint64_t)((k >> 2) * (BN * 8) + (k & 3) * 2), mma_desc(BN, false), k > 0);
      if constexpr (kLow) {
        const uint64_t bl = dk + (uint64_t)(sl * (H::kStage / 16));
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
          tc_mma_ts(d, a + k * 8, bl + (uint64_t)((k >> 2) * (BN * 8) + (k & 3) * 2), mma_desc(BN, false), 1);
      }
      tc_commit(&b_s[j & 1]);
      tc_commit(&b_empty[st]);
      if (kLow) tc_commit(&b_empty[sl]);
    };
    auto sums = [&](int j, int st, bool add) {
      const uint64_t b = dv + (uint64_t)(st * (H::kStage / 16));
      const uint32_t d = tm + H::cO, a = tm + H::cS(j & 1);
#pragma unroll
      for (int k = 0; k < BN / 16; ++k) tc_mma_ts(d, a + k * 8, b + (uint64_t)(k * 128), mma_desc(HD, true), add || k > 0);
      tc_commit(b_o);
      tc_commit(&b_empty[st]);
    };
    bool ok = true;
    int j = 0, nu = 0;
    auto keys = [&](int t) {                               // scores of tile t
      const int e = P * t;
      ok = ok && wait_warp(&b_full[e % ST], (e / ST) & 1) && (!kLow || wait_warp(&b_full[(e + 1) % ST], ((e + 1) / ST) & 1));
      tc_fence_after();
      if (ok && elect_one()) scores(t, e % ST, (e + 1) % ST);
      __syncwarp();
    };
    for (int u = unit_a; ok && j < tiles; ++u) {
      const int nt = min(end, s_first[u + 1]) - max(begin, s_first[u]);
      if (nt <= 0) continue;
      ok = wait_warp(b_q, nu & 1);
      keys(j);
      for (int i = 0; ok && i < nt; ++i, ++j) {
        if (i + 1 < nt) keys(j + 1);
        const int e = P * j + P - 1;
        ok = ok && wait_warp(&b_full[e % ST], (e / ST) & 1) && wait_warp(&b_p[j & 1], (j >> 1) & 1);
        tc_fence_after();
        if (ok && elect_one()) {
          sums(j, e % ST, i > 0);
          if (i + 1 == nt) tc_commit(b_f);
        }
        __syncwarp();
      }
      ++nu;
    }
    // nothing may be running when the accumulators are given back
    if (elect_one()) tc_commit(b_x);
    for (int it = 0; it < kWaitLimit && !mbar_try_wait(b_x, 0); ++it) {
    }
  } else if (warp == kGroupLoad) {
    // ---- key tiles of fp16 planes, codes of quantised ones
    if (lane == 0) {
      int j = 0;
      for (int u = unit_a; j < tiles; ++u) {
        if (min(end, s_first[u + 1]) <= max(begin, s_first[u])) continue;
        const Unit U = unit_of(u);
        for (int t = U.t0; t < U.t1; ++t, ++j) {
          int rows;
          const int r = tile_row(u, t, rows);
          if (!kq) {
            // hidden keys, and those past the last row, only reach logits that the mask replaces
            const int e = P * j;
            free_stage(e);
            if (!*s_abort) copy_tile<HD, BN>(stage(e), &map_k, U.row0 + r, &b_full[e % ST]);
          }
          if constexpr (kQuant) {
            const int x = j % slots;
            if (j >= slots) wait(&b_re[x], ((j / slots) - 1) & 1);
            if (*s_abort) continue;
            mbar_arrive_expect_tx(&b_rf[x], (kq ? rows * k_rb : 0) + (vq ? rows * v_rb : 0));
            if (kq) bulk_g2s(raw(j), A.k + (U.row0 + r) * k_rb, rows * k_rb, &b_rf[x]);
            if (vq) bulk_g2s(raw(j) + raw_v, A.v + (U.row0 + r) * v_rb, rows * v_rb, &b_rf[x]);
          }
        }
      }
      if (*s_abort) {                                      // waits, bounded, for copies still on their way
        for (int e = max(0, P * tiles - ST); e < P * tiles; ++e)
          for (int it = 0; it < 1024 && !kq && e % P == 0 && !mbar_try_wait(&b_full[e % ST], (e / ST) & 1); ++it) {
          }
        if constexpr (kQuant)
          for (int i = max(0, tiles - slots); i < tiles; ++i)
            for (int it = 0; it < 1024 && !mbar_try_wait(&b_rf[i % slots], (i / slots) & 1); ++it) {
            }
      }
    }
  } else if (wg >= 2 && wg < 4) {
    // ---- positions; value tiles of fp16 planes; codes into tiles
    const int tid = threadIdx.x & 255;
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGroupConv));
    uint16_t* s_scale = reinterpret_cast<uint16_t*>(smem + H::oScale);
    constexpr int NB = HD / 32;
    const int nb = A.hd / 32;
    int j = 0, looked = 0;
    for (int u = unit_a; j < tiles; ++u) {
      if (min(end, s_first[u + 1]) <= max(begin, s_first[u])) continue;
      const Unit U = unit_of(u);
      const AttendSeq& S = A.seq[U.s];
      const int32_t* rpos = A.cpos + U.row0;
      // the tokens' positions, and whether they hide rows
      const int tok_a = U.c0 / A.G, tok_b = (U.c0 + U.ncol - 1) / A.G;
      int pl = INT32_MAX, ph = INT32_MIN;
      if (tok_a + tid <= tok_b) pl = ph = A.pos[S.tok0 + tok_a + tid];
      const int newest = s_hi[u] > 0 ? rpos[s_hi[u] - 1] : INT32_MIN;
      pl = __reduce_min_sync(0xffffffffu, pl);
      ph = __reduce_max_sync(0xffffffffu, ph);
      if (lane == 0) {
        X.c_lo[warp & 7] = pl;
        X.c_hi[warp & 7] = ph;
      }
      asm volatile("bar.sync 3, 256;" ::: "memory");
      // (128 columns at most, so the first four warps hold all of the tokens)
      const int pmin = min(min(X.c_lo[0], X.c_lo[1]), min(X.c_lo[2], X.c_lo[3]));
      const int pmax = max(max(X.c_hi[0], X.c_hi[1]), max(X.c_hi[2], X.c_hi[3]));
      const bool need_pos = A.window > 0 || newest > pmin;
      int next_pos = INT32_MAX;                            // of this thread's row of the tile to come
      uint16_t next_k[NB], next_v[NB];                     // and its scales
      auto fetch = [&](int t) {
        int rows = 0;
        const int r = t < U.t1 ? tile_row(u, t, rows) : 0;
        next_pos = need_pos && tid < rows ? rpos[r + tid] : INT32_MAX;
        if constexpr (kQuant) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const int64_t at = (U.row0 + r + tid) * nb + b;
            const bool on = tid < rows && b < nb;
            next_k[b] = kq && on ? __ldg(reinterpret_cast<const uint16_t*>(A.ks) + at) : (uint16_t)0;
            next_v[b] = vq && on ? __ldg(reinterpret_cast<const uint16_t*>(A.vs) + at) : (uint16_t)0;
          }
        }
      };
      fetch(U.t0);
      for (int t = U.t0; t < U.t1; ++t, ++j) {
        int rows;
        const int r = tile_row(u, t, rows), ev = P * j + P - 1;
        if constexpr (kQuant) {
          if (tid < BN)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              s_scale[tid * NB + b] = next_k[b];
              s_scale[(BN + tid) * NB + b] = next_v[b];
            }
        }
        const int pos_now = next_pos;
        fetch(t + 1);
        if constexpr (kQuant) {
          wait(&b_rf[j % slots], (j / slots) & 1);
          asm volatile("bar.sync 3, 256;" ::: "memory");   // scales
          if (kq) {
            const int e = P * j;
            free_stage(e);
            if (kLow) free_stage(e + 1);
            __syncwarp();
            if (A.k_type == TRIA_Q8_0)
              widen_tile<HD, BN, true, kLow, false>(raw(j), k_rb, s_scale, stage(e), stage(e + 1), A.hd, rows, nullptr, tid);
            else
              widen_tile<HD, BN, false, kLow, false>(raw(j), k_rb, s_scale, stage(e), stage(e + 1), A.hd, rows, nullptr, tid);
            fence_proxy_async_smem();
            asm volatile("bar.sync 3, 256;" ::: "memory");
            if (tid == 0) {
              mbar_arrive(&b_full[e % ST]);
              if (kLow) mbar_arrive(&b_full[(e + 1) % ST]);
            }
          }
        }
        free_stage(ev);
        __syncwarp();
        // positions and marks go with the value tile, which stays until the weights are used
        int32_t* tp = s_pos + (j % H::kPosTiles) * BN;
        if (need_pos && tid < BN) tp[tid] = pos_now;
        if (tid < 4) X.junk[ev % ST][tid] = 0;
        asm volatile("bar.sync 3, 256;" ::: "memory");
        const bool all = rows == BN && (!need_pos || (tp[BN - 1] <= pmin && (A.window <= 0 || (int64_t)pmax - tp[0] < A.window ||
                                                                            r + BN <= A.sink)));   // seen whole by every token
        bool filled = false;
        if constexpr (kQuant) {
          if (vq) {
            filled = true;
            const uint8_t* codes = raw(j) + raw_v;
            uint32_t* marks = X.junk[ev % ST];
            if (A.v_type == TRIA_Q8_0) {
              if (all) widen_tile<HD, BN, true, false, false>(codes, v_rb, s_scale + BN * NB, stage(ev), nullptr, A.hd, rows, marks, tid);
              else widen_tile<HD, BN, true, false, true>(codes, v_rb, s_scale + BN * NB, stage(ev), nullptr, A.hd, rows, marks, tid);
            } else {
              if (all) widen_tile<HD, BN, false, false, false>(codes, v_rb, s_scale + BN * NB, stage(ev), nullptr, A.hd, rows, marks, tid);
              else widen_tile<HD, BN, false, false, true>(codes, v_rb, s_scale + BN * NB, stage(ev), nullptr, A.hd, rows, marks, tid);
            }
          }
        }
        if (!filled) {
          if (tid == 0 && !*s_abort) copy_tile<HD, BN>(stage(ev), &map_v, U.row0 + r, all ? &b_full[ev % ST] : b_v);
          if (!all) {
            wait(b_v, looked & 1);
            __syncwarp();
            ++looked;
            clean_tile<HD, BN, kConv>(stage(ev), rows, X.junk[ev % ST], tid);
            filled = true;
          }
        }
        if (filled || kQuant) {
          if (filled) fence_proxy_async_smem();
          asm volatile("bar.sync 3, 256;" ::: "memory");
          if (tid == 0) {
            if (filled) mbar_arrive(&b_full[ev % ST]);
            if (kQuant) mbar_arrive(&b_re[j % slots]);
          }
        }
      }
    }
    if (*s_abort && tid == 0 && !vq)                       // value copies still on their way
      for (int e = max(0, P * tiles - ST); e < P * tiles; ++e)
        for (int it = 0; it < 1024 && e % P == P - 1 && !mbar_try_wait(&b_full[e % ST], (e / ST) & 1); ++it) {
        }
  } else if (wg < 2) {
    // ---- softmax: a thread per row and half of a tile's columns
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGroupSoft));
    const int m = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    auto meet = [&] { asm volatile("bar.sync 4, 256;" ::: "memory"); };
    int j = 0, nu = 0, turn = 0;                           // turn: which half of the exchange is next
    auto swap = [&](float x) {                             // the other half's value of this row
      float* at = s_tops + (turn & 1) * 256;
      at[wg * 128 + m] = x;
      meet();
      ++turn;
      return at[(wg ^ 1) * 128 + m];
    };
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
      const int pmin = min(min(X.lo[4 * wg], X.lo[4 * wg + 1]), min(X.lo[4 * wg + 2], X.lo[4 * wg + 3]));
      const int pmax = max(max(X.hi[4 * wg], X.hi[4 * wg + 1]), max(X.hi[4 * wg + 2], X.hi[4 * wg + 3]));
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
      const uint32_t to = lane_base + H::cO + wg * (HD / 2);
      float M = -INFINITY, l = 0.f;
      bool poison = false;
      for (int t = U.t0; t < U.t1; ++t, ++j) {
        wait(&b_s[j & 1], (j >> 1) & 1);
        __syncwarp();
        tc_fence_after();
        const uint32_t ts = lane_base + H::cS(j & 1);
        uint32_t x[HALF];
#pragma unroll
        for (int c = 0; c < HALF; c += 32) tc_ld32(x + c, ts + wg * HALF + c);
        int rows;
        const int r = tile_row(u, t, rows);
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
        for (int c = 0; c < HALF; c += 32) tc_pin(x + c);
        if (masked) {
          // the row's token sees columns [cl, ch) and, of the first rows, [0, cf)
          int cl = 0, ch = rows, cf = 0;
          if (need_pos) {
            auto upto = [&](int pos) {                     // columns with a position <= pos
              int a = 0, b = rows;
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
#pragma unroll
          for (int c = 0; c < HALF; ++c) {
            const int at = wg * HALF + c;
            if (at >= ch || (at < cl && at >= cf)) x[c] = 0xFF800000u;   // -inf
          }
          const uint32_t* jm = X.junk[ev % ST];
          if (jm[0] | jm[1] | jm[2] | jm[3])
            for (int c = wg * HALF; c < min(rows, (wg + 1) * HALF); ++c)
              if (((jm[c >> 5] >> (c & 31)) & 1u) && c < ch && (c >= cl || c < cf)) poison = true;
        }
        float tops[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) tops[k] = __uint_as_float(x[k]);
#pragma unroll
        for (int c = 4; c < HALF; ++c) tops[c & 3] = fmaxf(tops[c & 3], __uint_as_float(x[c]));
        float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        top = fmaxf(top, swap(top));                       // (both halves' scores are in registers: weights may be written)
        top = top * sl - kShift;
        const bool move = (top > M + kLazy || M == -INFINITY) && top > -INFINITY;
        if (__any_sync(0xffffffffu, move)) {
          float a = 1.f;
          if (move) {
            a = exp2_fast(M - top);
            M = top;
            l *= a;
          }
          if (t > U.t0) {
            wait(b_o, (j - 1) & 1);                        // the sums of the tile before may be running
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < HD / 2; c += 16) {
              uint32_t o[16];
              tc_ld16(o, to + c);
              tc_wait_ld();
              tc_pin16(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
              tc_st16(to + c, o);
            }
          }
        }
        const float mb = M == -INFINITY ? 0.f : M;
        const float2 sl2 = make_float2(sl, sl), mb2 = make_float2(-mb, -mb);
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < HALF; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 e = __ffma2_rn(make_float2(__uint_as_float(x[c + 2 * k]), __uint_as_float(x[c + 2 * k + 1])), sl2, mb2);
            e.x = exp2_fast(e.x);
            e.y = exp2_fast(e.y);
            ls[k & 1] = __fadd2_rn(ls[k & 1], e);
            const __half2 h = __floats2half2_rn(e.x, e.y);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
          }
          tc_st16(ts + (wg * HALF + c) / 2, w);
        }
        l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&b_p[j & 1]);
      }
      // ---- the unit's part
      l += swap(l);
      poison = swap(poison ? 1.f : 0.f) != 0.f || poison;
      wait(b_f, nu & 1);
      __syncwarp();
      tc_fence_after();
      float* slot = A.part + (int64_t)(u + (int)blockIdx.x) * 128 * (HD + 2) + m;
      const bool write = __all_sync(0xffffffffu, *s_abort == 0);
      if (write && wg == 0 && on) {
        slot[0] = M;
        slot[128] = l;
      }
#pragma unroll 1
      for (int c = 0; c < HD / 2; c += 32) {
        uint32_t o[32];
        tc_ld32(o, to + c);
        tc_wait_ld();
        tc_pin(o);
        if (write && on)
#pragma unroll
          for (int k = 0; k < 32; ++k) slot[(int64_t)(2 + wg * (HD / 2) + c + k) * 128] = poison ? __uint_as_float(0x7FC00000u) : __uint_as_float(o[k]);
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

// Joins the parts of a unit with its tokens' own rows (o2, l2): a thread per
// column, a quarter of the parts and kJoinDims dims, whose loads are all in flight; the
// quarters meet in shared memory, in order. (A thread for all parts waited
// for memory again and again: 13 to 19 us.)
constexpr int kJoinDims = 8, kJoinQuarters = 4, kJoinLoads = 5;

template <int HD>
__global__ void __launch_bounds__(128 * kJoinQuarters) k_join_group(const __grid_constant__ AttendArgs A, const float* o2, const float* l2,
                                                                    const int32_t* own_live, const __grid_constant__ GroupOwn own, int grid) {
  __shared__ float s_m[kJoinQuarters][128], s_l[kJoinQuarters][128], s_v[kJoinQuarters][kJoinDims][128];
  const int u = blockIdx.x, d0 = blockIdx.y * kJoinDims, c = threadIdx.x & 127, quarter = threadIdx.x >> 7;
  int s = 0, hi_s = A.n_seqs - 1;
  while (s < hi_s) {
    const int mid = (s + hi_s + 1) >> 1;
    if (A.seq[mid].unit0 <= u) s = mid; else hi_s = mid - 1;
  }
  const AttendSeq& S = A.seq[s];
  const int ct = (S.t * A.G + 127) / 128, x = u - S.unit0, g = x / ct, col = (x - g * ct) * 128 + c;
  const bool on = col < S.t * A.G;
  const int tok = S.tok0 + (on ? col / A.G : 0), head = g * A.G + (on ? col % A.G : 0);
  const int64_t at = (int64_t)tok * A.nq + head;
  const int64_t total = A.table[A.units], t0 = A.table[u], t1 = A.table[u + 1];
  // the sequence's own rows join the first quarter
  float m = -INFINITY, l = 0.f, v[kJoinDims];
#pragma unroll
  for (int e = 0; e < kJoinDims; ++e) v[e] = 0.f;
  if (quarter == 0 && on) {
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
    const int64_t workers = min((int64_t)grid, total);
    c0 = (int)(((t0 + 1) * workers - 1) / total);
    parts = (int)((t1 * workers - 1) / total) - c0 + 1;
  }
  constexpr int64_t kSlot = 128 * (HD + 2);
  const float* p = A.part + (int64_t)(u + c0) * kSlot + c;
  if (on)
    for (int k0 = quarter; k0 < parts; k0 += kJoinQuarters * kJoinLoads) {
      float pm[kJoinLoads], pl[kJoinLoads], pv[kJoinLoads][kJoinDims];
#pragma unroll
      for (int k = 0; k < kJoinLoads; ++k) {
        const float* y = p + min(k0 + k * kJoinQuarters, parts - 1) * kSlot;   // (in the place of a part that is not there one that is)
        pm[k] = y[0];
        pl[k] = y[128];
#pragma unroll
        for (int e = 0; e < kJoinDims; ++e) pv[k][e] = y[(2 + d0 + e) * 128];
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kJoinLoads; ++k)
        if (k0 + k * kJoinQuarters < parts) top = fmaxf(top, pm[k]);
      const float tb = top == -INFINITY ? 0.f : top, f0 = exp2f(m - tb);
      l *= f0;
#pragma unroll
      for (int e = 0; e < kJoinDims; ++e) v[e] *= f0;
#pragma unroll
      for (int k = 0; k < kJoinLoads; ++k)
        if (k0 + k * kJoinQuarters < parts) {
          const float f = exp2f(pm[k] - tb);
          l = fmaf(pl[k], f, l);
#pragma unroll
          for (int e = 0; e < kJoinDims; ++e) v[e] = fmaf(pv[k][e], f, v[e]);
        }
      m = top;
    }
  s_m[quarter][c] = m;
  s_l[quarter][c] = l;
#pragma unroll
  for (int e = 0; e < kJoinDims; ++e) s_v[quarter][e][c] = v[e];
  __syncthreads();
  if (quarter != 0 || !on) return;
  int q = 0, hi_q = own.n_seqs - 1;                        // the token's sequence
  while (q < hi_q) {
    const int mid = (q + hi_q + 1) >> 1;
    if (own.tok0[mid] <= tok) q = mid; else hi_q = mid - 1;
  }
  const int n1 = *((volatile const int32_t*)(A.n_live + s)), n2 = *((volatile const int32_t*)(own_live + q));
  if (n1 < 0 || n1 > S.cap || n2 < 0 || n2 > own.cap[q]) return;
  float top = m;
#pragma unroll
  for (int k = 1; k < kJoinQuarters; ++k) top = fmaxf(top, s_m[k][c]);
  const float tb = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < kJoinDims; ++e) v[e] = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinQuarters; ++k) {
    const float f = exp2f(s_m[k][c] - tb);
    sum = fmaf(s_l[k][c], f, sum);
#pragma unroll
    for (int e = 0; e < kJoinDims; ++e) v[e] = fmaf(s_v[k][e][c], f, v[e]);
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

template <int HD>
cudaError_t launch_join_hd(const AttendArgs& A, const float* o2, const float* l2, const int32_t* own_live, const GroupOwn& own, int grid,
                           cudaStream_t st) {
  k_join_group<HD><<<dim3(A.units, A.hd / kJoinDims), 128 * kJoinQuarters, 0, st>>>(A, o2, l2, own_live, own, grid);
  return cudaGetLastError();
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
