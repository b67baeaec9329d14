// Attention of many new tokens over the cache (prompts and their chunks) on
// the fifth-generation tensor cores.
//
//   S = Q K^T (128 x BN, fp32 in TMEM), P = 2^(scale S - M) (fp16, written over
//   S in TMEM), O += P V (128 x head_dim, fp32 in TMEM), l = sum of P
//
// A tile's 128 rows are (token, head) pairs of one KV head's group, so that a
// key tile is read once for the whole group. Per CTA (one per SM): two such
// tiles with a softmax warpgroup each (one tile at head_dim 256, where two
// outputs would fill TMEM, with two score buffers), so that the tensor cores
// work on one tile while the other is in its softmax; threads that keep a ring
// of key and value tiles filled; one thread that issues the products. What
// bounds it is the tensor cores' rate together with one exponential per score.
//
// Heads of other sizes take the next larger kernel: a tile's dims past the
// plane's last one arrive as zeros.
//
// 8192 tokens of 32 heads x 128 dims over their own rows take 462 us, 1190
// TFLOP/s of the visible products (the hidden halves of diagonal tiles and each
// CTA's start and end included); far from the ends a pair of tiles takes 1.64
// us, 1490 TFLOP/s.
//
// A thread owns a row of S: maximum and sum need no shuffles. The reference M
// moves only when a row's maximum has grown by more than 2^8 (kLazy), since
// until then P stays inside fp16 (it is kept 2^-kShift below its limit) and
// the common factor cancels in O / l: rescaling O costs a pass over TMEM and is
// rare this way.
//
// Tiles come by TMA into 128-byte-swizzled shared memory, so the planes are
// fp16: 8- and 4-bit rows go into the workspace as fp16 (code x scale) first
// (k_widen), values rounded once, keys as the rounded value and the remainder,
// which takes a product of its own (kLow). The remainders are exact: a scale is a
// multiple of 2^-24 and a code whole, so what rounding leaves of their product has 8
// bits at most, all above 2^-24. lse is given out in fp32 and would show the keys'
// rounding (2e-3 at 230, 1e-5 with the remainders), which the output's own type
// hides: a caller who takes it (round_keys) saves the remainders. 3162 tokens in two
// chunks over 27081 rows take 975 us with them, 640 us without. Converting the rows
// tile by tile on their way into shared memory, which the products' operands
// already fill to its rate and where each row would be converted again for every
// 256 columns, held a pair of tiles at 2.3 (q4_0) and 3.2 us (q8_0) instead of 1.7.
//
// In tiles that some token does not see whole, value rows past the last one
// become zeros, and one that holds an infinity or NaN is replaced by zeros
// while the tokens that do see it get NaN, so that hidden junk never meets a
// weight of zero.
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "attend_tc.cuh"

namespace tria {

namespace {

template <int HD>
struct PromptShape {
  static constexpr int QT = HD == 256 ? 1 : 2;             // tiles of 128 rows per CTA
  static constexpr int BN = HD == 256 ? 64 : 128;          // rows of a key / value tile
  static constexpr int NB = HD == 256 ? 2 : 1;             // score buffers of a tile
  static constexpr int kQ = 128 * HD * 2;                  // bytes of a query tile
  static constexpr int kStage = BN * HD * 2;
  static constexpr int kStages = HD == 64 ? 8 : 5;
  static constexpr int kPosTiles = 4;                      // positions are kept of the last tiles: a tile's value
                                                           // stage is free once the fourth before it is done
  static constexpr int oQ = 0, oRing = QT * kQ, oPos = oRing + kStages * kStage;
  static constexpr int oBar = oPos + kPosTiles * BN * 4;   // barriers, then PromptShared
  static constexpr int kSmem = oBar + 512;
  // TMEM columns: score buffers, outputs
  static constexpr int cO = 256;
  static constexpr int cS(int q, int buf) { return (NB * q + buf) * BN; }
  static_assert(QT * NB * BN <= cO && cO + QT * HD <= 512, "TMEM");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct PromptShared {
  uint32_t junk[8][4];                                     // rows of a value tile that held junk, by stage
  uint32_t tmem, abort;
  int32_t pmin, pmax, hi, need_pos;
};
constexpr int kPromptBars = 2 * 8 + 4 + 4 + 2 + 2 + 3;
static_assert(kPromptBars * 8 + sizeof(PromptShared) <= 512, "barriers and shared state");

// two warpgroups of softmax; one whose first warp loads keys (the others only
// find the rows); one of which three warps load and look through values and
// the last issues the products
constexpr int kPromptThreads = 512, kIssueWarp = 15, kLoadV = 96, kPromptRegs = 128;
// registers of a thread in the softmax (a row of 128 scores stays in them) and
// in the other warpgroups, cut from what the block starts with
constexpr int kSoftRegs = 192, kOtherRegs = 64;
static_assert(2 * kSoftRegs + 2 * kOtherRegs == 4 * kPromptRegs, "register shares");

template <int HD, bool kLow>
__global__ void __launch_bounds__(kPromptThreads, 1) k_attend_prompt(const __grid_constant__ AttendArgs A,
                                                                     const __grid_constant__ CUtensorMap map_k,
                                                                     const __grid_constant__ CUtensorMap map_kl,
                                                                     const __grid_constant__ CUtensorMap map_v) {
  using H = PromptShape<HD>;
  // ring entries of tile i: keys P i, their remainders P i + 1 (kLow), values P i + P - 1
  constexpr int P = kLow ? 3 : 2;
  constexpr int QT = H::QT, BN = H::BN, NB = H::NB, ST = H::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + H::oBar);
  // full: a tile is in the ring; empty: its products are done; s: scores; p:
  // weights; q: queries; o: sums; f: the last sums; x: every product; raw: values that are
  // looked through before their tile is full
  uint64_t *b_full = bar, *b_empty = bar + ST, *b_s = bar + 2 * ST, *b_p = b_s + 4, *b_o = b_p + 4, *b_f = b_o + 2, *b_q = b_f + 2, *b_x = b_q + 1,
           *b_raw = b_x + 1;
  int32_t* s_pos = reinterpret_cast<int32_t*>(smem + H::oPos);
  PromptShared& X = *reinterpret_cast<PromptShared*>(smem + H::oBar + kPromptBars * 8);
  volatile uint32_t* s_abort = &X.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;

  // ---- the unit: QT x 128 columns (token x head) of one KV head; late tokens first
  const int part = blockIdx.x % A.split;
  const int y = A.units * A.n_kv - 1 - (int)(blockIdx.x / A.split);
  const int unit = y / A.n_kv, g = y - unit * A.n_kv;
  int s = 0;
  {
    int hi_s = A.n_seqs - 1;
    while (s < hi_s) {
      const int mid = (s + hi_s + 1) >> 1;
      if (A.seq[mid].unit0 <= unit) s = mid; else hi_s = mid - 1;
    }
  }
  const AttendSeq& S = A.seq[s];
  const int n = *((volatile const int32_t*)(A.n_live + s));
  if (n < 0 || n > S.cap) {
    if (threadIdx.x == 0) report(A.ctrl, TRIA_ERR_DEVICE_ARG, (uint32_t)s);
    return;
  }
  if (smem_u32(smem) & 1023u) {                            // the swizzled tiles need it
    if (threadIdx.x == 0) report(A.ctrl, TRIA_ERR_CUDA, (uint32_t)s);
    return;
  }
  const int c0 = (unit - S.unit0) * (QT * 128), ncol = min(QT * 128, S.t * A.G - c0);
  const int tok_a = c0 / A.G, tok_b = (c0 + ncol - 1) / A.G;   // its tokens (of the sequence)
  const int64_t row0 = S.row0 + (int64_t)g * S.cap, seg0 = (int64_t)g * S.cap;
  const int64_t key0 = seg0 + (A.wide_k ? S.wide0 : S.row0), value0 = seg0 + (A.wide_v ? S.wide0 : S.row0);
  const int32_t* rpos = A.cpos + row0;
  // loads that need nothing else are on their way before the set-up: a thread
  // per row of the softmax, its queries; the loading warpgroup, the tokens'
  // positions and those of the rows around the place where the newest of these
  // tokens should be (behind it, the later tokens' rows)
  const uint32_t q_row = threadIdx.x & 127;
  const int col = c0 + wg * 128 + (int)q_row;
  const bool on = wg < QT && wg * 128 + (int)q_row < ncol;
  const int tl = on ? col / A.G : tok_a;
  const int64_t tok = S.tok0 + tl;
  const int head = g * A.G + (on ? col - tl * A.G : 0);
  const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(A.q) + tok * A.q_stride + (int64_t)head * A.hd);
  auto piece = [&](int c) { return on && 8 * c < A.hd ? src[c] : make_uint4(0, 0, 0, 0); };
  constexpr int kPart = HD / 8 < 16 ? HD / 8 : 16;         // 16-byte pieces held at once
  uint4 v[kPart];
  int pl = INT32_MAX, ph = INT32_MIN, before = 0, after = 0;
  const int h = n - (S.t - 1 - tok_b);
  if (wg < QT) {
#pragma unroll
    for (int c = 0; c < kPart; ++c) v[c] = piece(c);
  } else if (wg == 2) {
    if (h > 0) before = rpos[h - 1];
    if (h >= 0 && h < n) after = rpos[h];
    for (int i = tok_a + (int)q_row; i <= tok_b; i += 128) {
      const int p = A.pos[S.tok0 + i];
      pl = min(pl, p);
      ph = max(ph, p);
    }
  }
  if (threadIdx.x == 480) {                                // the issuing warp's first thread
    X.pmin = INT32_MAX;
    X.pmax = INT32_MIN;
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
    }
    mbar_init(b_q, QT * 128);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b_o[i], 1);
      mbar_init(&b_f[i], 1);
    }
    mbar_init(b_x, 1);
    mbar_init(b_raw, 1);
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&X.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();
  // ---- queries into shared memory; the rows that these tokens see
  float sl = A.scale * 1.4426950408889634f;
  if (wg < QT) {
    // as fp16; bf16 ones times a power of two, undone in the logits
    uint8_t* dst = smem + H::oQ + wg * H::kQ;
    float f = 1.f;
    if (A.type == TRIA_BF16) {
      uint32_t am = 0;
#pragma unroll 1
      for (int c0q = 0; c0q < HD / 8; c0q += kPart) {
#pragma unroll
        for (int c = 0; c < kPart; ++c)
          if (c0q > 0) v[c] = piece(c0q + c);
#pragma unroll
        for (int c = 0; c < kPart; ++c) {
          const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) am = max(am, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
        }
      }
      const int ex = (int)(am >> 7) - 127;
      if (ex > -120 && ex < 120) {
        f = __uint_as_float((uint32_t)(127 - ex) << 23);
        sl *= __uint_as_float((uint32_t)(127 + ex) << 23);
      }
    }
    sl = fmaxf(sl, 0x1p-126f);                             // (times -inf stays -inf)
#pragma unroll 1
    for (int c0q = 0; c0q < HD / 8; c0q += kPart) {
#pragma unroll
      for (int c = 0; c < kPart; ++c)
        if (HD / 8 > kPart) v[c] = piece(c0q + c);
#pragma unroll
      for (int c = 0; c < kPart; ++c) {
        uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
        if (A.type == TRIA_BF16) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half2 h = __floats2half2_rn(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
        const int cc = c0q + c;
        *reinterpret_cast<uint4*>(dst + (cc >> 3) * (128 * 128) + swz(q_row, cc & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(b_q);
  } else if (wg == 2) {
    pl = __reduce_min_sync(0xffffffffu, pl);
    ph = __reduce_max_sync(0xffffffffu, ph);
    if (lane == 0) {
      atomicMin(&X.pmin, pl);
      atomicMax(&X.pmax, ph);
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (warp == 8) {
      // rows up to the newest token; where it is not as expected, by a search in 32 parts
      const int pmin = *(volatile int32_t*)&X.pmin, pmax = *(volatile int32_t*)&X.pmax;
      const bool there = h >= 0 && (h == 0 || before <= pmax) && (h == n || after > pmax);
      int lo = 0, hi = n;                                  // rows < lo are <= pmax, rows >= hi are not
      if (there) {
        lo = hi = h;
      } else {
        while (lo < hi) {
          const int step = (hi - lo + 31) / 32;
          const int r = min(hi, lo + (lane + 1) * step) - 1;   // last row of this lane's share
          const unsigned okm = __ballot_sync(0xffffffffu, rpos[r] <= pmax);
          const int k = __popc(okm);                       // whole shares at or below pmax
          lo = min(hi, lo + k * step);
          if (k < 32) hi = min(hi, lo + step - 1);
        }
      }
      if (!there && lo > 0) before = rpos[lo - 1];
      if (lane == 0) {
        X.hi = lo;
        X.need_pos = A.window > 0 || (lo > 0 && before > pmin);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int pmin = X.pmin, pmax = X.pmax;
  const int hi = X.hi;
  const int lo = A.window > 0 ? (int)max((int64_t)0, hi - (A.window + (int64_t)pmax - pmin)) : 0;
  const int sr = min(A.sink, lo), nt_sink = (sr + BN - 1) / BN;
  const int nt_all = nt_sink + (hi - lo + BN - 1) / BN;
  const int ta = (int)((int64_t)part * nt_all / A.split), nt = (int)((int64_t)(part + 1) * nt_all / A.split) - ta;
  const bool need_pos = X.need_pos != 0;
  auto tile_row = [&](int i, int& rows) {
    const int j = ta + i;
    if (j < nt_sink) {
      rows = min(BN, sr - j * BN);
      return j * BN;
    }
    const int r = lo + (j - nt_sink) * BN;
    rows = min(BN, hi - r);
    return r;
  };
  const uint32_t tmem = X.tmem;
  // bounded waits; after one gave up nobody waits any more, and the CTA writes no
  // results. The issuing warp goes on or gives up as one (wait_warp). Threads that
  // wait for themselves may learn different things near a limit, so none of them
  // leaves: the softmax and the loading warps run their loops to the end, past waits
  // that return at once, and a warp's lanes meet at every collective instruction.
  // (With votes at each of their waits a prompt of 8192 tokens took 530 us instead of 463.)
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

  if (wg >= 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kIssueWarp) {
    // ---- products
    if (nt > 0) {
      // results of waits and addresses are the same in all lanes and kept in
      // such a form (votes, a broadcast): operands of the products then live in
      // uniform registers, without which issuing them was the bottleneck
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t dq = tile_desc(smem_u32(smem + H::oQ), 16), dk = tile_desc(smem_u32(smem + H::oRing), 16),
                     dv = tile_desc(smem_u32(smem + H::oRing), BN * 128);
      auto scores = [&](int q, int i, int st, int sl) {    // address fields count 16 bytes
        const uint64_t a = dq + (uint64_t)(q * (H::kQ / 16)), b = dk + (uint64_t)(st * (H::kStage / 16));
        const uint32_t d = tm + H::cS(q, i % NB);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
          tc_mma_ss(d, a + (uint64_t)((k >> 2) * (128 * 8) + (k & 3) * 2), b + (uint64_t)((k >> 2) * (BN * 8) + (k & 3) * 2),
                    mma_desc(BN, false), k > 0);
        if constexpr (kLow) {
          const uint64_t bl = dk + (uint64_t)(sl * (H::kStage / 16));
#pragma unroll
          for (int k = 0; k < HD / 16; ++k)
            tc_mma_ss(d, a + (uint64_t)((k >> 2) * (128 * 8) + (k & 3) * 2), bl + (uint64_t)((k >> 2) * (BN * 8) + (k & 3) * 2),
                      mma_desc(BN, false), 1);
        }
        tc_commit(&b_s[NB * q + i % NB]);
      };
      auto sums = [&](int q, int i, int st) {
        const uint64_t b = dv + (uint64_t)(st * (H::kStage / 16));
        const uint32_t d = tm + H::cO + q * HD, a = tm + H::cS(q, i % NB);
#pragma unroll
        for (int k = 0; k < BN / 16; ++k) tc_mma_ts(d, a + k * 8, b + (uint64_t)(k * 128), mma_desc(HD, true), i > 0 || k > 0);
        tc_commit(&b_o[q]);
      };
      bool ok = wait_warp(b_q, 0) && wait_warp(&b_full[0], 0) && (!kLow || wait_warp(&b_full[1], 0));
      tc_fence_after();
      if (ok && elect_one()) {
#pragma unroll
        for (int q = 0; q < QT; ++q) scores(q, 0, 0, 1);
        tc_commit(&b_empty[0]);
        if (kLow) tc_commit(&b_empty[1]);
      }
      __syncwarp();
      int sv = P - 1, sk = P, pv = 0, pk = 0;              // ring stage and parity of V(i), K(i + 1)
      static_assert(P + 1 < ST, "the first ones lie in the ring's first round");
      for (int i = 0; ok && i < nt; ++i) {
        const bool more = i + 1 < nt;
        const int sl = sk + 1 == ST ? 0 : sk + 1, pl2 = sk + 1 == ST ? pk ^ 1 : pk;   // of the remainders of K(i + 1)
        if (more) ok = wait_warp(&b_full[sk], pk) && (!kLow || wait_warp(&b_full[sl], pl2));
        if constexpr (NB == 2) {
          // the other buffer's weights are those of tile i - 1, whose sums were issued before
          if (more) {
            tc_fence_after();
            if (ok && elect_one()) {
#pragma unroll
              for (int q = 0; q < QT; ++q) scores(q, i + 1, sk, sl);
              tc_commit(&b_empty[sk]);
              if (kLow) tc_commit(&b_empty[sl]);
            }
            __syncwarp();
          }
        }
        ok = ok && wait_warp(&b_full[sv], pv);
#pragma unroll
        for (int q = 0; q < QT; ++q) {
          ok = ok && wait_warp(&b_p[NB * q + i % NB], (i / NB) & 1);
          tc_fence_after();
          if (ok && elect_one()) {
            sums(q, i, sv);
            // products run in the order of their issue: the scores overwrite weights that the sums have used
            if (NB == 1 && more) scores(q, i + 1, sk, sl);
          }
          __syncwarp();
        }
        if (ok && elect_one()) {
          tc_commit(&b_empty[sv]);
          if (NB == 1 && more) {
            tc_commit(&b_empty[sk]);
            if (kLow) tc_commit(&b_empty[sl]);
          }
          if (!more)
#pragma unroll
            for (int q = 0; q < QT; ++q) tc_commit(&b_f[q]);
        }
        __syncwarp();
        sv += P;
        if (sv >= ST) {
          sv -= ST;
          pv ^= 1;
        }
        sk += P;
        if (sk >= ST) {
          sk -= ST;
          pk ^= 1;
        }
      }
      // nothing may be running when the accumulators are given back
      if (elect_one()) tc_commit(b_x);
      for (int it = 0; it < kWaitLimit && !mbar_try_wait(b_x, 0); ++it) {
      }
    }
  } else if (wg >= 2) {
    // ---- key tiles and value tiles
    const int tid = threadIdx.x & 127;
    auto stage = [&](int e) { return smem + H::oRing + (e % ST) * H::kStage; };
    auto free_stage = [&](int e) {
      if (e >= ST) wait(&b_empty[e % ST], ((e / ST) - 1) & 1);
    };
    // after a wait gave up the loops start no more copies, and wait, bounded, for
    // those still on their way
    auto go = [&] { return tid == 0 && !*s_abort; };
    auto drain = [&](bool values) {
      if (!*s_abort || tid != 0) return;
      for (int e = max(0, P * nt - ST); e < P * nt; ++e)
        for (int it = 0; it < 1024 && (e % P == P - 1) == values && !mbar_try_wait(&b_full[e % ST], (e / ST) & 1); ++it) {
        }
    };
    int rows;
    if (wg == 2) {
      if (tid == 0) {
        for (int i = 0; i < nt; ++i) {
          // hidden keys, and those past the last row, only reach logits that the mask replaces
          const int r = tile_row(i, rows), e = P * i;
          free_stage(e);
          if (go()) copy_tile<HD, BN>(stage(e), &map_k, key0 + r, &b_full[e % ST]);
          if constexpr (kLow) {
            free_stage(e + 1);
            if (go()) copy_tile<HD, BN>(stage(e + 1), &map_kl, key0 + r, &b_full[(e + 1) % ST]);
          }
        }
        drain(false);
      }
    } else {
      constexpr int kPos = (BN + kLoadV - 1) / kLoadV;
      int next_pos[kPos];                                  // of this thread's rows of the tile to come
      auto fetch_pos = [&](int i) {
        int n_rows;
        const int r = tile_row(i, n_rows);
#pragma unroll
        for (int k = 0; k < kPos; ++k) {
          const int c = k * kLoadV + tid;
          next_pos[k] = INT32_MAX;
          if (need_pos && i < nt && c < n_rows) next_pos[k] = rpos[r + c];
        }
      };
      fetch_pos(0);
      int looked = 0;
      for (int i = 0; i < nt; ++i) {
        const int r = tile_row(i, rows), e = P * i + P - 1;
        free_stage(e);
        __syncwarp();
        // positions and marks go with the value tile, which stays until the weights are used
        const int32_t* tp = s_pos + (i % H::kPosTiles) * BN;
#pragma unroll
        for (int k = 0; k < kPos; ++k)
          if (need_pos && k * kLoadV + tid < BN) s_pos[(i % H::kPosTiles) * BN + k * kLoadV + tid] = next_pos[k];
        fetch_pos(i + 1);
        if (tid < 4) X.junk[e % ST][tid] = 0;
        asm volatile("bar.sync 3, %0;" ::"n"(kLoadV) : "memory");
        const bool all = rows == BN && (!need_pos || (tp[BN - 1] <= pmin && (A.window <= 0 || (int64_t)pmax - tp[0] < A.window ||
                                                                            r + BN <= A.sink)));   // seen whole by every token
        if (go()) copy_tile<HD, BN>(stage(e), &map_v, value0 + r, all ? &b_full[e % ST] : b_raw);
        if (all) continue;
        wait(b_raw, looked & 1);
        __syncwarp();
        ++looked;
        clean_tile<HD, BN, kLoadV>(stage(e), rows, X.junk[e % ST], tid);
        fence_proxy_async_smem();
        asm volatile("bar.sync 3, %0;" ::"n"(kLoadV) : "memory");
        if (tid == 0) mbar_arrive(&b_full[e % ST]);
      }
      drain(true);
    }
  } else if (wg < QT) {
    // ---- softmax: a thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int q = wg, m = (int)q_row;
    const int p = on ? A.pos[tok] : INT32_MIN;
    // rows at or before it are outside the window
    const int pold = A.window > 0 ? (int)max((int64_t)INT32_MIN, (int64_t)p - A.window) : INT32_MIN;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = lane_base + H::cO + q * HD;
    float M = -INFINITY, l = 0.f;
    bool poison = false;
    for (int i = 0; i < nt; ++i) {
      const int buf = NB * q + i % NB;
      wait(&b_s[buf], (i / NB) & 1);
      __syncwarp();
      tc_fence_after();
      const uint32_t ts = lane_base + H::cS(q, i % NB);
      uint32_t x[BN];
#pragma unroll
      for (int c = 0; c < BN; c += 32) tc_ld32(x + c, ts + c);
      int rows;
      const int r = tile_row(i, rows);
      bool masked = rows < BN;
      const int ev = P * i + P - 1;
      if (need_pos || masked) {
        wait(&b_full[ev % ST], (ev / ST) & 1);       // positions and marks are there
        __syncwarp();
      }
      const int32_t* tp = s_pos + (i % H::kPosTiles) * BN;
      if (need_pos)
        masked = masked || tp[BN - 1] > pmin || (A.window > 0 && (int64_t)pmax - tp[0] >= A.window && r + BN > A.sink);
      tc_wait_ld();
#pragma unroll
      for (int c = 0; c < BN; c += 32) tc_pin(x + c);
      if (masked) {
        // the row's token sees columns [cl, ch) and, of the first rows, [0, cf)
        int cl = 0, ch = rows, cf = 0;
        if (need_pos) {
          auto upto = [&](int pos) {                       // columns with a position <= pos
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
        for (int c = 0; c < BN; ++c)
          if (c >= ch || (c < cl && c >= cf)) x[c] = 0xFF800000u;   // -inf
        const uint32_t* jm = X.junk[ev % ST];
        if (jm[0] | jm[1] | jm[2] | jm[3])
          for (int c = 0; c < rows; ++c)
            if (((jm[c >> 5] >> (c & 31)) & 1u) && c < ch && (c >= cl || c < cf)) poison = true;
      }
      float tops[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) tops[k] = __uint_as_float(x[k]);
#pragma unroll
      for (int c = 4; c < BN - 4; c += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tops[k] = fmaxf(fmaxf(tops[k], __uint_as_float(x[c + k])), __uint_as_float(x[c + 4 + k]));
#pragma unroll
      for (int k = 0; k < 4; ++k) tops[k] = fmaxf(tops[k], __uint_as_float(x[BN - 4 + k]));
      float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
      top = top * sl - kShift;
      const bool move = top > M + kLazy || M == -INFINITY;
      if (__any_sync(0xffffffffu, move && top > -INFINITY)) {
        float a = 1.f;
        if (move && top > -INFINITY) {
          a = exp2_fast(M - top);
          M = top;
          l *= a;
        }
        if (i > 0) {
          wait(&b_o[q], (i - 1) & 1);                // the sums of the tile before may be running
          __syncwarp();
          tc_fence_after();
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
          const __half2 h = __floats2half2_rn(e.x, e.y);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        tc_st16(ts + c / 2, w);
      }
      l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(&b_p[buf]);
    }
    // ---- results
    if (nt > 0) {
      wait(&b_f[q], 0);
      tc_fence_after();
    }
    if (__all_sync(0xffffffffu, *s_abort == 0)) {
      const bool split = A.split > 1;
      float* slot = A.part + ((int64_t)y * A.split + part) * (QT * 128) * (HD + 2) + (q * 128 + m);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      // a row leaves through shared memory in one copy (padded rows: no bank
      // conflicts), in the place of the queries: every score is done when
      // b_f is, and with the last tile's sums everything is,
      // whose rows reach past the queries into the ring
      uint8_t* row_out = smem + H::oQ + (q * 128 + m) * (HD * 2 + 16);
#pragma unroll 2
      for (int c = 0; c < HD; c += 32) {
        uint32_t o[32];
        if (nt > 0) {
          tc_ld32(o, to + c);
          tc_wait_ld();
          tc_pin(o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (poison) {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0x7FC00000u;
        }
        if (split) {
#pragma unroll
          for (int k = 0; k < 32; ++k) slot[(int64_t)(2 + c + k) * (QT * 128)] = __uint_as_float(o[k]);
        } else if (A.out_type == TRIA_F32) {               // results that are joined with others
          if (on && c < A.hd) {
            float4* to32 = reinterpret_cast<float4*>(reinterpret_cast<float*>(A.out) + tok * A.out_stride + (int64_t)head * A.hd + c);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              to32[k] = make_float4(__uint_as_float(o[4 * k]) * inv, __uint_as_float(o[4 * k + 1]) * inv, __uint_as_float(o[4 * k + 2]) * inv,
                                    __uint_as_float(o[4 * k + 3]) * inv);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_out(A.type, __uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(row_out + c * 2 + k * 16) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (!split && on && A.out_type != TRIA_F32) {
        fence_proxy_async_smem();
        bulk_s2g(reinterpret_cast<uint16_t*>(A.out) + tok * A.out_stride + (int64_t)head * A.hd, row_out, A.hd * 2);
        bulk_commit();
        bulk_wait_read_all();
      }
      if (split) {
        slot[0] = M;
        slot[QT * 128] = l;
      } else if (on && A.lse) {
        A.lse[tok * A.nq + head] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (threadIdx.x == 0 && *s_abort) report(A.ctrl, TRIA_ERR_TIMEOUT, (uint32_t)s);
  if (warp == kIssueWarp) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ---- parts of split units ------------------------------------------------------

constexpr int kJoinDims = 32;    // dims of a block

// Merges the parts of a unit in order: a thread per column, 32 dims a block.
// (One of the unit's own CTAs doing it alone took longer than all the parts.)
template <int HD>
__global__ void __launch_bounds__(PromptShape<HD>::QT * 128) k_join_parts(const __grid_constant__ AttendArgs A) {
  constexpr int kCols = PromptShape<HD>::QT * 128;
  const int y = blockIdx.x, unit = y / A.n_kv, g = y - unit * A.n_kv, d0 = blockIdx.y * kJoinDims, c = threadIdx.x;
  int s = 0, hi_s = A.n_seqs - 1;
  while (s < hi_s) {
    const int mid = (s + hi_s + 1) >> 1;
    if (A.seq[mid].unit0 <= unit) s = mid; else hi_s = mid - 1;
  }
  const AttendSeq& S = A.seq[s];
  const int n = *((volatile const int32_t*)(A.n_live + s)), col = (unit - S.unit0) * kCols + c;
  if (n < 0 || n > S.cap || col >= S.t * A.G) return;
  const int64_t stride = (int64_t)kCols * (HD + 2), tok = S.tok0 + col / A.G;
  const int head = g * A.G + col % A.G;
  const float* x = A.part + (int64_t)y * A.split * stride + c;
  float top = -INFINITY, sum = 0.f, v[kJoinDims];
#pragma unroll
  for (int e = 0; e < kJoinDims; ++e) v[e] = 0.f;
  for (int k = 0; k < A.split; ++k) top = fmaxf(top, x[k * stride]);
  const float tb = top == -INFINITY ? 0.f : top;
  for (int k = 0; k < A.split; ++k) {
    const float* p = x + k * stride;
    const float f = exp2_fast(p[0] - tb);
    sum = fmaf(p[kCols], f, sum);
#pragma unroll
    for (int e = 0; e < kJoinDims; ++e) v[e] = fmaf(p[(2 + d0 + e) * kCols], f, v[e]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (d0 == 0 && A.lse) A.lse[tok * A.nq + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  if (A.out_type == TRIA_F32) {
    float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(A.out) + tok * A.out_stride + (int64_t)head * A.hd + d0);
#pragma unroll
    for (int q = 0; q < kJoinDims / 4; ++q) o[q] = make_float4(v[4 * q] * inv, v[4 * q + 1] * inv, v[4 * q + 2] * inv, v[4 * q + 3] * inv);
    return;
  }
  uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(A.out) + tok * A.out_stride + (int64_t)head * A.hd + d0);
#pragma unroll
  for (int q = 0; q < kJoinDims / 8; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_out(A.type, v[8 * q + 2 * e] * inv, v[8 * q + 2 * e + 1] * inv);
    o[q] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---- quantised planes as fp16 ------------------------------------------------

constexpr int kWidenRows = 64;   // rows of a block

// Rows of the prompt's sequences as fp16 (code x scale, rounded once), eight
// values a thread; rows that no token sees are left out. Bound by the fp16
// rows' way to memory.
template <int T, bool kLow>
__device__ __forceinline__ void widen_rows(const uint8_t* data, const uint8_t* scale, uint16_t* out, uint16_t* low, int64_t src,
                                           int64_t dst, int rows, int hd) {
  const int per = hd / 8;
#pragma unroll 4
  for (int x = threadIdx.x; x < rows * per; x += blockDim.x) {
    const int r = x / per, c = x - r * per;
    const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(scale) + (src + r) * (hd / 32) + c / 4);
    const uint32_t sc = h | (h << 16);
    uint32_t o[4], lo[4];
    const float2 sf = make_float2(__half2float(__ushort_as_half((uint16_t)h)), __half2float(__ushort_as_half((uint16_t)h)));
    uint2 w;
    if constexpr (T == TRIA_Q8_0) {
      w = __ldg(reinterpret_cast<const uint2*>(data + (src + r) * hd + c * 8));
      w.x ^= 0x80808080u;                                  // 0x64, code + 128: 1152 + code
      w.y ^= 0x80808080u;
    } else {
      // dims 0..15 of a block in the low halves of its 16 bytes, 16..31 in the high ones
      w = __ldg(reinterpret_cast<const uint2*>(data + (src + r) * (hd / 2) + (c / 4) * 16 + (c & 1) * 8));
      if (c & 2) {
        w.x >>= 4;
        w.y >>= 4;
      }
      w.x &= 0x0F0F0F0Fu;
      w.y &= 0x0F0F0F0Fu;
    }
    const uint32_t bias = T == TRIA_Q8_0 ? 0x64806480u : 0x64086408u;
    const uint32_t b[4] = {__byte_perm(w.x, 0x64646464u, 0x4140), __byte_perm(w.x, 0x64646464u, 0x4342),
                           __byte_perm(w.y, 0x64646464u, 0x4140), __byte_perm(w.y, 0x64646464u, 0x4342)};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[k]) : "r"(b[k]), "r"(bias));
      const float2 code = __half22float2(*reinterpret_cast<const __half2*>(&o[k]));
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(o[k]) : "r"(o[k]), "r"(sc));
      if constexpr (kLow) {
        // code x scale fits fp32, and what fp16 left of it (8 bits at most, all above 2^-24) fits fp16
        const float2 x = __fmul2_rn(code, sf), hi = __half22float2(*reinterpret_cast<const __half2*>(&o[k]));
        const __half2 l = __floats2half2_rn(x.x - hi.x, x.y - hi.y);
        lo[k] = *reinterpret_cast<const uint32_t*>(&l);
      }
    }
    if constexpr (kLow) *reinterpret_cast<uint4*>(low + (dst + r) * hd + c * 8) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(out + (dst + r) * hd + c * 8) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

__global__ void __launch_bounds__(256) k_widen(const __grid_constant__ AttendArgs A) {
  __shared__ int s_min;
  const int g = blockIdx.y;
  // blocks of a sequence follow those of the ones before it
  int s = 0, b = blockIdx.x;
  for (; s < A.n_seqs; ++s) {
    const int nb = A.seq[s].t > 0 ? (A.seq[s].cap + kWidenRows - 1) / kWidenRows : 0;
    if (b < nb) break;
    b -= nb;
  }
  if (s == A.n_seqs) return;
  const AttendSeq& S = A.seq[s];
  const int n = *((volatile const int32_t*)(A.n_live + s)), r0 = b * kWidenRows;
  if (n > S.cap || r0 >= n) return;
  const int rows = min(kWidenRows, n - r0);
  const int64_t seg0 = (int64_t)g * S.cap;
  if (A.window > 0 && r0 >= A.sink) {
    if (threadIdx.x == 0) s_min = INT32_MAX;
    __syncthreads();
    int p = INT32_MAX;
    for (int i = threadIdx.x; i < S.t; i += blockDim.x) p = min(p, A.pos[S.tok0 + i]);
    p = __reduce_min_sync(0xffffffffu, p);
    if ((threadIdx.x & 31) == 0) atomicMin(&s_min, p);
    __syncthreads();
    if ((int64_t)s_min - A.cpos[S.row0 + seg0 + r0 + rows - 1] >= A.window) return;
  }
  const int64_t src = S.row0 + seg0 + r0, dst = S.wide0 + seg0 + r0;
  if (blockIdx.z == 0) {
    if (A.k_type == TRIA_Q8_0) {
      if (A.wide_kl) widen_rows<TRIA_Q8_0, true>(A.k, A.ks, A.wide_k, A.wide_kl, src, dst, rows, A.hd);
      else widen_rows<TRIA_Q8_0, false>(A.k, A.ks, A.wide_k, nullptr, src, dst, rows, A.hd);
    } else if (A.k_type == TRIA_Q4_0) {
      if (A.wide_kl) widen_rows<TRIA_Q4_0, true>(A.k, A.ks, A.wide_k, A.wide_kl, src, dst, rows, A.hd);
      else widen_rows<TRIA_Q4_0, false>(A.k, A.ks, A.wide_k, nullptr, src, dst, rows, A.hd);
    }
  } else {
    if (A.v_type == TRIA_Q8_0) widen_rows<TRIA_Q8_0, false>(A.v, A.vs, A.wide_v, nullptr, src, dst, rows, A.hd);
    else if (A.v_type == TRIA_Q4_0) widen_rows<TRIA_Q4_0, false>(A.v, A.vs, A.wide_v, nullptr, src, dst, rows, A.hd);
  }
}

template <int HD, bool kLow>
cudaError_t launch_prompt_hd(const AttendArgs& A, cudaStream_t st) {
  using H = PromptShape<HD>;
  auto kern = k_attend_prompt<HD, kLow>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, H::kSmem);
  if (e != cudaSuccess) return e;
  // the warpgroups' register shares are cut from what the block starts with
  cudaFuncAttributes attr;
  const cudaError_t e2 = cudaFuncGetAttributes(&attr, kern);
  if (e2 != cudaSuccess) return e2;
  if (attr.numRegs != kPromptRegs) return cudaErrorInvalidConfiguration;
  const int64_t grid = (int64_t)A.units * A.n_kv * A.split;
  CUtensorMap mk, ml, mv;
  memset(&mk, 0, sizeof(mk));
  memset(&ml, 0, sizeof(ml));
  memset(&mv, 0, sizeof(mv));
  int64_t rows = 0;
  for (int s = 0; s < A.n_seqs; ++s) rows = std::max(rows, A.seq[s].row0 + (int64_t)A.n_kv * A.seq[s].cap);
  if (!plane_map_f16(&mk, A.wide_k ? (const void*)A.wide_k : A.k, A.hd, A.wide_k ? A.wide_rows : rows, H::BN) ||
      !plane_map_f16(&mv, A.wide_v ? (const void*)A.wide_v : A.v, A.hd, A.wide_v ? A.wide_rows : rows, H::BN))
    return cudaErrorInvalidValue;
  if (kLow && !plane_map_f16(&ml, A.wide_kl, A.hd, A.wide_rows, H::BN)) return cudaErrorInvalidValue;
  kern<<<(unsigned)grid, kPromptThreads, H::kSmem, st>>>(A, mk, ml, mv);
  if (A.split > 1) {
    const cudaError_t e3 = cudaGetLastError();
    if (e3 != cudaSuccess) return e3;
    k_join_parts<HD><<<dim3((unsigned)(A.units * A.n_kv), A.hd / kJoinDims), H::QT * 128, 0, st>>>(A);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_prompt(const AttendArgs& A, cudaStream_t st) {
  if (A.wide_k || A.wide_v) {
    int64_t blocks = 0;
    for (int s = 0; s < A.n_seqs; ++s)
      if (A.seq[s].t > 0) blocks += (A.seq[s].cap + kWidenRows - 1) / kWidenRows;
    const dim3 grid((unsigned)blocks, A.n_kv, 2);
    if (blocks > 0) k_widen<<<grid, 256, 0, st>>>(A);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  switch (prompt_dims(A.hd)) {
    case 64: return A.wide_kl ? launch_prompt_hd<64, true>(A, st) : launch_prompt_hd<64, false>(A, st);
    case 128: return A.wide_kl ? launch_prompt_hd<128, true>(A, st) : launch_prompt_hd<128, false>(A, st);
    case 256: return A.wide_kl ? launch_prompt_hd<256, true>(A, st) : launch_prompt_hd<256, false>(A, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace tria
