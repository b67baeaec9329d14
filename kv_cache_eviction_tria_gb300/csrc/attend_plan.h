// Host arithmetic of rotation, append and attention that needs no GPU: grids and
// splits for a number of SMs, which sequences are prompts, and the rows of the
// fp16 copies that prompts over quantised planes read (k_widen). Plain C++, so that
// it can be checked by itself.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace tria {

// CTAs of k_rope, of which an SM holds one: warps take equal shares of the work
// (tokens x groups of heads), so no more than one wave.
inline int rope_grid(int64_t tokens, int64_t groups, int warps, int sms) {
  return (int)std::min<int64_t>(std::max<int64_t>((tokens * groups + warps - 1) / warps, 1), sms);
}

// Parts of a unit of the fp32 attention kernel (units: of all KV heads): three CTAs
// per SM, no part under 128 rows of the capacity. Units that are split count their
// arrivals: no more of them than there are counters.
inline int plain_split(int64_t units, int cap_max, int sms, int counters) {
  if (units > counters) return 1;
  const int64_t want = (3 * (int64_t)sms + units - 1) / std::max<int64_t>(units, 1);
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, ((int64_t)cap_max + 127) / 128, 64}));
}

// Columns (token x query head of a KV head's group) that a sequence may have
// as a decode step.
constexpr int kStepCols = 16;

inline bool prompt_cols_reached(int tokens, int group) { return (int64_t)tokens * group > kStepCols; }

// Rows of a widened plane: the segments of the prompts' sequences, one after
// the other; a sequence that is no prompt has none, wherever it stands in the
// batch. first (optional, [n_seqs]): the row at which a prompt's segments
// begin. The number is the space that the workspace holds for the plane and the
// height of its tensor map, whose bounds keep a tile that reaches past the last
// row inside the workspace: both have to be this one.
inline int64_t widened_rows(int n_seqs, int n_kv, int group, const int32_t* capacity, const int32_t* tok0, int64_t* first) {
  int64_t rows = 0;
  for (int s = 0; s < n_seqs; ++s) {
    const bool prompt = prompt_cols_reached(tok0[s + 1] - tok0[s], group);
    if (first) first[s] = prompt ? rows : 0;
    if (prompt) rows += (int64_t)n_kv * capacity[s];
  }
  return rows;
}

}  // namespace tria
