"""The host arithmetic of rotation, append and attention (csrc/attend_plan.h),
compiled by itself: the rows of the fp16 copies of quantised planes, grids and
splits for a number of SMs. No GPU."""
import os
import shutil
import subprocess

import numpy as np
import pytest

import kv_cache_eviction_tria_gb300 as tria

CSRC = os.path.join(os.path.dirname(os.path.abspath(tria.__file__)), "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "attend_plan.h"
// n_seqs n_kv group, capacities, token offsets -> rows, first rows
// 0 sms units, cap_max, counters, tokens, groups, warps -> parts of a unit, CTAs of a rotation
int main() {
  int n, kv, g;
  while (std::scanf("%d %d %d", &n, &kv, &g) == 3) {
    if (n == 0) {
      int cap_max, counters, groups, warps;
      long long tokens;
      if (std::scanf("%d %d %lld %d %d", &cap_max, &counters, &tokens, &groups, &warps) != 5) return 1;
      std::printf("%d %d\n", tria::plain_split(g, cap_max, kv, counters), tria::rope_grid(tokens, groups, warps, kv));
      continue;
    }
    std::vector<int32_t> cap(n), tok0(n + 1);
    std::vector<int64_t> first(n, -1);
    for (int& c : cap) if (std::scanf("%d", &c) != 1) return 1;
    for (int& t : tok0) if (std::scanf("%d", &t) != 1) return 1;
    const long long rows = tria::widened_rows(n, kv, g, cap.data(), tok0.data(), first.data());
    if (rows != tria::widened_rows(n, kv, g, cap.data(), tok0.data(), nullptr)) return 1;
    std::printf("%lld", rows);
    for (int64_t f : first) std::printf(" %lld", (long long)f);
    std::printf("\n");
  }
}
"""

# (KV heads, group, capacities, tokens): the steps and the empty sequences last, in the middle and first, with less and with
# more rows than the prompts
BATCHES = [(2, 4, [300, 20000], [50, 1]), (2, 4, [300, 20000], [50, 0]), (2, 4, [20000, 300], [1, 50]),
           (8, 4, [700, 65536, 90], [17, 1, 65]), (8, 4, [65536, 700, 0, 90], [4, 5, 0, 65]), (1, 8, [40, 40, 40], [2, 3, 2]),
           (2, 1, [500, 9], [17, 16]), (3, 2, [0, 64], [9, 9]), (2, 4, [100, 100], [1, 4]), (128, 1, [1 << 20, 1 << 22], [17, 0])]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    res = subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(d / "plan.cpp"), "-o",
                          str(d / "plan")], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr

    def ask(text):
        res = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True)
        return [[int(x) for x in line.split()] for line in res.stdout.splitlines()]
    return ask


@pytest.mark.parametrize("kv,group,cap,tokens", BATCHES)
def test_widened_rows_are_the_prompts_alone(plan, kv, group, cap, tokens):
    """The height of the tensor map is the rows of the prompts' segments, which lie one after the other: a tile that
    starts at any of their rows and reaches past the last one is filled by the map's bounds, not by what lies behind."""
    tok0 = [0] + list(np.cumsum(tokens))
    (rows, *first), = plan(f"{len(cap)} {kv} {group} {' '.join(map(str, cap))} {' '.join(map(str, tok0))}\n")
    at = 0
    for f, c, t in zip(first, cap, tokens):
        if t * group > 16:
            assert f == at
            at += kv * c
    assert rows == at


@pytest.mark.parametrize("k_type,v_type,planes", [("q8_0", "q4_0", 3), ("q4_0", "f16", 2), ("f16", "q8_0", 1)])
@pytest.mark.parametrize("kv,group,cap,tokens", BATCHES)
def test_the_workspace_holds_the_widened_rows(plan, kv, group, cap, tokens, k_type, v_type, planes):
    """What tria_attend_workspace_size reserves beyond an fp16 cache's is those rows, plane by plane (keys have two),
    whichever sequence of the batch has the most rows."""
    hd = 128
    tok0 = np.asarray([0] + list(np.cumsum(tokens)), np.int32)
    (rows, *_), = plan(f"{len(cap)} {kv} {group} {' '.join(map(str, cap))} {' '.join(map(str, tok0))}\n")
    row0 = np.concatenate([[0], np.cumsum(kv * np.asarray(cap, np.int64))[:-1]])

    def size(k, v):
        c = tria.LayerCache(k=0x10000, v=0x20000, pos=0x30000, n_live=0x40000, seq_row0=row0, capacity=cap, head_dim=hd,
                            n_kv_heads=kv, k_type=k, v_type=v, k_scale=None if k == "f16" else 0x50000,
                            v_scale=None if v == "f16" else 0x60000)
        return tria.attend_workspace_size(c, kv * group, tok0)
    if not os.path.exists(tria.LIB_PATH):
        from kv_cache_eviction_tria_gb300 import _build
        _build.build()
    assert size(k_type, v_type) - size("f16", "f16") == planes * ((rows * hd * 2 + 255) // 256 * 256)


@pytest.mark.parametrize("sms", [1, 38, 76, 152, 400])
def test_splits_and_grids_follow_the_sms(plan, sms):
    """Whatever the part of a GPU: units that are split are no more than their counters, the parts of a unit fill three
    CTAs per SM where the rows allow it, a rotation is one wave."""
    asked = [(u, cap, tok, g) for u in (0, 1, 7, 455, 456, 1024, 1025, 10 ** 6) for cap in (0, 100, 128, 129, 1 << 20)
             for tok, g in ((1, 1), (8191, 20), (0, 1))]
    got = plan("".join(f"0 {sms} {u} {cap} 1024 {tok} {g} 16\n" for u, cap, tok, g in asked))
    for (u, cap, tok, g), (split, grid) in zip(asked, got):
        assert 1 <= split <= 64 and (split == 1 or (u <= 1024 and (split - 1) * 128 < cap and u * (split - 1) < 3 * sms))
        assert split == 64 or u > 1024 or u == 0 or u * split >= 3 * sms or split * 128 >= cap
        assert 1 <= grid <= sms and (grid == sms or grid * 16 >= tok * g)
