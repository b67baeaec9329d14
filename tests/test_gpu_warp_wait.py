"""A bounded wait of a whole warp gives all of its lanes the same answer, whether
the barrier completes, another warp gives up or the limit runs out."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

HERE = os.path.dirname(os.path.abspath(__file__))
MET, ABORTED, RUNS_OUT, BOTH = range(4)


@pytest.fixture(scope="module")
def warp_wait(tmp_path_factory):
    from kv_cache_eviction_tria_gb300 import _build
    so = str(tmp_path_factory.mktemp("wait") / "warp_wait.so")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", _build.CSRC, "-I",
                    _build.INCLUDE, os.path.join(HERE, "warp_wait.cu"), "-o", so], check=True, capture_output=True)
    fn = ctypes.CDLL(so).warp_wait
    fn.argtypes = [ctypes.c_int] * 4 + [ctypes.c_void_p] * 2

    def ask(mode, limit, step, blocks):
        out = torch.full((blocks, 32), 7, dtype=torch.int32, device="cuda")
        assert fn(mode, limit, step, blocks, out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        return out.cpu().numpy()
    return ask


@pytest.mark.parametrize("mode,limit,step,blocks,answers", [(MET, 1 << 16, 7, 600, {1}), (ABORTED, 1 << 16, 7, 600, {-1}),
                                                            (RUNS_OUT, 2, 0, 4, {0}), (BOTH, 1 << 16, 7, 600, {1, -1})])
def test_lanes_agree(warp_wait, mode, limit, step, blocks, answers):
    got = warp_wait(mode, limit, step, blocks)
    assert np.all(got == got[:, :1])
    assert set(np.unique(got)) <= answers
