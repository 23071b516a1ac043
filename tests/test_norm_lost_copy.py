"""rms_norm_backward when a bulk copy does not come: the block that waited in vain leaves NaN in dx for the rows that it did not
finish, never what was there before.  The kernel's row loop runs on the host (tests/c/norm_rows.cpp)."""
import os
import shutil
import subprocess

import pytest

from combine_get_dispatch_histograms_gb300.build import CSRC, INCLUDE

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def norm_rows(tmp_path_factory):
    cxx = shutil.which("g++")
    cuda = os.path.join(os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc")), "include")
    if cxx is None or not os.path.exists(os.path.join(cuda, "cuda_bf16.h")):
        pytest.skip("no g++ or no CUDA headers")
    at = tmp_path_factory.mktemp("norm_rows")
    text = open(os.path.join(CSRC, "ep_norm.cu")).read()
    device, host = text.split("// ---- host ---")                # the kernels alone
    device = "\n".join(l for l in device.replace("extern __shared__", "extern").splitlines() if not l.startswith('#include "')) + "\n}\n"
    (at / "norm_kernels.inc").write_text(device)
    exe = at / "norm_rows"
    r = subprocess.run([cxx, "-std=c++20", "-O1", "-pthread", "-w", f'-DNORM_SOURCE="{at / "norm_kernels.inc"}"', "-I", INCLUDE, "-I", cuda,
                        os.path.join(HERE, "c", "norm_rows.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]

    def run(*args):
        r = subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        lines = r.stdout.split("\n")[:-1]
        return lines[:-1], lines[-1]
    return run


@pytest.mark.parametrize("stages", [1, 2, 4])
def test_every_copy_comes(norm_rows, stages):
    rows, dw = norm_rows(1032, 13, 2, stages, -1)
    assert rows == ["ok"] * 13 and dw == "dweight ok"


@pytest.mark.parametrize("stages", [1, 2, 4])
@pytest.mark.parametrize("lost", [0, 3, 6, 12])
def test_a_copy_is_lost(norm_rows, stages, lost):
    """Blocks take every second row: from the lost one on, that block's are NaN, all others right."""
    rows, dw = norm_rows(1032, 13, 2, stages, lost)
    assert rows == ["nan" if r >= lost and r % 2 == lost % 2 else "ok" for r in range(13)]
    assert dw == "dweight nan"
