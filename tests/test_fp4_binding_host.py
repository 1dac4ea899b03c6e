"""The Python binding without its call module: no part of the package needs it."""
import subprocess

import pytest
import torch

import blockwise_fp8_weight_b200 as fq
from blockwise_fp8_weight_b200 import build as B


def test_the_library_is_built_without_a_c_compiler(monkeypatch, tmp_path):
    """Only nvcc is asked for; a C compiler that is missing stops nothing."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd[0])
        if cmd[0] != B.nvcc():
            raise FileNotFoundError(cmd[0])
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(B.subprocess, "run", run)
    for name in ("LIB", "LIB_CHECKED", "CALLS"):
        monkeypatch.setattr(B, name, str(tmp_path / name))
    assert B.build() == str(tmp_path / "LIB")
    assert B.build(checked=True) == str(tmp_path / "LIB_CHECKED")
    assert ran == [B.nvcc()] * 2


@pytest.mark.parametrize("error", [FileNotFoundError("gcc"), RuntimeError("nvcc not found"),
                                   subprocess.CalledProcessError(1, "gcc"), ImportError("_calls")])
def test_a_call_module_that_cannot_be_built_is_done_without(monkeypatch, error):
    def fail(force=False):
        raise error

    monkeypatch.setattr(fq, "_calls", None)
    monkeypatch.setattr(B, "build_calls", fail)
    with pytest.warns(RuntimeWarning, match="call module"):
        assert fq._load_calls() is False
    assert fq._load_calls() is False                # said once

    class Cuda:
        is_cuda = True
    assert fq._fp4_quick("product", "matmul_fp4", Cuda(), "mxfp4", (0,), ()) is None
    with pytest.raises(ValueError, match="CUDA tensor"):
        fq.scaled_fp4_blockwise(torch.zeros(2, 32))
