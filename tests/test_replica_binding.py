"""The binding of the replica's operators, no GPU needed."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def v():
    pytest.importorskip("torch")
    from ring_allreduce_reduction_gb300 import build
    build.build()
    from ring_allreduce_reduction_gb300 import vrccl
    return vrccl


def test_imports_where_torch_has_no_cuda(v):
    """Host-side calls work with a torch that was built without CUDA (no raw stream to ask for)."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "from ring_allreduce_reduction_gb300 import vrccl as v\n"
            "assert v.vrcclLayerNormWorkspace(4, 64) > 0\n"
            "assert v.vrcclShardRange(100, 'float32', 4, 0)[1] > 0\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)


class NoLibrary:
    def __getattr__(self, name):
        def called(*args):
            raise AssertionError(f"{name} was called")
        return called


def test_tensors_that_do_not_fit_are_refused(v, monkeypatch):
    """Element types other than the call's, host tensors, vectors with gaps
    or too short, matrices of no known row stride: before the library is called."""
    import torch
    monkeypatch.setattr(v, "_lib", NoLibrary())
    x = torch.zeros(4, 64)
    norm = dict(x=4096, gamma=None, beta=None, y=8192, mean=None, rstd=None, rows=4, cols=64, dtype="float32", ptype="bfloat16")
    lin = dict(x=4096, w=8192, bias=None, residual=None, y=12288, z=None, rows=4, outs=8, ins=64, dtype="bfloat16")
    dis = dict(logits=4096, teacher=8192, index=12288, loss=16384, stats=None, rows=4, vocab=64, k=2, dtype="float32",
               teacher_dtype="float32", index_dtype="int64")
    for fn, base, change, why in (
            (v.vrcclLayerNormForward, norm, dict(x=x), "cpu"),
            (v.vrcclLayerNormForward, norm, dict(x=x.bfloat16()), "bfloat16"),
            (v.vrcclLayerNormForward, norm, dict(gamma=torch.zeros(64)), "float32"),
            (v.vrcclLayerNormForward, norm, dict(mean=torch.zeros(4).double()), "float64"),
            (v.vrcclLinearForward, lin, dict(w=torch.zeros(8, 64).half()), "float16"),
            (v.vrcclLinearForward, lin, dict(bias=torch.zeros(8).bfloat16()), "cpu"),
            (v.vrcclLinearForward, lin, dict(workspace=torch.zeros(16, dtype=torch.uint8)), "cpu"),
            (v.vrcclDistillForward, dis, dict(index=torch.zeros(4, 2, dtype=torch.int32)), "int32"),
            (v.vrcclDistillForward, dis, dict(stats=torch.zeros(4, 2)), "cpu"),
            (v.vrcclLayerNormForward, norm, dict(dtype="float8"), "float8")):
        with pytest.raises(ValueError, match=why):
            fn(**dict(base, **change))


def test_row_strides_of_tensors(v, monkeypatch):
    import torch
    f32 = torch.float32
    monkeypatch.setattr(v, "_misfit", lambda x, td: None)  # (host tensors stand in for the GPU's)
    wide = torch.zeros(6, 80)
    for x, rows, cols, ld in ((wide[:, :64], 6, 64, 80), (wide[:, 8:72], 6, 64, 80), (wide[::2, :64], 3, 64, 160),
                              (wide, 6, 80, 80), (wide.view(2, 3, 80), 6, 80, 80), (wide[:1, :64], 1, 64, 64)):
        assert v._mat(x, f32, rows, cols, None) == (x.data_ptr(), ld)
    assert v._mat(wide, f32, 3, 64, 160) == (wide.data_ptr(), 160)  # as the call says
    assert v._mat(4096, f32, 6, 64, None) == (4096, 64) and v._mat(None, f32, 6, 64, 70) == (None, 70)
    for x, rows, cols in ((wide.t(), 80, 6), (wide[:, ::2], 6, 40), (wide[:, :64], 3, 128), (wide, 7, 80),
                          (wide.view(2, 3, 80)[:, :, :64], 6, 64)):
        with pytest.raises(ValueError):
            v._mat(x, f32, rows, cols, None)
    with pytest.raises(ValueError):
        v._vec(wide[:, 0], f32)
    assert v._vec(None, f32) is None and v._vec(4096, f32) == 4096


def test_first_call_initialises_cuda(v, monkeypatch):
    """The first question for the current stream goes through torch's own
    initialisation, whose error is the caller's to see."""
    import torch

    def no_driver():
        raise RuntimeError("no driver")

    monkeypatch.setattr(torch.cuda, "current_device", no_driver)
    import importlib.util
    spec = importlib.util.spec_from_file_location(v.__name__ + "_again", v.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    for _ in range(2):
        with pytest.raises(RuntimeError, match="no driver"):
            again.vrcclLayerNormForward(4096, None, None, 8192, None, None, 4, 64, "float32", "float32")
