"""The binding's extension module: needed by its own entry points alone, and
only good for the torch it was built with (CPU)."""
import os

import pytest
import torch

import int4_weight_mixed_gb300 as w4
from int4_weight_mixed_gb300 import _build_lib


@pytest.fixture
def unloaded(monkeypatch):
    w4.build()
    monkeypatch.setattr(w4, "_lib", None)
    monkeypatch.setattr(w4, "_host", None)


CALLS = [lambda x: w4.rmsnorm(x), lambda x: w4.rmsnorm_quant(x),
         lambda x: w4.gemm(x, x, w4.INT4, 64, act=w4.ACT_SILU),
         lambda x: w4.gemm_dynamic(x, x, w4.INT4, 64, residual=x)]


def test_plain_calls_do_not_need_the_module(unloaded, monkeypatch, tmp_path):
    monkeypatch.setattr(_build_lib, "HOST", str(tmp_path / "w4_host.so"))
    assert w4.layout_version() == 1 and w4.num_schedules() > 0
    x = torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA tensor"):  # its arguments are looked at
        w4.gemm(x, x, w4.INT4, 64)
    for call in CALLS:
        with pytest.raises(RuntimeError, match="w4_host.so is not built"):
            call(x)


def test_a_module_of_another_torch_is_not_loaded(unloaded, monkeypatch):
    assert not _build_lib.host_lacks()
    monkeypatch.setattr(torch, "__version__", "1.0.other")
    x = torch.zeros(2, 64, dtype=torch.float16)
    for call in CALLS:
        with pytest.raises(RuntimeError, match="w4_host.so was built for torch"):
            call(x)


def test_build_makes_the_module_again_for_another_torch(monkeypatch, tmp_path):
    """Newer than its sources, but of another torch: it alone is built again."""
    w4.build()
    monkeypatch.setattr(_build_lib, "HOST_STAMP", str(tmp_path / "w4_host.for"))
    (tmp_path / "w4_host.for").write_text("torch 1.0.other")
    ran = []
    monkeypatch.setattr(_build_lib, "_run", lambda jobs, verbose: ran.extend(n for n, _ in jobs))
    monkeypatch.setattr(_build_lib.subprocess, "check_call", lambda cmd: ran.append("link"))
    monkeypatch.setattr(_build_lib.os, "replace", lambda a, b: ran.append(os.path.basename(b)))
    _build_lib.build()
    assert ran == ["w4_host.cpp", "link", "w4_host.so"]
    assert (tmp_path / "w4_host.for").read_text() == _build_lib._host_key()
    ran.clear()
    _build_lib.build()
    assert not ran
