"""The compiled module of the paged calls belongs to one torch: it is built anew for another, and
not used when it was built for another."""
import os
import sys
import types

import pytest
import torch

import compressed_sliding_window_b200 as hca
from compressed_sliding_window_b200 import build as B


def test_built_anew_for_another_torch(monkeypatch):
    B.build()
    assert B.calls_up_to_date()
    real = torch.__version__
    monkeypatch.setattr(torch, "__version__", real + ".other")
    assert not B.calls_up_to_date()
    monkeypatch.setattr(torch, "__version__", real)
    assert B.calls_up_to_date()


def test_stamp_and_sources(monkeypatch, tmp_path):
    B.build()
    stamp = tmp_path / "stamp"
    monkeypatch.setattr(B, "CALLS_STAMP", str(stamp))
    assert not B.calls_up_to_date()                    # no record of what it was built against
    stamp.write_text(B._built_against())
    assert B.calls_up_to_date()
    src = tmp_path / "paged_calls.cpp"
    src.write_text("")
    os.utime(src, (2e9, 2e9))
    monkeypatch.setattr(B, "CALLS_SRC", str(src))
    assert not B.calls_up_to_date()


def test_module_knows_its_torch(monkeypatch):
    B.build()
    monkeypatch.setattr(hca, "_CALLS", None)
    assert hca._calls().torch_version == torch.__version__
    name = hca.__name__ + "._paged_calls"
    for other in (types.SimpleNamespace(torch_version="1.0"), types.SimpleNamespace()):
        monkeypatch.setattr(hca, "_CALLS", None)
        monkeypatch.setitem(sys.modules, name, other)
        monkeypatch.setattr(hca, "_paged_calls", other, raising=False)
        with pytest.raises(RuntimeError, match="compressed_sliding_window_b200.build"):
            hca._calls()
        with pytest.raises(RuntimeError):
            hca.paged_append(*[None] * 11)
    monkeypatch.setattr(hca, "_CALLS", None)
    monkeypatch.setitem(sys.modules, name, None)       # cannot be imported
    monkeypatch.delattr(hca, "_paged_calls")
    with pytest.raises(RuntimeError, match="cannot be loaded"):
        hca._calls()
