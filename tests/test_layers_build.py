"""The torch binding is rebuilt for, and not loaded into, a torch other than the
one it was built against."""
import pytest
import torch

from sparse_communication_sharded_gb300 import build as B
from sparse_communication_sharded_gb300 import layers as L


@pytest.fixture(autouse=True)
def built():
    B.build()


def test_a_fresh_build_fits():
    assert B.binding_mismatch() is None
    assert not B.is_stale()


def test_another_torch(monkeypatch):
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert "torch 1.0.0" in B.binding_mismatch()
    assert B.is_stale()
    monkeypatch.setattr(L, "_binding", None)
    with pytest.raises(ImportError, match="built for"):
        L._lib()


def test_a_binding_without_a_record(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "BINDING_FOR", str(tmp_path / "none"))
    assert "unknown" in B.binding_mismatch()
    assert B.is_stale()
