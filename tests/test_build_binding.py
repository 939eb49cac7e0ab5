"""The row operators' compiled binding beside another torch than the one it was
built against: it is rebuilt by build(), and refused where it was not."""
import os

import pytest
import torch

import blockwise_fp8_linear_fp8bq_b200 as fp
from blockwise_fp8_linear_fp8bq_b200 import build


def test_another_torch_needs_another_binding(monkeypatch, tmp_path):
    build.build()
    assert not build.needs_binding()
    monkeypatch.setattr(build, "torch_version", lambda: "0.0.1+other")
    assert build.needs_binding() and build.needs_build()
    monkeypatch.undo()
    monkeypatch.setattr(build, "BINDING_TORCH", os.path.join(tmp_path, "none"))
    assert build.needs_binding()  # built before its torch was recorded


def test_a_binding_of_another_torch_is_refused(monkeypatch):
    build.build()
    assert fp._row_ops().torch_version == torch.__version__
    monkeypatch.setattr(fp, "_rows", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    with pytest.raises(ImportError, match="0.0.1"):
        fp._row_ops()
