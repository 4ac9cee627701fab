"""The library loads without the cache operators' marshalling module, which is
built for one torch and one interpreter (CPU)."""
import os
import subprocess
import sys

import pytest
import torch

import varlen_gqa_split_b200 as vg
from varlen_gqa_split_b200 import _binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_without_the_module():
    build.build()
    code = """
from varlen_gqa_split_b200 import _binding
_binding.MARSHAL_PATH += ".missing"
import varlen_gqa_split_b200 as vg
assert vg.lib() and vg.strerror(0) == "success"
rope = vg.Rope(8, *vg.rope_table(4))
import torch
_binding._raw_device = lambda: 0
_binding._raw_stream = lambda d: 0
try:
    rope.apply(torch.zeros(1, 1, 8), torch.zeros(1, 1, dtype=torch.int32))
except RuntimeError as e:
    assert "not built for this torch" in str(e), e
else:
    raise SystemExit("loaded")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=120)
    assert r.returncode == 0, r.stderr[-1500:]


def test_module_belongs_to_its_torch():
    build.build()
    assert os.path.exists(_binding.MARSHAL_PATH) and build.marshal_up_to_date()
    assert torch.__version__ in os.path.basename(_binding.MARSHAL_PATH)
    assert sys.implementation.cache_tag in os.path.basename(_binding.MARSHAL_PATH)


def test_another_torch_has_no_module(monkeypatch):
    build.build()
    monkeypatch.setattr(_binding, "MARSHAL_PATH", _binding.MARSHAL_PATH.replace(torch.__version__, "0.0.0"))
    assert not build.marshal_up_to_date()
    monkeypatch.setattr(_binding, "_marshal", _binding._Unloaded())
    with pytest.raises(RuntimeError, match="not built for this torch"):
        _binding._marshal.rope_apply
    assert vg.lib() is not None
