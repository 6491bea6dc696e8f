"""The binding without its compiled call layer, on the CPU: the package imports, and the named checks make the calls."""

import os
import shutil
import subprocess
import sys

import pytest

import block_sparse_attention_attngate_b200 as S
from block_sparse_attention_attngate_b200 import seer

PKG = os.path.dirname(S.__file__)
USE = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import torch
    import {name} as S
    S.version()
said = [str(w.message) for w in seen if "call layer" in str(w.message)]
assert len(said) == 1 and issubclass([w.category for w in seen if "call layer" in str(w.message)][0], RuntimeWarning), said
i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
calls = [lambda: S.page_plan(16, i32(4), i32(4), i32(4, 8), i32(64), i32(1), i32(5), i32(32), i32(32)),
         lambda: S.page_release(16, i32(4), i32(4), i32(4, 8), i32(64), i32(1)),
         lambda: S.qk_norm_rope(torch.zeros(2, 4, 64), None, i32(2), torch.zeros(2, 4, 64)),
         lambda: S.qk_norm_rope_backward(torch.zeros(2, 4, 64), None, torch.zeros(2, 4, 64), None, i32(2), torch.zeros(2, 4, 64), None),
         lambda: S.dense_decode(torch.zeros(2, 4, 64).bfloat16(),
                                *[S.KVCache(S.KVDesc(), (torch.zeros(2, 4, 8, 64).bfloat16(),))] * 2, i32(2),
                                torch.zeros(2, 4, 64).bfloat16(), torch.zeros(16, dtype=torch.uint8))]
for call in calls:
    try:
        call()
    except TypeError as e:
        assert "CUDA tensor" in str(e), e
    else:
        raise AssertionError("not refused")
print("used")
"""


@pytest.mark.parametrize("broken", [False, True])
def test_package_without_the_call_layer(tmp_path, broken):
    """The layer's file is not there, or is not a library that loads."""
    name = os.path.basename(PKG)
    os.makedirs(tmp_path / name)
    for f in ("__init__.py", "build.py", "seer.py"):
        shutil.copy(os.path.join(PKG, f), tmp_path / name / f)
    os.symlink(os.path.join(PKG, "libseer.so"), tmp_path / name / "libseer.so")
    if broken:
        for f in os.listdir(PKG):
            if f.startswith("_seer_call") and f.endswith(".so"):
                (tmp_path / name / f).write_bytes(b"not a library")
    r = subprocess.run([sys.executable, "-c", USE.format(name=name)], cwd=tmp_path, capture_output=True, text=True,
                       env={k: v for k, v in os.environ.items() if k != "SEER_LIBRARY"})
    assert r.returncode == 0 and r.stdout.strip() == "used", r.stderr


def test_the_call_layer_is_loaded_here():
    assert set(seer._call.entries()) == {"seer_page_plan", "seer_page_release", "seer_qk_norm_rope", "seer_qk_norm_rope_backward",
                                         "seer_dense_decode"}


# ---------------------------------------------------------------- building it
from block_sparse_attention_attngate_b200 import build as B   # noqa: E402


def test_a_layer_of_another_torch_is_not_used(monkeypatch):
    """The layer is compiled against one Python and one torch; both are in its name, so another's is neither taken for
    up to date nor loaded."""
    import torch
    here = B.call_layer_path()
    assert os.path.exists(here) and seer._call.__spec__.origin == here
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert B.call_layer_path() != here
    with pytest.warns(RuntimeWarning, match="call layer"):
        assert isinstance(seer._load_call_layer(), seer._NoCallLayer)
    monkeypatch.undo()
    monkeypatch.setattr(sys.implementation, "cache_tag", "other-11")
    assert B.call_layer_path() != here


def test_the_library_is_built_without_the_call_layer(monkeypatch):
    """No compiler for the layer, or no torch: the library is there all the same, and a warning tells of the layer."""
    def fails(*a, **k):
        raise RuntimeError("no g++")
    monkeypatch.setattr(B, "build_call_layer", fails)
    with pytest.warns(RuntimeWarning, match="no g[+][+]"):
        assert B.build() == B.LIB and os.path.exists(B.LIB)
