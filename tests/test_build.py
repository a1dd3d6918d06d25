"""What the build script makes, and what the package does without its extension (CPU)."""
import importlib.util
import os
import subprocess
import sys

import pytest

import kv_cache_vector_rope_b200 as tq

PKG = os.path.dirname(tq.__file__)


def _script():
    spec = importlib.util.spec_from_file_location("tq_build", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    return b


@pytest.fixture
def script(tmp_path, monkeypatch):
    """The build script over empty files in place of its libraries, its compilers' commands noted instead of run."""
    b = _script()
    for name in ("LIB", "BINDING", "BINDING_FOR"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    b.ran = []

    def run(cmd, check):
        b.ran.append(os.path.basename(cmd[0]))
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(b.subprocess, "run", run)
    return b


def test_one_call_builds_both_libraries(script):
    assert script.build() == script.LIB and script.ran == ["nvcc", "g++"]
    assert os.path.exists(script.LIB) and os.path.exists(script.BINDING)
    script.build()
    assert script.ran == ["nvcc", "g++"]                          # nothing is stale
    script.build(force=True)
    assert script.ran == ["nvcc", "g++"] * 2


def test_the_extension_is_stale_for_another_torch(script):
    script.build()
    script.ran.clear()
    with open(script.BINDING_FOR, "w") as f:
        f.write("python cpython-39-x86_64-linux-gnu, torch 1.0\n")
    script.build()
    assert script.ran == ["g++"]
    os.remove(script.BINDING_FOR)
    script.build_binding()
    assert script.ran == ["g++"] * 2
    script.build_binding()
    assert script.ran == ["g++"] * 2


def test_without_the_extension_only_its_calls_are_refused(tmp_path):
    pkg = tmp_path / "kv_cache_vector_rope_b200"
    pkg.mkdir()
    for name in ("__init__.py", "build.py", "libtq.so"):
        os.symlink(os.path.join(PKG, name), pkg / name)
    code = """
import kv_cache_vector_rope_b200 as tq
import torch
c, t, mse = tq.tq_make_codebook(64, 3)
assert c.shape[0] == 8 and tq.tq_cache8_bytes(64, 2, 16, 4) > 0
cache = tq.alloc_cache8(4, 2, 16, 64, device="cpu")
x, i = torch.zeros(3, 2, 64), torch.zeros(2, dtype=torch.int32)
for call in (lambda: tq.tq_cache8_write(cache, x, x, i, i), lambda: tq.tq_qk_norm_rope(x, None, x, None),
             lambda: tq.tq_cache8_attention(cache, x, i, x, x)):
    try:
        call()
    except ImportError as e:
        assert "_tq_torch.so" in str(e) and e.__cause__ is not None
    else:
        raise AssertionError("not refused")
print("fine")
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                         env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert out.returncode == 0 and out.stdout.strip() == "fine", out.stderr
