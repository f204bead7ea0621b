"""What build() builds: the library needs nvcc alone, the extension the torch that it was built for.  Compilers are
replaced here by functions that write the files."""
import os

import pytest


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """_build over an empty tree, and the list of what it makes."""
    from nvfp4_mixture_experts_expert_gb300 import _build as b
    made = []

    def write(name, tag):
        made.append(tag)
        (tmp_path / name).write_text(tag)
        return str(tmp_path / name)
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("1")
    (tmp_path / "a.cu").write_text("")
    (tmp_path / "calls.cpp").write_text("")
    for name, value in dict(BUILD=str(tmp_path), LIB=str(tmp_path / "lib.so"), EXT=str(tmp_path / "ext.so"),
                            EXT_SRC=str(tmp_path / "calls.cpp"), EXT_FOR=str(tmp_path / "ext.for"),
                            sources=lambda: [str(tmp_path / "a.cu")], torch_dir=lambda: str(torch),
                            _compile=lambda src, extra: (write("a.o", "object"), ""),
                            _link_lib=lambda objs: write("lib.so", "library"),
                            _compile_ext=lambda: write("calls.o", "extension object"),
                            _link_ext=lambda obj: write("ext.so", "extension")).items():
        monkeypatch.setattr(b, name, value)
    return b, made, torch


def test_both_once(tree):
    b, made, _ = tree
    assert not b.up_to_date()
    assert b.build() == b.LIB and sorted(made) == ["extension", "extension object", "library", "object"]
    made.clear()
    assert b.up_to_date() and b.build() == b.LIB and made == []


def test_the_library_alone_without_torch(tree, monkeypatch):
    b, made, _ = tree
    monkeypatch.setattr(b, "torch_dir", lambda: None)
    assert b.build() == b.LIB and made == ["object", "library"]
    assert b.up_to_date() and os.path.exists(b.LIB) and not os.path.exists(b.EXT)


def test_the_library_stands_where_the_extension_fails(tree, monkeypatch):
    b, made, _ = tree

    def fails():
        raise RuntimeError("no headers")
    monkeypatch.setattr(b, "_compile_ext", fails)
    with pytest.raises(RuntimeError, match="no headers"):
        b.build()
    assert os.path.exists(b.LIB) and not b.up_to_date()


def test_another_torch_rebuilds_the_extension_alone(tree):
    b, made, torch = tree
    b.build()
    made.clear()
    (torch / "version.py").write_text("2")
    assert not b.up_to_date()
    b.build()
    assert made == ["extension object", "extension"] and b.up_to_date()


def test_a_newer_kernel_rebuilds_the_library_alone(tree):
    b, made, _ = tree
    b.build()
    made.clear()
    later = os.path.getmtime(b.LIB) + 10
    os.utime(b.sources()[0], (later, later))
    b.build()
    assert made == ["object", "library"]


def test_torch_is_found_without_importing_it():
    pytest.importorskip("torch")
    import torch
    from nvfp4_mixture_experts_expert_gb300 import _build as b
    assert b.torch_dir() == os.path.dirname(torch.__file__)


def test_without_the_extension_the_older_calls_stay_and_its_own_fail_loudly(tmp_path):
    import shutil
    import subprocess
    import sys
    pytest.importorskip("torch")
    from nvfp4_mixture_experts_expert_gb300 import _build as b
    b.build()
    shutil.copytree(b.PKG, tmp_path / "nvfp4_mixture_experts_expert_gb300",
                    ignore=shutil.ignore_patterns("_torch_calls.so", "_build", "__pycache__", "csrc"))
    code = """
from nvfp4_mixture_experts_expert_gb300 import api
assert callable(api.MoEForward) and callable(api.quantize_moe_weights)
for call in (lambda: api.add_rms_norm_fp8(None, None, None), lambda: api.fp8_linear(None, None, None, None)):
    try:
        call()
    except ImportError as e:
        assert "_torch_calls" in str(e)
    else:
        raise SystemExit("no ImportError")
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env={**os.environ, "PYTHONPATH": str(tmp_path)},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["fine"], r.stdout + r.stderr
