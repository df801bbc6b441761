"""The native part of the Python binding: who needs it, and when it is built again (no GPU needed)."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "w8a8_post_quantization_calib_b200"


def _package_without_binding(tmp_path):
    d = tmp_path / PKG
    d.mkdir()
    for name in ("__init__.py", "layer.py", "libsq.so"):
        os.symlink(os.path.join(ROOT, PKG, name), d / name)
    return d


def _run(tmp_path, code):
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env={**os.environ, "PYTHONPATH": str(tmp_path)},
                          capture_output=True, text=True, timeout=300)


def test_other_calls_do_not_need_the_native_binding(tmp_path):
    _package_without_binding(tmp_path)
    r = _run(tmp_path, f"""
import {PKG} as sq, {PKG}.layer, torch
assert sq.__file__.startswith({str(tmp_path)!r})
assert sq.linear_workspace_size(16, 4096, 11008) == 0 and sq.fp4_scale_bytes(sq.MXFP4, 1, 1) == 512
try:
    sq.calib_absmax(torch.zeros(2, 8), torch.zeros(8))
except TypeError:
    pass
for _ in range(2):
    try:
        sq.dequant_fp4(None, None, sq.MXFP4, None)
    except ImportError as e:
        assert "build.py" in str(e)
    else:
        raise AssertionError("no error")
""")
    assert r.returncode == 0, r.stderr


def test_a_binding_of_another_torch_is_refused(tmp_path):
    d = _package_without_binding(tmp_path)
    (d / "_sqbind.py").write_text("TORCH_VERSION = '1.0.0'\n")
    r = _run(tmp_path, f"""
import {PKG} as sq
try:
    sq.dequant_fp4(None, None, sq.MXFP4, None)
except ImportError as e:
    assert "1.0.0" in str(e) and "build.py" in str(e)
else:
    raise AssertionError("no error")
""")
    assert r.returncode == 0, r.stderr


def test_a_prerelease_of_torch_has_its_release_number(tmp_path):
    d = _package_without_binding(tmp_path)
    (d / "_sqbind.py").write_text("TORCH_VERSION = '9.8.7'\ndef set_error(e): pass\ndef dequant_fp4(*a): pass\n")
    r = _run(tmp_path, f"""
import torch
import {PKG} as sq
torch.__version__ = "9.8.7a0+git1234567"
sq.dequant_fp4(None, None, sq.MXFP4, None)
""")
    assert r.returncode == 0, r.stderr


def test_the_binding_in_the_tree_loads():
    torch = pytest.importorskip("torch")
    sq = pytest.importorskip(PKG)
    with pytest.raises((TypeError, ValueError)):
        sq.dequant_fp4(None, None, sq.MXFP4, None)
    assert sq._bind.TORCH_VERSION == torch.__version__.split("+")[0]


def test_another_python_or_torch_makes_the_binding_stale(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("sq_build", os.path.join(ROOT, PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    so, stamp = tmp_path / "_sqbind.so", tmp_path / "versions"
    so.write_bytes(b"")
    assert b._bind_stale(str(so), str(stamp))                       # built by something that left no record
    stamp.write_text(b._bind_versions())
    assert not b._bind_stale(str(so), str(stamp))
    monkeypatch.setattr(b.importlib.metadata, "version", lambda name: "1.0.0")
    assert b._bind_stale(str(so), str(stamp))
    monkeypatch.undo()
    monkeypatch.setattr(b.sys, "version", "4.0")
    assert b._bind_stale(str(so), str(stamp))
    monkeypatch.undo()
    assert not b._bind_stale(str(so), str(stamp))
    os.utime(so, (0, 0))                                             # sources newer than the module
    assert b._bind_stale(str(so), str(stamp))


def test_tensors_of_the_wrong_kind_raise_what_the_other_calls_raise():
    """A tensor on the CPU is a TypeError, as in the INT8 and FP8 calls, and a ValueError."""
    torch = pytest.importorskip("torch")
    sq = pytest.importorskip(PKG)
    x, q, s = torch.zeros(4, 64), torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(64)
    kv, slots, i32 = torch.zeros(4, 2, 32), torch.arange(4), torch.zeros(1, 1, dtype=torch.int32)
    calls = [
        lambda: sq.smooth_quant_act(x, s, sq.ACT_STATIC, s, q),
        lambda: sq.smooth_quant_act_fp4(x, s, sq.MXFP4, q, q),
        lambda: sq.quant_weight_fp4(x, s, sq.MXFP4, q, q),
        lambda: sq.dequant_fp4(q, q, sq.MXFP4, x),
        lambda: sq.linear_fp4(q, q, q, q, sq.MXFP4, x),
        lambda: sq.smooth_scales_nvfp4(s, s, 0.5, s),
        lambda: sq.kv_cache_write(kv, kv, slots, sq.KV_INT8, q, s, q, s),
        lambda: sq.kv_cache_read(sq.KV_INT8, q, s, q, s, i32, i32[0], kv, kv),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
        if n:
            with pytest.raises(ValueError, match="CUDA tensor"):
                call()
