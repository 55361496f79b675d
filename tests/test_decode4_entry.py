"""The native module of the 4-bit operators' calls (_decode4.so): it is rebuilt,
and not used, where it was compiled against another torch or Python; and where
it is missing those operators raise and the rest of the package works."""

import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "activation_sparse_swiglu_b200")


@pytest.fixture()
def builder():
    spec = importlib.util.spec_from_file_location("_prox_build_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def python(code, path=ROOT):
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=path)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def test_entry_of_another_torch_is_stale(builder, monkeypatch):
    import torch
    assert builder.entry_tag() == f"torch {torch.__version__}, {sys.implementation.cache_tag}"
    assert builder.entry_up_to_date()
    monkeypatch.setattr(builder, "entry_tag", lambda: "torch 9.9.0, cpython-399")
    assert not builder.entry_up_to_date()


def test_entry_of_another_torch_is_refused():
    out = python("import torch; torch.__version__ = '9.9.0'\n"
                 "try:\n"
                 "    import activation_sparse_swiglu_b200 as p; p.plan_pages(*[None] * 7)\n"
                 "except ImportError as e:\n"
                 "    print('refused:', e)\n")
    assert "refused:" in out and "built for torch" in out and "9.9.0" in out


def test_package_without_the_entry(tmp_path):
    pkg = tmp_path / "activation_sparse_swiglu_b200"
    pkg.mkdir()
    for name in os.listdir(PKG):
        if name.endswith(".py") or name == "libprox.so":
            os.symlink(os.path.join(PKG, name), pkg / name)
    out = python("import activation_sparse_swiglu_b200 as p, activation_sparse_swiglu_b200.stack\n"
                 "assert p.__file__.startswith(%r) and p.Layer and 'sm_100a' in p.version()\n"
                 "for call in (lambda: p.plan_pages(*[None] * 7), p.Linear4, lambda: p.KVCache4(*[None] * 4)):\n"
                 "    try:\n"
                 "        call()\n"
                 "    except ImportError as e:\n"
                 "        print('refused:', e)\n" % str(tmp_path), tmp_path)
    assert out.count("refused:") == 3 and out.count("_decode4.so cannot be loaded") == 3
