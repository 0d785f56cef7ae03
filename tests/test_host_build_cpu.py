"""The optional host path's build and loading: where it cannot be built nothing of an older build stays to be loaded, a
module of other sources or another torch is built anew and not used, and the library and its binding do without."""
import importlib.util
import os
import subprocess
import sys
import types

import pytest
import torch

import gated_deltanet_03_b200 as g

PKG = os.path.dirname(g.LIB_PATH)


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build script with its outputs in a folder of the test's own, and a compiler that is a stand-in."""
    spec = importlib.util.spec_from_file_location("_host_build", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.HOST_OUT, b.HOST_KEY = str(tmp_path / "_gdn_host.x.so"), str(tmp_path / "key")
    b.calls = []

    def run(cmd, **kw):
        b.calls.append(cmd)
        if b.fails:
            return types.SimpleNamespace(returncode=1, stderr="no such thing", stdout="")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stderr="", stdout="")

    b.fails = False
    monkeypatch.setattr(b.subprocess, "run", run)
    return b


def test_built_once_for_the_same_sources_and_torch(build):
    assert build.build_host() == build.HOST_OUT and len(build.calls) == 1
    assert build.build_host() == build.HOST_OUT and len(build.calls) == 1
    build.build_host(force=True)
    assert len(build.calls) == 2
    build._torch_version = lambda d: "1.0"
    build.build_host()
    assert len(build.calls) == 3 and "torch-1.0" in open(build.HOST_KEY).read()


def test_another_header_is_another_build(build, tmp_path):
    build.build_host()
    build.ROOT = str(tmp_path)
    os.makedirs(tmp_path / "include")
    (tmp_path / "include" / "gdn.h").write_text("other")
    build.build_host()
    assert len(build.calls) == 2


@pytest.mark.parametrize("why", ["compiler", "no compiler", "no torch"])
def test_nothing_old_stays_where_it_cannot_be_built(build, monkeypatch, capsys, why):
    assert build.build_host()
    old = os.path.join(os.path.dirname(build.HOST_OUT), "_gdn_host.so")
    open(old, "w").close()
    if why == "compiler":
        build.fails = True
    elif why == "no compiler":
        def gone(*a, **k):
            raise OSError("no g++")
        monkeypatch.setattr(build.subprocess, "run", gone)
    else:
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build_host(force=True) is None
    assert not os.path.exists(build.HOST_OUT) and not os.path.exists(old)
    assert "host path not built" in capsys.readouterr().err


def test_the_whole_build_passes_force_on(build, monkeypatch):
    monkeypatch.setattr(build, "build_library", lambda *a: "lib")
    assert build.build() == "lib" and build.build(force=True) == "lib"
    assert len(build.calls) == 2


@pytest.mark.parametrize("key", ["other", None])
def test_a_module_of_other_sources_is_not_used(monkeypatch, key):
    stale = types.ModuleType("stale")
    stale.bind = lambda *a: pytest.fail("bound")
    if key:
        stale.KEY = key
    monkeypatch.setitem(sys.modules, g.__name__ + "._gdn_host", stale)
    assert g._load_host() is None


def test_the_built_one_is_used():
    from gated_deltanet_03_b200.build import HOST_OUT, host_key
    assert os.path.exists(HOST_OUT) and g._host.KEY == host_key(torch.__version__)


def test_the_binding_does_without():
    """With no host path there, the package loads and its calls check their arguments all the same."""
    code = ("import sys; sys.modules['gated_deltanet_03_b200._gdn_host'] = None\n"
            "import torch, gated_deltanet_03_b200 as g\n"
            "assert g._host is None\n"
            "try:\n    g.fp8_quantize_act(torch.zeros(4, 64))\n"
            "except ValueError as e:\n    assert 'must be a CUDA tensor' in str(e)\n"
            "else:\n    raise SystemExit(3)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(PKG), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
