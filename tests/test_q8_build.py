"""Where the package can be built and imported: the 8-bit cache's module _q8 is
asked of nobody who has no such cache."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

PACKAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decoder_only_transformer_sdpa_b200")


def in_copy(tmp_path, code):
    """Runs `code` where the package has its library but no _q8.so."""
    to = tmp_path / "decoder_only_transformer_sdpa_b200"
    to.mkdir()
    shutil.copy(os.path.join(PACKAGE, "__init__.py"), to)
    os.symlink(os.path.join(PACKAGE, "libattn.so"), to / "libattn.so")
    env = {k: v for k, v in os.environ.items() if k != "ATTN_LIBRARY"}
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env=env, capture_output=True, text=True, timeout=300)


def test_imports_without_the_cache_module(tmp_path):
    r = in_copy(tmp_path, "import decoder_only_transformer_sdpa_b200 as A\n"
                          "assert A.attn_version() == 1 and A.attn_bwd_workspace_bytes(1, 1, 1, 64) > 0\n"
                          "import sys; assert 'torch' not in sys.modules\n"
                          "try: A._binding()\n"
                          "except ImportError as e: assert '_q8.so is not built' in str(e) and 'build.py' in str(e)\n"
                          "else: raise SystemExit('no error')")
    assert r.returncode == 0, r.stderr


def build_module():
    """build.py as a module of its own, so that what a test changes in it is gone afterwards."""
    spec = importlib.util.spec_from_file_location("_attn_build_under_test", os.path.join(PACKAGE, "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def with_stub_compilers(m, tmp_path):
    """`m` building into tmp_path, with compilers that only write what they were asked for; returns what is built."""
    built = []
    m.HERE, m.BUILD, m.BUILD_DEBUG = str(tmp_path), str(tmp_path / "b"), str(tmp_path / "bd")
    m.LIB, m.LIB_DEBUG = str(tmp_path / "libattn.so"), str(tmp_path / "libattn_debug.so")

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        words = [x.split('"')[1] for x in cmd if x.startswith("-DATTN_BUILT_FOR")]
        open(out, "w").write("".join(f"built for {w}\0" for w in words))
        built.append(os.path.basename(out).split(".tmp")[0])
        return subprocess.CompletedProcess(cmd, 0, "", "")

    class Stub:
        CompletedProcess = subprocess.CompletedProcess
    Stub.run = Stub.check_call = staticmethod(run)
    m.subprocess = Stub
    return built


def test_the_library_is_built_without_torch(tmp_path, monkeypatch, capsys):
    m = build_module()
    built = with_stub_compilers(m, tmp_path)
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert m.build() == m.LIB and os.path.exists(m.LIB)
    assert "_q8.so" not in built and "torch" in capsys.readouterr().err


@pytest.mark.parametrize("debug", [False, True])
def test_the_library_is_there_when_the_module_fails(tmp_path, debug):
    """The library comes first: no compiler for the module, or no headers, leave it usable."""
    m = build_module()
    with_stub_compilers(m, tmp_path)
    m.CXX = "no-such-compiler"
    run = m.subprocess.run
    m.subprocess.run = staticmethod(lambda cmd, **kw: subprocess.CompletedProcess(cmd, 1, "", "no headers") if cmd[0] == m.CXX else run(cmd, **kw))
    with pytest.raises(RuntimeError, match="no headers"):
        m.build(debug=debug)
    assert os.path.exists(m.LIB_DEBUG if debug else m.LIB)


def test_the_module_is_built_anew_for_another_torch_or_python(tmp_path, monkeypatch):
    m = build_module()
    built = with_stub_compilers(m, tmp_path)
    version = m._torch_version(importlib.util.find_spec("torch").submodule_search_locations[0])
    count = lambda: built.count("_q8.so")
    for n in (1, 1):
        m.build_binding()
        assert count() == n
    monkeypatch.setattr(m, "_torch_version", lambda folder: version + "1")
    for n in (2, 2):
        m.build_binding()
        assert count() == n
    monkeypatch.setattr(sys.implementation, "cache_tag", "cpython-300")
    m.build_binding()
    assert count() == 3


def test_a_module_for_another_torch_is_not_used(monkeypatch):
    import torch

    import decoder_only_transformer_sdpa_b200 as A
    assert A._binding().built_for == f"torch {torch.__version__}, {sys.implementation.cache_tag}"
    monkeypatch.setattr(A, "_q8", None)
    monkeypatch.setattr(torch, "__version__", "0.0")
    with pytest.raises(ImportError, match="this is torch 0.0"):
        A._binding()
    assert A._q8 is None
