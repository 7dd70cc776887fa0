"""Where the package can be built and imported: the 8-bit cache's module _q8 is
asked of nobody who has no such cache."""
import os
import shutil
import subprocess
import sys

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
