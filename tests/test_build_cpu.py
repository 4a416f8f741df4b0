"""What each part of the build needs: libwq.so hipcc alone, the Python binding's compiled
part torch as well."""
import os
import shutil
import subprocess
import sys

import pytest

from w4a16_bit_matmul_amd import _build


def script_of(tmp_path):
    """A copy of the build script beside nothing, with a compiler that writes its name into its output."""
    cc = tmp_path / "cc"
    cc.write_text("#!/bin/sh\nwhile [ $# -gt 0 ]; do [ \"$1\" = -o ] && echo built > \"$2\"; shift; done\n")
    cc.chmod(0o755)
    shutil.copy(_build.__file__, tmp_path / "_build.py")
    return tmp_path / "_build.py", dict(os.environ, HIPCC=str(cc))


def test_the_library_is_built_without_torch(tmp_path):
    script, env = script_of(tmp_path)
    r = subprocess.run([sys.executable, "-S", str(script)], env=env, capture_output=True, text=True)  # (-S: no site packages)
    assert r.returncode == 0, r.stderr
    assert (tmp_path / "libwq.so").exists() and not (tmp_path / "_calls.so").exists()
    assert "binding" in r.stderr


def test_a_binding_that_fails_leaves_the_library(tmp_path):
    script, env = script_of(tmp_path)
    r = subprocess.run([sys.executable, str(script)], env=env, capture_output=True, text=True)  # (its source is missing)
    assert r.returncode != 0 and "wq_calls.cpp" in r.stderr
    assert (tmp_path / "libwq.so").exists() and not (tmp_path / "_calls.so").exists()


@pytest.mark.skipif(not os.path.exists(_build.OUT), reason="not built")
def test_the_library_does_not_need_the_binding():
    code = ("import sys; sys.modules['w4a16_bit_matmul_amd._calls'] = None\n"
            "import w4a16_bit_matmul_amd as wq\n"
            "assert wq.wq_version() and wq.wq_kv_attention_workspace_bytes(4, 8, 2, 128, 4, 16, 65536) > 0\n"
            "import torch\n"
            "try: wq.wq_verify_drafts(torch.zeros(1, 4), torch.zeros(1), torch.zeros(1))\n"
            "except ImportError as e: assert 'build it first' in str(e)\n"
            "else: raise AssertionError('not refused')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(_build.__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
