"""What the host code asks the runtime for once: answers are kept, failures returned and asked about again."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kv_cache_compression_snapkv_gb300", "csrc")


def test_failures_are_not_kept(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "ask_once_host")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", f"-I{CSRC}",
                    os.path.join(ROOT, "tests", "ask_once_host.cpp"), "-o", exe], check=True)
    lines = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    assert lines[:6] == ["2 0 1", "2 0 2", "0 5 3", "0 5 3", "0 5 3", "2 0 entry"]


@pytest.mark.parametrize("name", ["quant.cu", "window_tc.cu"])
def test_no_answer_is_kept_by_its_initialiser(name):
    """A static that a lambda fills in keeps whatever the first call returned, an error's stand-in too."""
    src = open(os.path.join(CSRC, name)).read()
    assert not re.findall(r"\bstatic\b[^;()]*=\s*\[", src)
    assert "ask_once" in src
