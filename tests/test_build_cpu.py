"""What a build leaves behind where a part of its tools is missing (no GPU, no compiler run)."""
import os
import stat
import subprocess
import sys

import pytest

from gated_delta_rule_93_b200 import build as B

FAKE_NVCC = """#!/bin/sh
# writes the file that -o names
while [ $# -gt 0 ]; do
  if [ "$1" = "-o" ]; then echo built > "$2"; fi
  shift
done
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The package's sources, with a stand-in for nvcc and all outputs elsewhere."""
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(FAKE_NVCC)
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(B, "NVCC", str(nvcc))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libgdr.so"))
    monkeypatch.setattr(B, "NATIVE", str(tmp_path / "front.so"))
    return tmp_path


@pytest.mark.parametrize("cxx", ["/nowhere/g++", "false"])
def test_the_library_is_built_without_the_front_end(tree, monkeypatch, cxx):
    """No g++, or one that fails: the C library, which needs neither, is there all the same,
    and no front end of an older source is left to be loaded."""
    monkeypatch.setattr(B, "CXX", cxx)
    (tree / "front.so").write_text("of an older source")
    with pytest.warns(RuntimeWarning, match="front end"):
        assert B.build(force=True) == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.NATIVE)


def test_a_failing_kernel_source_is_an_error(tree, monkeypatch):
    monkeypatch.setattr(B, "NVCC", "false")
    monkeypatch.setattr(B, "CXX", "false")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        B.build(force=True)
    assert not os.path.exists(B.LIB)


OTHER = """
import sys
import torch
{change}
from gated_delta_rule_93_b200 import binding
try:
    binding.native()
except RuntimeError as e:
    sys.exit(0 if "missing" in str(e) else 2)
sys.exit(1)  # loaded
"""


@pytest.mark.parametrize("change,loads", [
    ("", True), ("torch.__version__ = '2.99.0'", False),
    ("torch.version.git_version = '0123456789abcdef'", False),
    ("import sysconfig; sysconfig.get_config_vars()['EXT_SUFFIX'] = '.cpython-399-other.so'", False)])
def test_a_front_end_of_another_torch_is_not_loaded(change, loads):
    """The front end uses torch's C++ interfaces: what was compiled against another torch or
    Python is not this one's, whatever its file times say."""
    B.build()
    r = subprocess.run([sys.executable, "-c", OTHER.format(change=change)], cwd=B.ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == (1 if loads else 0), r.stderr
