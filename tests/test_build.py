"""The C-ABI library is built without torch, and before the compiled calls."""
import os
import subprocess
import sys

import pytest

from blockwise_fp8_linear_b200 import build as fbuild


def test_library_without_torch():
    # (up to date, so that nothing is compiled)
    lib = fbuild.build()
    r = subprocess.run([sys.executable, "-c", "import sys; sys.modules['torch'] = None\n"
                        "from blockwise_fp8_linear_b200 import build\nprint(build.build())"],
                       cwd=fbuild.ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == lib


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """The compilers' command lines, which only make their output files."""
    seen = []

    def run(cmd, check=False, **_):
        seen.append(os.path.basename(cmd[0]))
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(fbuild.subprocess, "run", run)
    monkeypatch.setattr(fbuild, "LIB", str(tmp_path / "libfp8bw.so"))
    monkeypatch.setattr(fbuild, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(fbuild, "BUILD_DIR", str(tmp_path / "objects"))
    return seen


def test_library_comes_first(commands):
    assert fbuild.build(force=True) == fbuild.LIB
    assert commands == ["nvcc"] * (len(fbuild.sources()) + 1) + ["g++"]
    assert os.path.exists(fbuild.LIB) and os.path.exists(fbuild.CALLS)
    fbuild.build()                       # both are newer than their sources
    assert commands.count("g++") == 1


def test_library_is_there_when_the_calls_fail(commands, monkeypatch):
    run = fbuild.subprocess.run

    def no_gxx(cmd, **kw):
        if os.path.basename(cmd[0]) == "g++":
            raise subprocess.CalledProcessError(1, cmd)
        run(cmd, **kw)

    monkeypatch.setattr(fbuild.subprocess, "run", no_gxx)
    with pytest.raises(subprocess.CalledProcessError):
        fbuild.build(force=True)
    assert os.path.exists(fbuild.LIB) and not os.path.exists(fbuild.CALLS)
