"""What the build compiles anew, and with which flags, with a compiler that writes its command into its output."""
import os
import stat
import sys

import pytest

from block_sparse_attention_moments_b200 import _build

COMPILER = """#!{python}
import os, sys
out = sys.argv[sys.argv.index("-o") + 1]
inputs = [a for a in sys.argv[1:] if a.endswith(".o") and a != out]
with open(out, "w") as f:
    f.write("partial")
    if os.environ.get("COMPILER_STOPS") and os.environ["COMPILER_STOPS"] in " ".join(sys.argv):
        f.flush()
        os._exit(1)
    f.seek(0)
    f.truncate()
    f.write(" ".join(a for a in sys.argv[1:] if a.startswith("-") and a != "-o") + "\\n")
    f.writelines(open(i).read() for i in inputs)
with open({log!r}, "a") as f:
    f.write(os.path.basename(sys.argv[-1]) + "\\n")
"""


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build(...) returns the library's text, the flags of every unit, and the number of compiler runs."""
    log, nvcc = str(tmp_path / "log"), tmp_path / "nvcc"
    nvcc.write_text(COMPILER.format(python=sys.executable, log=log))
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(_build, "nvcc_path", lambda: str(nvcc))
    monkeypatch.setattr(_build, "OBJ", str(tmp_path / "obj"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "PROFILE_LIB", str(tmp_path / "profile.so"))

    def run(**kw):
        open(log, "w").close()
        with open(_build.build(**kw)) as f:
            text = f.read()
        with open(log) as f:
            return text, len(f.read().splitlines())
    return run


UNITS = len(_build.UNITS)


def test_nothing_is_done_twice(build):
    assert build()[1] == UNITS + 1
    assert build()[1] == 0
    assert build(force=True)[1] == UNITS + 1


def test_flags_of_one_build_do_not_stay(build):
    plain, _ = build()
    marked, runs = build(extra_flags=["-DMARK"])
    assert runs == UNITS + 1 and marked.count("-DMARK") >= UNITS
    again, runs = build()
    assert runs == UNITS + 1 and again == plain
    build(force=True, extra_flags=["-DMARK"])
    assert build()[0] == plain


def test_changed_flags_and_defines_are_compiled(build, monkeypatch):
    build()
    name, source, defines = _build.UNITS[-1]
    monkeypatch.setattr(_build, "UNITS", _build.UNITS[:-1] + [(name, source, (*defines, "-DNEW"))])
    text, runs = build()
    assert runs == 2 and text.count("-DNEW") == 1
    monkeypatch.setattr(_build, "NVCC_FLAGS", [*_build.NVCC_FLAGS, "-DALL"])
    text, runs = build()
    assert runs == UNITS + 1 and text.count("-DALL") >= UNITS


def test_profile_shares_what_is_the_same(build):
    build(force=True)
    text, runs = build(force=True, profile=True)
    assert runs == 2 and text.count("-DSOL_ATTN_PROFILE") == 1
    text, runs = build(force=True, profile=True, extra_flags=["-DMARK"])
    assert runs == UNITS + 1 and text.count("-DMARK") >= UNITS


def test_a_stopped_compiler_leaves_nothing_that_looks_done(build, monkeypatch):
    plain, _ = build()
    for what in (os.path.join("csrc", "rope_launch.cu"), "-shared"):
        monkeypatch.setenv("COMPILER_STOPS", what)
        with pytest.raises(RuntimeError):
            build(force=True)
        monkeypatch.delenv("COMPILER_STOPS")
        assert build()[0] == plain
