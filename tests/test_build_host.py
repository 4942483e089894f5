"""What a build compiles again: sources and headers that changed, and files made with other compiler flags. The compiler is
a stand-in that copies its command line into its output."""
import os

import pytest

from bit_diffusion_transformer_svdquant_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Two sources that share a header, and the commands that ran."""
    csrc, commands = tmp_path / "csrc", []
    csrc.mkdir()
    (csrc / "shared.cuh").write_text("// shared\n")
    for name in ("a.cu", "b.cu"):
        (csrc / name).write_text('#include "shared.cuh"\n')
    sources = [str(csrc / name) for name in ("a.cu", "b.cu")]
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "SOURCES", sources)
    monkeypatch.setattr(build, "DEPS", [*sources, str(csrc / "shared.cuh")])
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")

    def run(cmd, verbose):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))

    monkeypatch.setattr(build, "_run", run)

    def made(**kw):
        """The files that a build writes, by name."""
        commands.clear()
        assert build.build(**kw) == build.LIB_PATH and os.path.exists(build.LIB_PATH)
        return sorted(os.path.basename(c[c.index("-o") + 1])[:-len(".tmp")] for c in commands)

    return made, csrc


ALL = ["a.o", "b.o", "lib.so"]


def _touch(path, seconds):
    t = os.path.getmtime(path) + seconds
    os.utime(path, (t, t))


def test_what_changed_is_made_again(tree):
    made, csrc = tree
    assert made() == ALL
    assert made() == []
    _touch(csrc / "b.cu", 5)
    assert made() == ["b.o", "lib.so"]
    _touch(csrc / "b.cu", -5)
    _touch(csrc / "shared.cuh", 5)
    assert made() == ALL
    _touch(csrc / "shared.cuh", -5)
    assert made(force=True) == ALL


def test_other_flags_make_everything_again(tree):
    """A library never holds objects of two sets of flags."""
    made, csrc = tree
    made()
    assert made(extra=["-G"]) == ALL
    assert made(extra=["-G"]) == []
    _touch(csrc / "a.cu", 5)
    assert made() == ALL                                    # b.o was made with -G
    _touch(csrc / "a.cu", -5)
    assert made() == []


def test_changed_default_flags(tree, monkeypatch):
    made, _ = tree
    made()
    monkeypatch.setattr(build, "NVCC_FLAGS", [*build.NVCC_FLAGS, "-DX"])
    assert made() == ALL and made() == []


def test_a_file_without_its_record_is_made_again(tree):
    made, csrc = tree
    made()
    os.remove(csrc / "a.o.flags")
    os.remove(build.LIB_PATH + ".flags")
    assert made() == ["a.o", "lib.so"]
