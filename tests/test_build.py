"""Building where the binding's native calls cannot be built (CPU)."""
import subprocess

import pytest

from sparse_attention_aware_b200 import build as B


@pytest.fixture
def place(monkeypatch, tmp_path):
    """A build that runs no compiler and leaves the tree's libraries alone."""
    ran = []

    def run(cmd, check):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libsa.so"))
    monkeypatch.setattr(B, "FAST", str(tmp_path / "_fastcall.so"))
    return ran, tmp_path


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), subprocess.CalledProcessError(1, "g++"),
                                   ImportError("torch")])
def test_the_library_is_built_without_the_native_calls(monkeypatch, place, error):
    ran, at = place
    (at / "_fastcall.so").write_bytes(b"of an earlier header")

    def fail(force=False):
        raise error

    monkeypatch.setattr(B, "build_fastcall", fail)
    with pytest.warns(RuntimeWarning, match="native calls"):
        assert B.build(force=True) == str(at / "libsa.so")
    assert len(ran) == 1 and (at / "libsa.so").exists() and not (at / "_fastcall.so").exists()


def test_a_library_that_does_not_build_is_an_error(monkeypatch, place):
    def run(cmd, check):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(subprocess, "run", run)
    with pytest.raises(subprocess.CalledProcessError):
        B.build(force=True)
