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


def test_native_calls_compiled_against_another_torch_are_built_again(monkeypatch, place):
    import torch
    ran, at = place
    made = B._made_for()
    monkeypatch.setattr(subprocess, "run", lambda cmd, check: (
        ran.append(cmd), open(cmd[cmd.index("-o") + 1], "wb").write(made.encode())))
    B.build_fastcall()
    assert len(ran) == 1 and B.fastcall_fits()
    B.build_fastcall()
    assert len(ran) == 1                                  # up to date
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not B.fastcall_fits()
    made = B._made_for()
    B.build_fastcall()
    assert len(ran) == 2 and "0.0.1" in " ".join(ran[-1]) and B.fastcall_fits()


@pytest.mark.parametrize("content", [None, b"of another torch"])
def test_native_calls_that_do_not_fit_are_not_loaded(monkeypatch, tmp_path, content):
    from sparse_attention_aware_b200 import api
    monkeypatch.setattr(B, "FAST", str(tmp_path / "_fastcall.so"))
    if content is not None:
        (tmp_path / "_fastcall.so").write_bytes(content)
    with pytest.warns(RuntimeWarning, match="native calls"):
        assert api._load_fast() is None


def test_the_built_native_calls_fit():
    B.build()
    assert B.fastcall_fits()


def test_a_forced_build_that_fails_leaves_native_calls_that_fit(monkeypatch, place):
    ran, at = place
    (at / "_fastcall.so").write_bytes(B._made_for().encode())

    def fail(force=False):
        raise FileNotFoundError("g++")

    monkeypatch.setattr(B, "build_fastcall", fail)
    with pytest.warns(RuntimeWarning, match="native calls"):
        B.build(force=True)
    assert B.fastcall_fits()
