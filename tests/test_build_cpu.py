"""CPU checks of the in-tree build: the C library needs nvcc alone.  The binding's
torch calls are built beside it, and where that fails the library is there all
the same.  (The compilers are replaced; nothing is built.)"""

import os

import pytest

build = pytest.importorskip("block_sparse_attention_masked_gb300.build")


@pytest.fixture
def steps(monkeypatch, tmp_path):
    done = []
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "_compile", lambda src, verbose, debug=False: src + (".debug" if debug else ""))
    monkeypatch.setattr(build, "_link", lambda objs, lib: done.append((os.path.basename(lib), list(objs))))
    return done


def _libraries():
    return [(os.path.basename(build.LIB), build.SOURCES),
            (os.path.basename(build.DEBUG_LIB), [s + ".debug" for s in build.SOURCES])]


def test_library_is_linked_without_torch(steps, monkeypatch, capsys):
    def no_torch(verbose=False):
        raise ModuleNotFoundError("No module named 'torch'", name="torch")

    monkeypatch.setattr(build, "_build_torch_calls", no_torch)
    assert build.build() == build.LIB
    assert steps == _libraries()
    assert "torch" in capsys.readouterr().err


def test_failure_of_the_torch_calls_is_its_own(steps, monkeypatch):
    def no_headers(verbose=False):
        raise RuntimeError("the compiler failed on torch_calls.cpp")

    monkeypatch.setattr(build, "_build_torch_calls", no_headers)
    with pytest.raises(RuntimeError, match="torch_calls.cpp"):
        build.build()
    assert steps == _libraries()  # (linked all the same)


def test_everything_is_built(steps, monkeypatch):
    monkeypatch.setattr(build, "_build_torch_calls", lambda verbose=False: steps.append("calls"))
    assert build.build(debug=False) == build.LIB
    assert "calls" in steps and [s for s in steps if s != "calls"] == _libraries()[:1]
