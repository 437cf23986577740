"""What the build needs for what (no GPU, nothing is compiled): the C library is free of torch, and
is built also where the Python binding's native half cannot be."""
import os

import pytest


@pytest.fixture
def built(tmp_path, monkeypatch):
    """The build module with its outputs in a folder of their own and a compiler that writes its
    output file only; the list of files built."""
    from blockwise_fp8_gemm_x128_amd import build
    hipcc = tmp_path / "hipcc"
    hipcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho built > "$2"\n')
    hipcc.chmod(0o755)
    monkeypatch.setattr(build, "HIPCC", str(hipcc))
    for name in ("LIB_PATH", "PROBE_PATH", "ARGS_PATH"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    return build


def there(b):
    return [os.path.exists(p) for p in (b.LIB_PATH, b.PROBE_PATH, b.ARGS_PATH)]


def test_whole_build(built, monkeypatch):
    monkeypatch.setattr(built, "_args", lambda verbose: open(built.ARGS_PATH, "w").close())
    assert built.build(verbose=False) == built.LIB_PATH
    assert there(built) == [True, True, True]


@pytest.mark.parametrize("error", [ImportError("no torch"), FileNotFoundError("no g++"),
                                   RuntimeError("no headers")])
def test_library_is_built_without_the_binding(built, monkeypatch, error):
    """build() says that the binding's half failed, with the library in place; build_library() does
    not ask for it."""
    def fail(verbose):
        raise error

    monkeypatch.setattr(built, "_args", fail)
    with pytest.raises(RuntimeError, match="native half.*libpuro.so is built"):
        built.build(verbose=False)
    assert there(built) == [True, True, False]
    os.remove(built.LIB_PATH)
    assert built.build_library(verbose=False) == built.LIB_PATH
    assert there(built) == [True, True, False]
