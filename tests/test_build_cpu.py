"""The build: the CUDA library does not depend on the feed-forward operators'
native binding, which needs torch with CUDA and g++."""
import ctypes
import os
import stat

import pytest

from async_copy_pipelined_gb300 import buildlib

SOURCE = 'extern "C" int seven() { return 7; }\n'


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """A library of one small source, a torch that is a folder, and a compiler that
    writes its output's name (or, with the file `broken` there, fails)."""
    out, torch_dir = tmp_path / "out", tmp_path / "torch"
    (torch_dir / "lib").mkdir(parents=True)
    (torch_dir / "include").mkdir()
    (torch_dir / "lib" / "libc10_cuda.so").write_text("")
    (torch_dir / "version.py").write_text("__version__ = '1.2.3+one'\n")
    out.mkdir()
    source = tmp_path / "seven.cu"
    source.write_text(SOURCE)
    compiler = tmp_path / "compiler"
    compiler.write_text("#!/bin/sh\n"
                        f"echo called >> {tmp_path}/calls\n"
                        f"if [ -e {tmp_path}/broken ]; then echo no such header >&2; exit 1; fi\n"
                        'while [ "$1" != -o ]; do shift; done\necho binding > "$2"\n')
    compiler.chmod(compiler.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("CXX", str(compiler))
    monkeypatch.setattr(buildlib, "OUT_DIR", str(out))
    monkeypatch.setattr(buildlib, "LIB_PATH", str(out / "lib.so"))
    monkeypatch.setattr(buildlib, "BINDING_PATH", str(out / "binding.so"))
    monkeypatch.setattr(buildlib, "BINDING_LOG", str(out / "binding.log"), raising=False)
    monkeypatch.setattr(buildlib, "_sources", lambda: [str(source)])
    monkeypatch.setattr(buildlib, "_torch_dir", lambda: str(torch_dir))
    return tmp_path


def _seven():
    return ctypes.CDLL(buildlib.LIB_PATH).seven()


def _calls(tree):
    at = tree / "calls"
    return len(at.read_text().split()) if at.exists() else 0


def test_both_are_built_once(tree, recwarn):
    buildlib.build()
    assert _seven() == 7 and os.path.exists(buildlib.BINDING_PATH) and buildlib.up_to_date()
    buildlib.build()
    assert _calls(tree) == 1 and not recwarn.list


def test_a_binding_that_does_not_compile_leaves_the_library(tree, monkeypatch):
    (tree / "broken").touch()
    with pytest.warns(RuntimeWarning, match="binding does not build"):
        buildlib.build()
    assert _seven() == 7 and not os.path.exists(buildlib.BINDING_PATH)
    with open(buildlib.BINDING_LOG) as f:
        assert "no such header" in f.read()
    # It is not tried again, nor the library built again, until asked or a source changes.
    compile_one = buildlib._compile
    monkeypatch.setattr(buildlib, "_compile", lambda src: pytest.fail("built again"))
    with pytest.warns(RuntimeWarning, match="--force"):
        buildlib.build()
    assert _calls(tree) == 1
    monkeypatch.setattr(buildlib, "_compile", compile_one)
    (tree / "broken").unlink()
    buildlib.build(force=True)
    assert os.path.exists(buildlib.BINDING_PATH) and buildlib.up_to_date()


def test_a_binding_of_other_sources_does_not_stay(tree, monkeypatch):
    buildlib.build()
    (tree / "broken").touch()
    with pytest.warns(RuntimeWarning):
        buildlib.build(force=True)
    assert _seven() == 7 and not os.path.exists(buildlib.BINDING_PATH)


def test_torch_without_cuda_needs_no_binding(tree, recwarn):
    (tree / "torch" / "lib" / "libc10_cuda.so").unlink()
    buildlib.build()
    assert _seven() == 7 and _calls(tree) == 0 and buildlib.up_to_date() and not recwarn.list


def test_no_torch_needs_no_binding(tree, monkeypatch, recwarn):
    monkeypatch.setattr(buildlib, "_torch_dir", lambda: None)
    buildlib.build()
    assert _seven() == 7 and _calls(tree) == 0 and buildlib.up_to_date() and not recwarn.list


def test_another_torch_is_given_a_binding_of_its_own(tree, monkeypatch):
    buildlib.build()
    assert buildlib.up_to_date()
    (tree / "torch" / "version.py").write_text("__version__ = '1.2.3+two'\n")
    assert not buildlib.up_to_date()
    monkeypatch.setattr(buildlib, "_compile", lambda src: pytest.fail("the library was built again"))
    buildlib.build()
    assert _calls(tree) == 2 and buildlib.up_to_date()


def test_a_binding_that_is_gone_is_built_again(tree):
    buildlib.build()
    os.remove(buildlib.BINDING_PATH)
    assert not buildlib.up_to_date()
    buildlib.build()
    assert os.path.exists(buildlib.BINDING_PATH)


def test_a_binding_of_another_build_of_the_same_release_is_refused(monkeypatch):
    import torch

    import async_copy_pipelined_gb300 as pg
    from async_copy_pipelined_gb300 import feedforward as ff
    pg.build()
    assert ff._load_native().torch_build == str(torch.__version__)
    release = str(torch.__version__).split("+")[0]
    for other in (release + "+another", release + ".dev20260101+cu130", release + "a0"):
        monkeypatch.setattr(torch, "__version__", other)
        with pytest.raises(RuntimeError, match="built for torch"):
            ff._load_native()
