"""Building of TokenSorter's extension module beside the library (host only; nothing is compiled but a stand-in)."""
import os
import sysconfig

import pytest
import torch

from sparse_moe_layer_biased_b200 import _abi, build


@pytest.fixture
def fresh(monkeypatch, tmp_path):
    """The libraries count as up to date, the module's place is an empty folder."""
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "LIB_DEBUG", str(tmp_path / "lib_debug.so"))
    for lib in (build.LIB, build.LIB_DEBUG):
        open(lib, "w").close()
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "_deps", lambda: 1.0)
    return tmp_path


@pytest.mark.parametrize("debug", [False, True])
@pytest.mark.parametrize("cxx", ["/bin/false", "/nowhere/g++"])
def test_the_library_does_not_need_the_module(fresh, monkeypatch, cxx, debug):
    """A compiler that fails, or none: the library is built all the same, with a warning."""
    monkeypatch.setenv("CXX", cxx)
    with pytest.warns(RuntimeWarning, match="TokenSorter's extension module is not built"):
        assert build.build(debug=debug) == (build.LIB_DEBUG if debug else build.LIB)
    with pytest.raises((RuntimeError, OSError)):
        build.build_calls()


def test_an_outdated_module_does_not_outlive_a_failed_build(fresh, monkeypatch):
    monkeypatch.setenv("CXX", "/bin/false")
    path = build.calls_path()
    open(path, "w").close()
    build.build()  # up to date: no compiler is asked for
    assert os.path.exists(path)
    os.utime(path, (0.5, 0.5))
    with pytest.warns(RuntimeWarning):
        build.build()
    assert not os.path.exists(path)


@pytest.mark.parametrize("debug", [False, True])
def test_both_builds_build_the_module(fresh, monkeypatch, debug):
    made = []
    monkeypatch.setattr(build, "build_calls", lambda force: made.append(force))
    build.build(debug=debug)
    assert made == [False]


def test_the_module_is_that_of_this_pytorch_and_python(monkeypatch):
    path = build.calls_path()
    assert torch.__version__ in os.path.basename(path) and path.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert os.path.exists(path) and _abi.calls().__file__ == path
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="0.0.1.*is not built"):
        _abi.calls.__wrapped__()
