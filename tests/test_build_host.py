"""The build of the call path, a CPython extension (no GPU)."""
import importlib.util
import os
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def build_module():
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, "scale_calibration_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


needs_headers = pytest.mark.skipif(not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")),
                                   reason="no Python headers: the extension is not built")


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build, putting the extension into a folder of its own."""
    b = build_module()
    monkeypatch.setattr(b, "CALL_LIB", str(tmp_path / os.path.basename(b.CALL_LIB)))
    if hasattr(b, "CALL_LIB_UNTAGGED"):
        monkeypatch.setattr(b, "CALL_LIB_UNTAGGED", str(tmp_path / "_lhcall.so"))
    return b


@needs_headers
def test_another_interpreter_does_not_find_the_extension(build, tmp_path):
    (tmp_path / "_lhcall.so").write_bytes(b"of an earlier build, for whichever interpreter made it")
    path = build.build_call()
    assert os.listdir(tmp_path) == ["_lhcall" + sysconfig.get_config_var("EXT_SUFFIX")] == [os.path.basename(path)]
    import scale_calibration_b200._lhcall as loaded
    assert loaded.__file__.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_the_library_builds_and_loads_without_python_headers(build, tmp_path, monkeypatch):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "nowhere")})
    assert not build.build_call(force=True) and os.listdir(tmp_path) == []


@needs_headers
def test_calls_without_the_extension_are_the_same(monkeypatch):
    import sys

    import scale_calibration_b200 as lh
    from scale_calibration_b200 import _binding
    fast = _binding._fast("lh_route_tokens", "piiippps")
    monkeypatch.setitem(sys.modules, "scale_calibration_b200._lhcall", None)  # its import fails
    monkeypatch.delattr(lh, "_lhcall", raising=False)
    slow = _binding._fast("lh_route_tokens", "piiippps")
    gather = _binding._fast("lh_gather_tokens", "ptiiipiipis")
    assert type(fast) is not type(slow)
    F = 0x10000000
    for args, want in [((None, 10, 4, 64, F, F, F, 0), 1), ((F, 10, 4, 2000, F, F + 8, F + 16, 0), 2),
                       ((F, 10, 0, 64, F, F + 8, F + 16, 0), 1)]:
        assert fast(*args) == slow(*args) == want
    assert gather(0, lh.LH_BF16, 0, 64, 64, 0, 2, 0, 0, 64, 0) == 0
    for call in (fast, slow):
        with pytest.raises(TypeError):
            call(F, 10)
        with pytest.raises(TypeError):
            call(F, 10, 4.0, 64, F, F, F, 0)
