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


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build, putting the extension into a folder of its own."""
    b = build_module()
    monkeypatch.setattr(b, "CALL_LIB", str(tmp_path / os.path.basename(b.CALL_LIB)))
    if hasattr(b, "CALL_LIB_UNTAGGED"):
        monkeypatch.setattr(b, "CALL_LIB_UNTAGGED", str(tmp_path / "_lhcall.so"))
    return b


def test_another_interpreter_does_not_find_the_extension(build, tmp_path):
    (tmp_path / "_lhcall.so").write_bytes(b"of an earlier build, for whichever interpreter made it")
    path = build.build_call()
    assert os.listdir(tmp_path) == ["_lhcall" + sysconfig.get_config_var("EXT_SUFFIX")] == [os.path.basename(path)]
    import scale_calibration_b200._lhcall as loaded
    assert loaded.__file__.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
