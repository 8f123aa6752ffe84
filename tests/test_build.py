"""The build's products (CPU): the marshalling module belongs to one interpreter."""
import importlib
import os
import sysconfig

from muon_newton_schulz_06_b200 import build as mbuild


def test_marshalling_module_is_built_for_this_interpreter():
    mbuild.build()
    assert mbuild.PY_LIB.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and os.path.exists(mbuild.PY_LIB)
    assert mbuild.up_to_date()
    mod = importlib.import_module("muon_newton_schulz_06_b200._muon_py")
    assert os.path.realpath(mod.__file__) == os.path.realpath(mbuild.PY_LIB)


def test_another_interpreter_finds_it_out_of_date(monkeypatch):
    mbuild.build()
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var",
                        lambda name: ".cpython-399-x86_64-linux-gnu.so" if name == "EXT_SUFFIX" else real(name))
    try:
        assert not importlib.reload(mbuild).up_to_date()
    finally:
        monkeypatch.undo()
        importlib.reload(mbuild)
    assert mbuild.up_to_date()
