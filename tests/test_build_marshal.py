"""The binding's compiled marshalling: whose file is loaded, and what works where it is missing."""
import os
import sysconfig

import pytest
import torch

from kv_cache_early_art_b200 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build_library()


def test_file_is_named_after_torch_and_python(monkeypatch):
    """Another torch, or another interpreter, looks for another file: the present one is stale for it."""
    here = build.marshal_path()
    assert os.path.exists(here) and here.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "9.1.0+other")
        torch_path = build.marshal_path()
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_config_var", lambda name: ".cpython-999-other.so")
        python_path = build.marshal_path()
    assert len({here, torch_path, python_path}) == 3
    assert not os.path.exists(torch_path) and not os.path.exists(python_path)


def test_another_torch_version_is_built_anew(monkeypatch):
    ran = []
    monkeypatch.setattr(build.subprocess, "check_call", lambda cmd, **kw: ran.append(cmd))
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    build.build_marshal()
    assert not ran                                       # this one's is up to date
    monkeypatch.setattr(torch, "__version__", "9.1.0+other")
    assert "9_1_0_other" in build.build_marshal()
    assert len(ran) == 1 and "9_1_0_other" in ran[0][ran[0].index("-o") + 1]


def test_the_binding_loads_that_file():
    from kv_cache_early_art_b200 import binding
    assert binding._marshal.__file__ == build.marshal_path()
