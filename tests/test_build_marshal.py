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


def test_the_library_is_built_where_the_marshalling_cannot_be(monkeypatch):
    def fails(**kw):
        raise FileNotFoundError("g++")
    monkeypatch.setattr(build, "build_marshal", fails)
    with pytest.warns(UserWarning, match="cache operators"):
        assert build.build_library() == build.LIB


@pytest.mark.parametrize("kind", ["missing", "broken"])
def test_the_walk_is_there_without_it(tmp_path, kind):
    """The package beside a library alone, or with a file that is no module: the walk's entry points answer (here with
    their refusal of CPU tensors), the cache operators name what they need."""
    import subprocess
    import sys
    at = tmp_path / "kv_cache_early_art_b200"
    at.mkdir()
    for f in ("__init__.py", "binding.py", "build.py", "workloads.py", "libart.so"):
        os.symlink(os.path.join(build.HERE, f), at / f)
    if kind == "broken":
        (at / os.path.basename(build.marshal_path())).write_bytes(b"not a library")
    code = """
import torch, kv_cache_early_art_b200 as art
assert art.LIB_PATH.startswith({0!r}) and art.art_version() >= 100
z, i = torch.zeros, torch.int32
try:
    art.art_decode_attention(z(1, 4, 64), z(2, 2, 64, 64), z(2, 2, 64, 64), z(1, 2, dtype=i), None, z(1, dtype=i), 0, 0, 1, 1)
except ValueError as e:
    assert "GPU" in str(e)
rope = art.art_rope_init(64)
for call in (lambda: art.art_decode_attention_split(z(1, 4, 64), z(9, 2, 16, 64), z(9, 2, 16, 64), z(1, 2, dtype=i), z(1, dtype=i)),
             lambda: art.art_rope_append(rope, *[z(1, 2, 64)] * 3, *[z(9, 2, 16, 64)] * 2, z(1, 2, dtype=i), z(1, dtype=i)),
             lambda: art.art_cache_evict(*[z(9, 2, 16, 64)] * 2, z(1, 2, dtype=i), z(1, dtype=i), z(1, 2, 32), 8)):
    try:
        call()
    except ImportError as e:
        assert "cache operators" in str(e) and "_marshal" in str(e)
    else:
        raise AssertionError("ran")
""".format(str(tmp_path))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=tmp_path, timeout=300)
