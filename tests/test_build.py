"""The build's two parts on the CPU, with fakes of the compilers: the library does
not depend on the Python module of its short calls, whose place ctypes takes."""
import os
import subprocess
import sysconfig

import pytest

import split_kv_decode_attn_b200 as fd
from split_kv_decode_attn_b200 import build

from test_fdcall import CALLS, REFUSED, test_refusals_are_those_of_the_c_entry_point as refusal


def test_the_module_is_named_for_its_interpreter():
    assert build.CALLS == fd.CALLS_PATH
    assert build.CALLS.endswith("_fdcall" + sysconfig.get_config_var("EXT_SUFFIX"))
    assert sysconfig.get_config_var("SOABI") in os.path.basename(build.CALLS)


@pytest.mark.parametrize("error", [FileNotFoundError("gcc"), subprocess.CalledProcessError(1, "gcc")])
def test_the_library_is_built_where_the_module_cannot_be(tmp_path, monkeypatch, error):
    made = []

    def nvcc_runs(cmd, **kw):
        made.append(cmd[cmd.index("-o") + 1])
        open(made[-1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def no_compiler(*a, **kw):
        raise error
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfd.so"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_fdcall.so"))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(build.subprocess, "run", nvcc_runs)
    monkeypatch.setattr(build.subprocess, "check_call", no_compiler)
    with pytest.warns(UserWarning, match="ctypes"):
        assert build.build() == str(tmp_path / "libfd.so")
    assert made == [str(tmp_path / "libfd.so")]


@pytest.fixture
def through_ctypes(monkeypatch):
    monkeypatch.setattr(fd, "CALLS_PATH", os.path.join(os.path.dirname(fd.CALLS_PATH), "missing.so"))
    monkeypatch.setattr(fd, "_calls", None)
    yield
    assert isinstance(fd._calls, fd._CtypesCalls)


@pytest.mark.parametrize("name,args", REFUSED)
def test_ctypes_calls_give_the_same_refusals(through_ctypes, name, args):
    refusal(name, args)


def test_ctypes_calls_take_every_argument(through_ctypes):
    """As many as the native calls, and numbers of the wrong kind raise."""
    for name, args in CALLS:
        call = getattr(fd._load_calls(), name[3:])
        with pytest.raises(Exception):
            call(*args)                    # without the stream
        for i in [i for i, x in enumerate(args) if type(x) is int]:
            with pytest.raises(Exception):
                call(*args[:i], "text", *args[i + 1:], 1)
