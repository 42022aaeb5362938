"""How the library and the small calls' host path are built (CPU): commands are
recorded, not run."""
import os
import subprocess
import sys

import pytest

from nvfp4_block_quantization_amax_b200 import build


class Recorder:
    """Stands in for subprocess.run; the host compiler can be made to fail."""
    def __init__(self, fail=False):
        self.commands, self.fail = [], fail

    def __call__(self, cmd, check):
        self.commands.append(cmd)
        if self.fail and "nvcc" not in os.path.basename(cmd[0]):
            raise subprocess.CalledProcessError(1, cmd)

    def compiled(self, compiler):
        return [c[-3] for c in self.commands if compiler in os.path.basename(c[0]) and "-c" in c]


@pytest.fixture
def record(monkeypatch):
    def start(fail=False):
        r = Recorder(fail)
        monkeypatch.setattr(subprocess, "run", r)
        monkeypatch.setattr(os, "replace", lambda a, b: None)
        monkeypatch.setattr(build, "_stale", lambda: True)
        return r
    return start


def test_library_is_built_without_torch(record, monkeypatch):
    r = record()
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(RuntimeWarning, match="_fastcall"):
        assert build.build(force=True) == build.LIB
    assert r.compiled("nvcc") == build.sources() and all("nvcc" in c[0] for c in r.commands)


def test_library_is_built_before_a_host_compiler_fails(record):
    r = record(fail=True)
    with pytest.warns(RuntimeWarning, match="_fastcall"):
        assert build.build(force=True) == build.LIB
    assert r.compiled("nvcc") == build.sources() and "nvcc" not in r.commands[-1][0]


def test_a_failing_library_is_an_error(record, monkeypatch):
    r = record()

    def fail(cmd, check):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(subprocess, "run", fail)
    with pytest.raises(subprocess.CalledProcessError):
        build.build(force=True)
    assert not r.commands


def test_host_path_belongs_to_one_torch_and_python(record, monkeypatch):
    """Another torch or Python has another file: the one of this torch does not
    count as built for it, nor is it taken in its place."""
    import torch
    here = build.build_fastcall()
    assert here == build.fastcall_path() and os.path.exists(here)
    r = record()
    assert build.build_fastcall() == here and not r.commands
    monkeypatch.setattr(torch, "__version__", "2.12.0+cu130")
    other = build.fastcall_path()
    assert other != here and build.build_fastcall() == other and len(r.commands) == 1
    monkeypatch.undo()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: ".cpython-313-x86_64-linux-gnu.so")
    assert build.fastcall_path() not in (here, other) and not os.path.exists(build.fastcall_path())


def test_binding_makes_the_calls_without_the_host_path(record, monkeypatch):
    """With another torch, say: one warning, and the binding's own checks."""
    import torch

    from nvfp4_block_quantization_amax_b200 import api
    monkeypatch.setattr(api, "_fast", None)
    monkeypatch.setattr(torch, "__version__", "2.12.0+cu130")
    with pytest.warns(RuntimeWarning, match="host path"):
        fast = api._load_fast()
    assert api._fast is fast
    for name in ("route", "route_backward", "dispatch", "combine", "combine_backward", "gemv"):
        assert getattr(fast, name)(1, 2, 3) is None
    with pytest.raises(TypeError, match="CUDA"):
        api.nvfp4_route(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError, match="CUDA"):
        api.nvfp4_combine(torch.zeros(4, 8).bfloat16(), None, torch.zeros(4, 1))
