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
