"""When the native host module is built again: it is missing, older than its
sources, or was built against another torch or Python."""
import os
import shutil

import torch

from precision_rl_rollout_nvfp4_b200 import binding as B
from precision_rl_rollout_nvfp4_b200 import build_lib


def test_host_module_names_what_it_was_built_against():
    assert B._host.built_against == build_lib.host_target()
    assert torch.__version__ in build_lib.host_target()


def test_when_the_host_module_is_rebuilt(tmp_path, monkeypatch):
    so = tmp_path / "_host.so"
    assert build_lib.host_needs_build(str(so))
    shutil.copy(build_lib.HOST, so)                         # (its time is now: newer than the sources)
    assert not build_lib.host_needs_build(str(so))
    monkeypatch.setattr(torch, "__version__", torch.__version__ + "1")
    assert build_lib.host_needs_build(str(so))
    monkeypatch.undo()
    os.utime(so, (1, 1))
    assert build_lib.host_needs_build(str(so))


def test_build_of_a_current_host_module_does_nothing(monkeypatch):
    build_lib.build_host()
    monkeypatch.setattr(build_lib.subprocess, "run", lambda *a, **k: 1 / 0)
    assert build_lib.build_host() == build_lib.HOST
