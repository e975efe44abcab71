"""Edges of the paged cache without a GPU."""
import os
import subprocess

import numpy as np
import pytest

import paged_ref as ref
from long_context_sparse_rtp_b200 import build, paged


def test_forced_pages_come_before_infinite_scores():
    """Ten pages, six of them of scale inf, four kept: the first and the last are among them."""
    zero = np.zeros((10, 128), dtype=np.int64)
    scale = np.ones(10, dtype=np.float32)
    scale[2:8] = np.inf
    q = np.ones((1, 128), dtype=np.float32)
    assert ref.select(q, zero, zero, scale, 4, 1, 1) == [0, 2, 3, 9]
    assert ref.select(q, zero, zero, scale, 1, 0, 1) == [9]
    assert ref.select(q, zero, zero, scale, 1, 1, 0) == [0]
    assert ref.select(q, zero, zero, scale, 4, 0, 0) == [2, 3, 4, 5]
    scale[[0, 9]] = -1  # not even a page outside the pool loses its place
    assert ref.select(q, zero, zero, scale, 3, 1, 1) == [0, 2, 9]


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The binding's files in a folder of their own, and a compiler that only notes its call."""
    calls = []

    def compile_(cmd, **kw):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "EXT", str(tmp_path / "_paged.so"))
    monkeypatch.setattr(build, "STAMP", str(tmp_path / "_paged.torch"), raising=False)
    monkeypatch.setattr(build, "build_lib", lambda *a: build.LIB)
    monkeypatch.setattr(subprocess, "check_call", compile_)
    return calls


def test_binding_is_built_again_for_another_torch(elsewhere, monkeypatch):
    import torch
    build.build()
    assert len(elsewhere) == 1 and os.path.exists(build.EXT)
    build.build()
    assert len(elsewhere) == 1
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    build.build()
    assert len(elsewhere) == 2
    os.remove(build.EXT)
    build.build()
    assert len(elsewhere) == 3


def test_library_is_built_without_what_the_binding_needs(elsewhere, monkeypatch, tmp_path):
    """Only the binding needs torch and Python's headers: without them it is left out, with a
    warning."""
    paths = dict(build.sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda *a, **kw: paths)
    with pytest.warns(UserWarning, match="Python.h"):
        assert build.build() == build.LIB
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    with pytest.warns(UserWarning, match="torch"):
        assert build.build() == build.LIB
    assert not elsewhere


def test_binding_of_another_torch_is_not_loaded(monkeypatch, tmp_path):
    build.build()
    stamp = tmp_path / "_paged.torch"
    stamp.write_text("python 3.0 torch 1.0.0 cxx11abi 0\n")
    monkeypatch.setattr(build, "STAMP", str(stamp))
    monkeypatch.setattr(paged, "_ext", None)
    with pytest.raises(RuntimeError, match="torch 1.0.0"):
        paged._native()
