"""A cache without the module of its calls on torch tensors: there is a warning, once, and calls go through ctypes."""
from __future__ import annotations

import warnings

import pytest

from entropy_coding_gb300 import build, kv


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), PermissionError("_lib"), RuntimeError("g++ failed"), ImportError("symbols")])
def test_a_module_that_cannot_be_had_leaves_the_other_path(monkeypatch, error):
    tries = []

    def load():
        tries.append(1)
        raise error

    monkeypatch.setattr(build, "load_module", load)
    monkeypatch.setattr(kv, "_torch", None)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert kv._quick(kv.KVCache._calls) is None
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert kv._quick(kv.KV4Cache._calls) is None
    assert len(tries) == 1
    cache, batch = object.__new__(kv.KVCache), object.__new__(kv.KVBatch)
    cache.__dict__.update(_many=False, _index=0, _quick=kv._quick(kv.KVCache._calls))
    batch.__dict__.update(_index=0)
    assert kv._at_once(cache, batch, None) is None


def test_a_compiler_that_is_not_there_is_one_of_these(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setenv("PATH", str(tmp_path))
    monkeypatch.setattr(kv, "_torch", None)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert kv._quick(kv.KVCache._calls) is None
