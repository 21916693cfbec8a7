"""The Python module of the cache's calls on torch tensors, without a GPU: it builds against the installed torch, and does
nothing where something is not as a call has it (the entry points here are fakes that must not run)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from entropy_coding_gb300 import build, kv


@pytest.fixture(scope="module")
def module():
    return build.load_module()


def _never(*_):
    raise AssertionError("an entry point ran")


FAKE = ctypes.CFUNCTYPE(ctypes.c_int)(_never)
ENTRY = ctypes.cast(FAKE, ctypes.c_void_p).value
CALL = (0, 0, 0, 0, 3, 2, 32)  # batch, status, stream, device, tokens, kv_heads, dim


def test_host_tensors_and_other_objects_are_left_to_the_python_layer(module):
    q, k = torch.zeros(3, 4, 32).half(), torch.zeros(3, 2, 32).half()
    for x in (q, None, 7, "q", q.numpy()):
        assert module.attend(ENTRY, 0, *CALL, x, 0.1, 1, 0, 0, 0) is None
        assert module.move(ENTRY, 0, *CALL, x, k) is None and module.move(ENTRY, 0, *CALL, k, x) is None
        assert module.rotate(ENTRY, *CALL, 0, 0, 0, x, k, None, None, 1e-6) is None
    assert module.rotate(ENTRY, *CALL, 0, 0, 0, q, k, torch.ones(32), 5, 1e-6) is None


def test_wrong_numbers_of_arguments_and_no_numbers_are_errors(module):
    q = torch.zeros(3, 4, 32).half()
    for f in (module.attend, module.read, module.move, module.rotate):
        with pytest.raises(TypeError):
            f()
        with pytest.raises(TypeError):
            f(ENTRY, 0, *CALL)
    with pytest.raises(TypeError):
        module.attend(ENTRY, 0, "batch", *CALL[1:], q, 0.1, 1, 0, 0, 0)
    with pytest.raises(TypeError):
        module.rotate(ENTRY, *CALL, 0, 0, 0, q, q, None, None, "eps")


def test_a_module_is_kept_for_each_torch(module):
    assert torch.__version__.replace("+", "_") in build._module_path() and build.build_module() == build._module_path()


def test_calls_are_made_at_once_only_on_the_caches_device(monkeypatch):
    """Fakes of two devices and of the module: a call on another stream, with another device current or with a batch of
    another device goes through the layer that sees to these."""
    cache, batch = object.__new__(kv.KVCache), object.__new__(kv.KVBatch)
    now = [0]
    monkeypatch.setattr(kv, "_current_device", lambda: now[0], raising=False)
    for many, mine, batchs, current, stream, at_once in ((False, 0, 0, 0, None, True), (False, 0, 0, 0, 7, False), (True, 1, 1, 1, None, True),
                                                         (True, 1, 1, 0, None, False), (True, 1, 0, 1, None, False), (True, 0, 0, 0, 7, False)):
        cache.__dict__.update(_many=many, _index=mine, _quick=(1, 2, 3, 4))
        batch.__dict__.update(_index=batchs)
        now[0] = current
        assert (kv._at_once(cache, batch, stream) is not None) == at_once
    del cache.__dict__["_quick"]
    assert kv._at_once(cache, batch, None) is None
