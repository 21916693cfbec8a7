"""Other threads of Python while a call of the cache is in its entry point, without a GPU. The entry point is a fake that
waits: a sleep of the C library, whose first argument stands where a cache's address would."""
from __future__ import annotations

import ctypes
import threading
import time
import warnings

import pytest
import torch

from entropy_coding_gb300 import build

fake_tensor = pytest.importorskip("torch._subclasses.fake_tensor")


def _stamps_during(call):
    """When another thread ran, apart from the call's beginning and end, as parts of its time."""
    stamps, done = [], threading.Event()

    def tick():
        while not done.wait(0.005):
            stamps.append(time.monotonic())

    thread = threading.Thread(target=tick)
    thread.start()
    time.sleep(0.03)
    t0 = time.monotonic()
    call()
    t1 = time.monotonic()
    done.set()
    thread.join()
    return t1 - t0, [t for t in stamps if t0 + 0.1 < t < t1 - 0.1]


def test_other_threads_run_while_an_entry_point_waits():
    module = build.load_module()
    sleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    with fake_tensor.FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")  # (no tokens: the address is not used)
        k = torch.empty(0, 2, 32, device="cuda:0", dtype=torch.float16)
        took, stamps = _stamps_during(lambda: module.move(sleep, 500000, 0, 0, 0, 0, 0, 2, 32, k, k))
    assert took >= 0.5 and len(stamps) >= 5, (took, stamps)
