"""The first calls of the 4-bit wrappers, from two threads at once or after a
load that failed: a thread that sees the module bound finds all of it bound
(no GPU)."""

import threading
import time

import pytest

from paged_kv_cache_357_b200 import _lib, cache4
from paged_kv_cache_357_b200 import build as pa_build


@pytest.fixture
def unbound(monkeypatch):
    pa_build.build()
    for name in ("torch", "_lib", "_raw_stream", "_current_device"):
        monkeypatch.setattr(cache4, name, None)
    monkeypatch.setattr(cache4, "_codes", {})


def test_two_threads(unbound, monkeypatch):
    entered, go = threading.Event(), threading.Event()

    def slow_load():
        entered.set()
        assert go.wait(10)
        return _lib.load()

    monkeypatch.setattr(cache4, "load", slow_load)
    errors = []

    def bind():
        try:
            cache4._bind()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    first = threading.Thread(target=bind)
    first.start()
    assert entered.wait(10)
    time.sleep(0.05)
    # what another thread's call looks at while the first one is loading
    seen = cache4.torch, cache4._lib
    second = threading.Thread(target=bind)
    second.start()
    go.set()
    first.join(10)
    second.join(10)
    assert not errors
    assert seen[0] is None or seen[1] is not None
    assert cache4.torch is not None and cache4._lib is not None and len(cache4._codes) == 2


def test_a_load_that_fails(unbound, monkeypatch):
    def missing():
        raise RuntimeError("libpa.so not found")

    monkeypatch.setattr(cache4, "load", missing)
    for _ in range(2):  # the second call tries again
        with pytest.raises(RuntimeError, match="libpa.so not found"):
            cache4._first(None, "k_pool", 4)
