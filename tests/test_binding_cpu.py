"""What the Python binding of the adapters and heads calls does on the host:
pools used by several threads at once, where memory comes from when a stream is
given, and refusals before anything is launched.  No GPU: stand-ins for tensors
and the library (tests/binding_stub.py)."""
import sys
import threading

import pytest
import torch

import binarized_rank_linear_b200 as lb
from binarized_rank_linear_b200 import build as lb_build
from tests.binding_stub import World


@pytest.fixture
def world(monkeypatch):
    lb_build.build()
    return World(monkeypatch)


def test_a_pool_is_whole_when_another_thread_finds_it(world):
    """`_c` is what tells a second thread that the pool is ready: whatever else
    the calls read of it is there before."""
    order = []
    pool = world.pool(2, 8, 64, 96)

    class Recorder:
        @staticmethod
        def __setattr__(obj, name, value):
            order.append(name)
            object.__setattr__(obj, name, value)

    lb.object = Recorder  # the module's `object` while as_c runs
    try:
        pool.as_c()
    finally:
        del lb.object
    assert order[-1] == "_c" and set(order[:-1]) == {"_p", "n_in", "n_out", "device"}


def test_fresh_pools_in_three_threads(world):
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    faults = []
    try:
        for _ in range(300):
            pools = [world.pool(2, 8, 64, 96) for _ in range(10)]
            start = threading.Barrier(3)

            def use():
                start.wait()
                for pool in pools:
                    try:
                        pool.as_c()
                        assert (pool.n_in, pool.n_out, pool.device.type, pool._p.contents.rank) == (64, 96, "cuda", 8)
                    except Exception as e:  # noqa: BLE001 - kept for the assertion below
                        faults.append(e)

            threads = [threading.Thread(target=use) for _ in range(3)]
            for th in threads:
                th.start()
            for th in threads:
                th.join()
    finally:
        sys.setswitchinterval(interval)
    assert not faults, faults[0]
