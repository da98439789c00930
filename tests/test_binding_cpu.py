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
from tests.binding_stub import Stream, World


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


def calls_of(world, stream, kept=None):
    """Every call that makes memory for itself, and what it returned."""
    x, dy, ids = world.tensor(5, 64), world.tensor(5, 96), world.tensor(5, dtype=torch.int32)
    path, pool = world.path(64, 96, 32), world.pool(3, 8, 64, 96)
    rot = lb.HeadRotation(32, world.tensor(16, dtype=torch.float32))
    w = world.tensor(32)
    z = world.tensor(5, 32, dtype=torch.float16)
    layer = lb.LittleBitLinear(path)
    if kept is not None:
        layer._ws = kept
    calls = [
        lambda: [lb.linear_forward(x, path, stream=stream)],
        lambda: lb.linear_forward_siblings(x, [(path, None)] * 2, adapters=[pool, None], ids=ids, rotation=rot, positions=ids,
                                           rotate={0: w}, stream=stream),
        lambda: [lb.latent_forward(x, path, stream=stream)],
        lambda: [lb.expand_forward(z, path, stream=stream)],
        lambda: [lb.linear_forward_fixed_scratch(x, path, stream=stream)],
        lambda: [v for v in lb.linear_backward(x, dy, path, adapters=pool, ids=ids, stream=stream).values()],
        lambda: lb.adapters_forward(x, ids, [pool], bases=[dy], stream=stream),
        lambda: [*lb.adapters_backward(x, dy, ids, pool, dx_base=x, stream=stream).values()],
        lambda: lb.heads_norm_rotate([dy], ids, rot, weights=[w], stream=stream),
        lambda: [*lb.heads_norm_rotate_backward([dy], [dy], ids, rot, weights=[w], stream=stream)[0].values()],
        lambda: [layer(x, adapters=pool, ids=ids, stream=stream)],
        lambda: [lb.pack_signs(world.tensor(96, 32), "U", stream=stream)],
    ]
    for call in calls:
        world.calls.clear()
        world.allocations.clear()
        yield call(), world.allocations, world.calls


def test_memory_for_a_stream_comes_from_it(world):
    """A block of the current stream's may still be read by kernels queued
    there; the call's stream is not ordered behind them."""
    side = Stream(77)
    scratch = world.tensor(1 << 16, dtype=torch.uint8)  # a layer's, from calls on the current stream
    kept = scratch.address
    for returned, made, calls in calls_of(world, side, scratch):
        assert made and calls
        for t in made:
            assert t.stream is side
        for t in returned:  # read on the current stream after the caller has waited there
            assert t in made and t.recorded == [world.default]
        assert not any(kept in args for _, args in calls)


def test_memory_without_a_stream_comes_from_the_current_one(world):
    for returned, made, _ in calls_of(world, None):
        assert all(t.stream is world.default and not t.recorded for t in made)


def group(world):
    """A sibling group with everything behind it, and the layer's other calls, as keyword arguments."""
    i32 = torch.int32
    return dict(x=world.tensor(5, 64), ids=world.tensor(5, dtype=i32), positions=world.tensor(5, dtype=i32),
                pools=[world.pool(3, 8, 64, 96), None], rot=lb.HeadRotation(32, world.tensor(16, dtype=torch.float32)),
                weight=world.tensor(32), path=world.path(64, 96, 32))


def siblings(world, g):
    return lb.linear_forward_siblings(g["x"], [(g["path"], None)] * 2, adapters=g["pools"], ids=g["ids"], rotation=g["rot"],
                                      positions=g["positions"], rotate={0: g["weight"]})


def layer(world, g):
    return lb.LittleBitLinear(g["path"])(g["x"], adapters=g["pools"][0], ids=g["ids"])


def backward(world, g):
    return lb.linear_backward(g["x"], world.tensor(5, 96), g["path"], adapters=g["pools"][0], ids=g["ids"], dx=g.get("dx"))


SOME = [siblings, layer, backward]
BAD_GROUPS = [  # what is wrong, the calls that see it, the error
    ("ids of another type", SOME, TypeError, lambda w, g: g.update(ids=w.tensor(5, dtype=torch.float32))),
    ("too few ids", SOME, ValueError, lambda w, g: g.update(ids=w.tensor(4, dtype=torch.int32))),
    ("no ids", SOME, ValueError, lambda w, g: g.update(ids=None)),
    ("ids on the host", SOME, ValueError, lambda w, g: g.update(ids=torch.zeros(5, dtype=torch.int32))),
    ("a pool for another x", SOME, ValueError, lambda w, g: g.update(pools=[w.pool(3, 8, 32, 96), None])),
    ("a pool for another y", SOME, ValueError, lambda w, g: g.update(pools=[w.pool(3, 8, 64, 64), None])),
    ("an odd rank", SOME, lb.LbError, lambda w, g: g.update(pools=[w.pool(3, 12, 64, 96), None])),
    ("too many adapters", SOME, lb.LbError, lambda w, g: g.update(pools=[w.pool(1025, 8, 64, 96), None])),
    ("a pool at an odd address", SOME, lb.LbError, lambda w, g: g.update(pools=[
        lb.AdapterPool(w.tensor(3, 8, 64, address=1 << 30 | 2), w.tensor(3, 96, 8)), None])),
    ("pools of unlike counts", [siblings], lb.LbError, lambda w, g: g.update(pools=[w.pool(3, 8, 64, 96), w.pool(4, 8, 64, 96)])),
    ("a dx of another shape", [backward], ValueError, lambda w, g: g.update(dx=w.tensor(5, 96))),
    ("positions of another type", [siblings], TypeError, lambda w, g: g.update(positions=w.tensor(5, dtype=torch.float32))),
    ("too few positions", [siblings], ValueError, lambda w, g: g.update(positions=w.tensor(4, dtype=torch.int32))),
    ("no positions", [siblings], ValueError, lambda w, g: g.update(positions=None)),
    ("a weight of another size", [siblings], ValueError, lambda w, g: g.update(weight=w.tensor(64))),
    ("a weight at an odd address", [siblings], lb.LbError, lambda w, g: g.update(weight=w.tensor(32, address=1 << 30 | 2))),
    ("heads that do not divide", [siblings], ValueError, lambda w, g: g.update(
        rot=lb.HeadRotation(40, w.tensor(16, dtype=torch.float32)))),
    ("more turned than a head has", [siblings], lb.LbError, lambda w, g: g.update(
        rot=lb.HeadRotation(32, w.tensor(24, dtype=torch.float32)))),
    ("a negative eps", [siblings], lb.LbError, lambda w, g: g.update(
        rot=lb.HeadRotation(32, w.tensor(16, dtype=torch.float32), eps=-1.0))),
]


@pytest.mark.parametrize("call,error,change", [pytest.param(c, e, f, id=f"{c.__name__}: {what}")
                                               for what, calls, e, f in BAD_GROUPS for c in calls])
def test_a_refused_call_launches_nothing(world, call, error, change):
    g = group(world)
    change(world, g)
    with pytest.raises(error):
        call(world, g)
    assert not world.calls


def test_a_group_that_is_right_launches_in_order(world):
    siblings(world, group(world))
    layer(world, group(world))
    backward(world, group(world))
    assert world.names() == ["lb_linear_forward_siblings", "lb_adapters_forward", "lb_heads_norm_rotate", "lb_linear_forward",
                             "lb_adapters_forward", "lb_linear_backward", "lb_adapters_backward"]


def test_wide_heads_are_refused_before_the_projections(world):
    x, path = world.tensor(5, 64), world.path(64, 4097 * 32, 32)
    with pytest.raises(lb.LbError) as e:
        lb.linear_forward_siblings(x, [(path, None)], rotation=lb.HeadRotation(32), positions=world.tensor(5, dtype=torch.int32),
                                   rotate={0: None})
    assert e.value.status == lb.LB_ERR_UNSUPPORTED_SHAPE and not world.calls


def test_no_tokens_launch_no_check(world):
    g = group(world)
    g.update(x=world.tensor(0, 64), ids=world.tensor(0, dtype=torch.int32))
    lb.linear_backward(g["x"], world.tensor(0, 96), g["path"], adapters=g["pools"][0], ids=g["ids"])
    assert world.names() == ["lb_linear_backward", "lb_adapters_backward"]


def test_a_norm_alone_needs_no_positions(world):
    """As heads_norm_rotate itself."""
    g = group(world)
    lb.linear_forward_siblings(g["x"], [(g["path"], None)], rotation=lb.HeadRotation(32), rotate={0: g["weight"]})
    lb.heads_norm_rotate([world.tensor(5, 96)], None, lb.HeadRotation(32), weights=[g["weight"]])
    assert world.names() == ["lb_linear_forward_siblings", "lb_heads_norm_rotate", "lb_heads_norm_rotate"]


def test_a_workspace_on_another_device_is_refused(world):
    g = group(world)
    far = world.tensor(1 << 22, dtype=torch.uint8, device=torch.device("cuda", 1))
    y, w = world.tensor(5, 96), [g["weight"]]
    for call in (lambda: lb.adapters_forward(g["x"], g["ids"], g["pools"][:1], ys=[y], workspace=far),
                 lambda: lb.adapters_backward(g["x"], y, g["ids"], g["pools"][0], want_dx=False, workspace=far),
                 lambda: lb.heads_norm_rotate_backward([y], [y], g["positions"], g["rot"], weights=w, workspace=far)):
        with pytest.raises(ValueError, match="workspace must be on cuda:0"):
            call()
    assert not world.calls
