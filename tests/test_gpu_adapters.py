"""lb_adapters_forward and lb_adapters_backward on the GPU against their plain
64-bit forms (tests/operators_ref.py), whose bounds are derived there."""
import pytest

import binarized_rank_linear_b200 as lb
from binarized_rank_linear_b200 import synth
from tests import gpu_util as gu
from tests import operators_ref as ref

pytestmark = pytest.mark.gpu


def torch_():
    import torch
    return torch


def gen(seed):
    t = torch_()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0):
    t = torch_()
    return (t.randn(*shape, generator=g, device="cuda") * scale).to(t.bfloat16)


def make_pool(g, count, rank, n_in, n_out, ranks=None, scale=True):
    t = torch_()
    s = t.rand(count, generator=g, device="cuda") + 0.5 if scale else None
    r = t.tensor(ranks, dtype=t.int32, device="cuda") if ranks is not None else None
    return lb.AdapterPool(normal(g, count, rank, n_in, scale=n_in ** -0.5), normal(g, count, n_out, rank, scale=0.3), s, r)


def make_ids(g, tokens, count, kind):
    t = torch_()
    if kind == "one":
        ids = t.full((tokens,), count - 1, device="cuda")
    elif kind == "none":
        ids = t.full((tokens,), -1, device="cuda")
    elif kind == "some":  # a fifth of the tokens without an adapter
        ids = t.randint(0, count, (tokens,), generator=g, device="cuda")
        ids = t.where(t.rand(tokens, generator=g, device="cuda") < 0.2, -3, ids)
    elif kind == "runs":
        ids = t.randint(0, count, (tokens,), generator=g, device="cuda").sort().values.roll(tokens // 3)
    else:
        ids = t.randint(0, count, (tokens,), generator=g, device="cuda")
    return ids.to(t.int32)


def check_forward(x, ids, pools, bases, ys, what):
    for j, (p, base, y) in enumerate(zip(pools, bases, ys)):
        exact, tol = ref.adapters(x, ids, p.a, p.b, p.scale, p.ranks, base)
        ref.within(y, exact, tol, f"{what} projection {j}")


FORWARD = [  # tokens, n_in, outputs, rank, count, ids, ranks
    (1, 32, [32], 8, 1, "one", None),
    (1, 4096, [4096, 4096, 4096], 16, 8, "mixed", None),
    (2, 64, [96], 8, 2, "none", None),
    (3, 1056, [32, 288], 24, 3, "mixed", [24, 0, 5]),
    (8, 256, [64], 16, 4, "one", None),
    (9, 288, [544], 128, 2, "one", [1, 127]),
    (33, 5120, [5120, 1024, 1024], 16, 64, "some", None),
    (100, 1024, [800, 64], 32, 7, "mixed", [32, 31, 17, 16, 1, 8, 0]),
    (128, 512, [256], 64, 128, "mixed", None),
    (129, 512, [256], 64, 128, "mixed", None),
    (200, 96, [160, 32, 64, 128], 8, 3, "runs", [8, 3, 7]),
    (257, 544, [288], 40, 5, "some", [40, 33, 32, 9, 0]),
    (300, 2080, [1056], 128, 2, "one", None),
    (1000, 1024, [2048], 16, 11, "runs", None),
    (1025, 160, [96], 72, 1, "one", [65]),
    (700, 64, [64], 8, 600, "mixed", None),
]


@pytest.mark.parametrize("tokens,n_in,outs,rank,count,kind,ranks", FORWARD)
def test_forward_against_64_bits(tokens, n_in, outs, rank, count, kind, ranks):
    g = gen(tokens * 131 + n_in)
    x = normal(g, tokens, n_in)
    ids = make_ids(g, tokens, count, kind)
    pools = [make_pool(g, count, rank, n_in, o, ranks, scale=j != 1) for j, o in enumerate(outs)]
    bases = [normal(g, tokens, o) for o in outs]
    ys = lb.adapters_forward(x, ids, pools, bases=bases)
    assert lb.device_status() == lb.LB_OK
    check_forward(x, ids, pools, bases, ys, f"M={tokens}")
    # in place, and a second time: the same bits
    own = [b.clone() for b in bases]
    lb.adapters_forward(x, ids, pools, ys=own)
    again = lb.adapters_forward(x, ids, pools, bases=bases)
    for y, z, w in zip(ys, own, again):
        assert torch_().equal(y, z) and torch_().equal(y, w)


@pytest.mark.parametrize("tokens", [5, 150, 300])
def test_strides_and_what_lies_around(tokens):
    t = torch_()
    g = gen(5)
    n_in, n_out, count = 96, 160, 3
    wide = normal(g, tokens, n_in + 40)
    x = wide[:, 8:8 + n_in]
    ids = make_ids(g, tokens, count, "some")
    pool = make_pool(g, count, 16, n_in, n_out)
    base = normal(g, tokens, n_out + 24)
    y = t.full((tokens + 2, n_out + 16), 7.0, dtype=t.bfloat16, device="cuda")
    lb.adapters_forward(x, ids, [pool], bases=[base[:, :n_out]], ys=[y[1:-1, :n_out]])
    check_forward(x, ids, [pool], [base[:, :n_out]], [y[1:-1, :n_out]], "strided")
    assert bool((y[0] == 7).all()) and bool((y[-1] == 7).all()) and bool((y[:, n_out:] == 7).all())


@pytest.mark.parametrize("tokens", [6, 140, 400])
def test_infinities_stay_in_their_rows(tokens):
    """A token's infinities and NaNs, and those of a token without an adapter,
    leave the other tokens' results as they were, bit for bit."""
    t = torch_()
    g = gen(6)
    n_in, n_out, count = 256, 96, 3
    x = normal(g, tokens, n_in)
    ids = make_ids(g, tokens, count, "some")
    ids[1], ids[tokens - 2] = 0, -1
    pool = make_pool(g, count, 8, n_in, n_out)
    base = normal(g, tokens, n_out)
    clean = lb.adapters_forward(x, ids, [pool], bases=[base])[0]
    x[1, 7], x[tokens - 2, 3], x[tokens - 2, 9] = float("nan"), float("inf"), float("nan")
    base[3, 5] = float("inf")
    y = lb.adapters_forward(x, ids, [pool], bases=[base])[0]
    keep = t.ones_like(y, dtype=t.bool)
    keep[1] = False
    keep[3, 5] = False
    assert t.equal(y[keep], clean[keep])
    assert bool(y[1].isnan().all()) and bool(y[3, 5].isinf())


@pytest.mark.parametrize("tokens", [3, 130, 300])
def test_an_id_past_the_pool_counts_as_none_and_is_reported(tokens):
    t = torch_()
    g = gen(7)
    pool = make_pool(g, 2, 8, 64, 64)
    x, base = normal(g, tokens, 64), normal(g, tokens, 64)
    ids = make_ids(g, tokens, 2, "mixed")
    ids[tokens // 2] = 2
    ids[0] = 2 ** 31 - 1
    y = lb.adapters_forward(x, ids, [pool], bases=[base])[0]
    assert lb.device_status() == lb.LB_ERR_INVALID_ARGUMENT
    assert lb.device_status() == lb.LB_OK
    assert t.equal(y[0], base[0]) and t.equal(y[tokens // 2], base[tokens // 2])
    check_forward(x, ids, [pool], [base], [y], "past the pool")
    dy = normal(g, tokens, 64)
    out = lb.adapters_backward(x, dy, ids, pool, dx_base=base)
    assert lb.device_status() == lb.LB_ERR_INVALID_ARGUMENT
    assert t.equal(out["dx"][0], base[0])


@pytest.mark.parametrize("tokens", [4, 160])
def test_adapters_past_32_bit_offsets(tokens):
    """The last of 1024 adapters lies past 2^31 elements of its pool."""
    t = torch_()
    n_in, rank, count = 17408, 128, 1024
    assert (count - 1) * rank * n_in > 2 ** 31
    g = gen(8)
    a = t.empty((count, rank, n_in), dtype=t.bfloat16, device="cuda")
    b = t.empty((count, 64, rank), dtype=t.bfloat16, device="cuda")
    for i in (0, count - 1):
        a[i], b[i] = normal(g, rank, n_in, scale=n_in ** -0.5), normal(g, 64, rank)
    pool = lb.AdapterPool(a, b)
    x, base = normal(g, tokens, n_in), normal(g, tokens, 64)
    ids = t.full((tokens,), count - 1, dtype=t.int32, device="cuda")
    ids[0] = 0
    y = lb.adapters_forward(x, ids, [pool], bases=[base])[0]
    small = t.where(ids == 0, 0, 1).to(t.int32)
    exact, tol = ref.adapters(x, small, a[[0, count - 1]], b[[0, count - 1]], None, None, base)
    ref.within(y, exact, tol, "offsets")


@pytest.mark.parametrize("tokens", [16, 300])
def test_captured_call_replays_with_new_ids(tokens):
    t = torch_()
    g = gen(9)
    n_in, n_out, count = 128, 192, 4
    pool = make_pool(g, count, 16, n_in, n_out)
    x, base = normal(g, tokens, n_in), normal(g, tokens, n_out)
    ids = make_ids(g, tokens, count, "mixed")
    y = t.empty_like(base)
    lb.adapters_forward(x, ids, [pool], bases=[base], ys=[y])
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        lb.adapters_forward(x, ids, [pool], bases=[base], ys=[y])
    for kind in ("none", "one", "some"):
        ids.copy_(make_ids(g, tokens, count, kind))
        y.fill_(3.0)
        graph.replay()
        t.cuda.synchronize()
        check_forward(x, ids, [pool], [base], [y], kind)


@pytest.mark.parametrize("tokens", [20, 300])
def test_two_streams_with_their_own_workspaces(tokens):
    t = torch_()
    g = gen(10)
    pool = make_pool(g, 3, 16, 512, 512)
    x, base = normal(g, tokens, 512), normal(g, tokens, 512)
    ids = make_ids(g, tokens, 3, "some")
    want = lb.adapters_forward(x, ids, [pool], bases=[base])[0]
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in range(2)]
    got = [lb.adapters_forward(x, ids, [pool], bases=[base], stream=s)[0] for _ in range(8) for s in streams]
    t.cuda.synchronize()
    assert all(t.equal(y, want) for y in got)


BACKWARD = [  # tokens, n_in, n_out, rank, count, ids, ranks
    (1, 32, 32, 8, 1, "one", None),
    (2, 64, 96, 16, 2, "none", None),
    (5, 288, 160, 24, 4, "mixed", [24, 0, 5, 23]),
    (64, 256, 512, 64, 1, "one", None),
    (65, 544, 96, 8, 3, "runs", None),
    (127, 128, 128, 128, 2, "some", [128, 77]),
    (333, 1056, 800, 8, 3, "runs", [8, 5, 2]),
    (513, 512, 1024, 72, 1, "one", None),
    (1000, 256, 256, 32, 40, "mixed", None),
    (2500, 512, 768, 16, 2, "some", [16, 9]),
    (3000, 96, 64, 40, 1, "one", None),
]


@pytest.mark.parametrize("tokens,n_in,n_out,rank,count,kind,ranks", BACKWARD)
def test_backward_against_64_bits(tokens, n_in, n_out, rank, count, kind, ranks):
    t = torch_()
    g = gen(tokens * 17 + n_in)
    x, dy, base = normal(g, tokens, n_in), normal(g, tokens, n_out), normal(g, tokens, n_in)
    ids = make_ids(g, tokens, count, kind)
    pool = make_pool(g, count, rank, n_in, n_out, ranks)
    out = lb.adapters_backward(x, dy, ids, pool, dx_base=base)
    assert lb.device_status() == lb.LB_OK
    exact, tol = ref.adapters_backward(x, dy, ids, pool.a, pool.b, pool.scale, pool.ranks, base)
    for name, e, w in zip(("dx", "da", "db"), exact, tol):
        ref.within(out[name], e, w, f"M={tokens} {name}")
    # in place, without dx, and into memory that holds NaN: the same bits
    own = base.clone()
    da, db = t.full_like(out["da"], float("nan")), t.full_like(out["db"], float("nan"))
    ws = t.full((max(16, lb.adapters_backward_workspace_bytes(tokens, n_in, n_out, count, rank)),), 255, dtype=t.uint8,
                device="cuda")
    lb.adapters_backward(x, dy, ids, pool, dx=own, da=da, db=db, workspace=ws)
    bare = lb.adapters_backward(x, dy, ids, pool, want_dx=False)
    assert bare["dx"] is None
    assert t.equal(own, out["dx"])
    for k, v in (("da", da), ("db", db)):
        assert t.equal(v, out[k]) and t.equal(bare[k], out[k])


def test_backward_keeps_infinities_with_their_adapter():
    """NaN in one adapter's tokens, and in tokens without one, leaves the
    other adapters' gradients and the other rows of dx as they were."""
    t = torch_()
    g = gen(11)
    tokens, n = 300, 128
    x, dy, base = normal(g, tokens, n), normal(g, tokens, n), normal(g, tokens, n)
    ids = make_ids(g, tokens, 4, "some")
    ids[10], ids[11] = 1, -1
    pool = make_pool(g, 4, 16, n, n)
    clean = lb.adapters_backward(x, dy, ids, pool, dx_base=base)
    x[10, 3], x[11, 4], dy[10, 5], dy[11, 6] = (float("nan"),) * 4
    out = lb.adapters_backward(x, dy, ids, pool, dx_base=base)
    others = [0, 2, 3]
    assert t.equal(out["da"][others], clean["da"][others]) and t.equal(out["db"][others], clean["db"][others])
    rows = [m for m in range(tokens) if m != 10]
    assert t.equal(out["dx"][rows], clean["dx"][rows])
    assert bool(out["da"][1].isnan().any()) and bool(out["db"][1].isnan().any())


def test_no_tokens():
    t = torch_()
    g = gen(12)
    pool = make_pool(g, 3, 8, 64, 96)
    x, ids = normal(g, 0, 64), t.zeros(0, dtype=t.int32, device="cuda")
    y = lb.adapters_forward(x, ids, [pool], bases=[normal(g, 0, 96)])[0]
    assert y.shape == (0, 96)
    da, db = t.full((3, 8, 64), 5.0, device="cuda"), t.full((3, 96, 8), 5.0, device="cuda")
    lb.adapters_backward(x, normal(g, 0, 96), ids, pool, dx_base=normal(g, 0, 64), da=da, db=db)
    assert bool((da == 0).all()) and bool((db == 0).all())


def test_gradients_against_differences():
    """The kernels' gradients along a direction against central differences of
    the 64-bit forward form: L = sum(y weight)."""
    t = torch_()
    g = gen(13)
    tokens, n_in, n_out, rank, count = 150, 64, 96, 16, 3
    x, base, dy = normal(g, tokens, n_in), normal(g, tokens, n_out), normal(g, tokens, n_out)
    ids = make_ids(g, tokens, count, "some")
    pool = make_pool(g, count, rank, n_in, n_out)
    zero = t.zeros_like(x)
    out = lb.adapters_backward(x, dy, ids, pool, dx_base=zero)
    loss = lambda x, a, b: float((ref.adapters(x, ids, a, b, pool.scale, None, base)[0] * dy.double()).sum())
    args = [x.double(), pool.a.double(), pool.b.double()]
    for k, name in enumerate(("dx", "da", "db")):
        d = t.randn(args[k].shape, generator=g, device="cuda", dtype=t.float64)
        h = 1e-3
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + h * d, args[k] - h * d
        slope = (loss(*up) - loss(*dn)) / (2 * h)  # exact but for rounding: the form is linear in each argument
        terms = (out[name].double() * d).abs().sum()
        got = float((out[name].double() * d).sum())
        # each element of dx is rounded to bf16; da and db carry the split's 2^-16 (and fp32 sums)
        bound = (ref.U16 if name == "dx" else 2.0 ** -14) * float(terms) + 1e-6 * abs(slope)
        assert abs(got - slope) <= bound, (name, got, slope, bound)


@pytest.mark.parametrize("tokens", [1, 24, 200])
def test_the_layer_with_adapters(tokens):
    """LittleBitLinear and linear_backward with a pool give what the layer and
    the adapters' own calls give, bit for bit."""
    t = torch_()
    layer = synth.make_layer(256, 512, [64, 32], tokens, config_id=1301)
    paths = gu.device_paths(layer)
    x = gu.bf16_tensor(layer["x"])
    g = gen(14)
    pool = make_pool(g, 4, 16, 256, 512)
    ids = make_ids(g, tokens, 4, "some")
    y = lb.LittleBitLinear(paths[0], paths[1])(x, adapters=pool, ids=ids)
    plain = lb.linear_forward(x, paths[0], paths[1])
    assert t.equal(y, lb.adapters_forward(x, ids, [pool], bases=[plain])[0])
    dy = normal(g, tokens, 512)
    out = lb.linear_backward(x, dy, paths[0], paths[1], adapters=pool, ids=ids)
    bare = lb.linear_backward(x, dy, paths[0], paths[1])
    more = lb.adapters_backward(x, dy, ids, pool, dx_base=bare["dx"])
    assert t.equal(out["dx"], more["dx"]) and t.equal(out["da"], more["da"]) and t.equal(out["db"], more["db"])
    assert all(t.equal(out[k], bare[k]) for k in ("dh", "dg", "dl"))
