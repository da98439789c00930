"""lb_heads_norm_rotate and its backward pass on the GPU against their plain
64-bit forms (tests/operators_ref.py), whose bounds are derived there, and the
whole of an attention block's query and key inputs: sibling projections,
adapters, head norms and rotation, forward and backward."""
import pytest

import binarized_rank_linear_b200 as lb
from tests import gpu_util as gu
from tests import operators_ref as ref
from tests.test_gpu_adapters import gen, make_ids, make_pool, normal, torch_

pytestmark = pytest.mark.gpu

CASES = [  # tokens, heads, head_dim, rotary_dim, rotation, norms, first position
    (1, [40, 8], 128, 128, "halves", [True, True], 131071),
    (1, [1], 8, 8, "pairs", [False], -5),
    (2, [1, 1, 1, 1], 64, 64, "halves", [True, False, True, False], 0),
    (7, [5, 3], 80, 40, "halves", [True, True], 2 ** 31 - 8),
    (7, [5, 3], 80, 40, "pairs", [True, True], 1000000),
    (13, [4, 2], 256, 256, "pairs", [True, False], 77),
    (13, [3], 200, 64, "halves", [True], 77),
    (50, [32, 32], 128, 64, "pairs", [False, False], 0),
    (129, [14, 2], 64, 64, "halves", [True, True], 4000),
    (300, [2, 1], 96, 0, "halves", [True, True], 0),
    (1000, [1, 1], 128, 128, "halves", [True, True], 30000),
    (1500, [6, 2], 128, 96, "halves", [True, True], 0),
]


def make(tokens, heads, d, rd, rotation, norms, first, seed):
    t = torch_()
    g = gen(seed)
    freq = (1e6 ** (-t.arange(0, rd, 2, dtype=t.float64, device="cuda") / max(rd, 1))).float() if rd else None
    pos = (t.arange(tokens, device="cuda") + first).to(t.int32)
    xs = [normal(g, tokens, h * d, scale=2.0) for h in heads]
    ws = [normal(g, d) if n else None for n in norms]
    return g, lb.HeadRotation(d, freq, rotation, 1e-6), pos, xs, ws


@pytest.mark.parametrize("tokens,heads,d,rd,rotation,norms,first", CASES)
def test_forward_against_64_bits(tokens, heads, d, rd, rotation, norms, first):
    t = torch_()
    g, rot, pos, xs, ws = make(tokens, heads, d, rd, rotation, norms, first, tokens + d)
    outs = lb.heads_norm_rotate(xs, pos, rot, weights=ws)
    assert lb.device_status() == lb.LB_OK
    for j, (x, w, o) in enumerate(zip(xs, ws, outs)):
        exact, tol = ref.heads(x, pos, rot.inv_freq, rotation, w, rot.eps, d)
        ref.within(o, exact, tol, f"tensor {j}")
    own = [x.clone() for x in xs]
    lb.heads_norm_rotate(own, pos, rot, weights=ws, outs=own)
    assert all(t.equal(a, b) for a, b in zip(own, outs))


@pytest.mark.parametrize("tokens,heads,d,rd,rotation,norms,first", CASES)
def test_backward_against_64_bits(tokens, heads, d, rd, rotation, norms, first):
    t = torch_()
    g, rot, pos, xs, ws = make(tokens, heads, d, rd, rotation, norms, first, tokens + d)
    douts = [normal(g, *x.shape) for x in xs]
    got = lb.heads_norm_rotate_backward(xs, douts, pos, rot, weights=ws)
    assert lb.device_status() == lb.LB_OK
    for j, (x, dy, w, o) in enumerate(zip(xs, douts, ws, got)):
        (din, dw), (tx, tw) = ref.heads_backward(x, dy, pos, rot.inv_freq, rotation, w, rot.eps, d)
        ref.within(o["din"], din, tx, f"tensor {j} din")
        assert ("dweight" in o) == (w is not None)
        if w is not None:
            ref.within(o["dweight"], dw, tw, f"tensor {j} dweight")
    # over dout, and a second time: the same bits; without dweight the same din
    own = [dy.clone() for dy in douts]
    again = lb.heads_norm_rotate_backward(xs, own, pos, rot, weights=ws, dins=own)
    bare = lb.heads_norm_rotate_backward(xs, douts, pos, rot, weights=ws, want_dweight=False)
    for o, p, q in zip(got, again, bare):
        assert t.equal(o["din"], p["din"]) and t.equal(o["din"], q["din"]) and "dweight" not in q
        assert "dweight" not in o or t.equal(o["dweight"], p["dweight"])


def test_strides_and_what_lies_around():
    t = torch_()
    tokens, d = 37, 64
    g, rot, pos, _, ws = make(tokens, [3], d, d, "halves", [True], 9, 3)
    wide = normal(g, tokens, 5 * d)
    out = t.full((tokens, 3 * d + 24), 7.0, dtype=t.bfloat16, device="cuda")
    lb.heads_norm_rotate([wide[:, d:4 * d]], pos, rot, weights=ws, outs=[out[:, :3 * d]])
    exact, tol = ref.heads(wide[:, d:4 * d].contiguous(), pos, rot.inv_freq, "halves", ws[0], rot.eps, d)
    ref.within(out[:, :3 * d], exact, tol, "strided")
    assert bool((out[:, 3 * d:] == 7).all())


def test_infinities_and_zero_heads_stay_in_their_heads():
    t = torch_()
    tokens, d = 40, 128
    g, rot, pos, (x,), ws = make(tokens, [4], d, d, "halves", [True], 5, 4)
    clean = lb.heads_norm_rotate([x], pos, rot, weights=ws)[0]
    x[3, d + 5], x[4, 0] = float("nan"), float("inf")
    x[5, 2 * d:3 * d] = 0
    y = lb.heads_norm_rotate([x], pos, rot, weights=ws)[0].view(tokens, 4, d)
    keep = t.ones((tokens, 4), dtype=t.bool, device="cuda")
    keep[3, 1] = keep[4, 0] = keep[5, 2] = False
    assert t.equal(y[keep], clean.view(tokens, 4, d)[keep])
    assert bool(y[3, 1].isnan().all()) and bool((y[5, 2] == 0).all())


def test_captured_call_replays_at_new_positions():
    t = torch_()
    g, rot, pos, xs, ws = make(24, [4, 2], 128, 128, "halves", [True, True], 0, 5)
    outs = [t.empty_like(x) for x in xs]
    lb.heads_norm_rotate(xs, pos, rot, weights=ws, outs=outs)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        lb.heads_norm_rotate(xs, pos, rot, weights=ws, outs=outs)
    for first in (100, 99999):
        pos.copy_(t.arange(24, device="cuda") + first)
        graph.replay()
        t.cuda.synchronize()
        for x, w, o in zip(xs, ws, outs):
            ref.within(o, *ref.heads(x, pos, rot.inv_freq, "halves", w, rot.eps, 128), f"from {first}")


def test_no_tokens():
    t = torch_()
    g, rot, pos, xs, ws = make(0, [4], 64, 64, "halves", [True], 0, 6)
    assert lb.heads_norm_rotate(xs, pos, rot, weights=ws)[0].shape == (0, 256)
    out = lb.heads_norm_rotate_backward(xs, xs, pos, rot, weights=ws)
    t.cuda.synchronize()
    assert bool((out[0]["dweight"] == 0).all())


def test_gradients_against_differences():
    t = torch_()
    d = 64
    g, rot, pos, (x,), (w,) = make(30, [3], d, 32, "pairs", [True], 1000, 7)
    dout = normal(g, *x.shape)
    out = lb.heads_norm_rotate_backward([x], [dout], pos, rot, weights=[w])[0]
    loss = lambda x, w: float((ref.heads(x, pos, rot.inv_freq, "pairs", w, rot.eps, d)[0] * dout.double()).sum())
    args = [x.double(), w.double()]
    for k, name in enumerate(("din", "dweight")):
        v = t.randn(args[k].shape, generator=g, device="cuda", dtype=t.float64)
        h = 1e-5
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + h * v, args[k] - h * v
        slope = (loss(*up) - loss(*dn)) / (2 * h)  # off by h^2 of a third derivative of order one, and 2^-52 / h
        got = out[name].double() * v
        bound = (ref.U16 if name == "din" else 2.0 ** -14) * float(got.abs().sum()) + 1e-6 * float(got.abs().sum())
        assert abs(float(got.sum()) - slope) <= bound, (name, float(got.sum()), slope, bound)


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_attention_inputs_together(tokens):
    """Queries, keys and values as a block computes them in one call: the
    sibling projections, each token's adapters, the norms and rotation of
    queries and keys; then the way back through the rotation, the adapters and
    the layers.  Each step against its 64-bit form on the step before."""
    from tests.test_gpu_siblings import group_layers
    t = torch_()
    n_in, d = 256, 64
    layers = group_layers([(512, [64, 32]), (128, [32]), (128, [32])], n_in, tokens, 1310)
    x = gu.bf16_tensor(layers[0]["x"])
    dev = [gu.device_paths(lay) for lay in layers]
    pairs = [(p[0], p[1] if len(p) > 1 else None) for p in dev]
    g, rot, pos, _, ws = make(tokens, [8, 2], d, d, "halves", [True, True], 500, 8)
    pools = [make_pool(g, 3, 8, n_in, 512), None, make_pool(g, 3, 8, n_in, 128)]
    ids = make_ids(g, tokens, 3, "some")
    q, k, v = lb.linear_forward_siblings(x, pairs, adapters=pools, ids=ids, rotation=rot, positions=pos,
                                         rotate={0: ws[0], 1: ws[1]})
    plain = lb.linear_forward_siblings(x, pairs)
    q0, v0 = lb.adapters_forward(x, ids, [pools[0], pools[2]], bases=[plain[0], plain[2]])
    for y, base, pool in ((q0, plain[0], pools[0]), (v0, plain[2], pools[2])):
        ref.within(y, *ref.adapters(x, ids, pool.a, pool.b, pool.scale, pool.ranks, base), "adapters")
    assert t.equal(v, v0)
    for y, before, w in ((q, q0, ws[0]), (k, plain[1], ws[1])):
        ref.within(y, *ref.heads(before, pos, rot.inv_freq, "halves", w, rot.eps, d), "heads")
    # back: dq -> the projection's output -> adapters and x
    dq = normal(g, tokens, 512)
    back = lb.heads_norm_rotate_backward([q0], [dq], pos, rot, weights=[ws[0]])[0]
    ref.within(back["din"], *[z[0] for z in ref.heads_backward(q0, dq, pos, rot.inv_freq, "halves", ws[0], rot.eps, d)])
    out = lb.linear_backward(x, back["din"], *pairs[0], adapters=pools[0], ids=ids)
    bare = lb.linear_backward(x, back["din"], *pairs[0])
    exact, tol = ref.adapters_backward(x, back["din"], ids, pools[0].a, pools[0].b, pools[0].scale, None, bare["dx"])
    for name, e, w in zip(("dx", "da", "db"), exact, tol):
        ref.within(out[name], e, w, name)
    assert lb.device_status() == lb.LB_OK


def test_the_most_heads_in_the_narrowest_chunks():
    """4096 heads of 136: 12 to a chunk, 342 chunks, and dweight from all of them."""
    t = torch_()
    tokens, d = 7, 136
    g, rot, pos, xs, ws = make(tokens, [4000, 96], d, 64, "halves", [True, True], 3, 9)
    douts = [normal(g, *x.shape) for x in xs]
    outs = lb.heads_norm_rotate(xs, pos, rot, weights=ws)
    got = lb.heads_norm_rotate_backward(xs, douts, pos, rot, weights=ws)
    assert lb.device_status() == lb.LB_OK
    for x, dy, w, y, o in zip(xs, douts, ws, outs, got):
        ref.within(y, *ref.heads(x, pos, rot.inv_freq, "halves", w, rot.eps, d), "out")
        (din, dw), (tx, tw) = ref.heads_backward(x, dy, pos, rot.inv_freq, "halves", w, rot.eps, d)
        ref.within(o["din"], din, tx, "din")
        ref.within(o["dweight"], dw, tw, "dweight")
