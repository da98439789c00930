"""Adapters and head norms/rotation at the borders of their kernels: the token
counts where another kernel takes over, groups of unlike ranks, orders that
break every run, long strides, captured calls, workspaces that captured graphs
share.  Against the 64-bit forms of tests/operators_ref.py."""
import pytest

import binarized_rank_linear_b200 as lb
from tests import operators_ref as ref
from tests.test_gpu_adapters import check_forward, gen, make_ids, make_pool, normal, torch_
from tests.test_gpu_heads import make

pytestmark = pytest.mark.gpu

FORWARD = [  # tokens, n_in, outputs, ranks of the pools, count, ids, ranks of the adapters
    (16, 1024, [256], [32], 1, "one", None),             # one full group
    (17, 1056, [288], [40], 1, "one", [33]),             # a group of one token behind a full one
    (33, 2080, [32, 544], [8, 128], 3, "mixed", None),   # pools of unlike ranks
    (250, 96, [64], [8], 600, "mixed", None),            # nearly as many groups as tokens
    (255, 32, [32], [128], 2, "some", [128, 3]),
    (256, 512, [256, 96, 32, 800], [64, 8, 72, 16], 128, "mixed", None),
    (256, 16384, [64], [16], 5, "mixed", [16, 0, 7, 8, 9]),
    (257, 512, [256, 96, 32, 800], [64, 8, 72, 16], 128, "mixed", None),
    (300, 96, [64], [8], 1024, "mixed", None),
    (416, 160, [96], [24], 6, "some", [24, 0, 1, 8, 23, 9]),
    (417, 160, [96], [24], 6, "some", [24, 0, 1, 8, 23, 9]),
    (511, 288, [64, 160], [32, 8], 16, "mixed", None),
    (512, 64, [288], [128], 64, "runs", None),
    (512, 1056, [32], [8], 8, "one", None),
    (513, 1056, [32], [8], 8, "one", None),
    (768, 96, [64, 32], [16, 128], 32, "mixed", [16] * 16 + [3] * 16),
    (769, 96, [64, 32], [16, 128], 32, "mixed", [16] * 16 + [3] * 16),
    (2047, 64, [288], [24], 1024, "some", None),
    (2048, 1056, [32], [8], 86, "one", None),           # a warp's tokens all of one adapter
    (2048, 64, [32, 64, 96, 32], [8, 16, 72, 128], 900, "runs", None),
    (2049, 64, [32], [8], 1000, "mixed", None),
    (385, 544, [160, 96], [128, 24], 3, "none", None),
    (600, 128, [96], [16], 4, "mixed", [0, 16, 0, 3]),
    (4096, 256, [160], [128], 5, "mixed", None),
    (9000, 64, [96, 32], [8, 72], 3, "mixed", [8, 5, 3]),  # more than the plan holds in shared memory
    (20001, 32, [32], [8], 700, "some", None),
    (1 << 20, 32, [32], [8], 1024, "some", None),  # the most tokens and adapters
]


@pytest.mark.parametrize("tokens,n_in,outs,pool_ranks,count,kind,ranks", FORWARD)
def test_adapters_forward_at_its_borders(tokens, n_in, outs, pool_ranks, count, kind, ranks):
    g = gen(tokens * 7 + n_in)
    x = normal(g, tokens, n_in)
    ids = make_ids(g, tokens, count, kind)
    pools = [make_pool(g, count, r, n_in, o, ranks, scale=j % 2 == 0) for j, (o, r) in enumerate(zip(outs, pool_ranks))]
    bases = [normal(g, tokens, o) for o in outs]
    ys = lb.adapters_forward(x, ids, pools, bases=bases)
    assert lb.device_status() == lb.LB_OK
    check_forward(x, ids, pools, bases, ys, f"M={tokens}")
    own = [b.clone() for b in bases]
    lb.adapters_forward(x, ids, pools, ys=own)
    assert all(torch_().equal(y, z) for y, z in zip(ys, own))


BACKWARD = [
    (256, 96, 64, 8, 600, "mixed", None),
    (700, 256, 160, 128, 5, "mixed", [128, 65, 64, 1, 0]),
    (4097, 64, 96, 72, 2, "mixed", None),
    (9000, 96, 64, 16, 7, "some", [16, 1, 2, 3, 0, 15, 8]),
]


@pytest.mark.parametrize("tokens,n_in,n_out,rank,count,kind,ranks", BACKWARD)
def test_adapters_backward_at_its_borders(tokens, n_in, n_out, rank, count, kind, ranks):
    g = gen(tokens * 19 + n_in)
    x, dy, base = normal(g, tokens, n_in), normal(g, tokens, n_out), normal(g, tokens, n_in)
    ids = make_ids(g, tokens, count, kind)
    pool = make_pool(g, count, rank, n_in, n_out, ranks)
    out = lb.adapters_backward(x, dy, ids, pool, dx_base=base)
    assert lb.device_status() == lb.LB_OK
    exact, tol = ref.adapters_backward(x, dy, ids, pool.a, pool.b, pool.scale, pool.ranks, base)
    for name, e, w in zip(("dx", "da", "db"), exact, tol):
        ref.within(out[name], e, w, f"M={tokens} {name}")


@pytest.mark.parametrize("tokens", [4, 200, 300])
def test_long_strides(tokens):
    """Rows so far apart that the last lies past 2^31 elements."""
    t = torch_()
    g = gen(31)
    ld = ((2 ** 31 // (tokens - 1)) // 8 + 1) * 8
    ld = min(ld, 2 ** 30)
    n_in, n_out, d = 64, 128, 64
    store = t.empty((tokens - 1) * ld + 1024, dtype=t.bfloat16, device="cuda")
    wide = store.as_strided((tokens, n_in), (ld, 1))
    wide.copy_(normal(g, tokens, n_in))
    y = store.as_strided((tokens, n_out), (ld, 1), 512)
    base = normal(g, tokens, n_out)
    ids, pool = make_ids(g, tokens, 3, "some"), make_pool(g, 3, 8, n_in, n_out)
    lb.adapters_forward(wide, ids, [pool], bases=[base], ys=[y])
    check_forward(wide.contiguous(), ids, [pool], [base], [y], "far rows")
    near = lb.adapters_backward(wide.contiguous(), y.contiguous(), ids, pool, dx_base=wide.contiguous())
    far = lb.adapters_backward(wide, y, ids, pool, dx_base=wide)
    assert all(t.equal(near[k], far[k]) for k in near)
    _, rot, pos, _, ws = make(tokens, [1], d, d, "halves", [True], 3, 32)
    want = lb.heads_norm_rotate([wide.contiguous()], pos, rot, weights=ws)[0]
    grad = lb.heads_norm_rotate_backward([wide], [want], pos, rot, weights=ws)[0]
    again = lb.heads_norm_rotate_backward([wide.contiguous()], [want], pos, rot, weights=ws)[0]
    assert all(t.equal(grad[k], again[k]) for k in grad)
    lb.heads_norm_rotate([wide], pos, rot, weights=ws, outs=[wide])
    assert t.equal(wide, want)


def test_a_pool_past_32_bit_offsets():
    """The last of 1024 adapters lies past 2^31 elements of its pool, and of
    its gradient; every other adapter's gradient is zero."""
    t = torch_()
    n_in, rank, count, tokens = 17408, 128, 1024, 300
    g = gen(33)
    a = t.zeros((count, rank, n_in), dtype=t.bfloat16, device="cuda")
    b = t.zeros((count, 64, rank), dtype=t.bfloat16, device="cuda")
    used = [0, count - 1]
    for i in used:
        a[i], b[i] = normal(g, rank, n_in, scale=n_in ** -0.5), normal(g, 64, rank)
    pool = lb.AdapterPool(a, b)
    x, base, dy = normal(g, tokens, n_in), normal(g, tokens, 64), normal(g, tokens, 64)
    ids = t.full((tokens,), count - 1, dtype=t.int32, device="cuda")
    ids[::3] = 0
    small = t.where(ids == 0, 0, 1).to(t.int32)
    y = lb.adapters_forward(x, ids, [pool], bases=[base])[0]
    ref.within(y, *ref.adapters(x, small, a[used], b[used], None, None, base), "offsets")
    out = lb.adapters_backward(x, dy, ids, pool, dx_base=x)
    exact, tol = ref.adapters_backward(x, dy, small, a[used], b[used], None, None, x)
    ref.within(out["dx"], exact[0], tol[0], "dx")
    ref.within(out["da"][used], exact[1], tol[1], "da")
    ref.within(out["db"][used], exact[2], tol[2], "db")
    assert not bool(out["da"][1:-1].any()) and not bool(out["db"][1:-1].any())


@pytest.mark.parametrize("tokens", [30, 400])
def test_captured_passes_share_a_workspace(tokens):
    """Two graphs over one workspace, each a forward and a backward pass,
    replayed in turn with new ids: what the calls give outside of a graph."""
    t = torch_()
    g = gen(34)
    n_in, n_out, count, d = 128, 256, 5, 64
    pool = make_pool(g, count, 16, n_in, n_out, [16, 9, 0, 1, 16])
    x, dy, base = normal(g, tokens, n_in), normal(g, tokens, n_out), normal(g, tokens, n_out)
    _, rot, pos, _, ws = make(tokens, [n_out // d], d, d, "pairs", [True], 11, 35)
    size = max(lb.adapters_workspace_bytes(tokens, n_in, count, (16,)),
               lb.adapters_backward_workspace_bytes(tokens, n_in, n_out, count, 16))
    ws_bytes = t.empty(size, dtype=t.uint8, device="cuda")

    def passes(ids):
        y = lb.adapters_forward(x, ids, [pool], bases=[base], workspace=ws_bytes)[0]
        q = lb.heads_norm_rotate([y], pos, rot, weights=ws)[0]
        back = lb.heads_norm_rotate_backward([y], [dy], pos, rot, weights=ws)[0]
        out = lb.adapters_backward(x, back["din"], ids, pool, dx_base=x, workspace=ws_bytes)
        return [q, back["din"], back["dweight"], out["dx"], out["da"], out["db"]]

    ids = [make_ids(g, tokens, count, k) for k in ("mixed", "runs")]
    passes(ids[0])
    t.cuda.synchronize()
    graphs, outs = [], []
    for k in range(2):
        graphs.append(t.cuda.CUDAGraph())
        with t.cuda.graph(graphs[k]):
            outs.append(passes(ids[k]))
    for kind in ("some", "one", "none"):
        for i in ids:
            i.copy_(make_ids(g, tokens, count, kind))
        for _ in range(3):
            for k in range(2):
                graphs[k].replay()
        t.cuda.synchronize()
        got = [[v.clone() for v in o] for o in outs]
        for k in range(2):
            assert all(t.equal(a, b) for a, b in zip(got[k], passes(ids[k]))), (kind, k)
    assert lb.device_status() == lb.LB_OK


@pytest.mark.parametrize("tokens", [20, 400])
def test_backward_on_two_streams(tokens):
    t = torch_()
    g = gen(36)
    n_in, n_out, d = 256, 512, 128
    pool = make_pool(g, 3, 16, n_in, n_out)
    x, dy = normal(g, tokens, n_in), normal(g, tokens, n_out)
    ids = make_ids(g, tokens, 3, "some")
    _, rot, pos, _, ws = make(tokens, [n_out // d], d, d, "halves", [True], 11, 37)

    def both(stream=None):
        out = lb.adapters_backward(x, dy, ids, pool, dx_base=x, stream=stream)
        return [*out.values(), *lb.heads_norm_rotate_backward([dy], [dy], pos, rot, weights=ws, stream=stream)[0].values()]

    want = both()
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in range(2)]
    got = [both(s) for _ in range(6) for s in streams]
    t.cuda.synchronize()
    assert all(t.equal(a, b) for o in got for a, b in zip(o, want))


HEADS = [  # tokens, heads, head_dim, rotary_dim, rotation, norms, first position
    (1, [128, 8], 128, 128, "halves", [True, True], 7),
    (3, [100], 64, 64, "halves", [True], 2 ** 31 - 3),
    (5, [49, 1], 256, 128, "pairs", [True, True], -9),
    (2, [300], 8, 8, "halves", [True], 1),
    (3000, [1], 8, 8, "pairs", [True], 0),
    (2049, [1, 2], 24, 16, "halves", [True, True], 0),
    (4001, [3], 64, 32, "halves", [True], 0),
    (149, [97, 3], 48, 48, "pairs", [False, True], 5),
]


@pytest.mark.parametrize("tokens,heads,d,rd,rotation,norms,first", HEADS)
def test_heads_at_their_borders(tokens, heads, d, rd, rotation, norms, first):
    t = torch_()
    g, rot, pos, xs, ws = make(tokens, heads, d, rd, rotation, norms, first, tokens + d)
    pos = pos[t.randint(0, tokens, (tokens,), generator=g, device="cuda")]  # any order, and one position twice
    outs = lb.heads_norm_rotate(xs, pos, rot, weights=ws)
    douts = [normal(g, *x.shape) for x in xs]
    got = lb.heads_norm_rotate_backward(xs, douts, pos, rot, weights=ws)
    assert lb.device_status() == lb.LB_OK
    for j, (x, dy, w, y, o) in enumerate(zip(xs, douts, ws, outs, got)):
        ref.within(y, *ref.heads(x, pos, rot.inv_freq, rotation, w, rot.eps, d), f"tensor {j}")
        (din, dw), (tx, tw) = ref.heads_backward(x, dy, pos, rot.inv_freq, rotation, w, rot.eps, d)
        ref.within(o["din"], din, tx, f"tensor {j} din")
        if w is not None:
            ref.within(o["dweight"], dw, tw, f"tensor {j} dweight")


def tiles_in_turn(segments, count):
    """ids whose tiles and K-blocks come now as consecutive tokens, now not:
    segments of 128 tokens of adapter 0, of 256 of 0 and 1 by turns, of 128 of
    the last adapter, and of 64 of adapter 0 with a token without one inside."""
    ids = []
    for k in segments:
        ids += {"run": [0] * 128, "turns": [0, 1] * 128, "last": [count - 1] * 128, "broken": [0] * 40 + [-1] + [0] * 23}[k]
    return torch_().tensor(ids, dtype=torch_().int32, device="cuda")


@pytest.mark.parametrize("rank", [16, 64, 128])
@pytest.mark.parametrize("segments", [
    ["run", "turns"] * 5, ["run"] * 9 + ["turns"] + ["run"] * 6, ["turns", "last"] * 4 + ["broken"],
    ["run", "broken", "broken", "turns", "run", "last", "last"] * 2, ["last"] * 8 + ["turns"] + ["last"] * 8,
])
def test_boxes_and_copies_in_turn(segments, rank):
    """The loaders of copied rows leave boxes alone and come back behind them:
    every gradient, and the same bits each time."""
    g = gen(41)
    n_in, n_out, count = 544, 160, 3
    ids = tiles_in_turn(segments, count)
    tokens = len(ids)
    x, dy, base = normal(g, tokens, n_in), normal(g, tokens, n_out), normal(g, tokens, n_in)
    pool = make_pool(g, count, rank, n_in, n_out)
    out = lb.adapters_backward(x, dy, ids, pool, dx_base=base)
    exact, tol = ref.adapters_backward(x, dy, ids, pool.a, pool.b, pool.scale, pool.ranks, base)
    for name, e, w in zip(("dx", "da", "db"), exact, tol):
        ref.within(out[name], e, w, name)
    for _ in range(30):
        again = lb.adapters_backward(x, dy, ids, pool, dx_base=base)
        assert all(torch_().equal(again[k], out[k]) for k in out)
    assert lb.device_status() == lb.LB_OK


@pytest.mark.parametrize("rank", [16, 64, 128])
@pytest.mark.parametrize("segments", [
    ["last"] * 8 + ["run"] + ["last"] * 8, ["turns", "last"] * 4 + ["broken"], ["last", "run"] * 5, ["last"] * 9,
    ["broken", "last", "broken", "turns", "last", "last"] * 2,
])
def test_copied_and_added_tiles_in_turn(segments, rank):
    """Where base is only copied (the last adapter has rank 0), tile after tile
    and between tiles with products: every row, and the same bits each time."""
    g = gen(42)
    n_in, outs, count = 160, [1056, 544], 3
    ids = tiles_in_turn(segments, count)
    tokens = len(ids)
    x, dy = normal(g, tokens, n_in), normal(g, tokens, outs[0])
    bases = [normal(g, tokens, o) for o in outs]
    pools = [make_pool(g, count, rank, n_in, o, [rank, rank - 3, 0]) for o in outs]
    ys = lb.adapters_forward(x, ids, pools, bases=bases)
    check_forward(x, ids, pools, bases, ys, "copied and added")
    out = lb.adapters_backward(x, dy, ids, pools[0], dx_base=x)
    exact, tol = ref.adapters_backward(x, dy, ids, pools[0].a, pools[0].b, pools[0].scale, pools[0].ranks, x)
    for name, e, w in zip(("dx", "da", "db"), exact, tol):
        ref.within(out[name], e, w, name)
    for _ in range(30):
        again = lb.adapters_forward(x, ids, pools, bases=bases)
        assert all(torch_().equal(a, b) for a, b in zip(again, ys))
    assert lb.device_status() == lb.LB_OK


@pytest.mark.parametrize("tokens", [10, 300])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_latents_between_the_largest_bf16_and_the_largest_fp32(tokens, sign):
    """A_i x (and B_i^T dy) of (255/128)^2 2^126 + 3 2^119 = 3.99224853515625
    2^126: finite in fp32 (24 bits hold it), but past the middle between the
    largest bf16, 3.984375 2^126, and 2^128."""
    t = torch_()
    n, rank = 32, 8
    big, latent = 255 / 128 * 2.0 ** 63, 3.99224853515625 * 2.0 ** 126
    bf16 = lambda *shape: t.zeros(shape, dtype=t.bfloat16, device="cuda")
    x, a, b, base = bf16(tokens, n), bf16(1, rank, n), bf16(1, n, rank), bf16(tokens, n)
    x[:, 0], x[:, 1] = big, 2.0 ** 60
    a[0, 0, 0], a[0, 0, 1] = sign * big, sign * 3 * 2.0 ** 59
    b[0, :, 0] = 2.0 ** -100
    ids = t.zeros(tokens, dtype=t.int32, device="cuda")
    pool = lb.AdapterPool(a, b)
    y = lb.adapters_forward(x, ids, [pool], bases=[base])[0]
    assert bool((y.double() == sign * 4.0 * 2.0 ** 26).all())  # 3.99224853515625 in bf16
    # db = dy v of one token with dy = 2^-100: exactly the latent over 2^100; the others' dy is zero
    dy = bf16(tokens, n)
    dy[0] = 2.0 ** -100
    db = lb.adapters_backward(x, dy, ids, pool, want_dx=False)["db"]
    assert bool((db[0, :, 0].double() == sign * latent * 2.0 ** -100).all())
    # u = B^T dy of the same size: da = u x and dx = A^T u
    pool = lb.AdapterPool(b.transpose(1, 2).contiguous(), a.transpose(1, 2).contiguous())
    small = bf16(tokens, n)
    small[0, 0] = 2.0 ** -100
    out = lb.adapters_backward(small, x, ids, pool, dx_base=base)
    assert bool((out["da"][0, 0, 0].double() == sign * latent * 2.0 ** -100).all())
    assert bool((out["dx"].double() == sign * 4.0 * 2.0 ** 26).all())
    assert lb.device_status() == lb.LB_OK


@pytest.mark.parametrize("tokens,n_in,n_out,rank", [(3, 1 << 20, 64, 16), (3, 64, 1 << 20, 128), (200, 1 << 20, 64, 8),
                                                    (200, 64, 1 << 20, 8)])
def test_the_widest_rows(tokens, n_in, n_out, rank):
    g = gen(tokens + rank)
    x, dy = normal(g, tokens, n_in), normal(g, tokens, n_out)
    ids, pool = make_ids(g, tokens, 2, "some"), make_pool(g, 1, rank, n_in, n_out)
    ids[ids == 1] = -1
    y = lb.adapters_forward(x, ids, [pool], bases=[dy])[0]
    check_forward(x, ids, [pool], [dy], [y], "wide")
    out = lb.adapters_backward(x, dy, ids, pool, dx_base=x)
    assert lb.device_status() == lb.LB_OK
    exact, tol = ref.adapters_backward(x, dy, ids, pool.a, pool.b, pool.scale, None, x)
    for name, e, w in zip(("dx", "da", "db"), exact, tol):
        ref.within(out[name], e, w, name)
