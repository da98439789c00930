"""The adapters calls where fp32 leaves nothing to chance: whole numbers whose
sums stay below 2^24 in any order, and latents that need all 24 bits.  What
arrives has to be equal, bit for bit, so that a lost part of a split or a few
lost bits of a sum show at any size."""
import pytest

import binarized_rank_linear_b200 as lb
from tests.test_gpu_adapters import gen, make_ids, torch_

pytestmark = pytest.mark.gpu


def whole(g, *shape, most):
    """Whole numbers from -most to most, in bf16 (exact up to 256)."""
    t = torch_()
    return t.randint(-most, most + 1, shape, generator=g, device="cuda").to(t.bfloat16)


def exact_forward(x, ids, pool, base):
    """In 64 bits; whole numbers, and scales that are powers of two, are exact there."""
    y = base.double().clone()
    for i in range(pool.a.shape[0]):
        m = ids == i
        y[m] += float(pool.scale[i]) * (x[m].double() @ pool.a[i].double().t()) @ pool.b[i].double().t()
    return y.to(torch_().bfloat16)  # rounded once, to nearest even


def make(g, count, rank, n_in, n_out, a, b):
    t = torch_()
    scale = 2.0 ** t.randint(-2, 1, (count,), generator=g, device="cuda").float()
    return lb.AdapterPool(whole(g, count, rank, n_in, most=a), whole(g, count, n_out, rank, most=b), scale)


# tokens, n_in, outputs, rank, count, ids, most in a.  |v| <= n_in a < 2^16, which two bf16 parts hold (8 bits each and
# the sign of the second), and y in units of its scale, 1/4 or more, is at most 4 * 3 + rank n_in a < 2^24.
FORWARD = [
    (1, 4096, [256], 16, 3, "one", 8), (7, 5120, [96, 288], 128, 2, "mixed", 8), (40, 16384, [64], 64, 5, "some", 3),
    (100, 1024, [544], 32, 16, "mixed", 63), (200, 4096, [128], 128, 1, "one", 15), (513, 5120, [160], 64, 4, "runs", 8),
    (1013, 4096, [288], 40, 5, "some", 15), (2048, 512, [64], 8, 80, "mixed", 100), (9001, 1056, [96], 72, 3, "mixed", 30),
]


@pytest.mark.parametrize("tokens,n_in,outs,rank,count,kind,most", FORWARD)
def test_whole_numbers_forward(tokens, n_in, outs, rank, count, kind, most):
    t = torch_()
    assert n_in * most < 2 ** 16 and rank * n_in * most + 4 * 3 < 2 ** 24
    g = gen(tokens + n_in)
    x = (t.randint(0, 2, (tokens, n_in), generator=g, device="cuda") * 2 - 1).to(t.bfloat16)
    ids = make_ids(g, tokens, count, kind)
    pools = [make(g, count, rank, n_in, o, most, 1) for o in outs]
    bases = [whole(g, tokens, o, most=3) for o in outs]
    ys = lb.adapters_forward(x, ids, pools, bases=bases)
    for pool, base, y in zip(pools, bases, ys):
        assert t.equal(y, exact_forward(x, ids, pool, base))


# tokens, n_in, n_out, rank, count, ids, most in a, in b, in dy; x is -1 or 1.  With n tokens of an adapter at most
# (all of them here): |u| <= n_out b dy, |da| <= n |u|, |v| <= n_in a, |db| <= n dy |v|, |dx| <= 4 * 3 + rank a |u| in units of
# the scale, all below 2^24; u into dx is two bf16 parts: |u| < 2^16.
BACKWARD = [
    (1, 64, 96, 16, 1, "one", 60, 20, 8), (5, 288, 160, 24, 4, "mixed", 20, 20, 8), (40, 4096, 512, 16, 3, "some", 4, 4, 4),
    (128, 1024, 1024, 8, 1, "one", 16, 8, 4), (333, 1056, 800, 8, 3, "runs", 8, 8, 4), (700, 256, 160, 128, 5, "mixed", 3, 8, 8),
    (1500, 256, 512, 64, 2, "runs", 8, 4, 4), (9001, 96, 64, 16, 3, "mixed", 4, 4, 4),
]


@pytest.mark.parametrize("tokens,n_in,n_out,rank,count,kind,a,b,d", BACKWARD)
def test_whole_numbers_backward(tokens, n_in, n_out, rank, count, kind, a, b, d):
    t = torch_()
    u, v = n_out * b * d, n_in * a
    assert u < 2 ** 16 and max(tokens * u, tokens * d * v, rank * a * u + 4 * 3) < 2 ** 24
    g = gen(tokens * 3 + n_in)
    x = (t.randint(0, 2, (tokens, n_in), generator=g, device="cuda") * 2 - 1).to(t.bfloat16)
    dy, base = whole(g, tokens, n_out, most=d), whole(g, tokens, n_in, most=3)
    ids = make_ids(g, tokens, count, kind)
    pool = make(g, count, rank, n_in, n_out, a, b)
    out = lb.adapters_backward(x, dy, ids, pool, dx_base=base)
    dx = base.double().clone()
    for i in range(count):
        m = ids == i
        s, ai, bi = float(pool.scale[i]), pool.a[i].double(), pool.b[i].double()
        ui = s * (dy[m].double() @ bi)
        dx[m] += ui @ ai
        assert t.equal(out["da"][i].double(), ui.t() @ x[m].double())
        assert t.equal(out["db"][i].double(), s * dy[m].double().t() @ (x[m].double() @ ai.t()))
    assert t.equal(out["dx"], dx.to(t.bfloat16))


def latents(g, count, rank):
    """Values of 24 bits, the first and the last of them set, and the three bf16 whose sum each is."""
    t = torch_()
    n = t.randint(0, 2 ** 22, (count, rank), generator=g, device="cuda").double() * 2 + 1 + 2 ** 23
    n = n * (t.randint(0, 2, (count, rank), generator=g, device="cuda") * 2 - 1) * 2.0 ** -23
    parts, left = [], n.clone()
    for _ in range(3):
        parts.append(left.to(t.bfloat16))
        left = left - parts[-1].double()
    assert not bool(left.any())
    return n, parts


@pytest.mark.parametrize("rank", [8, 40, 128])
@pytest.mark.parametrize("tokens", [12, 300, 9000])
def test_latents_of_24_bits_reach_the_gradients(tokens, rank):
    """u and v that need all of fp32: u from three elements of dy that are 1
    against rows of B that sum up to it, v likewise, met by powers of two of
    which each column of x or dy has one not zero (but for those three, which
    have one for every token of an adapter: a power of two of them)."""
    t = torch_()
    g = gen(71 + tokens + rank)
    count, n_in, n_out, each = 5, 160, 96, 4
    u, ub = latents(g, count, rank)
    v, va = latents(g, count, rank)
    a, b = (t.zeros(s, dtype=t.bfloat16, device="cuda") for s in ((count, rank, n_in), (count, n_out, rank)))
    for k in range(3):
        a[:, :, k], b[:, k, :] = va[k], ub[k]
    ids = t.full((tokens,), -1, dtype=t.int32, device="cuda")
    where = t.randperm(tokens, generator=g, device="cuda")[:min(tokens, count * each) // count * count]
    ids[where] = (t.arange(len(where), device="cuda") % count).to(t.int32)
    n = len(where) // count
    n = 1 << (n.bit_length() - 1)  # tokens of each adapter: 1, 2 or 4
    for i in range(count):
        ids[t.nonzero(ids == i)[n:, 0]] = -1

    def powers(cols):
        z = t.zeros((tokens, cols), dtype=t.float64, device="cuda")
        for i in range(count):
            m = t.nonzero(ids == i)[:, 0]
            owner = m[t.randint(0, n, (cols,), generator=g, device="cuda")]
            p = 2.0 ** t.randint(-30, 31, (cols,), generator=g, device="cuda").double()
            z[owner, t.arange(cols, device="cuda")] = p * (t.randint(0, 2, (cols,), generator=g, device="cuda") * 2 - 1)
            z[m, :3] = 1
        return z.to(t.bfloat16)

    x, dy = powers(n_in), powers(n_out)
    # A and B are zero in the other columns, so u and v are what they were made to be
    out = lb.adapters_backward(x, dy, ids, lb.AdapterPool(a, b), want_dx=False)
    for i in range(count):
        m = ids == i
        assert t.equal(out["da"][i].double(), u[i][:, None] * x[m].double().sum(0)[None, :])
        assert t.equal(out["db"][i].double(), dy[m].double().sum(0)[:, None] * v[i][None, :])


@pytest.mark.parametrize("tokens", [1, 16, 100, 176, 177, 1000])
def test_latents_of_24_bits_reach_small_batches(tokens):
    """y = v - (the first two parts of v): the third part in small batches, which
    keep v in fp32, and within 2^-16 of v in larger ones."""
    t = torch_()
    g = gen(81)
    rank, n_in, n_out = 8, 64, 32
    v, parts = latents(g, 1, 1)
    a, b = (t.zeros(s, dtype=t.bfloat16, device="cuda") for s in ((1, rank, n_in), (1, n_out, rank)))
    for k in range(3):
        a[0, 0, k] = parts[k]
        if k < 2:
            a[0, 1, k] = -parts[k]
    b[0, :, :2] = 1
    x, base = t.ones((tokens, n_in), dtype=t.bfloat16, device="cuda"), t.zeros((tokens, n_out), dtype=t.bfloat16, device="cuda")
    ids = t.zeros(tokens, dtype=t.int32, device="cuda")
    y = lb.adapters_forward(x, ids, [lb.AdapterPool(a, b)], bases=[base])[0].double()
    if tokens <= 176:
        assert bool((y == parts[2].double()).all())
    else:
        assert bool(((y - parts[2].double()).abs() <= 2.0 ** -16 * v.abs()).all())
