"""The adapters and heads calls on a machine without a GPU: what they refuse
before they touch CUDA, their workspace queries, and the 64-bit forms that the
GPU tests compare with, held against differences."""
import ctypes

import pytest
import torch

import binarized_rank_linear_b200 as lb
from binarized_rank_linear_b200 import build as lb_build
from tests import operators_ref as ref

FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    lb_build.build()
    return lb.lib()


def pool(**over):
    d = dict(a=FAKE, b=FAKE, scale=FAKE, ranks=FAKE, count=4, rank=16)
    d.update(over)
    return lb.LbAdapters(**d)


def forward(L, x=FAKE, tokens=5, n_in=64, ldx=64, ids=FAKE, nproj=None, ws=FAKE, ws_bytes=1 << 24, projs=None, **over):
    projs = [dict(over)] if projs is None else projs
    arr = (lb.LbAdapterProjection * max(1, len(projs)))()
    for e, o in zip(arr, projs):
        o = dict(dict(n_out=96, pool=pool(), base=FAKE, ldbase=96, y=FAKE, ldy=96), **o)
        e.n_out, e.base, e.ldbase, e.y, e.ldy = o["n_out"], o["base"], o["ldbase"], o["y"], o["ldy"]
        e.adapters = ctypes.pointer(o["pool"]) if o["pool"] is not None else None
    return L.lb_adapters_forward(x, tokens, n_in, ldx, ids, len(projs) if nproj is None else nproj, arr, ws, ws_bytes, None)


BAD, SHAPE, ALIGN = lb.LB_ERR_INVALID_ARGUMENT, lb.LB_ERR_UNSUPPORTED_SHAPE, lb.LB_ERR_MISALIGNED


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0, x=0, ids=0), lb.LB_OK), (dict(tokens=-1), BAD), (dict(x=0), BAD), (dict(ids=0), BAD),
    (dict(nproj=0), BAD), (dict(nproj=5), BAD), (dict(n_in=0), BAD), (dict(n_in=40, ldx=40), SHAPE), (dict(ldx=56), BAD),
    (dict(ldx=68), ALIGN), (dict(x=FAKE + 2), ALIGN), (dict(ids=FAKE + 2), ALIGN), (dict(tokens=(1 << 20) + 1), SHAPE),
    (dict(pool=None), BAD), (dict(pool=pool(a=0)), BAD), (dict(pool=pool(b=0)), BAD), (dict(pool=pool(count=0)), BAD),
    (dict(pool=pool(count=1025)), SHAPE), (dict(pool=pool(rank=0)), BAD), (dict(pool=pool(rank=12)), SHAPE),
    (dict(pool=pool(rank=136)), SHAPE), (dict(pool=pool(a=FAKE + 8)), ALIGN), (dict(pool=pool(scale=FAKE + 2)), ALIGN),
    (dict(pool=pool(ranks=FAKE + 1)), ALIGN), (dict(n_out=100, ldy=104), SHAPE), (dict(y=0), BAD), (dict(ldy=64), BAD),
    (dict(ldy=100, base=0), ALIGN), (dict(y=FAKE + 2), ALIGN), (dict(base=FAKE + 2), ALIGN), (dict(ldbase=64), BAD),
    (dict(ldbase=100), BAD), (dict(base=2 * FAKE, ldbase=100), ALIGN), (dict(ws=0), BAD), (dict(ws=FAKE + 8), ALIGN),
    (dict(ws_bytes=16), lb.LB_ERR_WORKSPACE_TOO_SMALL),
    (dict(projs=[{}, dict(pool=pool(count=5))]), BAD),  # pools of one call have one count
])
def test_forward_refuses_before_any_cuda_call(L, kw, status):
    assert forward(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), BAD), (dict(x=0), BAD), (dict(dy=0), BAD), (dict(ids=0), BAD), (dict(pool=None), BAD),
    (dict(da=0), BAD), (dict(db=0), BAD), (dict(n_in=40), SHAPE), (dict(n_out=90, lddy=96), SHAPE), (dict(lddy=64), BAD),
    (dict(lddx=32), BAD), (dict(ldbase=32), BAD), (dict(ldbase=72), BAD), (dict(base=2 * FAKE, ldbase=68), ALIGN),
    (dict(dx=FAKE + 2, base=0), ALIGN), (dict(da=FAKE + 4), ALIGN), (dict(db=FAKE + 8), ALIGN), (dict(dy=FAKE + 2), ALIGN),
    (dict(pool=pool(rank=20)), SHAPE), (dict(ws=0), BAD), (dict(ws=FAKE + 8), ALIGN),
    (dict(ws_bytes=16), lb.LB_ERR_WORKSPACE_TOO_SMALL),
])
def test_backward_refuses_before_any_cuda_call(L, kw, status):
    o = dict(x=FAKE, dy=FAKE, tokens=5, n_in=64, n_out=96, ldx=64, lddy=96, ids=FAKE, pool=pool(), base=FAKE, ldbase=64,
             dx=FAKE, lddx=64, da=FAKE, db=FAKE, ws=FAKE, ws_bytes=1 << 24)
    o.update(kw)
    p = ctypes.byref(o["pool"]) if o["pool"] is not None else None
    assert L.lb_adapters_backward(o["x"], o["dy"], o["tokens"], o["n_in"], o["n_out"], o["ldx"], o["lddy"], o["ids"], p,
                                  o["base"], o["ldbase"], o["dx"], o["lddx"], o["da"], o["db"], o["ws"], o["ws_bytes"],
                                  None) == status


def test_workspace_queries(L):
    assert lb.adapters_workspace_bytes(32, 5120, 64, (16, 16, 16)) > 0
    assert lb.adapters_workspace_bytes(0, 5120, 64, (16,)) == 0
    assert lb.adapters_workspace_bytes(32, 5120, 0, (16,)) == 0
    assert lb.adapters_workspace_bytes(32, 5000, 64, (16,)) == 0
    assert lb.adapters_workspace_bytes(8192, 5120, 8, (64,)) > 0
    assert lb.adapters_backward_workspace_bytes(333, 4096, 4096, 3, 8) > 0
    assert lb.adapters_backward_workspace_bytes(0, 4096, 4096, 3, 8) == 0
    assert lb.adapters_backward_workspace_bytes(333, 4096, 4096, 3, 9) == 0
    assert lb.heads_backward_workspace_bytes(128) > 0 and lb.heads_backward_workspace_bytes(12) == 0


def heads(L, tokens=3, d=64, rd=64, rotation=0, pos=FAKE, freq=FAKE, eps=1e-6, n=1, ws=FAKE, ws_bytes=1 << 22, back=False,
          **over):
    t = lb.LbHeadsGrad if back else lb.LbHeads
    o = dict(heads=2, in_=FAKE, ld_in=128, weight=FAKE)
    o.update(dict(dout=2 * FAKE, ld_dout=128, din=3 * FAKE, ld_din=128, dweight=FAKE) if back else dict(out=FAKE, ld_out=128))
    o.update(over)
    arr = (t * 1)(t(**o))
    if back:
        return L.lb_heads_norm_rotate_backward(tokens, d, rd, rotation, pos, freq, eps, n, arr, ws, ws_bytes, None)
    return L.lb_heads_norm_rotate(tokens, d, rd, rotation, pos, freq, eps, n, arr, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), BAD), (dict(d=0), BAD), (dict(d=60, rd=0), SHAPE), (dict(d=264, rd=0), SHAPE), (dict(rd=72), BAD),
    (dict(rd=12), SHAPE), (dict(rd=-8), BAD), (dict(rotation=2), BAD), (dict(pos=0), BAD), (dict(freq=0), BAD),
    (dict(pos=FAKE + 2), ALIGN), (dict(freq=FAKE + 1), ALIGN), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(eps=float("inf")), BAD), (dict(n=0), BAD), (dict(n=5), BAD), (dict(heads=0), BAD), (dict(heads=4097), SHAPE),
    (dict(in_=0), BAD), (dict(ld_in=120), BAD), (dict(in_=FAKE + 2), ALIGN), (dict(in_=2 * FAKE, ld_in=132), ALIGN),
    (dict(weight=FAKE + 8), ALIGN),
])
def test_heads_refuse_before_any_cuda_call(L, kw, status):
    assert heads(L, **kw) == status
    assert heads(L, back=True, **kw) == status


def test_heads_refuse_their_own_outputs(L):
    assert heads(L, tokens=0, in_=0, out=0) == lb.LB_OK
    assert heads(L, out=0) == BAD and heads(L, ld_out=136) == BAD  # in place with another stride
    assert heads(L, out=FAKE + 2) == ALIGN
    assert heads(L, back=True, dout=0) == BAD and heads(L, back=True, din=0) == BAD
    assert heads(L, back=True, weight=0) == BAD  # a dweight without a weight
    assert heads(L, back=True, din=2 * FAKE, ld_din=136) == BAD and heads(L, back=True, din=FAKE, ld_din=136) == BAD
    assert heads(L, back=True, ws=0) == BAD and heads(L, back=True, ws=FAKE + 4) == ALIGN
    assert heads(L, back=True, ws_bytes=64) == lb.LB_ERR_WORKSPACE_TOO_SMALL


def test_binding_refuses_wrong_tensors(L):
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    ids = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device memory"):
        lb.adapters_forward(x, ids, [], bases=[])
    with pytest.raises(ValueError, match="device memory"):
        lb.adapters_backward(x, x, ids, None)
    with pytest.raises(TypeError, match="bfloat16"):
        lb.AdapterPool(torch.zeros((2, 8, 64)), torch.zeros((2, 64, 8))).as_c()
    with pytest.raises(ValueError, match="3-D device"):
        lb.AdapterPool(torch.zeros((2, 8, 64), dtype=torch.bfloat16), torch.zeros((2, 64, 8), dtype=torch.bfloat16)).as_c()
    with pytest.raises(ValueError, match="halves"):
        lb.HeadRotation(64, None, "both")
    with pytest.raises(ValueError, match="inv_freq"):
        lb.HeadRotation(64, torch.zeros(32))
    with pytest.raises(ValueError, match="device memory"):
        lb.heads_norm_rotate([x], ids, lb.HeadRotation(64))
    with pytest.raises(ValueError, match="1 to 4"):
        lb.heads_norm_rotate([], ids, lb.HeadRotation(64))


def differences(f, args, grads, dout, seed):
    """Each gradient along a direction against the central difference of sum(f dout)."""
    g = torch.Generator().manual_seed(seed)
    for k, grad in enumerate(grads):
        v = torch.randn(args[k].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + h * v, args[k] - h * v
        slope = float(((f(*up) - f(*dn)) * dout).sum()) / (2 * h)
        assert abs(slope - float((grad * v).sum())) <= 1e-6 * (1 + float((grad * v).abs().sum()))


def test_adapters_form_against_differences():
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, a, b, base, dy = n(9, 12), n(3, 4, 12), n(3, 10, 4), n(9, 10), n(9, 10)
    ids = torch.tensor([0, 2, 2, -1, 0, 2, 5, 0, 2])
    scale, ranks = torch.tensor([0.5, 2.0, 1.5]), [4, 2, 3]
    (dx, da, db), _ = ref.adapters_backward(x, dy, ids, a, b, scale, ranks, torch.zeros_like(x))
    differences(lambda x, a, b: ref.adapters(x, ids, a, b, scale, ranks, base)[0], [x, a, b], [dx, da, db], dy, 2)


@pytest.mark.parametrize("rotation,rd", [("halves", 8), ("pairs", 8), ("halves", 16), ("pairs", 16)])
def test_heads_form_against_differences(rotation, rd):
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, w, dout, d = n(5, 48), n(16), n(5, 48), 16
    pos, freq = torch.arange(5) + 100, torch.rand(rd // 2, generator=g)
    (din, dw), _ = ref.heads_backward(x, dout, pos, freq, rotation, w, 1e-6, d)
    differences(lambda x, w: ref.heads(x, pos, freq, rotation, w, 1e-6, d)[0], [x, w], [din, dw], dout, 4)
    # a rotation keeps lengths: backward of the form without a norm undoes the forward pass
    y, _ = ref.heads(x, pos, freq, rotation, None, 1e-6, d)
    (back, _), _ = ref.heads_backward(None, y, pos, freq, rotation, None, 1e-6, d)
    assert float((back - x).abs().max()) < 1e-12


FAR = (1 << 30) + 8


@pytest.mark.parametrize("kw", [dict(ldx=FAR), dict(base=0, ldy=FAR), dict(ldy=FAR, ldbase=FAR), dict(base=2 * FAKE, ldbase=FAR)])
def test_forward_refuses_rows_too_far_apart(L, kw):
    assert forward(L, **kw) == SHAPE


@pytest.mark.parametrize("name", ["ldx", "lddy", "lddx", "ldbase"])
def test_backward_refuses_rows_too_far_apart(L, name):
    ld = dict(ldx=64, lddy=96, lddx=64, ldbase=64)
    ld[name] = FAR
    p = pool()
    assert L.lb_adapters_backward(FAKE, FAKE, 5, 64, 96, ld["ldx"], ld["lddy"], FAKE, ctypes.byref(p), 2 * FAKE, ld["ldbase"],
                                  FAKE, ld["lddx"], FAKE, FAKE, FAKE, 1 << 24, None) == SHAPE


@pytest.mark.parametrize("kw", [dict(ld_in=FAR), dict(ld_out=FAR)])
def test_heads_refuse_rows_too_far_apart(L, kw):
    assert heads(L, **kw) == SHAPE


def test_workspace_follows_the_kernels(L):
    """Small batches need partial sums alone, more tokens than the pool allows
    for them the plan and tiles too; the query knows both sides of the border."""
    for count, border in ((1, 176), (6, 416), (16, 512), (64, 1536), (1000, 2048)):
        sizes = [lb.adapters_workspace_bytes(t, 64, count, (16,)) for t in (1, border, border + 1)]
        assert 0 < sizes[0] <= sizes[1] < sizes[2]


@pytest.mark.parametrize("n_in,count,ranks", [(16384, 64, (64,) * 4), (28672, 86, (16,)), (64, 3, (8,)), (1 << 20, 1, (128,) * 4),
                                              (5120, 1024, (16, 8, 128)), (4096, 8, (16,) * 3)])
def test_a_workspace_serves_every_smaller_batch(L, n_in, count, ranks):
    tokens = sorted({*range(1, 200, 13), *range(160, 2200, 61), 512, 513, 1536, 1537, 1736, 2048, 2049, 4096, 1 << 20})
    sizes = [lb.adapters_workspace_bytes(t, n_in, count, ranks) for t in tokens]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    back = [lb.adapters_backward_workspace_bytes(t, n_in, 64, count, ranks[0]) for t in tokens]
    assert back[0] > 0 and back == sorted(back)
