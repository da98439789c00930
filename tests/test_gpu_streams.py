"""Calls on a stream of the caller's, and behind kernels that let the next
launch start early, on the GPU."""
import ctypes
import os
import subprocess

import pytest

import binarized_rank_linear_b200 as lb
from binarized_rank_linear_b200 import build as lb_build
from tests.test_gpu_adapters import gen, make_ids, make_pool, normal, torch_
from tests.test_gpu_heads import make

pytestmark = pytest.mark.gpu


def sleep(seconds):
    """A kernel on the current stream that takes about this long."""
    t = torch_()
    t.cuda._sleep(int(seconds * 1.9e9))


@pytest.mark.parametrize("tokens", [20, 400])
def test_memory_that_the_current_stream_still_reads(tokens):
    """Blocks freed while kernels queued on the current stream still read them
    are not what a call on another stream writes to."""
    t = torch_()
    g = gen(61)
    n_in, n_out, d = 256, 512, 128
    pool = make_pool(g, 3, 16, n_in, n_out)
    x, dy = normal(g, tokens, n_in), normal(g, tokens, n_out)
    ids = make_ids(g, tokens, 3, "some")
    _, rot, pos, _, ws = make(tokens, [n_out // d], d, d, "halves", [True], 11, 62)
    calls = [
        lambda s: lb.adapters_forward(x, ids, [pool], bases=[dy], stream=s),
        lambda s: [*lb.adapters_backward(x, dy, ids, pool, dx_base=x, stream=s).values()],
        lambda s: lb.heads_norm_rotate([dy], pos, rot, weights=ws, stream=s),
        lambda s: [*lb.heads_norm_rotate_backward([dy], [dy], pos, rot, weights=ws, stream=s)[0].values()],
    ]
    sizes = [lb.adapters_workspace_bytes(tokens, n_in, 3, (16,)), lb.heads_backward_workspace_bytes(d),
             lb.adapters_backward_workspace_bytes(tokens, n_in, n_out, 3, 16)]
    side = t.cuda.Stream()
    for call in calls:
        want = call(None)
        like = sizes + [v.numel() * v.element_size() for v in want]
        kept = [t.empty(n, dtype=t.uint8, device="cuda") for n in like]
        t.cuda.synchronize()
        sleep(0.05)
        temporary = [t.full((n,), 7, dtype=t.uint8, device="cuda") for n in like]
        for k, v in zip(kept, temporary):
            k.copy_(v)
        del temporary, v
        got = call(side)
        t.cuda.synchronize()
        assert all(bool((k == 7).all()) for k in kept)
        assert all(t.equal(a, b) for a, b in zip(got, want))


@pytest.fixture(scope="module")
def early_copy(tmp_path_factory):
    """copy(dst, src, seconds): dst = src by a kernel that lets the launch behind
    it start at once and writes only when `seconds` have passed."""
    so = str(tmp_path_factory.mktemp("early") / "early_writer.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "early_writer.cu")
    subprocess.run([lb_build.NVCC, *lb_build.ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", so, src], check=True)
    launch = ctypes.CDLL(so).early_copy_launch
    launch.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p]

    def copy(dst, src, seconds=1e-3):
        t = torch_()
        words = dst.numel() * dst.element_size() // 4
        assert words == src.numel() * src.element_size() // 4 and dst.is_contiguous() and src.is_contiguous()
        assert launch(dst.data_ptr(), src.data_ptr(), words, int(seconds * 1e9), t.cuda.current_stream().cuda_stream) == 0

    return copy


def behind(copy, fields, call, what):
    """`call()` with each of `fields` written directly ahead of it gives what it gives with them in place."""
    t = torch_()
    new = {k: v.clone() for k, v in fields.items()}
    t.cuda.synchronize()
    want = [v.clone() for v in call()]
    for name, field in fields.items():
        field.copy_(new[name].flatten().roll(1).view_as(field))
        t.cuda.synchronize()
        copy(field, new[name])
        got = call()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(got, want)), f"{what}: {name} was read before it was written"
    assert lb.device_status() == lb.LB_OK


@pytest.mark.parametrize("tokens", [1, 30, 400, 9001])
def test_adapters_behind_an_early_writer(early_copy, tokens):
    t = torch_()
    g = gen(63)
    n_in, n_out = 512, 1024
    pool = make_pool(g, 5, 16, n_in, n_out, [16, 3, 8, 12, 15])
    x, dy, base = normal(g, tokens, n_in), normal(g, tokens, n_out), normal(g, tokens, n_out)
    ids = t.arange(tokens, device="cuda", dtype=t.int32) * 2 % 5
    y, dx = t.empty_like(base), t.empty_like(x)
    fields = dict(ids=ids, a=pool.a, b=pool.b, scale=pool.scale, ranks=pool.ranks, x=x)
    if tokens == 1:  # rolled by one it would be what it was
        stale = t.tensor([3], dtype=t.int32, device="cuda")
        fields.pop("ids")
        want = lb.adapters_forward(x, ids, [pool], bases=[base])[0].clone()
        new = ids.clone()
        ids.copy_(stale)
        t.cuda.synchronize()
        early_copy(ids, new)
        assert t.equal(lb.adapters_forward(x, ids, [pool], bases=[base])[0], want)
    behind(early_copy, dict(fields, base=base), lambda: lb.adapters_forward(x, ids, [pool], bases=[base], ys=[y]), "forward")
    behind(early_copy, dict(fields, dy=dy), lambda: [*lb.adapters_backward(x, dy, ids, pool, dx_base=x, dx=dx).values()],
           "backward")


@pytest.mark.parametrize("tokens,rotation", [(2, "halves"), (300, "pairs"), (2000, "halves")])
def test_heads_behind_an_early_writer(early_copy, tokens, rotation):
    t = torch_()
    g, rot, pos, (x,), (w,) = make(tokens, [3], 128, 64, rotation, [True], 1000, 64)
    dout = normal(g, *x.shape)
    out = t.empty_like(x)
    fields = dict(positions=pos, inv_freq=rot.inv_freq, weight=w, x=x)
    behind(early_copy, fields, lambda: lb.heads_norm_rotate([x], pos, rot, weights=[w], outs=[out]), "forward")
    behind(early_copy, dict(fields, dout=dout), lambda: [*lb.heads_norm_rotate_backward([x], [dout], pos, rot, weights=[w],
                                                                                      dins=[out])[0].values()], "backward")


def test_heads_behind_a_launch_that_takes_longer_than_their_waits(early_copy):
    """The kernels' own waits give up after 2 s; the time until the launch ahead
    has finished is not theirs."""
    t = torch_()
    g, rot, pos, (x,), (w,) = make(40, [3], 128, 128, "halves", [True], 7, 65)
    out = t.empty_like(x)
    want = lb.heads_norm_rotate([x], pos, rot, weights=[w])[0].clone()
    late = x.clone()
    x.zero_()
    t.cuda.synchronize()
    early_copy(x, late, seconds=2.6)
    lb.heads_norm_rotate([x], pos, rot, weights=[w], outs=[out])
    assert lb.device_status() == lb.LB_OK
    assert t.equal(out, want)


@pytest.mark.parametrize("tokens", [5, 700, 8192, 9001])
def test_ids_past_the_pool_that_are_written_over_in_time(early_copy, tokens):
    """What ids held before their writer has finished is not reported, what it
    writes is."""
    t = torch_()
    g = gen(66)
    pool = make_pool(g, 3, 8, 64, 96)
    x, base = normal(g, tokens, 64), normal(g, tokens, 96)
    good = make_ids(g, tokens, 3, "mixed")
    bad = good.clone()
    bad[tokens // 2] = 3
    ids = t.full_like(good, 99)
    want = lb.adapters_forward(x, good, [pool], bases=[base])[0]
    assert lb.device_status() == lb.LB_OK
    early_copy(ids, good)
    y = lb.adapters_forward(x, ids, [pool], bases=[base])[0]
    assert lb.device_status() == lb.LB_OK and t.equal(y, want)
    early_copy(ids, bad)
    y = lb.adapters_forward(x, ids, [pool], bases=[base])[0]
    assert lb.device_status() == lb.LB_ERR_INVALID_ARGUMENT
    assert t.equal(y[tokens // 2], base[tokens // 2])
    y[tokens // 2] = want[tokens // 2]
    assert t.equal(y, want)


@pytest.mark.parametrize("tokens,count", [(2, 5), (17, 64), (100, 16), (368, 5), (1500, 64), (2048, 1000)])
def test_small_batches_behind_an_early_writer(early_copy, tokens, count):
    """What the groups of tokens were found from before it was written."""
    t = torch_()
    g = gen(67)
    n_in, outs = 2080, [288, 64]
    ranks = [(7 * i) % 17 for i in range(count)]
    pools = [make_pool(g, count, 16, n_in, o, ranks) for o in outs]
    x, bases = normal(g, tokens, n_in), [normal(g, tokens, o) for o in outs]
    ids = t.randint(-1, count, (tokens,), generator=g, device="cuda").to(t.int32)
    ids[0], ids[1] = 1, 0
    ys = [t.empty_like(b) for b in bases]
    fields = dict(ids=ids, ranks=pools[1].ranks, a=pools[0].a, b=pools[1].b, x=x, base=bases[1])
    behind(early_copy, fields, lambda: lb.adapters_forward(x, ids, pools, bases=bases, ys=ys), "forward")
    # from all tokens without an adapter to all of one, and back
    for old, new in ((-1, 1), (1, -1)):
        ids.fill_(new)
        want = [y.clone() for y in lb.adapters_forward(x, ids, pools, bases=bases)]
        late = ids.clone()
        ids.fill_(old)
        t.cuda.synchronize()
        early_copy(ids, late)
        got = lb.adapters_forward(x, ids, pools, bases=bases)
        assert all(t.equal(a, b) for a, b in zip(got, want))
