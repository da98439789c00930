"""Calls on a stream of the caller's, and behind kernels that let the next
launch start early, on the GPU."""
import pytest

import binarized_rank_linear_b200 as lb
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
