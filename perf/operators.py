"""Cases for the operators beside the factored projection: low-rank adapters of many requests (forward and backward) and
per-head norms with the position rotation (forward and backward).

``listed()`` and ``draw()`` give cases, ``prepare()`` the inputs a caller holds, ``run()`` one pass (plain torch, or the
library's calls where ``own`` is true), ``work()`` the bytes and operations a pass cannot do without, and ``exact()`` the
definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 1e6


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one request decoding through Llama-2-7B's query, key and value projections, its adapter of rank 16
        dict(name="adapters 1 token", op="adapters", tokens=1, n_in=4096, n_out="4096,4096,4096", rank=16, count=8,
             order="mixed", ragged=False, without=False),
        # a decode batch of 32 requests over Qwen3-14B's attention inputs, 64 adapters of ranks 4 to 16 loaded, some
        # requests without one
        dict(name="adapters 32 tokens", op="adapters", tokens=32, n_in=5120, n_out="5120,1024,1024", rank=16, count=64,
             order="mixed", ragged=True, without=True),
        # a large decode batch at the gate and up projections
        dict(name="adapters 100 tokens", op="adapters", tokens=100, n_in=5120, n_out="17408,17408", rank=32, count=16,
             order="mixed", ragged=False, without=False),
        # a ragged prefill of a few prompts, an odd number of tokens, ranks of every size up to 40
        dict(name="adapters 1013 tokens", op="adapters", tokens=1013, n_in=4096, n_out="11008", rank=40, count=5,
             order="runs", ragged=True, without=True),
        # a full prefill batch of prompts over Qwen3-14B's query projection
        dict(name="adapters 8192 tokens", op="adapters", tokens=8192, n_in=5120, n_out="5120", rank=64, count=8,
             order="runs", ragged=False, without=False),
        # fine-tuning three small adapters on a short batch
        dict(name="adapters backward 333", op="adapters_backward", tokens=333, n_in=4096, n_out="4096", rank=8, count=3,
             order="runs", ragged=True, without=True),
        # fine-tuning four adapters at the gate projection of Qwen3-14B on 8192 tokens
        dict(name="adapters backward 8192", op="adapters_backward", tokens=8192, n_in=5120, n_out="17408", rank=64,
             count=4, order="runs", ragged=False, without=False),
        # one decoded token of Qwen3-14B: 40 query and 8 key heads, normed and rotated at a far position
        dict(name="heads 1 token", op="heads", tokens=1, heads="40,8", head_dim=128, rotary_dim=128, rotation="halves",
             norm=True, far=True),
        # a Llama-2-7B prompt (no norms), neighbouring pairs rotated, half of each head
        dict(name="heads 777 tokens", op="heads", tokens=777, heads="32,32", head_dim=128, rotary_dim=64,
             rotation="pairs", norm=False, far=False),
        # Qwen3-14B prefill
        dict(name="heads 8192 tokens", op="heads", tokens=8192, heads="40,8", head_dim=128, rotary_dim=128,
             rotation="halves", norm=True, far=False),
        # a short training batch with narrow heads
        dict(name="heads backward 129", op="heads_backward", tokens=129, heads="14,2", head_dim=64, rotary_dim=64,
             rotation="halves", norm=True, far=False),
        # a training batch of Qwen3-14B
        dict(name="heads backward 8192", op="heads_backward", tokens=8192, heads="40,8", head_dim=128, rotary_dim=128,
             rotation="halves", norm=True, far=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "adapters_backward", "heads", "heads_backward"])
    if op in ("heads", "heads_backward"):
        d = rng.choice([64, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        q = kv * rng.choice([1, 3, 4, 5])
        tokens = _log(rng, 1 if op == "heads" else 16, 8192)
        if tokens * (q + kv) * d > 8192 * 48 * 128:
            tokens = 8192 * 48 * 128 // ((q + kv) * d)
        return dict(op=op, tokens=tokens, heads="%d,%d" % (q, kv), head_dim=d,
                    rotary_dim=rng.choice([d, d, d // 2]), rotation=rng.choice(["halves", "halves", "pairs"]),
                    norm=rng.random() < 0.7, far=rng.random() < 0.5)
    n_in = 32 * _log(rng, 16, 160)
    rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
    count = _log(rng, 1, 64 if op == "adapters" else 8)
    if op == "adapters":
        tokens = _log(rng, 1, 8192)
        outs = [32 * _log(rng, 16, 160) for _ in range(rng.choice([1, 1, 2, 3]))]
        if tokens > 512:  # a plain pass over every adapter of the pool stays within the largest listed case
            outs, count = outs[:1], min(count, 8)
        rank = min(rank, 64) if tokens > 512 else rank
    else:
        tokens = _log(rng, 16, 8192)
        outs = [32 * _log(rng, 16, 544)]
        if tokens > 512:
            rank, count = min(rank, 64), min(count, 4)
    return dict(op=op, tokens=tokens, n_in=n_in, n_out=",".join(map(str, outs)), rank=rank, count=count,
                order=rng.choice(["mixed", "runs"]), ragged=rng.random() < 0.5, without=rng.random() < 0.5)


def _numbers(text):
    return [int(v) for v in str(text).split(",")]


def _ranks(case):
    """The rank of each adapter of the pool: all of them, or from 1/4 of the stored rank up to it, odd ones among them."""
    r, n = case["rank"], case["count"]
    return [r - (3 * i * r) // (4 * n) for i in range(n)] if case["ragged"] else [r] * n


# ------------------------------------------------------------------------------------------------ inputs

def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _pool(g, case, n_out, ranks):
    """A pool as it is loaded: A and B zero past each adapter's rank."""
    n, r, n_in = case["count"], case["rank"], case["n_in"]
    keep = torch.arange(r, device="cuda")[None, :] < ranks[:, None].to(torch.int64)
    a = _normal(g, n, r, n_in, scale=n_in ** -0.5) * keep[:, :, None]
    b = _normal(g, n, n_out, r, scale=0.05) * keep[:, None, :]
    scale = torch.rand(n, generator=g, device="cuda") + 0.5
    return a.contiguous(), b.contiguous(), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = case["tokens"]
    s = {"case": case}
    if case["op"] in ("adapters", "adapters_backward"):
        outs, n = _numbers(case["n_out"]), case["count"]
        ids = torch.randint(0, n, (t,), generator=g, device="cuda")
        if case["without"]:
            ids = torch.where(torch.rand(t, generator=g, device="cuda") < 0.125, -1, ids)
        if case["order"] == "runs":  # the tokens of a prompt stand together, the prompts in any order
            ids = torch.sort(ids).values.roll(t // 3)
        s["ids"] = ids.to(torch.int32)
        s["x"] = _normal(g, t, case["n_in"])
        ranks = torch.tensor(_ranks(case), dtype=torch.int32, device="cuda")
        s["ranks"] = ranks if case["ragged"] else None
        s["pools"] = [_pool(g, case, o, ranks) for o in outs]
        if case["op"] == "adapters":
            s["base"] = [_normal(g, t, o) for o in outs]
        else:
            s["dy"] = _normal(g, t, outs[0])
            s["dx_base"] = _normal(g, t, case["n_in"])
    else:
        d = case["head_dim"]
        heads = _numbers(case["heads"])
        first = int(torch.randint(0, 200000 if case["far"] else 2000, (1,), generator=g, device="cuda"))
        s["positions"] = (torch.arange(t, device="cuda") + first).to(torch.int32)
        rd = case["rotary_dim"]
        s["inv_freq"] = (THETA ** (-torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd)).float()
        s["heads"] = heads
        s["in"] = [_normal(g, t, h * d) for h in heads]
        s["weight"] = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] else None
                       for _ in heads]
        if case["op"] == "heads_backward":
            s["dout"] = [_normal(g, t, h * d) for h in heads]
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program of the library keeps from call to call: the loaded pools, the model's rotation."""
    import binarized_rank_linear_b200 as lb
    c = s["case"]
    if "pools" in s:
        s["handles"] = [lb.AdapterPool(a, b, scale, s["ranks"]) for a, b, scale in s["pools"]]
    else:
        s["handle"] = lb.HeadRotation(c["head_dim"], s["inv_freq"], rotation=c["rotation"], eps=EPS)


# ------------------------------------------------------------------------------------------------ plain forms

# Up to this many tokens the plain form gathers each token's own adapter; past it that copy would be far larger than
# the products of every token with every adapter of the pool.
GATHER = 128


def _latent(x, a, s, ids, used):
    """s_i A_i x of each token in fp32: [tokens, rank] from the token's own adapter, or [tokens, count, rank] with
    zeros at the adapters a token does not use."""
    if x.shape[0] <= GATHER:
        i = ids.clamp(min=0)
        v = torch.bmm(a[i].float(), x.float()[:, :, None])[:, :, 0] * s[i, None]
        return torch.where((ids >= 0)[:, None], v, 0.0)
    v = (x.float() @ a.float().flatten(0, 1).t()).view(x.shape[0], a.shape[0], a.shape[1]) * s[None, :, None]
    return torch.where(used[:, :, None], v, 0.0)


def _plain_adapters(st):
    ids = st["ids"].long()
    x = st["x"]

    def one(pool, base):
        a, b, s = pool
        used = ids[:, None] == torch.arange(a.shape[0], device=x.device)[None, :]
        v = _latent(x, a, s, ids, used)
        if v.dim() == 2:
            d = torch.bmm(b[ids.clamp(min=0)].float(), v[:, :, None])[:, :, 0]
        else:
            d = v.flatten(1) @ b.float().transpose(1, 2).flatten(0, 1)
        return (base.float() + d).to(base.dtype)

    return [one(p, y) for p, y in zip(st["pools"], st["base"])]


def _plain_adapters_backward(st):
    ids, x, dy = st["ids"].long(), st["x"].float(), st["dy"].float()
    a, b, s = st["pools"][0]
    n, r, n_in = a.shape
    used = ids[:, None] == torch.arange(n, device=x.device)[None, :]
    v = torch.where(used[:, :, None], (x @ a.float().flatten(0, 1).t()).view(-1, n, r) * s[None, :, None], 0.0).flatten(1)
    u = (dy @ b.float().transpose(1, 2).flatten(0, 1).t()).view(-1, n, r) * s[None, :, None]
    u = torch.where(used[:, :, None], u, 0.0).flatten(1)
    keep = (v.new_tensor(_ranks(st["case"]))[:, None] > torch.arange(r, device=x.device)[None, :])
    da = (u.t() @ x).view(n, r, n_in) * keep[:, :, None]
    db = (dy.t() @ v).view(-1, n, r).transpose(0, 1).contiguous() * keep[:, None, :]
    dx = st["dx_base"].float() + u @ a.float().flatten(0, 1)
    return {"dx": dx.to(torch.bfloat16), "da": da, "db": db}


def _angles(st):
    a = st["positions"].double()[:, None] * st["inv_freq"].double()[None, :]
    return a.cos().float()[:, None, :], a.sin().float()[:, None, :]


def _turn(v, cos, sin, rotary, rotation):
    """Turns the first `rotary` elements of each head by the angles."""
    p, rest = v[..., :rotary], v[..., rotary:]
    if rotation == "halves":
        a, b = p[..., : rotary // 2], p[..., rotary // 2:]
        p = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = p[..., 0::2], p[..., 1::2]
        p = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([p, rest], -1)


def _plain_heads(st):
    c = st["case"]
    cos, sin = _angles(st)

    def one(x, w, h):
        v = x.float().view(x.shape[0], h, c["head_dim"])
        if w is not None:
            v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w.float()
        return _turn(v, cos, sin, c["rotary_dim"], c["rotation"]).flatten(1).to(x.dtype)

    return [one(*z) for z in zip(st["in"], st["weight"], st["heads"])]


def _plain_heads_backward(st):
    c = st["case"]
    cos, sin = _angles(st)

    def one(x, dy, w, h):
        v = x.float().view(x.shape[0], h, c["head_dim"])
        g = _turn(dy.float().view_as(v), cos, -sin, c["rotary_dim"], c["rotation"])  # the rotation's transpose
        if w is None:
            return {"din": g.flatten(1).to(x.dtype)}
        rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        n = v * rstd
        dw = (g * n).sum((0, 1), dtype=torch.float64).float()
        g = g * w.float()
        din = rstd * (g - n * (g * n).mean(-1, keepdim=True))
        return {"din": din.flatten(1).to(x.dtype), "dweight": dw}

    return [one(*z) for z in zip(st["in"], st["dout"], st["weight"], st["heads"])]


# ------------------------------------------------------------------------------------------------ one pass

def _own(st):
    import binarized_rank_linear_b200 as lb
    op = st["case"]["op"]
    if op == "adapters":
        return lb.adapters_forward(st["x"], st["ids"], st["handles"], bases=st["base"])
    if op == "adapters_backward":
        return lb.adapters_backward(st["x"], st["dy"], st["ids"], st["handles"][0], dx_base=st["dx_base"])
    if op == "heads":
        return lb.heads_norm_rotate(st["in"], st["positions"], st["handle"], weights=st["weight"])
    return lb.heads_norm_rotate_backward(st["in"], st["dout"], st["positions"], st["handle"], weights=st["weight"])


def run(state):
    if own:
        return _own(state)
    plain = {"adapters": _plain_adapters, "adapters_backward": _plain_adapters_backward, "heads": _plain_heads,
             "heads_backward": _plain_heads_backward}
    return plain[state["case"]["op"]](state)


def work(case):
    t = case["tokens"]
    if case["op"] in ("adapters", "adapters_backward"):
        outs, n_in = _numbers(case["n_out"]), case["n_in"]
        used = min(case["count"], t)
        ranks = _ranks(case)
        mean = sum(ranks) / len(ranks)
        weights = sum(2 * mean * used * (n_in + o) for o in outs)
        flops = sum(2 * t * mean * (n_in + o) for o in outs)
        if case["op"] == "adapters":
            return {"bytes": weights + 2 * t * n_in + 4 * t * sum(outs) + 4 * t, "flops": flops}
        grads = 4 * case["count"] * case["rank"] * (n_in + outs[0])
        return {"bytes": weights + grads + 2 * t * (n_in + outs[0]) + 4 * t * n_in + 4 * t,
                "flops": 2 * flops + 2 * t * mean * n_in}
    n = t * sum(_numbers(case["heads"])) * case["head_dim"]
    if case["op"] == "heads":
        return {"bytes": 4 * n + 4 * t, "flops": 8 * n}
    read = 3 if case["norm"] else 2
    return {"bytes": 2 * read * n + 4 * t, "flops": 16 * n}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("adapters", "adapters_backward"):
        ids, x = st["ids"].long(), st["x"].double()
        if case["op"] == "adapters":
            out = []
            for (a, b, s), base in zip(st["pools"], st["base"]):
                y = base.double()
                for i, r in enumerate(_ranks(case)):
                    m = torch.nonzero(ids == i)[:, 0]
                    y[m] += s[i].double() * ((x[m] @ a[i, :r].double().t()) @ b[i, :, :r].double().t())
                out.append(y)
            return out
        (a, b, s), dy, dx = st["pools"][0], st["dy"].double(), st["dx_base"].double()
        da = torch.zeros_like(a, dtype=torch.float64)
        db = torch.zeros_like(b, dtype=torch.float64)
        for i, r in enumerate(_ranks(case)):
            m = torch.nonzero(ids == i)[:, 0]
            ai, bi, si = a[i, :r].double(), b[i, :, :r].double(), s[i].double()
            da[i, :r] = si * (bi.t() @ dy[m].t()) @ x[m]
            db[i, :, :r] = si * dy[m].t() @ (x[m] @ ai.t())
            dx[m] += si * (dy[m] @ bi) @ ai
        return {"dx": dx, "da": da, "db": db}
    d, rd = case["head_dim"], case["rotary_dim"]
    k = torch.arange(rd // 2, device="cuda")
    lo, hi = (k, k + rd // 2) if case["rotation"] == "halves" else (2 * k, 2 * k + 1)
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                    st["positions"].double()[:, None] * st["inv_freq"].double())[:, None, :]
    out = []
    for j, h in enumerate(st["heads"]):
        x = st["in"][j].double().view(-1, h, d)
        w = st["weight"][j]
        norm = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() if w is not None else torch.ones_like(x[..., :1])
        scale = w.double() if w is not None else torch.ones(d, dtype=torch.float64, device="cuda")
        v = (x / norm * scale) if case["op"] == "heads" else st["dout"][j].double().view(-1, h, d).clone()
        turned = torch.complex(v[..., lo], v[..., hi]) * (z if case["op"] == "heads" else z.conj())
        v[..., lo], v[..., hi] = turned.real, turned.imag
        if case["op"] == "heads":
            out.append(v.flatten(1))
        elif w is None:
            out.append({"din": v.flatten(1)})
        else:
            n = x / norm
            g = v * scale
            out.append({"din": ((g - n * (g * n).sum(-1, keepdim=True) / d) / norm).flatten(1),
                        "dweight": (v * n).sum((0, 1))})
    return out
