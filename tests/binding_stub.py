"""Stand-ins for device tensors, streams and the library, so that what the
Python binding checks, allocates and launches, and in which order, can be
tested on a machine without a GPU."""
import contextlib
import ctypes
import types

import torch

import binarized_rank_linear_b200 as lb

CUDA = torch.device("cuda", 0)


class Stream:
    def __init__(self, number):
        self.cuda_stream = number


class Tensor:
    """A dense device tensor without memory."""

    def __init__(self, world, shape, dtype, device=CUDA, strides=None, address=None):
        self.world, self.shape, self.dtype, self.device = world, torch.Size(shape), dtype, device
        self.is_cuda, self.ndim = device.type == "cuda", len(self.shape)
        dense = [1]
        for n in reversed(self.shape[1:]):
            dense.insert(0, dense[0] * n)
        self.strides = tuple(dense if strides is None else strides)
        self.contiguous_, self.stream, self.recorded = strides is None, world.current, []
        world.top += 1 << 24
        self.address = world.top if address is None else address

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def dim(self):
        return self.ndim

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self.contiguous_

    def data_ptr(self):
        return self.address

    def record_stream(self, stream):
        self.recorded.append(stream)

    def new_empty(self, *shape, dtype=None):
        shape = shape[0] if isinstance(shape[0], (tuple, list)) else shape
        return self.world.made(Tensor(self.world, shape, dtype or self.dtype, self.device))


class World:
    """The torch module and the library as the binding sees them.  `calls` are
    the library calls by name with their arguments, `allocations` the tensors
    that the binding made; `refuse` maps a call's name to a status."""

    def __init__(self, monkeypatch):
        self.top, self.calls, self.allocations, self.refuse = 1 << 32, [], [], {}
        self.current = self.default = Stream(0)
        self.lib = lb.lib()
        cuda = types.SimpleNamespace(current_device=lambda: 0, current_stream=lambda device=None: self.current, stream=self.on)
        stub = types.SimpleNamespace(
            empty=lambda shape, dtype, device: self.made(Tensor(self, (shape,) if isinstance(shape, int) else shape, dtype, torch.device(device))),
            empty_strided=lambda shape, strides, dtype, device: self.made(Tensor(self, shape, dtype, torch.device(device))),
            cuda=cuda, _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda index: self.current.cuda_stream),
            **{k: getattr(torch, k) for k in ("bfloat16", "float32", "float16", "int32", "uint8", "float64", "int8")})
        monkeypatch.setattr(lb, "_torch_module", stub)
        monkeypatch.setattr(lb, "_lib", self)

    def __getattr__(self, name):
        """A library call.  What the library answers on the host goes to it
        (queries, and calls without workspace or tokens, which it only checks);
        the others are noted."""
        if not name.startswith("lb_"):
            raise AttributeError(name)
        if name.endswith("_bytes") or name == "lb_status_string":
            return getattr(self.lib, name)

        def call(*args):
            if (name.startswith("lb_adapters") and args[-2] == 0) or (name == "lb_heads_norm_rotate" and args[0] == 0):
                return getattr(self.lib, name)(*args)
            self.calls.append((name, args))
            return self.refuse.get(name, lb.LB_OK)
        return call

    @contextlib.contextmanager
    def on(self, stream):
        before, self.current = self.current, stream
        try:
            yield
        finally:
            self.current = before

    def made(self, tensor):
        self.allocations.append(tensor)
        return tensor

    def tensor(self, *shape, dtype=torch.bfloat16, **kw):
        return Tensor(self, shape, dtype, **kw)

    def path(self, n_in, n_out, rank):
        words = lambda n: (n + 31) // 32
        i32, f16 = torch.int32, torch.float16
        return lb.PackedPath(self.tensor(n_out, words(rank), dtype=i32), self.tensor(rank, words(n_in), dtype=i32),
                             self.tensor(n_out, dtype=f16), self.tensor(n_in, dtype=f16), self.tensor(rank, dtype=f16), rank)

    def pool(self, count, rank, n_in, n_out, **kw):
        return lb.AdapterPool(self.tensor(count, rank, n_in), self.tensor(count, n_out, rank), **kw)

    def names(self):
        return [name for name, _ in self.calls]
