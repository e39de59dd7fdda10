"""The checks of tensor arguments that the expert and cache calls share, on the host."""
import random
import subprocess
import sys

import pytest
import torch
import torch.autograd.forward_ad as fw

from sparse_selection_primitive_b200 import _launch
from tests.conftest import ROOT


def test_tangents_are_refused():
    x, y = torch.randn(3), torch.randn(3)
    _launch.no_tangents("call", x, y)
    with fw.dual_level():
        _launch.no_tangents("call", x, y)
        dual = fw.make_dual(x, torch.ones(3))
        for args in ((dual,), (y, dual), (dual, y)):
            with pytest.raises(NotImplementedError, match="call"):
                _launch.no_tangents("call", *args)
    _launch.no_tangents("call", x, y)

    def inner(t):
        _launch.no_tangents("call", t)
        return t

    with pytest.raises(NotImplementedError):
        torch.func.jvp(inner, (x,), (torch.ones(3),))


def test_import_without_cuda():
    """The package and its host-side parts are imported with a torch that was built without CUDA,
    which has none of the device calls."""
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda_get')]:\n"
            "    delattr(torch._C, name)\n"
            "import sparse_selection_primitive_b200\n"
            "import sparse_selection_primitive_b200.sharded\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


def _memory(x):
    """The bytes that x's elements take, as a set."""
    starts = torch.zeros((), dtype=torch.int64)
    for n, step in zip(x.shape, x.stride()):
        starts = starts[..., None] + torch.arange(n) * step
    first = x.data_ptr() + starts.reshape(-1) * x.element_size()
    return set((first[:, None] + torch.arange(x.element_size())).reshape(-1).tolist())


def test_apart_of_views():
    """Tensors called apart share no byte, over random pairs of views of one piece of memory;
    the layouts that callers use are told apart."""
    base = torch.zeros(4096, dtype=torch.uint8)
    rng = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        steps = [rng.choice([512, 1024]), rng.choice([64, 128, 256]), rng.choice([8, 16, 32])]
        pair = []
        for _ in range(2):
            dtype = rng.choice([torch.float32, torch.bfloat16])
            es = 4 if dtype is torch.float32 else 2
            shape = (rng.choice([1, 2]), rng.choice([1, 2, 3]), rng.choice([1, 2, 4]), rng.choice([1, 2, 4, 8]))
            if rng.random() < 0.3:
                steps[2] = rng.choice([8, 16, 32])
            at = rng.choice([0, 4, 8, 16, 32, 64]) // es
            pair.append(base.view(dtype).as_strided(shape, [s // es for s in steps] + [1], at))
        a, b = pair
        said = _launch.apart(a, b)
        seen[said] += 1
        assert not said or not (_memory(a) & _memory(b)), (a.shape, a.stride(), b.shape, b.stride())
        assert _launch.apart(b, a) == said
    assert min(seen.values()) > 200
    kv = torch.zeros((2, 3, 10, 2, 8))                 # rows of k and v by turns
    assert _launch.apart(kv[:, :, :, 0], kv[:, :, :, 1])
    assert not _launch.apart(kv[:, :, :, 0], kv[:, :, :, 0])
    heads = torch.zeros((2, 3, 2 * 10 * 8 + 10))       # a head's k, v and scores in one piece
    k, v = (heads[:, :, i * 80:i * 80 + 80].unflatten(2, (10, 8)) for i in (0, 1))
    s = heads[:, :, 160:]
    assert _launch.apart(k, v) and _launch.apart(v, s) and _launch.apart(k, s)
    assert not _launch.apart(k, heads[:, :, 79:89])
    one = torch.zeros((2, 3, 11, 8))                   # a row further on
    assert not _launch.apart(one[:, :, :10], one[:, :, 1:])
