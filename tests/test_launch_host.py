"""The checks of tensor arguments that the expert and cache calls share, on the host."""
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
