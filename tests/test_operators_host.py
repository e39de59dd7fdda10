"""Refusals of the routing, expert-row, cache-attention and eviction calls that need
no GPU: every one is decided on the host, before anything is launched."""
import ctypes

import pytest
import torch

import sparse_selection_primitive_b200 as L
from sparse_selection_primitive_b200 import _build, _launch

BAD, WS = 1, 2


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return L._lib()


D = 1 << 20  # stands for a device address; no call below gets as far as using it


def refuses(fn, ok, changes, code=BAD):
    for at, value in changes:
        args = list(ok)
        for i, x in zip(at, value) if isinstance(at, tuple) else ((at, value),):
            args[i] = x
        assert fn(*args) == code, (fn.__name__, at, value)


def test_route(lib):
    ok = (D, 0, 256, 16, 256, 8, 0, None, 1, 1, 2, 1, 1.0, D, D, None)
    refuses(lib.lapsum_route, ok, [
        (0, None), (13, None), (14, None), (1, 3), (1, -1), (2, 255), (3, 0), (3, -1), (4, 0),
        (4, 1025), (5, 0), (5, 33), (6, 2), (6, -1), (8, 0), (8, 33), (8, 3), ((8, 9), (8, 9)),
        ((8, 9), (8, 0)), (10, 0), (10, 3), (12, 0.0), (12, -1.0), (12, float("nan")),
        (12, float("inf")), ((4, 5), (4, 5)), ((8, 9, 5), (64, 1, 8)), ((8, 9, 5), (32, 1, 9)),
        (0, D + 2), (7, D + 1), (13, D + 2), (14, D + 2), ((0, 1), (D + 1, 1))])
    ok = (D, 0, 256, 16, 256, 8, 0, 1, 1.0, D, D, D, D, 256, None)
    refuses(lib.lapsum_route_backward, ok, [
        (0, None), (9, None), (10, None), (11, None), (12, None), (1, 5), (2, 255), (13, 255),
        (3, 0), (5, 0), (6, 9), (8, 0.0), (12, D + 2), (11, D + 1)])


def test_experts(lib):
    size = lib.lapsum_expert_plan_workspace_bytes
    assert size(0, 8) == 0 and size(8, 0) == 0 and size(8, 1025) == 0 and size(1 << 31, 8) == 0
    assert size(1, 1) > 0 and size(1 << 20, 1024) % 256 == 0
    need = size(100000, 64)
    ok = (D, 100000, 64, D, D, D, D, need, None)
    refuses(lib.lapsum_expert_plan, ok, [(0, None), (3, None), (4, None), (5, None), (1, 0),
                                         (2, 0), (2, 1025), (1, 1 << 31), (0, D + 2), (5, D + 1)])
    refuses(lib.lapsum_expert_plan, ok, [(6, None), (6, D + 8), (7, need - 1)], WS)
    ok = (D, 1, 64, 10, 4, 64, D, D, D, None)
    refuses(lib.lapsum_expert_gather, ok, [
        (0, None), (6, None), (7, None), (8, None), (1, 3), (2, 63), (3, 0), (4, 0), (4, 33), (5, 0),
        ((3, 4), (1 << 30, 2)), (0, D + 1), (8, D + 1), (6, D + 2), (7, D + 2)])
    ok = (D, 1, 10, 4, 64, D, D, D, D, None)
    refuses(lib.lapsum_expert_combine, ok, [
        (0, None), (5, None), (6, None), (8, None), (1, 7), (2, 0), (3, 0), (3, 33), (4, 0),
        (7, D + 2), (8, D + 1)])
    ok = (D, 1, 64, D, 10, 4, 64, D, D, D, D, D, None)
    refuses(lib.lapsum_expert_combine_backward, ok, [
        (0, None), (3, None), (7, None), (8, None), (9, None), (10, None), (11, None), (1, 4),
        (2, 63), (4, 0), (5, 33), (6, 0), (11, D + 2)])


def test_attend(lib):
    size = lib.lapsum_attend_workspace_bytes
    for bad in ((0, 1, 8, 2, 100, 64), (1, 0, 8, 2, 100, 64), (1, 1, 8, 3, 100, 64),
                (1, 1, 8, 2, 0, 64), (1, 1, 8, 2, 100, 8), (1, 1, 8, 2, 100, 24),
                (1, 1, 8, 2, 100, 272), (1, 1, 0, 2, 100, 64), (1, 1, 8, 0, 100, 64),
                (1, 1, 8, 2, 1 << 31, 64), (65535, 65535, 8, 2, 100, 64)):
        assert size(*bad) == 0, bad
    need = size(2, 1, 8, 2, 100, 64)
    assert need > 0 and need % 256 == 0
    strides = (ctypes.c_int64 * 13)(512, 64, 512, 12800, 6400, 64, 12800, 6400, 64, 200, 100, 200, 100)
    ok = (D, D, D, 1, D, strides, 2, 1, 8, 2, 100, 64, 0.125, None, D, D, D, need, None)
    refuses(lib.lapsum_attend_accumulate, ok, [
        (0, None), (1, None), (2, None), (4, None), (5, None), (14, None), (15, None), (3, 0), (3, 3),
        (9, 3), (11, 60), (11, 0), (10, 0), (6, 0), (7, 0), (12, float("nan")), (12, float("inf")),
        (0, D + 8), (1, D + 2), (2, D + 4), (15, D + 8), (4, D + 2), (13, D + 1), (14, D + 2)])
    refuses(lib.lapsum_attend_accumulate, ok, [(16, None), (16, D + 128), (17, need - 1)], WS)
    for i, x in ((0, 508), (5, 68), (8, -64), (9, -1)):
        s = (ctypes.c_int64 * 13)(*strides)
        s[i] = x
        refuses(lib.lapsum_attend_accumulate, ok, [(5, s)])


def test_evict(lib):
    strides = (ctypes.c_int64 * 16)(*([100] * 16))
    ok = (D, D, 1, D, D, strides, 2, 2, 100, 64, 10, 2, 3, D, D, D, D, D, None)
    refuses(lib.lapsum_evict, ok, [
        (0, None), (1, None), (3, None), (4, None), (5, None), (13, None), (14, None), (15, None),
        (16, None), (17, None), (2, 3), (6, 0), (7, 0), (8, 0), (9, 0), (10, 0), (11, -1), (12, -1),
        (11, 11), ((11, 12), (6, 5)), (8, 1 << 31), (0, D + 1), (14, D + 1), (3, D + 2), (16, D + 2)])
    s = (ctypes.c_int64 * 16)(*strides)
    s[7] = -1
    refuses(lib.lapsum_evict, ok, [(5, s)])


def test_python_calls_refuse_host_tensors():
    x = torch.zeros((4, 8))
    i = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(TypeError):
        L.route_experts(x, 2)
    with pytest.raises(TypeError):
        L.expert_plan(i, 8)
    c = torch.zeros((1, 2, 4, 16), dtype=torch.bfloat16)
    s, n = torch.zeros((1, 2, 4)), torch.ones(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        L.attend_accumulate(c[:, :, :1], c, c, n, s)
    with pytest.raises(TypeError):
        L.evict(c, c, s, n, 2)


def test_memory_checks():
    x = torch.zeros((4, 6, 8))
    assert _launch.distinct(x) and _launch.distinct(x.transpose(0, 2)) and _launch.distinct(x[:, ::2])
    assert not _launch.distinct(x[:1].expand(4, 6, 8))
    assert not _launch.distinct(x.as_strided((4, 6, 8), (48, 4, 1)))
    assert _launch.distinct(x[:1, :1])
    flat = x.view(-1)
    assert _launch.overlap(flat[:10], flat[9:20]) and not _launch.overlap(flat[:10], flat[10:20])
