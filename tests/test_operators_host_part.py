"""Refusals of lapsum_expert_combine_backward_part that need no GPU."""
from tests.test_operators_host import D, lib, refuses  # noqa: F401


def test_combine_backward_part(lib):  # noqa: F811
    ok = (D, 1, 64, D, 10, 4, 64, D, D, D, D, D, None)
    refuses(lib.lapsum_expert_combine_backward_part, ok, [
        (0, None), (3, None), (7, None), (8, None), (9, None), ((10, 11), (None, None)), (1, 4),
        (2, 63), (4, 0), (5, 33), (6, 0), (11, D + 2), (10, D + 1), ((3, 11), (D + 1, None))])
