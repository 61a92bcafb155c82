"""The size query of the router gradient and the call it is for have the same limits."""
import ctypes
import itertools

import pytest

from w4a16_grouped_expert_amd import _lib

P = 256  # a pointer that is never dereferenced
SIZES = [(T, d, E, k) for T, d, E, k in itertools.product(
    (-1, 0, 1, 4, 1 << 24, (1 << 24) + 1), (-8, 0, 4, 8, 60, 64, 1 << 20, (1 << 20) + 8), (-1, 0, 1, 8, 1024, 1025),
    (-1, 0, 1, 2, 8, 9, 16, 17))]


@pytest.mark.parametrize("T,d,E,k", [(4, 64, 8, 17), (4, 64, 64, 17), (4, 64, 8, 9), (4, 60, 8, 2), (0, 60, 8, 2)])
def test_sizes_that_the_call_refuses(T, d, E, k):
    assert _lib.lib().moe_route_backward_workspace_bytes(T, d, E, k) == -1


def test_query_and_call_agree():
    """Without a workspace the call is refused for its sizes, or else for the workspace."""
    L = _lib.lib()
    a = _lib.RouteBackwardArgs()
    for f in ("x", "w_router", "logits", "topk_ids", "topk_weights", "dweights", "dx", "dw_router"):
        setattr(a, f, P)
    a.renormalize = 1
    for T, d, E, k in SIZES:
        need = L.moe_route_backward_workspace_bytes(T, d, E, k)
        assert need == -1 or (need > 0 and need % 256 == 0), (T, d, E, k)
        if T == 0:
            continue  # nothing to do within the limits: the call would go on to launch
        a.T, a.d, a.E, a.k = T, d, E, k
        status = L.moe_route_backward(ctypes.byref(a), None)
        assert status == (3 if need > 0 else 1 if min(T, d, E, k) < 0 or min(d, E, k) == 0 else 2), (T, d, E, k)
