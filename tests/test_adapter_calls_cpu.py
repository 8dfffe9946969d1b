"""Calls of the adapter path that have nothing to do, and their limits, on the host."""

import ctypes

from bit_grouped_moe_e4b_b200 import e4b
from test_adapters_cpu import INVALID, OK, P, UNSUPPORTED, lora_args


def test_results_without_rows_need_no_address():
    # an empty tensor's address is NULL
    L = e4b.lib()

    def grad(R, dys=None, dg=None):
        return L.e4b_unpermute_backward(P, 64, None, 64, R, 64, P, P, 4, 2, dys, 64, dg, None)

    assert grad(0) == OK and grad(8) == INVALID
    n = e4b.e4b_lora_workspace_size(4, 16, 64, 128, 0, True)
    empty = {"x": None, "s": None, "dy": None, "dx_base": None, "dx": None, "da": None, "db": None}
    for R, status in ((0, OK), (8, INVALID)):
        a = lora_args(R_max=R, **empty)
        assert L.e4b_lora_backward(ctypes.byref(a), P, n, 0, None) == status


def test_sizes_up_to_the_limits_are_accepted():
    def size(G, r, N, K, R):
        return [e4b.e4b_lora_workspace_size(G, r, N, K, R, backward) for backward in (False, True)]

    for G, r, N, K, R in ((1024, 64, 1 << 30, 64, 1 << 14), (1024, 8, 64, 1 << 30, 1 << 14), (1, 8, 1 << 14, 1 << 14, 1 << 30),
                          (1024, 64, 1 << 14, 8, 1 << 30)):
        s, t = size(G, r, N, K, R)
        assert s >= R * r * 4 and t >= 2 * R * r * 4
    for G, r, N, K, R in ((4, 16, 1 << 30, 64, (1 << 14) + 1), (4, 16, 64, (1 << 14) + 8, 1 << 30), (4, 16, (1 << 30) + 8, 64, 8),
                          (4, 16, 64, 64, (1 << 30) + 1)):
        for backward in (0, 1):
            n = ctypes.c_size_t(0)
            assert e4b.lib().e4b_lora_workspace_size(G, r, N, K, R, backward, ctypes.byref(n)) == UNSUPPORTED
