"""Calls of the adapter path that have nothing to do, and their limits, on the host."""

import ctypes

from bit_grouped_moe_e4b_b200 import e4b
from test_adapters_cpu import INVALID, OK, P, lora_args


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
