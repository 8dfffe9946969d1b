"""The adapter path's calls at their edges: workspaces of other batches."""

import pytest
import torch

from bit_grouped_moe_e4b_b200 import e4b
from test_gpu_adapter_tiles import Case

pytestmark = pytest.mark.gpu

GUARD = 8 << 20


@pytest.mark.parametrize("counts,r,K,N", [
    ([700, 0, 85], 16, 4096, 1032), ([33] * 16, 16, 264, 2064), ([1900], 64, 520, 1160), ([1500, 1], 8, 1000, 4104),
    ([2, 1, 0, 9], 32, 2056, 264)], ids=str)
def test_one_workspace_for_smaller_batches(counts, r, K, N):
    # as many rows in the workspace as the largest batch has; nothing is written behind it
    c = Case(counts, r, K, N, seed=21)
    s = c.s()
    for most in (c.R, c.R + 1, 3 * c.R, 8192):
        def ws(backward):
            n = e4b.e4b_lora_workspace_size(c.G, c.r, c.N, c.K, most, backward)
            assert n >= e4b.e4b_lora_workspace_size(c.G, c.r, c.N, c.K, c.R, backward)
            whole = torch.full((n + GUARD,), 255, dtype=torch.uint8, device="cuda")
            held.append((whole, n))
            return whole[:n]
        held = []
        c.ws = ws
        c.check_forward(c.forward())
        c.check_backward(s, c.backward(s))
        assert len(held) == 2
        for whole, n in held:
            assert bool((whole[n:] == 255).all())
    assert int(c.status) == 0
