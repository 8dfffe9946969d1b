"""The adapters' workspace: one sized for the largest batch serves the others."""

import random

import pytest

from bit_grouped_moe_e4b_b200 import e4b

SHAPES = [  # G, r, N, K
    (8, 16, 28672, 4096), (1, 16, 4096, 4096), (16, 16, 4096, 4096), (128, 32, 1536, 2048), (32, 64, 2880, 2880),
    (1024, 8, 64, 64), (3, 48, 8, 100000), (2, 64, 100000, 8), (7, 24, 328, 1096),
]


def sizes_of_rows(limit, rng):
    """Every row count at first, then counts around whole tiles and between."""
    rows, R = [], 0
    while R < limit:
        R += 1 if R < 70 else max(1, R // rng.choice([9, 30, 100]))
        rows += [R, R // 128 * 128 + 127, R // 128 * 128 + 128]
    return sorted(set(rows))


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_size_never_falls_with_the_rows(shape, backward):
    before = e4b.e4b_lora_workspace_size(*shape, 0, backward)
    for R in sizes_of_rows(300000, random.Random(sum(shape))):
        n = e4b.e4b_lora_workspace_size(*shape, R, backward)
        assert n >= before, (R, n, before)
        assert n >= R * shape[1] * 4 * (2 if backward else 1)  # s; t and its parts
        before = n


def test_size_stays_within_what_the_rows_are_worth():
    # beside x and y, or dy and dx, of the layer's own batches
    for G, r, N, K, R in ((8, 16, 28672, 4096, 8192), (128, 32, 1536, 2048, 65536)):
        for backward in (False, True):
            assert e4b.e4b_lora_workspace_size(G, r, N, K, R, backward) <= 2 * R * (N + K) // 4
