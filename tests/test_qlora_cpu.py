"""The reference of the adapter layer against automatic differentiation in 64
bits, and the shapes that qlora refuses before any launch."""

import pytest
import torch

import adapter_ref as ref
import qlora_ref
from bit_grouped_moe_e4b_b200 import e4b, qlora


def case(E, H, I, r, T, k, seed):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, std=1.0):
        return torch.randn(*shape, generator=g, dtype=torch.float64) * std
    ad = [(rnd(E, r, K, std=K ** -0.5), rnd(E, N, r, std=0.5 * r ** -0.5), 0.5 + torch.rand(E, generator=g).double())
          for N, K in ((2 * I, H), (H, I))]
    ids = torch.randint(0, E, (T, k), generator=g)
    return (rnd(E, 2 * I, H, std=H ** -0.5), rnd(E, H, I, std=I ** -0.5), rnd(E, 2 * I, std=0.1), rnd(E, H, std=0.1),
            ad[0], ad[1], rnd(T, H), ids, torch.rand(T, k, generator=g), rnd(T, H))


@pytest.mark.parametrize("layout", ["halves", "interleaved"])
@pytest.mark.parametrize("act", ["swiglu", "clamped_glu"])
def test_reference_is_the_gradient(layout, act):
    c = case(3, 16, 12, 4, 9, 2, 1)
    got = qlora_ref.step(*c, layout, act, stored=lambda t: t)
    w_gu, w_dn, b_gu, b_dn, (A1, B1, s1), (A2, B2, s2), x, ids, gates, dy = c
    leaves = [t.detach().clone().requires_grad_() for t in (A1, B1, A2, B2, x, gates.double())]
    A1, B1, A2, B2, x, gates = leaves
    y = []
    for t in range(x.shape[0]):
        row = 0
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            gu = w_gu[e] @ x[t] + b_gu[e] + s1[e] * (B1[e] @ (A1[e] @ x[t]))
            h = ref.glu(*(v[0] for v in ref.split_gu(gu[None], layout)), act)[0]
            row = row + gates[t, j] * (w_dn[e] @ h + b_dn[e] + s2[e] * (B2[e] @ (A2[e] @ h)))
        y.append(row)
    y = torch.stack(y)
    assert torch.allclose(y, got["y"], rtol=1e-10, atol=1e-12)
    for want, name in zip(torch.autograd.grad((y * dy).sum(), leaves), ("gu_a", "gu_b", "dn_a", "dn_b", "dx", "dgates")):
        assert torch.allclose(want, got[name], rtol=1e-9, atol=1e-11), name


def test_adapters_of_other_shapes_are_refused():
    layer = e4b.PackedLayer("nf4", 2, 64, 128, *[torch.zeros(1)] * 4)
    good = [qlora.Adapter(torch.zeros(2, 8, 64), torch.zeros(2, 256, 8)),
            qlora.Adapter(torch.zeros(2, 8, 128), torch.zeros(2, 64, 8))]
    x, ids, gates = torch.zeros(1, 64), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1)
    for i, bad in ((0, qlora.Adapter(torch.zeros(3, 8, 64), torch.zeros(3, 256, 8))),
                   (0, qlora.Adapter(torch.zeros(2, 8, 64), torch.zeros(2, 128, 8))),
                   (1, qlora.Adapter(torch.zeros(2, 8, 64), torch.zeros(2, 64, 8))),
                   (1, qlora.Adapter(torch.zeros(2, 8, 128), torch.zeros(2, 64, 16)))):
        ads = list(good)
        ads[i] = bad
        with pytest.raises(ValueError):
            qlora.forward(layer, *ads, x, ids, gates)
    with pytest.raises(ValueError):
        qlora.forward(e4b.PackedLayer("int4b32", 2, 64, 128, *[torch.zeros(1)] * 4), *good, x, ids, gates)
    with pytest.raises(ValueError):
        qlora.backward(layer, *good, None, x, accumulate=True)
