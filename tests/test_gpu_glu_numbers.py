"""The gated activation on stored rows where gates and ups are of any size: the
forward kernel, the h that its gradient writes again, and the definition."""

import pytest
import torch

import adapter_ref as ref
from bit_grouped_moe_e4b_b200 import e4b

pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64


def both(g, u, layout, act):
    """h of e4b_glu and of e4b_glu_backward for pairs [n]."""
    gu = ref.join_gu(g[None], u[None], layout).contiguous()
    h = torch.empty(1, len(g), dtype=BF16, device="cuda")
    again, dgu = torch.empty_like(h), torch.empty_like(gu)
    e4b.e4b_glu(gu, h, layout=layout, act=act)
    e4b.e4b_glu_backward(torch.ones_like(h), gu, dgu, h=again, layout=layout, act=act)
    return h[0], again[0]


@pytest.mark.parametrize("layout", ["halves", "interleaved"])
@pytest.mark.parametrize("act", ["swiglu", "clamped_glu"])
def test_huge_pairs_do_not_overflow_on_the_way(layout, act):
    side = torch.tensor([0.0, 1e-30, 0.5, 2.0, 7.0, 8.0, 30.0, 80.0, 1e3, 1e20, 3e38])
    side = torch.cat([side, -side]).to(BF16).cuda()
    g, u = (t.reshape(-1) for t in torch.meshgrid(side, side, indexing="ij"))
    n = len(g) // 8 * 8
    g, u = g[:n].contiguous(), u[:n].contiguous()
    h, again = both(g, u, layout, act)
    want = ref.glu(g, u, act)[0]
    fine = want.abs() <= 3.38e38  # bf16's range
    assert bool(torch.isfinite(h[fine].float()).all())
    assert bool((torch.isinf(h[~fine].float()) & (h[~fine].double().sign() == want[~fine].sign())).all())
    # half a bf16 step and 2^-18 of the value; a sigmoid below 2^-126 counts as zero, which leaves 2^-124 of |g u'| at most
    up = torch.clamp(u.double().abs(), max=7.0) + 1 if act == "clamped_glu" else u.double().abs()
    err = (h.double() - want).abs()[fine]
    # bf16's steps end at 2^-133 (smallest exponent -126, seven bits behind it): half of that below 2^-126, where the
    # relative bound would ask for more bits than the type has (1e-30 * 1e-30 / 2 is 0)
    step = 2.0 ** -134
    assert bool((err <= (2 ** -8 + 2 ** -18) * want.abs()[fine] + 2.0 ** -124 * (g.double().abs() * up)[fine] + step).all())
    assert torch.equal(h, again)


@pytest.mark.parametrize("layout", ["halves", "interleaved"])
@pytest.mark.parametrize("act", ["swiglu", "clamped_glu"])
def test_the_gradient_writes_the_forward_h_again(layout, act):
    gen = torch.Generator(device="cuda").manual_seed(3)
    g, u = (torch.randn(40960, generator=gen, device="cuda").mul_(6.0).to(BF16) for _ in range(2))
    h, again = both(g, u, layout, act)
    assert torch.equal(h, again)
