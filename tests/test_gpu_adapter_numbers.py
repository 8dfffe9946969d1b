"""The numbers of the adapters' products: how many bits of the fp32 factors they
keep, and what infinities become. Against the definitions in 64 bits."""

import pytest
import torch

import adapter_ref as ref
from bit_grouped_moe_e4b_b200 import e4b

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def workspace(G, r, N, K, R, backward):
    return torch.empty(e4b.e4b_lora_workspace_size(G, r, N, K, R, backward), dtype=torch.uint8, device="cuda")


def even_groups(G, each):
    return torch.arange(G + 1, dtype=torch.int64, device="cuda") * each


# -------------------------------------------------- factors with 24 bits
class Cancelling:
    """out = base + v_0 W_0 + v_1 W_1 where base takes nearly all of v_0 W_0 away
    and v_1 W_1 nearly all of what is left: out is near 2^-17 of the terms, so
    that an error of the factor v_0 shows. v has 24 bits: each is the sum of
    three bf16 values 8 bits apart, times ones, exact in fp32 in any order."""

    def __init__(self, r, C, G=24, each=20):
        g = torch.Generator().manual_seed(r + C)
        self.G, self.r, self.C, self.each, self.R = G, r, C, each, G * each
        v = 1 + 0.25 * torch.rand(G, 2, generator=g)  # fp32 in [1, 1.25)
        self.pieces = torch.zeros(G, r, 8)            # of the two factors that are not zero
        self.at = (0, r - 1)
        for j, f in zip(self.at, v.unbind(1)):
            left = f.clone()
            for k in range(3):
                # cut, not rounded: 8 bits a piece
                self.pieces[:, j, k] = (left.view(torch.int32) & -65536).view(F32)
                left = left - self.pieces[:, j, k]
            assert not bool(left.any())
        v = v.double()
        w = torch.zeros(G, C, r, dtype=F64)
        w[:, :, 0] = (1 + 0.25 * torch.rand(G, C, generator=g)).to(BF16).double()
        base = -(v[:, :1] * w[:, :, 0]).to(BF16).double()
        left = base + v[:, :1] * w[:, :, 0]
        w[:, :, r - 1] = (-left / v[:, 1:]).to(BF16).double()
        self.want = (left + v[:, 1:] * w[:, :, r - 1]).repeat_interleave(each, 0)
        self.w, self.base = w.to(BF16), base.to(BF16).repeat_interleave(each, 0)
        assert float(self.want.abs().max()) <= 2.0 ** -16  # half a bf16 step of half a bf16 step, below 2

    def check(self, got):
        """At most six MMAs have products that are not zero, of at most three
        addends below 2, each cut at 2^-23 of its binade; three more such cuts
        where the terms themselves end (2^-24 of a factor below 2). Two terms of
        a factor alone are off by up to 2^-17, three times this and more."""
        err = (6 * 3 + 3) * 2.0 ** -23
        assert ref.off_bf16(got.cpu(), self.want, torch.full_like(self.want, err)) <= 1


@pytest.mark.parametrize("r", [8, 16, 24, 64])
@pytest.mark.parametrize("layout", [None, "halves", "interleaved"])
def test_expanded_rows_keep_24_bits_of_s(r, layout):
    c = Cancelling(r, 96)
    x = torch.zeros(c.R, 8, dtype=BF16, device="cuda")
    x[:, :3] = 1
    y = torch.empty(c.R, c.C, dtype=BF16, device="cuda")
    h = torch.empty(c.R, c.C // 2, dtype=BF16, device="cuda") if layout else None
    e4b.e4b_lora(c.pieces.to(BF16).cuda(), c.w.cuda(), x, even_groups(c.G, c.each), workspace(c.G, r, c.C, 8, c.R, False),
                 base=c.base.cuda(), y=y, h=h, layout=layout or "halves")
    c.check(y)


@pytest.mark.parametrize("r", [8, 16, 24, 64])
def test_row_gradients_keep_24_bits_of_t(r):
    c = Cancelling(r, 96)
    dy = torch.zeros(c.R, 8, dtype=BF16, device="cuda")
    dy[:, :3] = 1
    dx = torch.empty(c.R, c.C, dtype=BF16, device="cuda")
    a = c.w.transpose(1, 2).contiguous()
    b = c.pieces.transpose(1, 2).contiguous().to(BF16)
    e4b.e4b_lora_backward(a.cuda(), b.cuda(), None, None, dy, even_groups(c.G, c.each),
                          workspace(c.G, r, 8, c.C, c.R, True), dx=dx, dx_base=c.base.cuda())
    c.check(dx)


# ------------------------------------------------------------- infinities
def same_kind(got, want):
    """Infinite, with the sign, and NaN at the same places."""
    got, want = got.cpu().double(), want.cpu()
    return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want)) and \
        torch.equal(got[torch.isinf(got)].sign(), want[torch.isinf(want)].sign())


def infinite_case(r, seed=0):
    """Factors of every kind: of 24 bits, of 8 (whose lower terms would be zero),
    powers of two, of both signs."""
    g = torch.Generator().manual_seed(seed + r)
    G, each, K, N = 3, 37, 72, 80
    R = G * each
    a, b = torch.randn(G, r, K, generator=g).to(BF16), torch.randn(G, N, r, generator=g).to(BF16)
    x, dy = torch.randn(R, K, generator=g).to(BF16), torch.randn(R, N, generator=g).to(BF16)
    s = torch.randn(R, r, generator=g)
    s[::3] = s[::3].to(BF16).float()
    s[::5] = torch.sign(s[::5]) * 0.25
    return G, each, K, N, R, a, b, x, dy, s, g


@pytest.mark.parametrize("r", [8, 16, 40, 64])
def test_infinite_rows_make_infinite_gradients(r):
    G, each, K, N, R, a, b, x, dy, s, _ = infinite_case(r)
    # t of 24 bits, of 8 and of one: of rows of dy with all, one and one simple value
    dy[::3] = 0
    dy[::3, 0] = 1.5
    b[:, 0] = 0.5
    t = torch.stack([dy[p].double() @ b[p // each].double() for p in range(R)])
    x[5, 3], x[40, 9], x[42, 10], x[42, 11] = float("inf"), -float("inf"), float("inf"), -float("inf")
    x[80, 20], x[81, 20] = float("inf"), float("inf")
    da, db = torch.empty(G, r, K, device="cuda"), torch.empty(G, N, r, device="cuda")
    off = even_groups(G, each)
    ws = workspace(G, r, N, K, R, True)
    e4b.e4b_lora_backward(a.cuda(), b.cuda(), x.cuda(), None, dy.cuda(), off, ws, da=da)
    want = torch.stack([t[g * each:(g + 1) * each].T @ x[g * each:(g + 1) * each].double() for g in range(G)])
    assert bool(torch.isinf(want).any()) and same_kind(da, want)
    dy[6, 4], dy[41, 8], dy[45, 7] = float("inf"), -float("inf"), float("inf")
    e4b.e4b_lora_backward(a.cuda(), b.cuda(), None, s.cuda(), dy.cuda(), off, ws, db=db)
    want = torch.stack([dy[g * each:(g + 1) * each].double().T @ s[g * each:(g + 1) * each].double() for g in range(G)])
    assert bool(torch.isinf(want).any()) and same_kind(db, want)


@pytest.mark.parametrize("r", [8, 16, 40, 64])
def test_infinite_weights_and_factors_make_infinite_rows(r):
    G, each, K, N, R, a, b, x, dy, s, _ = infinite_case(r, 1)
    off = even_groups(G, each)
    x[::4] = 0
    x[::4, 0] = 2.0  # s of few bits
    a[:, :, 0] = a[:, :, 0].sign() * 0.5
    b[1, 7, 2], b[1, 20, r - 1], b[2, 9, 0] = float("inf"), -float("inf"), float("inf")
    x[30, 5] = float("inf")  # an infinite factor
    y = torch.empty(R, N, dtype=BF16, device="cuda")
    e4b.e4b_lora(a.cuda(), b.cuda(), x.cuda(), off, workspace(G, r, N, K, R, False), y=y)
    xa = torch.stack([a[p // each].double() @ x[p].double() for p in range(R)])
    want = torch.stack([b[p // each].double() @ xa[p] for p in range(R)])
    assert bool(torch.isinf(want).any()) and same_kind(y, want)
    b[~torch.isfinite(b.float())] = 1.0
    dy[::4] = 0
    dy[::4, 0] = 2.0
    b[:, 0] = 0.25
    a[0, 3, 7], a[1, 0, 9], a[2, r - 1, 11] = float("inf"), -float("inf"), float("inf")
    dx = torch.empty(R, K, dtype=BF16, device="cuda")
    e4b.e4b_lora_backward(a.cuda(), b.cuda(), None, None, dy.cuda(), off, workspace(G, r, N, K, R, True), dx=dx)
    t = torch.stack([dy[p].double() @ b[p // each].double() for p in range(R)])
    want = torch.stack([t[p] @ a[p // each].double() for p in range(R)])
    assert bool(torch.isinf(want).any()) and same_kind(dx, want)
