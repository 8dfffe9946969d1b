"""Buffers of more than 2^31 values: rows at their far ends, against the
definitions in 64 bits."""

import pytest
import torch

import adapter_ref as ref
from bit_grouped_moe_e4b_b200 import e4b
from test_gpu_adapters import glu_tol

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def filled(shape, g):
    t = torch.empty(shape, dtype=BF16, device="cuda")
    return t.normal_(0.0, 1.0, generator=g)


def some(n):
    return torch.tensor([0, 1, n // 3, n // 2 + 5, n - 130, n - 2, n - 1], device="cuda")


def test_rows_by_expert_and_back():
    g, T, k, H = gen(1), 300000, 2, 4096
    R = T * k
    assert R * H > 1 << 31
    x = filled((T, H), g)
    inv = torch.randperm(R, generator=g, device="cuda").to(torch.int32)
    perm = torch.empty_like(inv)
    perm[inv.long()] = torch.arange(R, dtype=torch.int32, device="cuda")
    xs = torch.empty(R, H, dtype=BF16, device="cuda")
    e4b.e4b_permute(x, perm, torch.tensor([0, R // 2, R], device="cuda"), xs, top_k=k)
    p = some(R)
    assert torch.equal(xs[p], x[perm[p].long() // k])
    gates, t = torch.rand(T, k, generator=g, device="cuda"), some(T)
    y = torch.empty_like(x)
    e4b.e4b_unpermute(xs, inv, gates, y, top_k=k)
    rows = xs[inv.view(T, k)[t].long()].double()
    want = (rows * gates[t].double()[:, :, None]).sum(1)
    assert ref.off_bf16(y[t], want, 3 * ref.U_SUM * want.abs()) <= 1  # both rows of a token are the same here
    dgates = torch.empty_like(gates)
    e4b.e4b_unpermute_backward(y, xs, inv, gates, None, dgates, top_k=k)
    prod = rows * y[t].double()[:, None]
    assert ref.off_f32(dgates[t], prod.sum(2), (H / 32 + 16) * ref.U_SUM * prod.abs().sum(2)) <= 1
    dys = torch.empty_like(xs)
    e4b.e4b_unpermute_backward(y, None, inv, gates, dys, None, top_k=k)
    at = inv.view(T, k)[t].long()
    want = gates[t].double()[:, :, None] * y[t].double()[:, None]
    assert ref.off_bf16(dys[at].flatten(0, 1), want.flatten(0, 1), ref.U_SUM * want.flatten(0, 1).abs()) <= 1


@pytest.mark.parametrize("layout", ["halves", "interleaved"])
def test_activation(layout):
    g, R, I = gen(2), 80000, 14336
    assert R * 2 * I > 1 << 31
    gu, dh = filled((R, 2 * I), g), filled((R, I), g)
    h, dgu, p = torch.empty_like(dh), torch.empty_like(gu), some(R)
    e4b.e4b_glu(gu, h, layout=layout)
    e4b.e4b_glu_backward(dh, gu, dgu, layout=layout)
    pair = ref.split_gu(gu[p], layout)
    want, dg, du = ref.glu(*pair, "swiglu")
    eh, edg, edu = glu_tol("swiglu", *pair)
    assert ref.off_bf16(h[p], want, eh) <= 1
    d = dh[p].double()
    err = ref.join_gu(d.abs() * edg + 2 ** -20 * (d * dg).abs(), d.abs() * edu + 2 ** -20 * (d * du).abs(), layout)
    assert ref.off_bf16(dgu[p], ref.join_gu(d * dg, d * du, layout), err) <= 1


@pytest.mark.parametrize("mapped", [False, True])
def test_adapters(mapped):
    g, G, r, K, N, R = gen(3), 2, 8, 64, 28672, 80000
    assert R * N > 1 << 31
    off = torch.tensor([0, 100, R], device="cuda")
    row = torch.randperm(R, generator=g, device="cuda").to(torch.int32) if mapped else None
    a, b = filled((G, r, K), g), filled((G, N, r), g)
    x, base = filled((R, K), g), filled((R, N), g)
    y, s = torch.empty_like(base), torch.empty(R, r, device="cuda")
    ws = torch.empty(e4b.e4b_lora_workspace_size(G, r, N, K, R, True), dtype=torch.uint8, device="cuda")
    e4b.e4b_lora(a, b, x, off, ws, base=base, y=y, s=s, row=row)
    p = some(R)
    i = p if row is None else row[p].long()
    grp = (p >= 100).long()
    ag, bg = a[grp].double(), b[grp].double()
    xd = x[i].double()
    want = torch.einsum("prk,pk->pr", ag, xd)
    mag = torch.einsum("prk,pk->pr", ag.abs(), xd.abs())
    assert ref.off_f32(s[p], want, (K / 16 + 24) * ref.U_SUM * mag) <= 1
    add, size = torch.einsum("pnr,pr->pn", bg, want), torch.einsum("pnr,pr->pn", bg.abs(), mag)
    err = (K / 16 + r / 8 + 60) * ref.U_SUM * (size + base[i].double().abs())
    assert ref.off_bf16(y[i], base[i].double() + add, err) <= 1
    # the gradients, of y as dy
    dx, db = torch.empty_like(x), torch.empty(G, N, r, device="cuda")
    e4b.e4b_lora_backward(a, b, None, s, y, off, ws, dx=dx, dx_base=x, db=db, row=row)
    dy = y[i].double()
    t, mag = torch.einsum("pnr,pn->pr", bg, dy), torch.einsum("pnr,pn->pr", bg.abs(), dy.abs())
    want, size = torch.einsum("prk,pr->pk", ag, t), torch.einsum("prk,pr->pk", ag.abs(), mag)
    assert ref.off_bf16(dx[i], xd + want, (N / 16 + r / 8 + 60) * ref.U_SUM * (size + xd.abs())) <= 1
    for e, (lo, hi) in enumerate(((0, 100), (100, R))):
        at = torch.arange(lo, hi, device="cuda") if row is None else row[lo:hi].long()
        cols, sd = y[:, -40:][at].double(), s[lo:hi].double()
        assert ref.off_f32(db[e, -40:], cols.T @ sd, ((hi - lo) / 8 + 28) * ref.U_SUM * (cols.abs().T @ sd.abs())) <= 1
