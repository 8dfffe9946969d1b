"""The adapter path's entry points without a GPU: argument checks on the host,
the argument structs' layout, and the 64-bit reference of the GPU tests."""

import ctypes
import os
import subprocess

import pytest
import torch

import adapter_ref as ref
from conftest import ROOT
from bit_grouped_moe_e4b_b200 import e4b

P = 4096  # a pointer that is never followed: every call below is refused or does nothing
OK, INVALID, UNSUPPORTED, SMALL, MISALIGNED = 0, 1, 2, 3, 7


def test_structs_match_the_header(tmp_path):
    structs = {"e4b_glu_args": e4b.GluArgs, "e4b_lora_args": e4b.LoraArgs}
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "e4b.h"', "int main(void) {"]
    for cname, py in structs.items():
        src.append(f'printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        src += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src += ["return 0; }"]
    c, exe = tmp_path / "layout.c", tmp_path / "layout"
    c.write_text("\n".join(src))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    got = {}
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        s, f, v = line.split()
        got[(s, f)] = int(v)
    for cname, py in structs.items():
        assert got[(cname, "sizeof")] == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)


def test_rows_refusals():
    L = e4b.lib()

    def permute(x=P, ld_x=64, T=4, H=64, perm=P, k=2, off=P, E=8, R=8, xs=P, ld_xs=64):
        return L.e4b_permute(x, ld_x, T, H, perm, k, off, E, R, xs, ld_xs, None)

    assert permute(T=0) == OK and permute(R=0) == OK
    assert permute(T=-1) == INVALID and permute(k=0) == INVALID and permute(H=0) == INVALID and permute(E=0) == INVALID
    assert permute(H=60) == UNSUPPORTED and permute(T=1 << 30, k=2) == UNSUPPORTED
    assert permute(x=None) == INVALID and permute(perm=None) == INVALID and permute(off=None) == INVALID
    assert permute(xs=None) == INVALID and permute(ld_x=56) == INVALID and permute(ld_xs=0) == INVALID
    assert permute(ld_x=68) == MISALIGNED and permute(x=P + 8) == MISALIGNED and permute(xs=P + 2) == MISALIGNED

    def back(ys=P, ld=64, R=8, H=64, inv=P, g=P, T=4, k=2, y=P, ld_y=64, f=L.e4b_unpermute):
        return f(ys, ld, R, H, inv, g, T, k, y, ld_y, None)

    assert back(T=0) == OK
    assert back(inv=None) == INVALID and back(y=None) == INVALID and back(ys=None) == INVALID
    assert back(ld=32) == INVALID and back(R=-1) == INVALID
    assert back(H=12) == UNSUPPORTED and back(ys=P + 4) == MISALIGNED and back(ld_y=66) == MISALIGNED
    assert L.e4b_permute_backward(P + 8, 64, 8, 64, P, 4, 2, P, 64, None) == MISALIGNED
    assert L.e4b_permute_backward(P, 64, 8, 64, None, 4, 2, P, 64, None) == INVALID

    def grad(dy=P, ys=P, inv=P, dys=P, dg=P, H=64, ld_dys=64, T=4):
        return L.e4b_unpermute_backward(dy, 64, ys, 64, 8, H, inv, P, T, 2, dys, ld_dys, dg, None)

    assert grad(T=0) == OK
    assert grad(dys=None, dg=None) == INVALID and grad(dy=None) == INVALID and grad(inv=None) == INVALID
    assert grad(ys=None) == INVALID  # needed for dgates
    assert grad(ld_dys=8) == INVALID and grad(dys=P + 8) == MISALIGNED and grad(H=20) == UNSUPPORTED


def test_glu_refusals():
    L = e4b.lib()

    def call(backward=True, **kw):
        a = e4b.GluArgs(4, 0, 0, 1.702, 7.0, 64, 8, P, P, 128, P, 64, P, 64, P, 128)
        for k, v in kw.items():
            setattr(a, k, v)
        return (L.e4b_glu_backward if backward else L.e4b_glu)(ctypes.byref(a), None)

    for b in (False, True):
        assert call(b, R_max=0) == OK
        assert call(b, I=0) == INVALID and call(b, R_max=-1) == INVALID and call(b, E=0) == INVALID
        assert call(b, I=60) == UNSUPPORTED
        assert call(b, gate_up_layout=2) == INVALID and call(b, activation=3) == INVALID
        assert call(b, activation=1, glu_limit=-1.0) == INVALID
        assert call(b, activation=1, glu_limit=float("nan")) == INVALID
        assert call(b, gu=None) == INVALID and call(b, ld_gu=120) == INVALID
        assert call(b, gu=P + 2) == MISALIGNED and call(b, ld_gu=132) == MISALIGNED
        assert call(b, h=P + 8) == MISALIGNED
    assert call(False, h=None) == INVALID
    assert call(dh=None) == INVALID and call(dgu=None) == INVALID and call(ld_dgu=64) == INVALID
    assert call(ld_gu=136) == INVALID  # in place (dgu is gu) with another stride
    assert L.e4b_glu(None, None) == INVALID and L.e4b_glu_backward(None, None) == INVALID


def lora_args(**kw):
    a = e4b.LoraArgs(4, 16, 64, 128, 8, P, P, None, P, None, 0, P, 128, P, P, 64, P, 64, None, 32, 0, 0, 1.702, 7.0,
                     P, 64, P, 128, P, 128, P, P)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("backward", [False, True])
def test_lora_refusals(backward):
    L = e4b.lib()
    f = L.e4b_lora_backward if backward else L.e4b_lora
    n = e4b.e4b_lora_workspace_size(4, 16, 64, 128, 8, backward)

    def call(ws=P, ws_bytes=n, flags=0, **kw):
        return f(ctypes.byref(lora_args(**kw)), ws, ws_bytes, flags, None)

    assert f(None, P, n, 0, None) == INVALID
    for bad in ({"G": 0}, {"r": 0}, {"N": 0}, {"K": -8}, {"R_max": -1}, {"a": None}, {"b": None}, {"offsets": None},
                {"ws": None}, {"flags": 0x40}, {"row": P, "rows": -1}):
        assert call(**bad) == INVALID, bad
    for bad in ({"r": 4}, {"r": 12}, {"r": 72}, {"N": 60}, {"K": 100}, {"G": 2000}, {"R_max": 1 << 31}):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in ({"a": P + 8}, {"b": P + 2}, {"s": P + 4}, {"ws": P + 8}):
        assert call(**bad) == MISALIGNED, bad
    assert call(ws_bytes=n - 1) == SMALL
    if backward:
        assert call(dx=None, da=None, db=None) == INVALID
        assert call(dy=None) == INVALID and call(x=None) == INVALID and call(s=None) == INVALID
        assert call(ld_dy=32) == INVALID and call(ld_dx=64) == INVALID
        assert call(ld_dx_base=136) == INVALID  # in place with another stride
        assert call(dx=P + 8) == MISALIGNED and call(da=P + 4) == MISALIGNED and call(ld_dy=68) == MISALIGNED
        assert call(dx_base=P + 2) == MISALIGNED
    else:
        assert call(R_max=0) == OK
        assert call(flags=e4b.FLAG_ACCUMULATE) == INVALID
        assert call(y=None, s=None) == INVALID
        assert call(x=None) == INVALID and call(ld_x=64) == INVALID and call(ld_y=32) == INVALID
        assert call(ld_base=72) == INVALID
        assert call(x=P + 8) == MISALIGNED and call(y=P + 2) == MISALIGNED and call(base=P + 4) == MISALIGNED
        assert call(h=P, gate_up_layout=5) == INVALID and call(h=P, activation=1, glu_limit=-2.0) == INVALID
        assert call(h=P, N=72, ld_y=72, ld_base=72, ws_bytes=1 << 30) == UNSUPPORTED  # N / 2 not a multiple of 8
        assert call(h=P, ld_h=16) == INVALID and call(h=P + 2) == MISALIGNED


def test_lora_workspace_size_refusals():
    for bad in ((0, 16, 64, 64, 8), (4, 16, -1, 64, 8)):
        with pytest.raises(e4b.E4BError) as e:
            e4b.e4b_lora_workspace_size(*bad)
        assert e.value.status == INVALID
    for bad in ((4, 20, 64, 64, 8), (4, 128, 64, 64, 8), (4, 16, 68, 64, 8), (1025, 16, 64, 64, 8),
                (4, 16, 1 << 30, 1 << 30, 1 << 30)):
        with pytest.raises(e4b.E4BError) as e:
            e4b.e4b_lora_workspace_size(*bad)
        assert e.value.status == UNSUPPORTED, bad
    # grows with the rows, and holds t of every row for the backward pass
    one = e4b.e4b_lora_workspace_size(8, 16, 256, 512, 1000, True)
    two = e4b.e4b_lora_workspace_size(8, 16, 256, 512, 2000, True)
    assert one >= 1000 * 16 * 4 and two > one


def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    bf = torch.bfloat16
    i32, i64 = torch.int32, torch.int64
    with pytest.raises(ValueError, match="CUDA"):
        e4b.e4b_permute(z(4, 8, dtype=bf), z(8, dtype=i32), z(3, dtype=i64), z(8, 8, dtype=bf), top_k=2)
    with pytest.raises(ValueError, match="CUDA"):
        e4b.e4b_unpermute(z(8, 8, dtype=bf), z(8, dtype=i32), None, z(4, 8, dtype=bf), top_k=2)
    with pytest.raises(ValueError, match="CUDA"):
        e4b.e4b_glu(z(4, 16, dtype=bf), z(4, 8, dtype=bf))
    with pytest.raises(ValueError, match="CUDA"):
        e4b.e4b_lora(z(2, 8, 16, dtype=bf), z(2, 8, 8, dtype=bf), z(4, 16, dtype=bf), z(3, dtype=i64),
                     z(256, dtype=torch.uint8), y=z(4, 8, dtype=bf))


# ----------------------------------------------- the reference of the GPU tests
def test_reference_gradients_by_autograd():
    g = torch.Generator().manual_seed(0)
    G, r, K, N, R = 3, 8, 24, 32, 11
    a = torch.randn(G, r, K, generator=g, dtype=torch.float64).requires_grad_()
    b = torch.randn(G, N, r, generator=g, dtype=torch.float64).requires_grad_()
    x = torch.randn(R, K, generator=g, dtype=torch.float64).requires_grad_()
    off, w = torch.tensor([0, 4, 4, 11]), torch.tensor([0.5, 1.0, -2.0])
    dy = torch.randn(R, N, generator=g, dtype=torch.float64)
    s, y = [], []
    for e in range(G):
        s.append(x[off[e]:off[e + 1]] @ a[e].T)
        y.append(w[e].double() * (s[-1] @ b[e].T))
    torch.cat(y).backward(dy)
    m = ref.Lora(a.detach(), b.detach(), off, w)
    s_ref, _, y_ref, _ = m.forward(x.detach(), None, R, R)
    assert torch.allclose(s_ref, torch.cat(s).detach()) and torch.allclose(y_ref, torch.cat(y).detach())
    dx, _, da, _, db, _ = m.backward(x.detach(), s_ref, dy, None, R)
    assert torch.allclose(dx, x.grad) and torch.allclose(da, a.grad) and torch.allclose(db, b.grad)


@pytest.mark.parametrize("act", ["swiglu", "clamped_glu"])
def test_reference_activation_gradient_by_autograd(act):
    g = torch.randn(500, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * 5
    u = g.flip(0).clone()
    g.requires_grad_(), u.requires_grad_()
    h, dg, du = ref.glu(g, u, act)
    h.sum().backward()
    assert torch.allclose(g.grad, dg.detach()) and torch.allclose(u.grad, du.detach())


def test_reference_routing_against_the_oracle():
    import oracle
    ids = torch.randint(0, 9, (40, 3), generator=torch.Generator().manual_seed(2))
    counts, offsets, perm, inv = ref.routing(ids, 9)
    rc, ro, rp, ri = oracle.route_ref(ids.numpy().astype("int32"), 9)
    assert (counts.numpy() == rc).all() and (offsets.numpy() == ro).all()
    assert (perm.numpy() == rp).all() and (inv.numpy() == ri).all()
