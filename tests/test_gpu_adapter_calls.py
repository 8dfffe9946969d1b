"""The adapter path's calls at their edges: workspaces of other batches, waits
that give up in every kind of pass, no rows at all."""

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


FORMS = [("da", "db", "dx"), ("da",), ("db",), ("dx",)]  # passes of both kinds, of gradients alone, of rows alone


def only(c, s, form, **kw):
    """c's backward with the results that `form` names."""
    return c.backward(s, **{k: None for k in ("dx", "da", "db") if k not in form}, **kw)


@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("mapped", [False, True])
@pytest.mark.parametrize("r", [16, 64])
def test_waits_that_give_up_anywhere_leave_the_next_call_right(r, mapped, form):
    # which role gives up first is a matter of timing: each must drain its own work
    c = Case([900, 130, 0, 2300], r, 1096, 1544, mapped=mapped, seed=22)
    s = c.s()
    want = only(c, s, form)
    torch.cuda.synchronize()
    for _ in range(10):
        only(c, s, form, flags=e4b.FLAG_TEST_TIMEOUT)
        assert e4b.e4b_status_string(int(c.status)) == "device wait timed out"
        c.status.zero_()
        got = only(c, s, form)
        assert int(c.status) == 0
        for k in form:
            same = (lambda t: t[c.used]) if k == "dx" else (lambda t: t)
            assert torch.equal(same(got[k]), same(want[k])), k


@pytest.mark.parametrize("form", [("da",), ("db",), ("da", "db")], ids=str)
def test_mapped_gradients_alone_over_many_stages(form):
    # nothing comes by TMA in these passes; stages go round many times
    c = Case([9000, 0, 3000], 16, 1544, 1288, mapped=True, seed=23)
    s = c.s()
    want = c.backward(s)
    c.check_backward(s, want)
    for _ in range(5):
        got = only(c, s, form)
        for k in form:
            assert float((got[k] - want[k]).norm()) <= 2 ** -20 * float(want[k].norm()), k  # cut otherwise, in fp32
    assert int(c.status) == 0


def test_without_rows_tokens_and_gates_get_zeros():
    T, k, H = 5, 3, 72
    BF16, F32 = torch.bfloat16, torch.float32
    inv = torch.arange(T * k, dtype=torch.int32, device="cuda")  # every position is behind the last row
    gates = torch.full((T, k), float("nan"), device="cuda")      # of dropped slots: not read
    rows = torch.empty(0, H, dtype=BF16, device="cuda")
    for g in (gates, None):
        y = torch.full((T, H), 3.0, dtype=BF16, device="cuda")
        e4b.e4b_unpermute(rows, inv, g, y, top_k=k)
        assert not bool(y.any())
    dx = torch.full((T, H), 3.0, dtype=BF16, device="cuda")
    e4b.e4b_permute_backward(rows, inv, dx, top_k=k)
    assert not bool(dx.any())
    dy, dgates = torch.ones(T, H, dtype=BF16, device="cuda"), torch.full((T, k), 3.0, device="cuda")
    e4b.e4b_unpermute_backward(dy, rows, inv, gates, torch.empty_like(rows), dgates, top_k=k)
    assert not bool(dgates.any())
    e4b.e4b_unpermute_backward(dy, rows, inv, gates, torch.empty_like(rows), None, top_k=k)
    e4b.e4b_permute(torch.ones(T, H, dtype=BF16, device="cuda"), inv, torch.zeros(3, dtype=torch.int64, device="cuda"),
                    torch.empty_like(rows), top_k=k)


def test_adapters_without_rows():
    G, r, K, N = 3, 16, 64, 96
    BF16 = torch.bfloat16
    a, b = torch.ones(G, r, K, dtype=BF16, device="cuda"), torch.ones(G, N, r, dtype=BF16, device="cuda")
    off = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
    x, y = torch.empty(0, K, dtype=BF16, device="cuda"), torch.empty(0, N, dtype=BF16, device="cuda")
    s = torch.empty(0, r, device="cuda")
    ws = torch.empty(e4b.e4b_lora_workspace_size(G, r, N, K, 0, True), dtype=torch.uint8, device="cuda")
    e4b.e4b_lora(a, b, x, off, ws, base=y, y=y, s=s)
    e4b.e4b_lora_backward(a, b, None, None, y, off, ws, dx=x, dx_base=x)
    da, db = torch.full((G, r, K), 3.0, device="cuda"), torch.full((G, N, r), 3.0, device="cuda")
    e4b.e4b_lora_backward(a, b, x, s, y, off, ws, dx=x, dx_base=x, da=da, db=db, accumulate=True)
    assert bool((da == 3.0).all()) and bool((db == 3.0).all())
    e4b.e4b_lora_backward(a, b, x, s, y, off, ws, dx=x, dx_base=x, da=da, db=db)
    assert not bool(da.any()) and not bool(db.any())


@pytest.mark.parametrize("mapped", [False, True])
@pytest.mark.parametrize("r", [16, 64])
def test_rows_with_strides_on_whole_tiles(r, mapped):
    # every row buffer with a padding of its own, on another stream; the padding is neither read nor written
    c = Case([6000, 131, 0, 2000], r, 2312, 520, mapped=mapped, seed=24)
    assert c.R * c.K * c.r > 2e8  # s on tiles
    want_f = c.forward()
    s = c.s()
    want_b = c.backward(s)
    pads = []

    def wide(t, pad):
        whole = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
        whole[:, :t.shape[1]] = t
        pads.append(whole[:, t.shape[1]:])
        return whole[:, :t.shape[1]]
    x, dy, base, dx_base = wide(c.x, 8), wide(c.dy, 24), wide(c.base, 40), wide(c.dx_base, 16)
    y, dx = wide(want_f["y"], 56), wide(want_b["dx"], 8)
    y.fill_(123.0)
    dx.fill_(123.0)
    da, db, sf = torch.empty_like(want_b["da"]), torch.empty_like(want_b["db"]), torch.empty_like(want_f["s"])
    ws = [c.ws(False), c.ws(True)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kw = dict(scale=c.scale, row=c.row, status=c.status, stream=side)
    e4b.e4b_lora(c.a, c.b, x, c.offsets, ws[0], base=base, y=y, s=sf, **kw)
    e4b.e4b_lora_backward(c.a, c.b, x, s, dy, c.offsets, ws[1], dx=dx, dx_base=dx_base, da=da, db=db, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want_f["y"]) and torch.equal(dx, want_b["dx"]) and torch.equal(sf[:c.n], want_f["s"][:c.n])
    assert torch.equal(da, want_b["da"]) and torch.equal(db, want_b["db"])
    assert all(bool(torch.isnan(p).all()) for p in pads) and int(c.status) == 0
