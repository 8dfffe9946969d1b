"""Token rows by expert and back, the gated activation on stored rows and the
grouped low-rank adapters, with their gradients, against their definitions in
64 bits (adapter_ref.py). Every bound counts the roundings of the path: half a
bf16 step of a bf16 result, fp32 sums, two bf16 terms for a value between two
products, 2^-18 for the activation's exp2 and reciprocal."""

import pytest
import torch

import adapter_ref as ref
from bit_grouped_moe_e4b_b200 import e4b

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SENTINEL = 123.0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF16)


def strided(t, pad, fill=SENTINEL):
    """t on the GPU in rows with `pad` more values between them."""
    out = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    out[:, :t.shape[1]] = t.cuda()
    return out[:, :t.shape[1]]


def padding_untouched(t, pad):
    if not pad or t.shape[0] < 2:
        return True
    full = t.as_strided((t.shape[0], t.shape[1] + pad), (t.stride(0), 1))
    return bool((full[:, t.shape[1]:] == SENTINEL).all())


# ------------------------------------------------------------------- rows
ROW_CASES = [  # T, k, E, H, dropped share, row padding
    (1, 1, 1, 8, 0.0, 0), (1, 2, 8, 4096, 0.0, 0), (16, 2, 8, 4096, 0.0, 8), (7, 3, 5, 72, 0.3, 8),
    (33, 8, 128, 2048, 0.1, 0), (130, 4, 32, 2880, 0.0, 0), (257, 1, 3, 256, 0.5, 16), (5, 5, 9, 1000, 0.0, 0),
    (64, 2, 8, 120, 1.0, 0), (301, 7, 11, 16, 0.2, 0),
]


def row_case(T, k, E, H, drop, seed):
    g = gen(seed)
    ids = torch.randint(0, E, (T, k), generator=g)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    _, offsets, perm, inv = ref.routing(ids, E)
    return g, offsets, perm, inv


@pytest.mark.parametrize("T,k,E,H,drop,pad", ROW_CASES)
def test_permute_copies_the_rows(T, k, E, H, drop, pad):
    g, offsets, perm, inv = row_case(T, k, E, H, drop, T * 7 + H)
    R, n = T * k, int(offsets[-1])
    x = randn(g, T, H)
    xs = strided(torch.full((R, H), SENTINEL, dtype=BF16), pad)
    e4b.e4b_permute(strided(x, pad), perm.cuda(), offsets.cuda(), xs, top_k=k)
    got = xs.cpu()
    assert torch.equal(got[:n], x[perm[:n].long() // k])
    assert bool((got[n:] == SENTINEL).all())
    assert padding_untouched(xs, pad)


@pytest.mark.parametrize("T,k,E,H,drop,pad", ROW_CASES)
@pytest.mark.parametrize("weighted", [False, True])
def test_rows_back_to_tokens(T, k, E, H, drop, pad, weighted):
    g, offsets, perm, inv = row_case(T, k, E, H, drop, T * 11 + H)
    R, n = T * k, int(offsets[-1])
    rows = randn(g, R, H)
    rows[n:] = float("nan")  # rows of no slot are not read
    gates = torch.randn(T, k, generator=g)
    gates.view(-1)[inv < 0] = float("nan")  # nor are gates of dropped slots
    y = strided(torch.full((T, H), SENTINEL, dtype=BF16), pad)
    if weighted:
        e4b.e4b_unpermute(strided(rows, pad), inv.cuda(), gates.cuda(), y, top_k=k)
    else:
        e4b.e4b_permute_backward(strided(rows, pad), inv.cuda(), y, top_k=k)
    want, mag = ref.sum_slots(rows, inv, gates if weighted else None, T, k)
    assert ref.off_bf16(y.cpu(), want, (k + 1) * ref.U_SUM * mag) <= 1
    assert padding_untouched(y, pad)


@pytest.mark.parametrize("T,k,E,H,drop,pad", ROW_CASES)
@pytest.mark.parametrize("which", ["both", "rows", "gates", "unweighted"])
def test_unpermute_backward(T, k, E, H, drop, pad, which):
    g, offsets, perm, inv = row_case(T, k, E, H, drop, T * 13 + H)
    R, n = T * k, int(offsets[-1])
    dy, ys = randn(g, T, H), randn(g, R, H)
    ys[n:] = float("nan")
    gates = torch.randn(T, k, generator=g) if which != "unweighted" else None
    dys = strided(torch.full((R, H), SENTINEL, dtype=BF16), pad) if which != "gates" else None
    dgates = torch.full((T, k), SENTINEL, device="cuda") if which != "rows" else None
    e4b.e4b_unpermute_backward(strided(dy, pad), None if which == "rows" else strided(ys, pad), inv.cuda(),
                               None if gates is None else gates.cuda(), dys, dgates, top_k=k)
    tok = perm[:n].long() // k
    w = gates.view(-1)[perm[:n].long()].double()[:, None] if gates is not None else 1.0
    if dys is not None:
        got = dys.cpu()
        want = w * dy[tok].double()
        assert ref.off_bf16(got[:n], want, ref.U_SUM * want.abs()) <= 1
        assert bool((got[n:] == SENTINEL).all())
        assert padding_untouched(dys, pad)
    if dgates is not None:
        prod = dy[tok].double() * ys[:n].double()
        want, mag = torch.zeros(R, dtype=torch.float64), torch.zeros(R, dtype=torch.float64)
        want[perm[:n].long()], mag[perm[:n].long()] = prod.sum(1), prod.abs().sum(1)
        got = dgates.cpu().view(-1)
        assert bool((got[inv < 0] == 0).all())
        # each lane adds H / 32 products, five more additions join the lanes
        assert ref.off_f32(got, want, (H / 32 + 16) * ref.U_SUM * mag) <= 1


def test_unpermute_backward_is_the_gradient_by_differences():
    T, k, E, H = 5, 2, 4, 16
    g, offsets, perm, inv = row_case(T, k, E, H, 0.2, 3)
    ys, dy, gates = randn(g, T * k, H), randn(g, T, H), torch.randn(T, k, generator=g)
    dys = torch.zeros(T * k, H, dtype=BF16, device="cuda")
    dg = torch.zeros(T, k, device="cuda")
    e4b.e4b_unpermute_backward(dy.cuda(), ys.cuda(), inv.cuda(), gates.cuda(), dys, dg, top_k=k)

    def f(rows, gs):
        return float((ref.sum_slots(rows, inv, gs, T, k)[0] * dy.double()).sum())
    for s in range(T * k):  # the function is linear in each of its arguments
        e = torch.zeros(T * k)
        e[s] = 1.0
        slope = (f(ys, gates + e.view(T, k)) - f(ys, gates - e.view(T, k))) / 2
        assert abs(slope - float(dg.cpu().view(-1)[s])) <= 1e-5 * (1 + abs(slope))


def test_rows_repeat_bit_for_bit_and_run_on_another_stream():
    T, k, E, H = 300, 4, 16, 520
    g, offsets, perm, inv = row_case(T, k, E, H, 0.1, 5)
    rows, gates = randn(g, T * k, H).cuda(), torch.randn(T, k, generator=g).cuda()
    inv_d = inv.cuda()
    y = [torch.empty(T, H, dtype=BF16, device="cuda") for _ in range(3)]
    for o in y[:2]:
        e4b.e4b_unpermute(rows, inv_d, gates, o, top_k=k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    e4b.e4b_unpermute(rows, inv_d, gates, y[2], top_k=k, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


# -------------------------------------------------------------- activation
GLU_CASES = [(1, 8, 0), (3, 32, 8), (64, 512, 0), (37, 2880, 0), (5, 14336, 24), (1025, 40, 0), (700, 768, 16)]


def glu_inputs(R, I, seed, std=3.0):
    g = gen(seed)
    gu = randn(g, R, 2 * I, std=std)
    flat = gu.view(-1)
    edge = torch.tensor([7.0, -7.0, 7.03125, -7.03125, 0.0, -0.0, 88.0, -88.0, -120.0, 120.0, 1e-30, -1.28125],
                        dtype=BF16)
    n = min(flat.numel(), 8 * edge.numel())
    flat[:n] = edge.repeat(8)[:n]
    return g, gu


def glu_tol(act, g, u, dh=None):
    """Bounds on h, dg, du before their bf16 rounding: 2^-18 of each factor."""
    e = 2.0 ** -18
    h, dg, du = ref.glu(g, u, act)
    uc = u.double().abs() + 1
    gc = g.double().abs()
    if act == "clamped_glu":
        gc, uc = torch.where(g.double() > 7, torch.full_like(gc, 7.0), gc), torch.clamp(u.double().abs(), max=7) + 1
    sg = torch.sigmoid((1.702 if act == "clamped_glu" else 1.0) * torch.where(g > 0, gc, -gc))
    tiny = 2.0 ** -124  # the reciprocal flushes results below 2^-126 to zero
    eh = 4 * e * h.abs() + tiny * gc * uc
    edg = 8 * e * uc * sg * (1 + 1.702 * gc) + tiny * uc * (1 + gc)
    edu = 4 * e * du.abs() + tiny * gc
    return eh, edg, edu


@pytest.mark.parametrize("R,I,pad", GLU_CASES)
@pytest.mark.parametrize("layout", ["halves", "interleaved"])
@pytest.mark.parametrize("act", ["swiglu", "clamped_glu"])
def test_glu_and_its_gradient(R, I, pad, layout, act):
    gen_, gu = glu_inputs(R, I, R + I)
    g, u = ref.split_gu(gu, layout)
    h_ref, dg, du = ref.glu(g, u, act)
    eh, edg, edu = glu_tol(act, g, u)
    gu_d = strided(gu, pad)
    h = strided(torch.full((R, I), SENTINEL, dtype=BF16), pad)
    e4b.e4b_glu(gu_d, h, layout=layout, act=act)
    assert ref.off_bf16(h.cpu(), h_ref, eh) <= 1
    assert padding_untouched(h, pad)

    dh = randn(gen_, R, I)
    d = dh.double()
    dgu = strided(torch.full((R, 2 * I), SENTINEL, dtype=BF16), pad)
    h2 = strided(torch.full((R, I), SENTINEL, dtype=BF16), pad)
    e4b.e4b_glu_backward(strided(dh, pad), gu_d, dgu, h=h2, layout=layout, act=act)
    want = ref.join_gu(d * dg, d * du, layout)
    err = ref.join_gu(d.abs() * edg + 2 ** -20 * (d * dg).abs(), d.abs() * edu + 2 ** -20 * (d * du).abs(), layout)
    assert ref.off_bf16(dgu.cpu(), want, err) <= 1
    assert ref.off_bf16(h2.cpu(), h_ref, eh) <= 1
    assert padding_untouched(dgu, pad) and padding_untouched(h2, pad)
    e4b.e4b_glu_backward(strided(dh, pad), gu_d, gu_d, layout=layout, act=act)  # in place, without h
    assert torch.equal(gu_d, dgu)


@pytest.mark.parametrize("act", ["swiglu", "clamped_glu"])
def test_glu_gradient_by_differences(act):
    R, I = 16, 64
    g = gen(9)
    gu, dh = randn(g, R, 2 * I, std=2.0), randn(g, R, I)
    gu = torch.where((gu.abs() - 7).abs() < 0.1, torch.ones_like(gu), gu)  # away from the clamps' corners
    dgu = torch.empty(R, 2 * I, dtype=BF16, device="cuda")
    e4b.e4b_glu_backward(dh.cuda(), gu.cuda(), dgu, act=act)
    a, b = ref.split_gu(gu.double(), "halves")
    eps = 1e-6
    sg = (ref.glu(a + eps, b, act)[0] - ref.glu(a - eps, b, act)[0]) / (2 * eps) * dh.double()
    su = (ref.glu(a, b + eps, act)[0] - ref.glu(a, b - eps, act)[0]) / (2 * eps) * dh.double()
    want = torch.cat([sg, su], 1)
    # half a bf16 step, and the difference quotient's own error
    assert float(((dgu.cpu().double() - want).abs() / (ref.U_BF16 * want.abs() + 1e-4)).max()) <= 1


def test_glu_nan_stays_and_rows_past_the_last_are_left():
    R, I = 12, 64
    gu = randn(gen(1), R, 2 * I)
    gu[2, 5] = float("nan")
    gu[3, I + 7] = float("nan")
    offsets = torch.tensor([0, 4, 4, 9]).cuda()
    for act in ("swiglu", "clamped_glu"):
        h = torch.full((R, I), SENTINEL, dtype=BF16, device="cuda")
        dgu = torch.full((R, 2 * I), SENTINEL, dtype=BF16, device="cuda")
        e4b.e4b_glu(gu.cuda(), h, offsets=offsets, act=act)
        e4b.e4b_glu_backward(torch.ones(R, I, dtype=BF16).cuda(), gu.cuda(), dgu, offsets=offsets, act=act)
        nan = torch.isnan(h.cpu())
        assert nan[2, 5] and nan[3, 7] and int(nan.sum()) == 2
        assert bool((h[9:] == SENTINEL).all()) and bool((dgu[9:] == SENTINEL).all())
        assert not bool((h[:9] == SENTINEL).any())


# ----------------------------------------------------------------- adapters
LORA_CASES = [  # rows per group, r, K, N, row map, scale, row padding
    ([1], 8, 8, 16, False, False, 0),
    ([1], 16, 4096, 4096, False, True, 0),
    ([0, 1, 0, 2, 1], 16, 520, 264 + 8, True, True, 8),
    ([16, 17, 31, 0, 33, 1], 16, 256, 512, False, True, 0),
    ([5, 130, 64], 32, 776, 1040, True, False, 8),
    ([129, 0, 700], 64, 600, 560, False, True, 0),
    ([40, 3], 24, 72, 48, True, True, 0),
    ([300, 20], 48, 136, 1104, False, True, 16),
    ([3000, 1], 16, 64, 2064, False, True, 0),
    ([1] * 70, 8, 264, 80, True, True, 0),
    ([0, 0], 16, 64, 64, False, True, 0),
    ([2900], 8, 1032, 64, False, False, 0),
]


class LoraCase:
    def __init__(self, counts, r, K, N, mapped, scaled, pad, seed=0, tail=3):
        g = gen(seed + sum(counts) * 3 + r + K + N)
        G, n = len(counts), sum(counts)
        self.G, self.r, self.K, self.N, self.n, self.pad = G, r, K, N, n, pad
        self.R = n + tail  # positions past the last group
        self.offsets = torch.zeros(G + 1, dtype=torch.int64)
        self.offsets[1:] = torch.tensor(counts).cumsum(0)
        self.rows = self.R + 5 if mapped else self.R
        self.row = torch.randperm(self.rows, generator=g)[:self.R].to(torch.int32) if mapped else None
        self.a, self.b = randn(g, G, r, K, std=K ** -0.5), randn(g, G, N, r, std=r ** -0.5)
        self.scale = torch.rand(G, generator=g) * 2 - 0.5 if scaled else None
        self.x, self.base = randn(g, self.rows, K), randn(g, self.rows, N)
        self.dy, self.dx_base = randn(g, self.rows, N), randn(g, self.rows, K)
        self.ref = ref.Lora(self.a, self.b, self.offsets, self.scale, self.row, self.rows)
        used = torch.arange(n) if self.row is None else self.row[:n].long()
        self.used = torch.zeros(self.rows, dtype=torch.bool)
        self.used[used] = True
        for t in (self.x, self.dy, self.base, self.dx_base):
            t[~self.used] = float("nan")  # rows of no position are not read

    def dev(self, t):
        return None if t is None else t.cuda()

    def ws(self, backward):
        n = e4b.e4b_lora_workspace_size(self.G, self.r, self.N, self.K, self.R, backward)
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns

    def forward(self, base=True, y=True, h=False, s=True, layout="halves", act="swiglu", inplace=False):
        out = {"y": strided(torch.full((self.rows, self.N), SENTINEL, dtype=BF16), self.pad) if y else None,
               "h": strided(torch.full((self.rows, self.N // 2), SENTINEL, dtype=BF16), self.pad) if h else None,
               "s": torch.full((self.R, self.r), SENTINEL, device="cuda") if s else None}
        b = strided(self.base, self.pad) if base else None
        if inplace:
            out["y"] = b
        e4b.e4b_lora(self.dev(self.a), self.dev(self.b), strided(self.x, self.pad), self.dev(self.offsets),
                     self.ws(False), base=b, scale=self.dev(self.scale), row=self.dev(self.row), layout=layout,
                     act=act, **out)
        return out

    def backward(self, s, dx=True, da=True, db=True, base=True, accumulate=False, inplace=False, fill=SENTINEL):
        out = {"dx": strided(torch.full((self.rows, self.K), SENTINEL, dtype=BF16), self.pad) if dx else None,
               "da": torch.full((self.G, self.r, self.K), fill, device="cuda") if da else None,
               "db": torch.full((self.G, self.N, self.r), fill, device="cuda") if db else None}
        b = strided(self.dx_base, self.pad) if base else None
        if inplace:
            out["dx"] = b
        e4b.e4b_lora_backward(self.dev(self.a), self.dev(self.b), strided(self.x, self.pad) if da else None,
                              s.to(F32).cuda() if db else None, strided(self.dy, self.pad), self.dev(self.offsets),
                              self.ws(True), dx_base=b, accumulate=accumulate, scale=self.dev(self.scale),
                              row=self.dev(self.row), **out)
        return out


@pytest.mark.parametrize("case", LORA_CASES, ids=str)
def test_lora_forward(case):
    c = LoraCase(*case)
    out = c.forward()
    s, es, y, ey = c.ref.forward(c.x, c.base, c.R, c.rows)
    got = out["s"].cpu()
    assert ref.off_f32(got[:c.n], s[:c.n], es[:c.n]) <= 1
    assert bool((got[c.n:] == SENTINEL).all())
    got = out["y"].cpu()
    assert ref.off_bf16(got[c.used], y[c.used], ey[c.used]) <= 1
    assert bool((got[~c.used] == SENTINEL).all()) and padding_untouched(out["y"], c.pad)
    same = c.forward(inplace=True)["y"].cpu()
    assert torch.equal(same[c.used], got[c.used])
    # without base, s or y
    alone = c.forward(base=False, s=False)["y"].cpu()
    _, _, y0, ey0 = c.ref.forward(c.x, None, c.R, c.rows)
    assert ref.off_bf16(alone[c.used], y0[c.used], ey0[c.used]) <= 1
    assert torch.equal(c.forward(y=False)["s"].cpu(), out["s"].cpu())


@pytest.mark.parametrize("case", [k for k in LORA_CASES if k[3] % 16 == 0], ids=str)
@pytest.mark.parametrize("layout", ["halves", "interleaved"])
@pytest.mark.parametrize("act", ["swiglu", "clamped_glu"])
def test_lora_with_the_activation(case, layout, act):
    c = LoraCase(*case, seed=1)
    c.base = (c.base.float() * 3).to(BF16)
    out = c.forward(h=True, layout=layout, act=act)
    _, _, y, ey = c.ref.forward(c.x, c.base, c.R, c.rows)
    got = out["h"].cpu()
    y, ey = y[c.used], ey[c.used]
    assert ref.off_bf16(out["y"].cpu()[c.used], y, ey) <= 1
    g, u = ref.split_gu(y, layout)
    eg, eu = ref.split_gu(ey, layout)
    h = ref.glu(g, u, act)[0]
    # |dh/dg| <= 1.1 |u'|, |dh/du| <= |g'| (the sigmoid factor is below 1.1 and 1)
    err = glu_tol(act, g, u)[0] + 1.1 * (u.abs() + 1) * eg + g.abs() * eu + 1.1 * eg * eu
    assert ref.off_bf16(got[c.used], h, err) <= 1
    assert bool((got[~c.used] == SENTINEL).all()) and padding_untouched(out["h"], c.pad)
    only = c.forward(y=False, s=False, h=True, layout=layout, act=act)["h"].cpu()
    assert torch.equal(only, got)


@pytest.mark.parametrize("case", LORA_CASES, ids=str)
def test_lora_backward(case):
    c = LoraCase(*case, seed=2)
    s = c.ref.s(c.x, c.R)[0].to(F32)
    s[c.n:] = float("nan")
    out = c.backward(s)
    dx, edx, da, eda, db, edb = c.ref.backward(c.x, s, c.dy, c.dx_base, c.rows)
    got = out["dx"].cpu()
    assert ref.off_bf16(got[c.used], dx[c.used], edx[c.used]) <= 1
    assert bool((got[~c.used] == SENTINEL).all()) and padding_untouched(out["dx"], c.pad)
    assert ref.off_f32(out["da"].cpu(), da, eda) <= 1
    assert ref.off_f32(out["db"].cpu(), db, edb) <= 1
    # in place; each result alone; added to what is there
    assert torch.equal(c.backward(s, inplace=True)["dx"].cpu()[c.used], got[c.used])
    assert torch.equal(c.backward(s, dx=False, da=False)["db"], out["db"])
    assert torch.equal(c.backward(s, dx=False, db=False)["da"], out["da"])
    assert torch.equal(c.backward(s, da=False, db=False)["dx"].cpu(), got)
    more = c.backward(s, accumulate=True, fill=0.5)
    assert ref.off_f32(more["da"].cpu(), da + 0.5, eda + 2 * ref.U_SUM * (da.abs() + 0.5)) <= 1
    assert ref.off_f32(more["db"].cpu(), db + 0.5, edb + 2 * ref.U_SUM * (db.abs() + 0.5)) <= 1


def test_lora_backward_without_base():
    c = LoraCase([20, 5], 16, 128, 256, False, True, 0)
    s = c.ref.s(c.x, c.R)[0].to(F32)
    got = c.backward(s, base=False)["dx"].cpu()
    dx, edx = c.ref.backward(c.x, s, c.dy, None, c.rows)[:2]
    assert ref.off_bf16(got[c.used], dx[c.used], edx[c.used]) <= 1


def test_lora_gradients_by_differences():
    # loss = <y, dy> is linear in A and in B: differences of any step are exact
    c = LoraCase([6, 4], 8, 16, 32, False, True, 0, seed=4)
    s = c.ref.s(c.x, c.R)[0].to(F32)
    out = c.backward(s)
    u = c.used

    def loss(a, b):
        y = ref.Lora(a, b, c.offsets, c.scale).forward(c.x, c.base, c.R, c.rows)[2]
        return float((y[u] * c.dy[u].double()).sum())
    g = gen(8)
    for _ in range(20):
        e = int(torch.randint(0, c.G, (1,), generator=g))
        j, k, n = (int(torch.randint(0, m, (1,), generator=g)) for m in (c.r, c.K, c.N))
        da = torch.zeros_like(c.a, dtype=torch.float64)
        db = torch.zeros_like(c.b, dtype=torch.float64)
        da[e, j, k], db[e, n, j] = 1, 1
        a, b = c.a.double(), c.b.double()
        sa = (loss(a + da, b) - loss(a - da, b)) / 2
        sb = (loss(a, b + db) - loss(a, b - db)) / 2
        assert abs(sa - float(out["da"][e, j, k])) <= 1e-4 * (1 + abs(sa))
        assert abs(sb - float(out["db"][e, n, j])) <= 1e-4 * (1 + abs(sb))


def test_lora_map_entries_outside_the_rows_are_left_out():
    c = LoraCase([4, 3], 16, 64, 96, True, True, 0, seed=5)
    dropped = [1, 5]
    lost = c.row[dropped].long()
    c.row[1], c.row[5] = -1, c.rows
    c.used[lost] = False
    c.ref = ref.Lora(c.a, c.b, c.offsets, c.scale, c.row, c.rows)
    out = c.forward()
    s, es, y, ey = c.ref.forward(c.x, c.base, c.R, c.rows)
    assert bool((out["s"].cpu()[dropped] == 0).all())
    got = out["y"].cpu()
    assert ref.off_bf16(got[c.used], y[c.used], ey[c.used]) <= 1
    assert bool((got[~c.used] == SENTINEL).all())
    back = c.backward(s.to(F32))
    dx, edx, da, eda, db, edb = c.ref.backward(c.x, s.to(F32), c.dy, c.dx_base, c.rows)
    assert ref.off_f32(back["da"].cpu(), da, eda) <= 1 and ref.off_f32(back["db"].cpu(), db, edb) <= 1
    assert ref.off_bf16(back["dx"].cpu()[c.used], dx[c.used], edx[c.used]) <= 1
    assert bool((back["dx"].cpu()[~c.used] == SENTINEL).all())


def test_lora_an_infinite_row_stays_in_its_row_and_group():
    c = LoraCase([3, 4], 16, 64, 96, False, True, 0, seed=6)
    c.x[1, 5] = float("inf")
    c.dy[2, 7] = float("nan")
    y = c.forward()["y"].cpu()
    ok = torch.ones(c.rows, dtype=torch.bool)
    ok[1] = False
    _, _, want, ey = c.ref.forward(c.x, c.base, c.R, c.rows)
    ok &= c.used
    assert ref.off_bf16(y[ok], want[ok], ey[ok]) <= 1
    assert not bool(torch.isfinite(y[1].float()).any())
    s = torch.randn(c.R, c.r, generator=gen(1))
    out = c.backward(s)
    assert bool(torch.isfinite(out["da"][1]).all()) and bool(torch.isfinite(out["db"][1]).all())
    assert bool(torch.isnan(out["dx"][2].float()).all()) and bool(torch.isfinite(out["dx"][3:c.n].float()).all())


def test_lora_repeats_bit_for_bit():
    c = LoraCase([2000, 77, 0, 3], 16, 520, 1032, False, True, 0, seed=7)
    s = c.ref.s(c.x, c.R)[0].to(F32)
    one, two = c.backward(s), c.backward(s)
    for k in ("da", "db"):
        assert torch.equal(one[k], two[k])
    assert torch.equal(one["dx"][c.used.cuda()], two["dx"][c.used.cuda()])
    f1, f2 = c.forward(), c.forward()
    assert torch.equal(f1["s"][:c.n], f2["s"][:c.n]) and torch.equal(f1["y"][c.used.cuda()], f2["y"][c.used.cuda()])


def test_lora_wide_rank_as_two_adapters():
    # a rank of 128 as the sum of two rank-64 adapters, the second on the first's y
    c = LoraCase([40, 9], 64, 256, 320, False, False, 0, seed=8)
    d = LoraCase([40, 9], 64, 256, 320, False, False, 0, seed=9)
    y = c.forward()["y"]
    out = torch.empty_like(y)
    e4b.e4b_lora(d.a.cuda(), d.b.cuda(), c.x.cuda(), c.offsets.cuda(), c.ws(False), base=y, y=out)
    y1 = c.ref.forward(c.x, c.base, c.R, c.rows)
    y2 = d.ref.forward(c.x, None, c.R, c.rows)
    u = c.used
    # two bf16 roundings of y
    err = y1[3][u] + y2[3][u] + ref.U_BF16 * (y1[2][u].abs() + y1[3][u])
    assert ref.off_bf16(out.cpu()[u], y1[2][u] + y2[2][u], err) <= 1


def test_lora_captured_and_replayed():
    c = LoraCase([33, 0, 12], 16, 128, 160, True, True, 0, seed=10)
    ws, ws_b = c.ws(False), c.ws(True)
    a, b, x, base = c.a.cuda(), c.b.cuda(), c.x.cuda(), c.base.cuda()
    off, row, scale, dy, dxb = c.offsets.cuda(), c.row.cuda(), c.scale.cuda(), c.dy.cuda(), c.dx_base.cuda()
    y, s = torch.zeros_like(base), torch.zeros(c.R, c.r, device="cuda")
    dx, da, db = torch.zeros_like(x), torch.zeros(c.G, c.r, c.K, device="cuda"), torch.zeros(c.G, c.N, c.r, device="cuda")

    def step():
        e4b.e4b_lora(a, b, x, off, ws, base=base, y=y, s=s, scale=scale, row=row)
        e4b.e4b_lora_backward(a, b, x, s, dy, off, ws_b, dx=dx, dx_base=dxb, da=da, db=db, scale=scale, row=row)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.where(torch.isnan(x), x, -x))  # new inputs in the captured buffers
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, s, dx, da, db)]
    for t in (y, s, dx, da, db):
        t.zero_()
    step()
    u = c.used.cuda()
    assert torch.equal(got[0][u], y[u]) and torch.equal(got[1][:c.n], s[:c.n]) and torch.equal(got[2][u], dx[u])
    assert torch.equal(got[3], da) and torch.equal(got[4], db)
