"""The adapters where they run on whole tiles of 128 positions: tiles that end
inside a group, groups that several CTAs share, long chains of tiles, mapped
rows, partial column blocks, all ranks; the waits that give up; calls side by
side. Against the formulas in 64 bits on the GPU, with the bounds of
adapter_ref.py (its sums run in the kernels' number of steps)."""

import pytest
import torch

import adapter_ref as ref
from bit_grouped_moe_e4b_b200 import e4b

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
SENTINEL = 123.0


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)


class Case:
    """counts: positions of the groups; rows: of the buffers (a map if more)."""

    def __init__(self, counts, r, K, N, mapped=False, tail=3, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + r + K + N + sum(counts))
        G, n = len(counts), sum(counts)
        self.G, self.r, self.K, self.N, self.n, self.R = G, r, K, N, n, n + tail
        self.offsets = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
        self.offsets[1:] = torch.tensor(counts, device="cuda").cumsum(0)
        self.rows = self.R + (7 if mapped else 0)
        self.row = torch.randperm(self.rows, generator=g, device="cuda")[:self.R].to(torch.int32) if mapped else None
        self.used = torch.zeros(self.rows, dtype=torch.bool, device="cuda")
        self.used[torch.arange(n, device="cuda") if self.row is None else self.row[:n].long()] = True
        self.a, self.b = randn(g, G, r, K, std=K ** -0.5), randn(g, G, N, r, std=r ** -0.5)
        self.scale = torch.rand(G, generator=g, device="cuda") + 0.5
        self.x, self.dy = randn(g, self.rows, K), randn(g, self.rows, N)
        self.base, self.dx_base = randn(g, self.rows, N), randn(g, self.rows, K)
        for t in (self.x, self.dy, self.base, self.dx_base):
            t[~self.used] = float("nan")  # rows of no position are not read
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def ws(self, backward):
        n = e4b.e4b_lora_workspace_size(self.G, self.r, self.N, self.K, self.R, backward)
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns

    def full(self, *shape, dtype=BF16):
        return torch.full(shape, SENTINEL, dtype=dtype, device="cuda")

    def forward(self, **kw):
        out = {"y": self.full(self.rows, self.N), "s": self.full(self.R, self.r, dtype=F32)}
        e4b.e4b_lora(self.a, self.b, self.x, self.offsets, self.ws(False), base=self.base, scale=self.scale,
                     row=self.row, status=self.status, **out, **kw)
        return out

    def backward(self, s, **kw):
        out = {"dx": self.full(self.rows, self.K), "da": self.full(self.G, self.r, self.K, dtype=F32),
               "db": self.full(self.G, self.N, self.r, dtype=F32)}
        out.update({k: v for k, v in kw.items() if k in out})
        rest = {k: v for k, v in kw.items() if k not in out}
        e4b.e4b_lora_backward(self.a, self.b, self.x, s, self.dy, self.offsets, self.ws(True), dx_base=self.dx_base,
                              scale=self.scale, row=self.row, status=self.status, **out, **rest)
        return out

    def groups(self):
        off = self.offsets.tolist()
        for g in range(self.G):
            p = torch.arange(off[g], off[g + 1], device="cuda")
            yield g, p, p if self.row is None else self.row[p].long()

    def check_forward(self, out):
        """s within the sums' bound, y within s' and its own."""
        u, steps = ref.U_SUM, self.K / 16 + 24
        for g, p, i in self.groups():
            if not len(p):
                continue
            x, a, b, w = self.x[i].double(), self.a[g].double(), self.b[g].double(), float(self.scale[g])
            s, es = x @ a.T, steps * u * (x.abs() @ a.abs().T)
            assert ref.off_f32(out["s"][p], s, es) <= 1
            add, mag = w * (s @ b.T), w * (s.abs() @ b.abs().T)
            base = self.base[i].double()
            ey = w * (es @ b.abs().T) + (ref.U_SPLIT + (self.r / 8 + 24) * u) * mag + 4 * u * (base.abs() + mag)
            assert ref.off_bf16(out["y"][i], base + add, ey) <= 1
        assert bool((out["s"][self.n:] == SENTINEL).all()) and bool((out["y"][~self.used] == SENTINEL).all())

    def check_backward(self, s, out, before=None):
        u = ref.U_SUM
        for g, p, i in self.groups():
            a, b, w = self.a[g].double(), self.b[g].double(), float(self.scale[g])
            d, x, sg = self.dy[i].double(), self.x[i].double(), s[p].double()
            t, et = w * (d @ b), w * (self.N / 16 + 28) * u * (d.abs() @ b.abs())
            da, db = t.T @ x, w * (d.T @ sg)
            sums = (len(p) / 8 + 26) * u  # positions by sixteens, three terms, the parts
            eda = et.T @ x.abs() + sums * (t.abs().T @ x.abs())
            edb = (sums + u) * w * (d.abs().T @ sg.abs())
            if before is not None:
                da, db = da + before, db + before
                eda, edb = eda + 2 * u * (da.abs() + abs(before)), edb + 2 * u * (db.abs() + abs(before))
            assert ref.off_f32(out["da"][g], da, eda) <= 1
            assert ref.off_f32(out["db"][g], db, edb) <= 1
            if len(p):
                base, mag = self.dx_base[i].double(), t.abs() @ a.abs()
                edx = et @ a.abs() + (ref.U_SPLIT + (self.r / 8 + 24) * u) * mag + 4 * u * (base.abs() + mag)
                assert ref.off_bf16(out["dx"][i], base + t @ a, edx) <= 1
        assert bool((out["dx"][~self.used] == SENTINEL).all())

    def s(self):
        s = torch.full((self.R, self.r), float("nan"), device="cuda")
        for g, p, i in self.groups():
            s[p] = (self.x[i].double() @ self.a[g].double().T).float()
        return s


TILES = [  # counts, r, K, N, mapped
    ([600], 16, 128, 128, False),                   # whole tiles and one that ends early
    ([129, 127, 128, 1, 0, 256], 16, 264, 1032, False),
    ([513, 2], 8, 72, 4104, False),                 # rank below the operand's width, many column blocks
    ([300, 300, 0, 1], 24, 520, 264, True),
    ([700, 40], 32, 1000, 520, False),
    ([640, 15, 33], 48, 648, 1160, True),
    ([1025], 64, 2056, 8, False),                   # one column block of eight columns
    ([16] * 40, 64, 136, 200, False),
    ([1] * 600, 16, 64, 96, True),                  # more groups than CTAs
    ([5000], 16, 64, 64, False),                    # a group over all CTAs
    ([9000, 0, 3000], 64, 200, 136, True),
]
WIDE = [  # enough work for s to run on tiles
    ([6000, 131], 16, 2312, 72, True),
    ([700] * 9 + [0, 1, 259], 24, 2048, 144, False),
    ([2100, 900], 64, 1096, 328, False),
    ([130] * 30, 48, 1160, 64, True),
    ([12345], 8, 2056, 16, False),
]


@pytest.mark.parametrize("case", TILES, ids=str)
def test_tiles_forward_and_backward(case):
    c = Case(*case)
    c.check_forward(c.forward())
    s = c.s()
    c.check_backward(s, c.backward(s))
    assert int(c.status) == 0


@pytest.mark.parametrize("case", WIDE, ids=lambda c: f"{len(c[0])} groups {c[1:]}")
def test_wide_rows_forward_and_backward(case):
    c = Case(*case, seed=11)
    assert c.R * c.K * c.r > 2e8
    c.check_forward(c.forward())
    s = c.s()
    c.check_backward(s, c.backward(s))
    assert int(c.status) == 0


ROWS = [(1, 1), (15, 2), (17, 1), (64, 3), (100, 1), (200, 2), (500, 1), (1500, 3)]


@pytest.mark.parametrize("r", [8, 16, 32, 64])
@pytest.mark.parametrize("rows,G", ROWS)
def test_few_rows_take_smaller_tiles(rows, G, r):
    # one long group and short ones, so that tiles of every size end inside a group
    c = Case([rows] + [rows // 7 + 1] * (G - 1), r, 264, 520, seed=12)
    c.check_forward(c.forward())
    s = c.s()
    c.check_backward(s, c.backward(s))


@pytest.mark.parametrize("case", [TILES[1], TILES[4], TILES[9]], ids=str)
def test_tiles_accumulate(case):
    c = Case(*case, seed=1)
    s = c.s()
    filled = {"da": torch.full((c.G, c.r, c.K), 0.25, device="cuda"), "db": torch.full((c.G, c.N, c.r), 0.25, device="cuda")}
    c.check_backward(s, c.backward(s, accumulate=True, **filled), before=0.25)


def test_long_chains_of_tiles():
    # more row tiles in a CTA's run than one accumulator takes, and a long K
    c = Case([32768, 5], 16, 1024, 1024, seed=2)
    c.check_forward(c.forward())
    s = c.s()
    out = c.backward(s)
    c.check_backward(s, out)
    for g, p, i in c.groups():  # as exact as fp32 products and sums: 2-norms
        w = float(c.scale[g])
        t = w * (c.dy[i].double() @ c.b[g].double())
        for got, want in ((out["da"][g], t.T @ c.x[i].double()), (out["db"][g], w * (c.dy[i].double().T @ s[p].double()))):
            # truncation: 1.2e-8 a step, 64 steps a chain, t's 16 on top (2^-26 each), and the products' 2^-24
            assert float((got.double() - want).norm() / want.norm()) <= (64 + 16) * 2 ** -26 + 4 * 2 ** -24


def test_values_of_other_groups_do_not_meet():
    # the tile behind group 0's last row holds rows of group 1, all NaN
    c = Case([130, 140, 7], 16, 136, 264, seed=3)
    s = c.s()
    c.dy[130:270] = float("nan")
    c.x[130:270] = float("inf")
    out, fwd = c.backward(s), c.forward()
    for g in (0, 2):
        assert bool(torch.isfinite(out["da"][g]).all()) and bool(torch.isfinite(out["db"][g]).all())
    rows = torch.ones(c.R, dtype=torch.bool, device="cuda")
    rows[130:270] = False
    rows &= c.used
    assert bool(torch.isfinite(out["dx"][rows].float()).all()) and bool(torch.isfinite(fwd["y"][rows].float()).all())
    assert not bool(torch.isfinite(out["db"][1]).any())


def test_a_wait_that_gives_up_is_reported_and_the_next_call_works():
    c = Case([6000, 2300], 16, 2048, 512, seed=4)  # s on tiles too
    s = c.s()
    c.forward(flags=e4b.FLAG_TEST_TIMEOUT)
    first = int(c.status)
    assert e4b.e4b_status_string(first) == "device wait timed out"
    c.status.zero_()
    c.backward(s, flags=e4b.FLAG_TEST_TIMEOUT)
    assert int(c.status) == first
    c.status.zero_()
    c.check_forward(c.forward())
    c.check_backward(s, c.backward(s))
    assert int(c.status) == 0


def test_calls_side_by_side_and_repeated():
    cases = [Case(*TILES[1], seed=5), Case(*TILES[4], seed=6), Case(*TILES[10], seed=7)]
    s = [c.s() for c in cases]
    alone = [{**c.forward(), **c.backward(v)} for c, v in zip(cases, s)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    both = [None] * len(cases)
    for i, (c, v) in enumerate(zip(cases, s)):
        with torch.cuda.stream(streams[i]):
            both[i] = {**c.forward(), **c.backward(v)}
    torch.cuda.synchronize()
    for c, a, b in zip(cases, alone, both):
        for k in a:
            x, y = (t[c.used] if k in ("y", "dx") else t for t in (a[k], b[k]))
            assert torch.equal(x, y), k


def test_two_graphs_share_a_workspace_one_after_the_other():
    c, d = Case(*TILES[1], seed=8), Case(*TILES[1], seed=9)
    s = [c.s(), d.s()]
    ws = c.ws(True)
    outs, graphs = [], []
    for k, v in ((c, s[0]), (d, s[1])):
        out = {"dx": k.full(k.rows, k.K), "da": k.full(k.G, k.r, k.K, dtype=F32), "db": k.full(k.G, k.N, k.r, dtype=F32)}

        def call(k=k, v=v, out=out):
            e4b.e4b_lora_backward(k.a, k.b, k.x, v, k.dy, k.offsets, ws, dx_base=k.dx_base, scale=k.scale, row=k.row, **out)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        outs.append(out)
        graphs.append(graph)
    for o in outs:
        for t in o.values():
            t.fill_(SENTINEL)
    for g in (0, 1, 0, 1):
        graphs[g].replay()
    torch.cuda.synchronize()
    c.check_backward(s[0], outs[0])
    d.check_backward(s[1], outs[1])


def test_without_rows_gradients_are_zero_and_nothing_else_is_written():
    c = Case([0, 0, 0], 16, 64, 96, seed=10, tail=700)
    out = c.backward(c.s())
    assert not bool(out["da"].any()) and not bool(out["db"].any())
    assert bool((out["dx"] == SENTINEL).all())
    fwd = c.forward()
    assert bool((fwd["y"] == SENTINEL).all()) and bool((fwd["s"] == SENTINEL).all())


def test_a_map_without_any_row_in_range():
    # every position is left out: s is zero, gradients are zero, no row is written
    c = Case([200, 57], 16, 72, 136, mapped=True, seed=13)
    c.row.fill_(-1)
    c.used[:] = False
    fwd = c.forward()
    assert not bool(fwd["s"][:c.n].any()) and bool((fwd["y"] == SENTINEL).all())
    out = c.backward(torch.ones(c.R, c.r, device="cuda"))
    assert not bool(out["da"].any()) and not bool(out["db"].any()) and bool((out["dx"] == SENTINEL).all())


def test_largest_group_count_and_single_positions():
    # 1024 groups, most of them empty, the rest of one position
    counts = [1 if g % 7 == 3 else 0 for g in range(1024)]
    c = Case(counts, 8, 40, 24, seed=14)
    c.check_forward(c.forward())
    s = c.s()
    c.check_backward(s, c.backward(s))


@pytest.mark.parametrize("layout", ["halves", "interleaved"])
@pytest.mark.parametrize("act", ["swiglu", "clamped_glu"])
def test_activation_of_huge_values_does_not_overflow_on_the_way(layout, act):
    # a gate far below zero closes whatever the up value is; no adapter term (scale 0)
    c = Case([40], 8, 16, 64, seed=15)
    c.scale.zero_()
    g = torch.tensor([-1e20, -300.0, -3e38, -100.0, 2.0, -1e3], device="cuda").to(BF16)
    u = torch.tensor([1e20, 1e37, -3e38, 1e30, 3.0, 3e38], device="cuda").to(BF16)
    reps = c.N // 2 // len(g) + 1
    gu = ref.join_gu(g.repeat(reps)[None, :c.N // 2], u.repeat(reps)[None, :c.N // 2], layout)
    c.base = gu.expand(c.rows, -1).contiguous()
    h = c.full(c.rows, c.N // 2)
    c.forward(h=h, layout=layout, act=act)
    want = ref.glu(*ref.split_gu(gu, layout), act)[0].to(F32)
    assert bool(torch.isfinite(want).all())
    got = h[:c.n].to(F32)
    assert bool(torch.isfinite(got).all())
    # half a bf16 step and 2^-18 of the value; a sigmoid that the reciprocal flushes leaves 2^-124 of |g u'| at most
    a, b = (v.double().abs() for v in ref.split_gu(gu, layout))
    flushed = 2.0 ** -124 * a * (torch.clamp(b, max=7.0) + 1 if act == "clamped_glu" else b)
    assert bool(((got - want).abs().double() <= (2 ** -8 + 2 ** -18) * want.abs().double() + flushed).all())


@pytest.mark.parametrize("layout", ["halves", "interleaved"])
@pytest.mark.parametrize("act", ["swiglu", "clamped_glu"])
def test_activation_gradient_of_huge_values_does_not_overflow_on_the_way(layout, act):
    g = torch.tensor([-1e20, -300.0, -3e38, -100.0, 2.0, -1e3, 5.0, -3e38], device="cuda").to(BF16)
    u = torch.tensor([1e20, 1e37, -3e38, 1e30, 3.0, 3e38, -2.0, 0.0], device="cuda").to(BF16)
    dh = torch.tensor([1e20, -1e30, 1e10, 2.0, 1.5, 3e38, -0.5, 3e38], device="cuda").to(BF16)
    R = 9
    gu = ref.join_gu(g[None], u[None], layout).expand(R, -1).contiguous()
    d = dh.expand(R, -1).contiguous()
    dgu, h = torch.empty_like(gu), torch.empty_like(d)
    e4b.e4b_glu_backward(d, gu, dgu, h=h, layout=layout, act=act)
    h_ref, dg, du = ref.glu(g.double()[None], u.double()[None], act)
    open_ = (g.float() > -90)[None]  # elsewhere the gate is closed: nothing passes
    got_g, got_u = ref.split_gu(dgu, layout)
    for got, want in ((h, h_ref), (got_g, dg * dh.double()), (got_u, du * dh.double())):
        assert bool(torch.isfinite(got.float()).all())
        err = (got.double() - want).abs()
        # half a bf16 step and 2^-16 for the gradient's few roundings
        assert bool((err <= (2 ** -8 + 2 ** -16) * want.abs())[open_.expand_as(err)].all())
        assert not bool(got[~open_.expand_as(err)].any())
