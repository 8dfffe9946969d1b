"""The adapter layer as a training step runs it, forward and backward, on
packed experts, against the same steps in 64 bits with the same tensors stored
in bf16 (qlora_ref.py).

Bounds. Both sides round the same tensors to bf16; the fp32 sums before a
rounding differ from exact ones by less than 2^-16 of the values (2^-23 a sum,
hundreds of sums; 2^-16 for a factor of two bf16 terms). A bf16 step is at least
2^-8 of the value, so at most one value in 256 rounds to the other neighbour, by
a step, at most 2^-7: a 2-norm error of 2^-7 / sqrt(256) = 2^-11 for each stored
tensor on the way. Eight lie on the longest way (gu, h, ys, dys, dh twice, dgu,
dxs), and the matrices between them pass an error on with a gain near that of the
values themselves, two at most with the activation's slope: 8 * 2 * 2^-11 = 2^-7
for fp32 results, and half a step, 2^-8, more for the bf16 ones."""

import pytest
import torch

import qlora_ref
from bit_grouped_moe_e4b_b200 import e4b, qlora

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16

CASES = [  # fmt, E, H, I, r of the two adapters, T, k, layout, act, bias
    ("nf4", 4, 128, 192, 16, 8, 37, 2, "halves", "swiglu", False),
    ("nf4", 8, 256, 320, 16, 32, 400, 2, "halves", "swiglu", False),
    ("mxfp4", 5, 160, 96, 64, 24, 131, 3, "interleaved", "clamped_glu", True),
    ("mxfp4", 32, 320, 256, 8, 16, 3, 4, "halves", "swiglu", False),
    ("nf4", 3, 64, 64, 8, 8, 1, 1, "halves", "swiglu", False),
]


class Case:
    def __init__(self, fmt, E, H, I, r1, r2, T, k, layout, act, bias):
        g = torch.Generator().manual_seed(E * 7 + T)

        def rnd(*shape, std=1.0):
            return torch.randn(*shape, generator=g) * std
        w_gu, w_dn = rnd(E, 2 * I, H, std=H ** -0.5), rnd(E, H, I, std=I ** -0.5)
        (gc, gs), (dc, ds) = e4b.quantize(fmt, w_gu.cuda()), e4b.quantize(fmt, w_dn.cuda())
        self.w = [e4b.dequantize(fmt, c, s, E, n, m).double().cpu() for c, s, n, m in ((gc, gs, 2 * I, H), (dc, ds, H, I))]
        self.b = [rnd(E, 2 * I, std=0.1) if bias else torch.zeros(E, 2 * I), rnd(E, H, std=0.1) if bias else torch.zeros(E, H)]
        self.layer = e4b.PackedLayer(fmt, E, H, I, gc, gs, dc, ds, layout=layout, act=act,
                                     gate_up_bias=self.b[0].cuda() if bias else None,
                                     down_bias=self.b[1].cuda() if bias else None)
        self.ad = [(rnd(E, r, K, std=K ** -0.5).to(BF16), rnd(E, N, r, std=0.5 * r ** -0.5).to(BF16),
                    0.5 + torch.rand(E, generator=g)) for r, N, K in ((r1, 2 * I, H), (r2, H, I))]
        self.dev = [qlora.Adapter(*(t.cuda() for t in a)) for a in self.ad]
        self.x, self.dy = rnd(T, H).to(BF16), rnd(T, H).to(BF16)
        self.ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
        self.ids[self.ids == 1] = 0  # an expert without rows
        self.gates = torch.rand(T, k, generator=g)
        self.layout, self.act = layout, act

    def reference(self):
        return qlora_ref.step(*self.w, *(b.double() for b in self.b), *(tuple(t.double() for t in a) for a in self.ad),
                              self.x.double(), self.ids, self.gates, self.dy.double(), self.layout, self.act)

    def step(self, buffers=None, **kw):
        y, kept = qlora.forward(self.layer, *self.dev, self.x.cuda(), self.ids.cuda(), self.gates.cuda(), buffers)
        dx, dgates, gu, dn = qlora.backward(self.layer, *self.dev, kept, self.dy.cuda(), buffers=buffers, **kw)
        return {"y": y, "dx": dx, "dgates": dgates, "gu_a": gu.a, "gu_b": gu.b, "dn_a": dn.a, "dn_b": dn.b}


def off(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


@pytest.mark.parametrize("case", CASES, ids=str)
def test_step_against_the_formulas(case):
    c = Case(*case)
    want, got = c.reference(), c.step()
    for name, t in got.items():
        assert off(t, want[name]) <= 2 ** -7 + (2 ** -8 if t.dtype == BF16 else 0), name
    if c.layer.E > 1:
        assert not bool(got["gu_a"][1].any()) and not bool(got["dn_b"][1].any())


def test_gradients_accumulate_over_micro_batches():
    c = Case(*CASES[1])
    one = c.step()
    grads = tuple(qlora.Gradient(one[f"{n}_a"].clone(), one[f"{n}_b"].clone()) for n in ("gu", "dn"))
    two = c.step(grads=grads, accumulate=True)
    for n in ("gu_a", "gu_b", "dn_a", "dn_b"):
        # twice the same sum: exact up to one fp32 addition and the order of the parts
        assert float((two[n] - 2 * one[n]).norm()) <= 2 ** -20 * float(two[n].norm())


def test_step_captured_and_replayed_with_new_inputs():
    c = Case(*CASES[1])
    buf = qlora.Buffers()
    x, ids, gates, dy = c.x.cuda(), c.ids.cuda(), c.gates.cuda(), c.dy.cuda()

    def step():
        y, kept = qlora.forward(c.layer, *c.dev, x, ids, gates, buf)
        return y, qlora.backward(c.layer, *c.dev, kept, dy, buffers=buf)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, (dx, dgates, gu, dn) = step()
    # other routing and rows in the captured buffers
    ids.copy_((ids + 3) % c.layer.E)
    x.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, dx, dgates, gu.a, gu.b, dn.a, dn.b)]
    y, (dx, dgates, gu, dn) = step()
    for a, b in zip(got, (y, dx, dgates, gu.a, gu.b, dn.a, dn.b)):
        assert torch.equal(a, b)


def test_two_steps_on_two_streams():
    cases = [Case(*CASES[1]), Case(*CASES[2])]
    alone = [c.step() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    both = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            both.append(c.step())
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for n in a:
            assert torch.equal(a[n], b[n]), n
