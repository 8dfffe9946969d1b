"""The adapter layer as programs call it beside the plain step: other batch sizes
between a graph's replays, no tokens, dropped slots."""

import pytest
import torch

from bit_grouped_moe_e4b_b200 import qlora
from test_gpu_qlora import CASES, Case, off

pytestmark = pytest.mark.gpu


def tensors(y, back):
    dx, dgates, gu, dn = back
    return [y, dx, dgates, gu.a, gu.b, dn.a, dn.b]


def test_another_batch_size_between_replays():
    c = Case(*CASES[1])
    buf = qlora.Buffers()
    x, ids, gates, dy = c.x.cuda(), c.ids.cuda(), c.gates.cuda(), c.dy.cuda()

    def step(n):
        y, kept = qlora.forward(c.layer, *c.dev, x[:n], ids[:n], gates[:n], buf)
        return tensors(y, qlora.backward(c.layer, *c.dev, kept, dy[:n], buffers=buf))
    T = x.shape[0]
    step(T)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(T)
    graph.replay()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    small = [t.clone() for t in step(T // 3)]
    # memory that was free after the smaller step
    held = [torch.full((1 << 18,), 7.0, device="cuda") for _ in range(40)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(bool((h == 7.0).all()) for h in held)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.equal(a, b) for a, b in zip(step(T // 3), small))


def test_a_batch_without_tokens():
    c = Case(*CASES[2])
    empty = lambda t: t[:0].cuda().contiguous()  # noqa: E731
    for buf in (None, qlora.Buffers()):
        y, kept = qlora.forward(c.layer, *c.dev, empty(c.x), empty(c.ids), empty(c.gates), buf)
        dx, dgates, gu, dn = qlora.backward(c.layer, *c.dev, kept, empty(c.dy), buffers=buf)
        assert y.shape == dx.shape == (0, c.layer.H) and dgates.shape == (0, c.ids.shape[1])
        for t in (gu.a, gu.b, dn.a, dn.b):
            assert not bool(t.any())
    grads = tuple(qlora.Gradient(torch.ones_like(d.a), torch.ones_like(d.b)) for d in (gu, dn))
    qlora.backward(c.layer, *c.dev, kept, empty(c.dy), grads=grads, accumulate=True)
    assert all(bool((t == 1).all()) for d in grads for t in (d.a, d.b))


@pytest.mark.parametrize("case", [CASES[1], CASES[2]], ids=str)
def test_dropped_slots_have_no_part_in_any_result(case):
    c = Case(*case)
    g = torch.Generator().manual_seed(5)
    drop = torch.rand(c.ids.shape, generator=g) < 0.3
    drop[0] = True  # a token without any expert
    c.ids[drop] = torch.where(torch.rand(c.ids.shape, generator=g) < 0.5, -1, c.layer.E)[drop].to(torch.int32)
    c.gates[drop] = 0.0
    want = c.reference()
    c.gates[drop] = float("nan")  # gates of dropped slots are not read
    buf = qlora.Buffers()
    c.step(buf)
    for t in buf.held.values():  # nor are rows behind the routed ones, or anything of the step before
        t.fill_(float("nan") if t.dtype.is_floating_point else 255 if t.dtype == torch.uint8 else 0)
    got = c.step(buf)
    for name, t in got.items():
        assert off(t, want[name]) <= 2 ** -7 + (2 ** -8 if t.dtype == torch.bfloat16 else 0), name
    assert not bool(got["y"][0].any()) and not bool(got["dx"][0].any()) and not bool(got["dgates"].cpu()[drop].any())
