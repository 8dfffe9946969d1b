"""Low-rank adapters on the frozen packed experts: the layer's forward with
what a training step keeps of it, and its backward pass ("experts4bit-qlora"
README: adapters on 4-bit experts that stay packed).

For routed row p of expert e, with B A the adapter of each projection:

    gu[p] = W_gu x + w_e B_gu A_gu x          h[p] = act(gu[p])
    ys[p] = W_dn h[p] + w_e B_dn A_dn h[p]    y[t] = sum_j gates[t, j] ys[p(t, j)]

The packed weights are never unpacked to memory: both projections and their
input gradients run on the packed bytes (e4b_grouped_gemm, e4b_grouped_dgrad),
the steps between them are e4b_permute / e4b_unpermute, e4b_lora and e4b_glu.
gu is kept in bf16, since the backward pass needs it. All work is enqueued on
the current stream of x's (dy's) device; no call synchronises, so forward and
backward can be captured into a CUDA graph with buffers that the caller keeps
(``Buffers``).
"""

from __future__ import annotations

from dataclasses import dataclass, field

import torch

from . import e4b


@dataclass
class Adapter:
    """One projection's adapters: a [E, r, K] and b [E, N, r] bf16, the weight
    of each expert's product (fp32 [E], or None for 1)."""
    a: torch.Tensor
    b: torch.Tensor
    scale: torch.Tensor | None = None


@dataclass
class Gradient:
    """fp32 gradients of an Adapter's a and b."""
    a: torch.Tensor
    b: torch.Tensor


@dataclass
class Kept:
    """What backward() needs of a forward() call."""
    ids_shape: tuple
    gates: torch.Tensor
    offsets: torch.Tensor
    inv: torch.Tensor
    xs: torch.Tensor
    gu: torch.Tensor
    h: torch.Tensor
    ys: torch.Tensor
    s_gu: torch.Tensor
    s_dn: torch.Tensor


@dataclass
class Buffers:
    """Named device buffers, allocated at their first use and kept for as long as
    this object lives, so that a CUDA graph may hold their addresses: one of each
    name, shape, type and device. Results and kept rows of a step overwrite those of
    the step before it of the same shapes; one Buffers serves one step at a time, on
    one stream (two streams, or a graph beside an eager step, take two). Every batch
    size that comes up keeps its own buffers: a program whose sizes vary without end
    calls without, and lets the allocator serve it."""
    held: dict = field(default_factory=dict)

    def __call__(self, name, shape, dtype, device):
        key = (name, tuple(shape), dtype, torch.device(device))
        t = self.held.get(key)
        if t is None:
            t = self.held[key] = torch.empty(shape, dtype=dtype, device=device)
        return t


def _fresh(name, shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


def _lora_ws(ad: Adapter, R, backward, new, name, device):
    E, r, K = ad.a.shape
    n = e4b.e4b_lora_workspace_size(E, r, ad.b.shape[1], K, R, backward)
    return new(name, (n,), torch.uint8, device)


def _check(layer: e4b.PackedLayer, gate_up: Adapter, down: Adapter):
    if layer.fmt not in ("nf4", "mxfp4"):
        raise ValueError("adapters run beside NF4 and MXFP4 experts")
    for name, ad, N, K in (("gate_up", gate_up, 2 * layer.I, layer.H), ("down", down, layer.H, layer.I)):
        if ad.a.dim() != 3 or ad.b.dim() != 3 or ad.a.shape[0] != layer.E or ad.a.shape[2] != K:
            raise ValueError(f"{name}.a: expected [{layer.E}, r, {K}], got {tuple(ad.a.shape)}")
        if ad.b.shape != (layer.E, N, ad.a.shape[1]):
            raise ValueError(f"{name}.b: expected [{layer.E}, {N}, {ad.a.shape[1]}], got {tuple(ad.b.shape)}")


def forward(layer: e4b.PackedLayer, gate_up: Adapter, down: Adapter, x, ids, gates, buffers: Buffers | None = None):
    """y bf16 [T, H] and the Kept rows of x bf16 [T, H] with routing ids int32
    and gates fp32 [T, k]."""
    _check(layer, gate_up, down)
    # the routing pass takes an address: other types would be read as int32
    if ids.dtype != torch.int32 or ids.dim() != 2 or ids.shape[0] != x.shape[0] or ids.device != x.device:
        raise ValueError(f"ids: expected int32 [{x.shape[0]}, k] on {x.device}, got {ids.dtype} {tuple(ids.shape)} on {ids.device}")
    with torch.cuda.device(x.device):  # the packed projections run on the current device
        return _forward(layer, gate_up, down, x, ids, gates, buffers or _fresh)


def _forward(layer, gate_up, down, x, ids, gates, new):
    (T, k), dev = ids.shape, x.device
    E, H, I, R = layer.E, layer.H, layer.I, T * k
    bf16 = torch.bfloat16
    counts = new("counts", (E,), torch.int32, dev)
    offsets = new("offsets", (E + 1,), torch.int64, dev)
    perm, inv = new("perm", (R,), torch.int32, dev), new("inv", (R,), torch.int32, dev)
    ws = new("route_ws", (e4b.e4b_route_workspace_size(T, k, E),), torch.uint8, dev)
    e4b.e4b_route(ids, E, counts, offsets, perm, inv, ws)
    xs = new("xs", (R, H), bf16, dev)
    e4b.e4b_permute(x, perm, offsets, xs, top_k=k)

    gu, h = new("gu", (R, 2 * I), bf16, dev), new("h", (R, I), bf16, dev)
    s_gu = new("s_gu", (R, gate_up.a.shape[1]), torch.float32, dev)
    if R:  # the packed projections take no empty batch
        e4b.e4b_grouped_gemm(layer.fmt, e4b.E4B_EPI_STORE, layer.gate_up_codes, layer.gate_up_scales, xs, offsets, gu, E=E,
                             N=2 * I, K=H, R_max=R, bias=layer.gate_up_bias)
    e4b.e4b_lora(gate_up.a, gate_up.b, xs, offsets, _lora_ws(gate_up, R, False, new, "ws_gu", dev), base=gu, y=gu, h=h,
                 s=s_gu, scale=gate_up.scale, layout=layer.layout, act=layer.act, alpha=layer.alpha, limit=layer.limit)

    ys = new("ys", (R, H), bf16, dev)
    s_dn = new("s_dn", (R, down.a.shape[1]), torch.float32, dev)
    if R:
        e4b.e4b_grouped_gemm(layer.fmt, e4b.E4B_EPI_STORE, layer.down_codes, layer.down_scales, h, offsets, ys, E=E, N=H, K=I,
                             R_max=R, bias=layer.down_bias)
    e4b.e4b_lora(down.a, down.b, h, offsets, _lora_ws(down, R, False, new, "ws_dn", dev), base=ys, y=ys, s=s_dn,
                 scale=down.scale)
    y = new("y", (T, H), bf16, dev)
    e4b.e4b_unpermute(ys, inv, gates, y, top_k=k)
    return y, Kept((T, k), gates, offsets, inv, xs, gu, h, ys, s_gu, s_dn)


def backward(layer: e4b.PackedLayer, gate_up: Adapter, down: Adapter, kept: Kept, dy, *, grads=None, accumulate=False,
             buffers: Buffers | None = None):
    """dx bf16 [T, H], dgates fp32 [T, k] and the Gradients of gate_up and down
    for dy bf16 [T, H]. grads: the pair of Gradients to write (accumulate: to
    add to)."""
    if accumulate and grads is None:
        raise ValueError("accumulate needs the gradients to add to")
    with torch.cuda.device(dy.device):
        return _backward(layer, gate_up, down, kept, dy, grads, accumulate, buffers or _fresh)


def _backward(layer, gate_up, down, kept, dy, grads, accumulate, new):
    (T, k), dev = kept.ids_shape, dy.device
    E, H, I, R = layer.E, layer.H, layer.I, T * k
    bf16, f32 = torch.bfloat16, torch.float32
    if grads is None:
        grads = tuple(Gradient(new(f"d{n}_a", ad.a.shape, f32, dev), new(f"d{n}_b", ad.b.shape, f32, dev))
                      for n, ad in (("gu", gate_up), ("dn", down)))
    d_gu, d_dn = grads

    dys, dgates = new("dys", (R, H), bf16, dev), new("dgates", (T, k), f32, dev)
    e4b.e4b_unpermute_backward(dy, kept.ys, kept.inv, kept.gates, dys, dgates, top_k=k)
    dh = new("dh", (R, I), bf16, dev)
    if R:
        e4b.e4b_grouped_dgrad(layer.fmt, layer.down_codes, layer.down_scales, dys, kept.offsets, dh, E=E, N=H, K=I, R_max=R)
    e4b.e4b_lora_backward(down.a, down.b, kept.h, kept.s_dn, dys, kept.offsets,
                          _lora_ws(down, R, True, new, "ws_ddn", dev), dx=dh, dx_base=dh, da=d_dn.a, db=d_dn.b,
                          accumulate=accumulate, scale=down.scale)

    dgu = new("dgu", (R, 2 * I), bf16, dev)
    e4b.e4b_glu_backward(dh, kept.gu, dgu, offsets=kept.offsets, layout=layer.layout, act=layer.act, alpha=layer.alpha,
                         limit=layer.limit)
    dxs = new("dxs", (R, H), bf16, dev)
    if R:
        e4b.e4b_grouped_dgrad(layer.fmt, layer.gate_up_codes, layer.gate_up_scales, dgu, kept.offsets, dxs, E=E, N=2 * I,
                              K=H, R_max=R)
    e4b.e4b_lora_backward(gate_up.a, gate_up.b, kept.xs, kept.s_gu, dgu, kept.offsets,
                          _lora_ws(gate_up, R, True, new, "ws_dgu", dev), dx=dxs, dx_base=dxs, da=d_gu.a, db=d_gu.b,
                          accumulate=accumulate, scale=gate_up.scale)
    dx = new("dx", (T, H), bf16, dev)
    e4b.e4b_permute_backward(dxs, kept.inv, dx, top_k=k)
    return dx, dgates, d_gu, d_dn
