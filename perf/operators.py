"""The operators of the adapter path around the packed experts, case by case.

Three families, as a training step or a serving step of one MoE layer with
low-rank adapters calls them:

  permute, permute_bwd, unpermute, unpermute_bwd
      token rows sorted by expert and back, with the gate weights applied, and
      the gradients of both;
  glu, glu_bwd
      the gated activation on stored gate_up rows, and its gradient;
  lora, lora_glu, lora_bwd
      low-rank adapters of many groups of rows (experts, or requests) beside a
      shared projection, with or without the gated activation behind it, and
      their gradients.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU,
``run`` is one call, in elementary torch operations where ``own`` is false and
through the library where it is true, ``exact`` the same from the definition in
64 bits, ``work`` what a pass cannot do without.
"""

import math

import torch

own = False

_F32 = torch.float32
_F64 = torch.float64
_BF16 = torch.bfloat16


# ------------------------------------------------------------------ the cases
def _rows(name, op, T, top_k, E, H, skew=0.0):
    return {"name": name, "op": op, "T": T, "top_k": top_k, "E": E, "H": H, "skew": skew}


def _glu(name, op, R, I, layout="halves", act="swiglu", pad=0):
    return {"name": name, "op": op, "R": R, "I": I, "layout": layout, "act": act, "pad": pad}


def _lora(name, op, R, G, r, K, N, skew=0.0, scattered=False, layout="halves", act="swiglu", keep=False):
    return {"name": name, "op": op, "R": R, "G": G, "r": r, "K": K, "N": N, "skew": skew, "scattered": scattered,
            "layout": layout, "act": act, "keep": keep}


def listed():
    return [
        # 16 decoding requests of the E=8, H=4096 layer: the rows the experts read, a latency case
        _rows("permute_decode16", "permute", 16, 2, 8, 4096),
        # the many-expert layer's batch (E=128, top-8, uneven experts) sorted before its first projection
        _rows("permute_skewed", "permute", 8192, 8, 128, 2048, skew=1.5),
        # the gradient of that sorting on the MXFP4 layer's sizes (H not a power of two)
        _rows("permute_bwd_mx", "permute_bwd", 8192, 4, 32, 2880),
        # expert outputs back to an odd number of prefill tokens, weighted
        _rows("unpermute_prefill", "unpermute", 4097, 2, 8, 4096),
        # the gradient of the weighted sum for rows and gates on the many-expert layer
        _rows("unpermute_bwd_skewed", "unpermute_bwd", 8192, 8, 128, 2048, skew=1.5),
        # stored gate_up rows of the prefill layer (T=4096, top-2, I=14336)
        _glu("glu_prefill", "glu", 8192, 14336),
        # the clamped, interleaved variant's gradient on the MXFP4 layer (T=8191, top-4: an odd row count)
        _glu("glu_bwd_clamped", "glu_bwd", 32764, 2880, layout="interleaved", act="clamped_glu"),
        # 16 requests, each with one of 16 adapters, beside a shared H=4096 projection, in request order
        _lora("lora_requests16", "lora", 16, 16, 16, 4096, 4096, scattered=True),
        # adapters on the prefill layer's gate_up projection, one per expert
        _lora("lora_gate_up_prefill", "lora", 8192, 8, 16, 4096, 28672),
        # serving the many-expert layer: adapters and activation in one pass, uneven experts
        _lora("lora_glu_skewed", "lora_glu", 65536, 128, 32, 2048, 1536, skew=1.5),
        # one training step's adapter gradients on the prefill layer's gate_up projection
        _lora("lora_bwd_gate_up", "lora_bwd", 8192, 8, 16, 4096, 28672),
        # the same on the MXFP4 layer's down projection, a small ragged batch, a wide rank
        _lora("lora_bwd_down_mx", "lora_bwd", 2047, 32, 64, 2880, 2880, skew=0.7),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi // step, max(-(-lo // step), round(v / step)))) * step


def draw(rng):
    op = rng.choice(["permute", "permute_bwd", "unpermute", "unpermute_bwd", "glu", "glu_bwd", "lora", "lora",
                     "lora_glu", "lora_bwd", "lora_bwd"])
    skew = rng.choice([0.0, 0.7, 1.5])
    if op in ("permute", "permute_bwd", "unpermute", "unpermute_bwd"):
        E = _log(rng, 2, 256)
        k = rng.randint(1, min(8, E))
        H = _log(rng, 64, 8192, 8)
        T = _log(rng, 1, max(2, min(32768, (1 << 27) // (H * k))))
        return {"op": op, "T": T, "top_k": k, "E": E, "H": H, "skew": skew}
    layout, act = rng.choice(["halves", "interleaved"]), rng.choice(["swiglu", "clamped_glu"])
    if op in ("glu", "glu_bwd"):
        I = _log(rng, 32, 14336, 8)
        R = _log(rng, 1, max(2, min(65536, (1 << 27) // (2 * I))))
        return {"op": op, "R": R, "I": I, "layout": layout, "act": act, "pad": rng.choice([0, 0, 8, 24])}
    G = _log(rng, 1, 128)
    r = rng.choice([8, 16, 16, 32, 48, 64])
    K = _log(rng, 64, 8192, 8)
    N = _log(rng, 64, 8192, 16)
    G = min(G, max(1, (1 << 25) // (r * (K + N))))  # the gradients of all groups stay below 128 MiB
    R = _log(rng, 1, max(2, min(32768, 100_000_000 // (K + 2 * N))))
    return {"op": op, "R": R, "G": G, "r": r, "K": K, "N": N, "skew": skew, "scattered": rng.random() < 0.4,
            "layout": layout, "act": act, "keep": op == "lora_glu" and rng.random() < 0.5}


# ------------------------------------------------------------------- the work
def work(case):
    op = case["op"]
    if "T" in case:
        T, k, H = case["T"], case["top_k"], case["H"]
        R = T * k
        if op == "permute":  # tokens read, routed rows written, the order
            return {"bytes": 2 * (T + R) * H + 4 * R, "flops": 0}
        if op == "permute_bwd":
            return {"bytes": 2 * (T + R) * H + 4 * R, "flops": R * H}
        if op == "unpermute":
            return {"bytes": 2 * (T + R) * H + 8 * R, "flops": 2 * R * H}
        # dy and the expert outputs read, their gradient written
        return {"bytes": 2 * (T + 2 * R) * H + 12 * R, "flops": 3 * R * H}
    if "I" in case:
        n = case["R"] * case["I"]
        return {"bytes": 2 * n * (3 if op == "glu" else 5), "flops": n * (6 if op == "glu" else 16)}
    R, G, r, K, N = (case[k] for k in ("R", "G", "r", "K", "N"))
    g = min(G, R)  # groups that can hold a row
    weights = 2 * g * r * (K + N) + 4 * g
    if op == "lora":  # x and the projection read, the sum and x A^T written
        return {"bytes": 2 * R * (K + 2 * N) + 4 * R * r + weights, "flops": 2 * R * r * (K + N)}
    if op == "lora_glu":
        out = N // 2 + (N if case["keep"] else 0)
        return {"bytes": 2 * R * (K + N + out) + 4 * R * r + weights, "flops": 2 * R * r * (K + N) + 3 * R * N}
    # x, dy, dx in and out, x A^T; the adapters and their fp32 gradients (of every group)
    return {"bytes": 2 * R * (3 * K + N) + 4 * R * r + weights + 4 * G * r * (K + N), "flops": 4 * R * r * (K + N)}


# ----------------------------------------------------------------- the inputs
class _Inputs:
    """Draws of one seed on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=_BF16):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        out.normal_(0.0, std, generator=self.g)
        return out

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.g, device="cuda")

    def order(self, n):
        return torch.argsort(self.uniform(n))


def _sorted_by(ids, E):
    """The routing pass' arrays for the ids of all slots: positions grouped by
    expert, slots in increasing order within one."""
    perm = torch.argsort(ids, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(ids.numel(), device=ids.device)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.bincount(ids, minlength=E).cumsum(0)
    return perm.to(torch.int32), inv.to(torch.int32), offsets


def prepare(case, seed):
    op, ins = case["op"], _Inputs(seed)
    s = {"op": op, "case": case}
    if "T" in case:
        T, k, E, H = case["T"], case["top_k"], case["E"], case["H"]
        logits = ins.normal(T, E, dtype=_F32) + case["skew"] * ins.normal(E, dtype=_F32)
        top, ids = logits.topk(k, dim=1)
        s["gates"] = torch.softmax(top, 1).contiguous()
        s["perm"], s["inv"], s["offsets"] = _sorted_by(ids.reshape(-1), E)
        if op in ("permute", "unpermute_bwd"):  # x, or dy
            s["x"] = ins.normal(T, H)
        if op != "permute":  # dxs, ys
            s["rows"] = ins.normal(T * k, H)
        if op in ("permute", "unpermute_bwd"):
            s["out_rows"] = torch.zeros(T * k, H, dtype=_BF16, device="cuda")
        if op in ("permute_bwd", "unpermute"):
            s["out"] = torch.empty(T, H, dtype=_BF16, device="cuda")
        if op == "unpermute_bwd":
            s["dgates"] = torch.empty(T, k, dtype=_F32, device="cuda")
        return s
    if "I" in case:
        R, I, pad = case["R"], case["I"], case["pad"]
        std = 3.0 if case["act"] == "clamped_glu" else 1.5  # some gates past the limit of 7
        s["gu"] = ins.normal(R, 2 * I + pad, std=std)[:, :2 * I]
        s["h"] = torch.empty(R, I + pad, dtype=_BF16, device="cuda")[:, :I]
        if op == "glu_bwd":
            s["dh"] = ins.normal(R, I + pad)[:, :I]
            s["dgu"] = torch.empty(R, 2 * I + pad, dtype=_BF16, device="cuda")[:, :2 * I]
        return s
    R, G, r, K, N = (case[k] for k in ("R", "G", "r", "K", "N"))
    bias = case["skew"] * ins.normal(G, dtype=_F32)
    ids = torch.multinomial(torch.softmax(bias, 0), R, replacement=True, generator=ins.g)
    perm, _, s["offsets"] = _sorted_by(ids, G)
    s["most"] = int(torch.bincount(ids, minlength=G).max())  # rows of the largest group
    s["row"] = perm if case["scattered"] else None
    s["x"] = ins.normal(R, K)
    s["a"] = ins.normal(G, r, K, std=K ** -0.5)
    s["b"] = ins.normal(G, N, r, std=0.5 * r ** -0.5)
    s["scale"] = 0.5 + 1.5 * ins.uniform(G)
    if op == "lora_bwd":
        s["dy"] = ins.normal(R, N, std=0.25)
        s["dx_base"] = ins.normal(R, K, std=0.25)
        s["s"] = _plain_s(s, *_padded(s)[::2])  # kept from the forward pass
        s["dx"] = torch.empty(R, K, dtype=_BF16, device="cuda")
        s["da"] = torch.empty(G, r, K, dtype=_F32, device="cuda")
        s["db"] = torch.empty(G, N, r, dtype=_F32, device="cuda")
    else:
        s["base"] = ins.normal(R, N, std=3.0 if case["act"] == "clamped_glu" else 1.0)
        s["s"] = torch.empty(R, r, dtype=_F32, device="cuda")
        s["y"] = torch.empty(R, N, dtype=_BF16, device="cuda") if op == "lora" or case["keep"] else None
        s["h"] = torch.empty(R, N // 2, dtype=_BF16, device="cuda") if op == "lora_glu" else None
    s["ws"] = {}  # the workspace, once its size is asked
    return s


# ------------------------------------------------------------ the plain forms
_ALPHA, _LIMIT = 1.702, 7.0


def _split(gu, layout):
    if layout == "halves":
        n = gu.shape[1] // 2
        return gu[:, :n], gu[:, n:]
    return gu[:, 0::2], gu[:, 1::2]


def _join(dg, du, layout):
    return torch.cat([dg, du], 1) if layout == "halves" else torch.stack([dg, du], 2).flatten(1)


def _act(g, u, act):
    if act == "swiglu":
        return g * torch.sigmoid(g) * u
    g, u = torch.clamp(g, max=_LIMIT), torch.clamp(u, -_LIMIT, _LIMIT)
    return (u + 1) * g * torch.sigmoid(_ALPHA * g)


def _act_grad(g, u, dh, act):
    if act == "swiglu":
        sg = torch.sigmoid(g)
        return dh * u * sg * (1 + g * (1 - sg)), dh * g * sg
    gin, uin = g <= _LIMIT, (u >= -_LIMIT) & (u <= _LIMIT)
    g, u = torch.clamp(g, max=_LIMIT), torch.clamp(u, -_LIMIT, _LIMIT)
    sg = torch.sigmoid(_ALPHA * g)
    return dh * (u + 1) * sg * (1 + _ALPHA * g * (1 - sg)) * gin, dh * g * sg * uin


def _padded(s):
    """Positions of the groups' rows as [G, most], and for each position its
    place in the padded form; rows past a group's end are those that follow."""
    off, R = s["offsets"], s["case"]["R"]
    p = torch.arange(R, device=off.device)
    g = torch.searchsorted(off[1:], p, right=True)
    at = off[:-1, None] + torch.arange(s["most"], device=off.device)
    inside = at < off[1:, None]
    return at.clamp(max=R - 1), inside, g * s["most"] + p - off[g]


def _by_group(t, at, s):
    """Rows of t in the padded form, in 32 bits."""
    rows = at if s["row"] is None else s["row"].long()[at]
    return t[rows].to(_F32)


def _back(t, s):
    """Rows by position to rows by their place."""
    if s["row"] is None:
        return t
    return torch.empty_like(t).index_copy_(0, s["row"].long(), t)


def _plain_s(s, at, place):
    xa = torch.bmm(_by_group(s["x"], at, s), s["a"].to(_F32).transpose(1, 2))
    return xa.flatten(0, 1)[place]


def _plain_lora(s):
    at, _, place = _padded(s)
    xa = _plain_s(s, at, place)
    add = torch.bmm(xa[at] * s["scale"][:, None, None], s["b"].to(_F32).transpose(1, 2))
    y = s["base"].to(_F32) + _back(add.flatten(0, 1)[place], s)
    if s["op"] == "lora":
        return {"y": y.to(_BF16), "s": xa}
    out = {"h": _act(*_split(y, s["case"]["layout"]), s["case"]["act"]).to(_BF16), "s": xa}
    if s["case"]["keep"]:
        out["y"] = y.to(_BF16)
    return out


def _plain_lora_bwd(s):
    at, inside, place = _padded(s)
    x, dy = _by_group(s["x"], at, s), _by_group(s["dy"], at, s) * inside[:, :, None]
    t = torch.bmm(dy, s["b"].to(_F32)) * s["scale"][:, None, None]
    da = torch.bmm(t.transpose(1, 2), x)
    db = torch.bmm(dy.transpose(1, 2), s["s"][at] * s["scale"][:, None, None])
    dx = s["dx_base"].to(_F32) + _back(torch.bmm(t, s["a"].to(_F32)).flatten(0, 1)[place], s)
    return {"dx": dx.to(_BF16), "da": da, "db": db}


def _plain(s):
    op, c = s["op"], s["case"]
    if op == "permute":
        return s["x"][(s["perm"] // c["top_k"]).long()]
    if op == "permute_bwd":
        rows = s["rows"][s["inv"].long()].to(_F32)
        return rows.view(c["T"], c["top_k"], c["H"]).sum(1).to(_BF16)
    if op == "unpermute":
        rows = s["rows"][s["inv"].long()].to(_F32).view(c["T"], c["top_k"], c["H"])
        return (rows * s["gates"][:, :, None]).sum(1).to(_BF16)
    if op == "unpermute_bwd":
        dy = s["x"][(s["perm"] // c["top_k"]).long()].to(_F32)
        dgates = (dy * s["rows"].to(_F32)).sum(1)[s["inv"].long()].view(c["T"], c["top_k"])
        return {"dys": (dy * s["gates"].view(-1)[s["perm"].long()][:, None]).to(_BF16), "dgates": dgates}
    if op == "glu":
        return _act(*_split(s["gu"].to(_F32), c["layout"]), c["act"]).to(_BF16)
    if op == "glu_bwd":
        g, u = _split(s["gu"].to(_F32), c["layout"])
        dg, du = _act_grad(g, u, s["dh"].to(_F32), c["act"])
        return {"dgu": _join(dg, du, c["layout"]).to(_BF16), "h": _act(g, u, c["act"]).to(_BF16)}
    return _plain_lora_bwd(s) if op == "lora_bwd" else _plain_lora(s)


# ------------------------------------------------------- the library's calls
def _workspace(e4b, s, backward):
    if "ws" not in s["ws"]:
        c = s["case"]
        n = e4b.e4b_lora_workspace_size(c["G"], c["r"], c["N"], c["K"], c["R"], backward=backward)
        s["ws"]["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s["ws"]["ws"]


def _library(s):
    from bit_grouped_moe_e4b_b200 import e4b

    op, c = s["op"], s["case"]
    if op == "permute":
        e4b.e4b_permute(s["x"], s["perm"], s["offsets"], s["out_rows"], top_k=c["top_k"])
        return s["out_rows"]
    if op == "permute_bwd":
        e4b.e4b_permute_backward(s["rows"], s["inv"], s["out"], top_k=c["top_k"])
        return s["out"]
    if op == "unpermute":
        e4b.e4b_unpermute(s["rows"], s["inv"], s["gates"], s["out"], top_k=c["top_k"])
        return s["out"]
    if op == "unpermute_bwd":
        e4b.e4b_unpermute_backward(s["x"], s["rows"], s["inv"], s["gates"], s["out_rows"], s["dgates"],
                                   top_k=c["top_k"])
        return {"dys": s["out_rows"], "dgates": s["dgates"]}
    if op == "glu":
        e4b.e4b_glu(s["gu"], s["h"], layout=c["layout"], act=c["act"])
        return s["h"]
    if op == "glu_bwd":
        e4b.e4b_glu_backward(s["dh"], s["gu"], s["dgu"], h=s["h"], layout=c["layout"], act=c["act"])
        return {"dgu": s["dgu"], "h": s["h"]}
    ws = _workspace(e4b, s, op == "lora_bwd")
    if op == "lora_bwd":
        e4b.e4b_lora_backward(s["a"], s["b"], s["x"], s["s"], s["dy"], s["offsets"], ws, dx=s["dx"],
                              dx_base=s["dx_base"], da=s["da"], db=s["db"], scale=s["scale"], row=s["row"])
        return {"dx": s["dx"], "da": s["da"], "db": s["db"]}
    e4b.e4b_lora(s["a"], s["b"], s["x"], s["offsets"], ws, base=s["base"], y=s["y"], h=s["h"], s=s["s"],
                 scale=s["scale"], row=s["row"], layout=c["layout"], act=c["act"])
    if op == "lora":
        return {"y": s["y"], "s": s["s"]}
    out = {"h": s["h"], "s": s["s"]}
    if c["keep"]:
        out["y"] = s["y"]
    return out


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------- the same from the definition, 64 bits
def _exact_act(y, c):
    n = y.shape[1] // 2
    u_at = torch.arange(n, device=y.device)
    g_at, u_at = (u_at, n + u_at) if c["layout"] == "halves" else (2 * u_at, 2 * u_at + 1)
    g, u = y[:, g_at], y[:, u_at]
    if c["act"] == "swiglu":
        return g / (1 + torch.exp(-g)) * u, g, u, g_at, u_at
    g2, u2 = torch.where(g > _LIMIT, _LIMIT, g), torch.where(u.abs() > _LIMIT, _LIMIT * u.sign(), u)
    return (u2 + 1) * g2 / (1 + torch.exp(-_ALPHA * g2)), g, u, g_at, u_at


def _exact_glu_grad(gu, dh, c):
    """By the product rule on h = v(u) * f(g), f(g) = g' / (1 + exp(-b g'))."""
    h, g, u, g_at, u_at = _exact_act(gu, c)
    b, lim = (1.0, math.inf) if c["act"] == "swiglu" else (_ALPHA, _LIMIT)
    gc = torch.clamp(g, max=lim)
    den = 1 + torch.exp(-b * gc)
    f, df = gc / den, (1 / den + gc * b * torch.exp(-b * gc) / den ** 2) * (g <= lim)
    v = u if c["act"] == "swiglu" else torch.clamp(u, -lim, lim) + 1
    out = torch.empty_like(gu)
    out[:, g_at] = dh * v * df
    out[:, u_at] = dh * f * (u.abs() <= lim)
    return out, h


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def groups():  # of each group with rows: its number, its positions and its places
        off = s["offsets"].tolist()
        for g in range(len(off) - 1):
            if off[g + 1] > off[g]:
                p = torch.arange(off[g], off[g + 1], device="cuda")
                yield g, p, p if s["row"] is None else s["row"][p].long()

    if "T" in case:
        T, k = case["T"], case["top_k"]
        perm, inv = s["perm"].long(), s["inv"].long().view(T, k)
        if op == "permute":
            return s["x"].double().index_select(0, torch.div(perm, k, rounding_mode="floor"))
        rows = s["rows"].double()
        if op in ("permute_bwd", "unpermute"):
            out = torch.zeros(T, case["H"], dtype=_F64, device="cuda")
            for j in range(k):
                w = s["gates"][:, j:j + 1].double() if op == "unpermute" else 1.0
                out += w * rows[inv[:, j]]
            return out
        dy = s["x"].double()
        dys, dgates = torch.zeros_like(rows), torch.zeros(T, k, dtype=_F64, device="cuda")
        for j in range(k):
            dys[inv[:, j]] = s["gates"][:, j:j + 1].double() * dy
            dgates[:, j] = torch.einsum("th,th->t", dy, rows[inv[:, j]])
        return {"dys": dys, "dgates": dgates}
    if op == "glu":
        return _exact_act(s["gu"].double(), case)[0]
    if op == "glu_bwd":
        dgu, h = _exact_glu_grad(s["gu"].double(), s["dh"].double(), case)
        return {"dgu": dgu, "h": h}
    if op == "lora_bwd":
        dx, da, db = s["dx_base"].double(), torch.zeros_like(s["da"], dtype=_F64), torch.zeros_like(s["db"], dtype=_F64)
        for g, p, rows in groups():
            w = s["scale"][g].double()
            dy, x = s["dy"][rows].double(), s["x"][rows].double()
            t = w * (dy @ s["b"][g].double())
            dx[rows] += t @ s["a"][g].double()
            da[g] = t.T @ x
            db[g] = w * (dy.T @ s["s"][p].double())
        return {"dx": dx, "da": da, "db": db}
    y = s["base"].double()
    xa = torch.zeros(case["R"], case["r"], dtype=_F64, device="cuda")
    for g, p, rows in groups():
        xa[p] = s["x"][rows].double() @ s["a"][g].double().T
        y[rows] += s["scale"][g].double() * (xa[p] @ s["b"][g].double().T)
    if op == "lora":
        return {"y": y, "s": xa}
    out = {"h": _exact_act(y, case)[0], "s": xa}
    if case["keep"]:
        out["y"] = y
    return out
