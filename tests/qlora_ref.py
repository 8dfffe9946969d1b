"""The packed layer with adapters, forward and backward, in 64 bits: the formulas
of qlora.py expert by expert. `stored` is applied to every tensor that the path
stores in bf16 (identity: the mathematics alone)."""

import torch

import adapter_ref as ref


def bf16(t):
    return t.to(torch.bfloat16).double()


def step(w_gu, w_dn, b_gu, b_dn, gu_ad, dn_ad, x, ids, gates, dy, layout, act, stored=bf16):
    """w_gu [E, 2I, H], w_dn [E, H, I] and biases in 64 bits; adapters as
    (a [E, r, K], b [E, N, r], scale [E]). Returns a dict of results."""
    E, _, H = w_gu.shape
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    out = {n: torch.zeros_like(t) for n, t in (("gu_a", gu_ad[0]), ("gu_b", gu_ad[1]), ("dn_a", dn_ad[0]),
                                               ("dn_b", dn_ad[1]))}
    ys = torch.zeros(T * k, H, dtype=torch.float64)
    dxs = torch.zeros(T * k, H, dtype=torch.float64)
    dgates = torch.zeros(T * k, dtype=torch.float64)
    g = gates.reshape(-1).double()
    for e in range(E):
        s = torch.nonzero(flat == e).flatten()
        if not len(s):
            continue
        (A1, B1, w1), (A2, B2, w2) = ((t[0][e], t[1][e], t[2][e]) for t in (gu_ad, dn_ad))
        xe, d = x[s // k], dy[s // k]
        s1 = xe @ A1.T
        y32 = stored(xe @ w_gu[e].T + b_gu[e]) + w1 * (s1 @ B1.T)
        gu, h = stored(y32), stored(ref.glu(*ref.split_gu(y32, layout), act)[0])
        s2 = h @ A2.T
        ys[s] = stored(stored(h @ w_dn[e].T + b_dn[e]) + w2 * (s2 @ B2.T))
        dgates[s] = (d * ys[s]).sum(1)
        dys = stored(g[s][:, None] * d)
        t = w2 * (dys @ B2)
        out["dn_a"][e], out["dn_b"][e] = t.T @ h, w2 * (dys.T @ s2)
        dh = stored(stored(dys @ w_dn[e]) + t @ A2)
        _, dg, du = ref.glu(*ref.split_gu(gu, layout), act)
        dgu = stored(ref.join_gu(dh * dg, dh * du, layout))
        t = w1 * (dgu @ B1)
        out["gu_a"][e], out["gu_b"][e] = t.T @ xe, w1 * (dgu.T @ s1)
        dxs[s] = stored(stored(dgu @ w_gu[e]) + t @ A1)
    out["y"] = (ys * g[:, None]).view(T, k, H).sum(1)
    out["dx"] = dxs.view(T, k, H).sum(1)
    out["dgates"] = dgates.view(T, k)
    return out
