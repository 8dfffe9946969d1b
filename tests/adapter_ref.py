"""The adapter path's operators from their definitions in 64 bits (torch on the
CPU), with bounds on the error of fp32 sums and bf16 results."""

import torch

U_BF16 = 2.0 ** -8    # half a bf16 step, relative
U_SPLIT = 2.0 ** -16  # a value as two bf16 terms: half a step of half a step
U_SUM = 2.0 ** -23    # one fp32 addition (an MMA's may truncate: a whole step)


def routing(ids, E):
    """(counts, offsets, perm, inv) of the routing pass; ids outside [0, E) are
    dropped (inv -1)."""
    flat = ids.reshape(-1).long()
    slots = torch.nonzero((flat >= 0) & (flat < E)).reshape(-1)
    order = slots[torch.argsort(flat[slots], stable=True)]
    counts = torch.bincount(flat[slots], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64)
    offsets[1:] = counts.cumsum(0)
    inv = torch.full((flat.numel(),), -1, dtype=torch.int64)
    inv[order] = torch.arange(order.numel())
    perm = torch.full((flat.numel(),), -7, dtype=torch.int64)  # the tail is not defined
    perm[:order.numel()] = order
    return counts, offsets, perm.to(torch.int32), inv.to(torch.int32)


def sum_slots(rows, inv, gates, T, k):
    """(the weighted sums [T, H], the sums of their terms' magnitudes)."""
    H = rows.shape[1]
    y, mag = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            p = int(inv[t * k + j])
            if p < 0 or p >= rows.shape[0]:
                continue
            v = rows[p].double() * (float(gates[t, j]) if gates is not None else 1.0)
            y[t] += v
            mag[t] += v.abs()
    return y, mag


def split_gu(gu, layout):
    n = gu.shape[1] // 2
    return (gu[:, :n], gu[:, n:]) if layout == "halves" else (gu[:, 0::2], gu[:, 1::2])


def join_gu(g, u, layout):
    return torch.cat([g, u], 1) if layout == "halves" else torch.stack([g, u], 2).flatten(1)


def glu(g, u, act, alpha=1.702, limit=7.0):
    """(h, dh/dg, dh/du) in 64 bits."""
    g, u = g.double(), u.double()
    if act == "swiglu":
        sg = torch.sigmoid(g)
        return g * sg * u, u * sg * (1 + g * (1 - sg)), g * sg
    gc, uc = torch.clamp(g, max=limit), torch.clamp(u, -limit, limit)
    sg = torch.sigmoid(alpha * gc)
    zero = torch.zeros_like(g)
    dg = torch.where(g > limit, zero, (uc + 1) * sg * (1 + alpha * gc * (1 - sg)))
    du = torch.where(u.abs() > limit, zero, gc * sg)
    return (uc + 1) * gc * sg, dg, du


class Lora:
    """Forward and backward of the grouped adapters in 64 bits, each result with
    a bound on the kernels' error before its own rounding."""

    def __init__(self, a, b, offsets, scale=None, row=None, rows=None):
        self.a, self.b = a.double(), b.double()
        self.off = [int(o) for o in offsets]
        self.w = scale.double() if scale is not None else torch.ones(a.shape[0], dtype=torch.float64)
        self.row, self.rows = row, rows

    def groups(self):
        for g in range(len(self.off) - 1):
            p = torch.arange(self.off[g], self.off[g + 1])
            i = p if self.row is None else self.row[p].long()
            ok = (i >= 0) & (i < (self.rows if self.row is not None else 1 << 40))
            yield g, p[ok], i[ok]

    @staticmethod
    def _sum_err(n):
        # n / 16 chained MMAs, the sums inside one and the few that join chains
        return (n / 16 + 24) * U_SUM

    def s(self, x, R_max):
        G, r, K = self.a.shape
        s, err = torch.zeros(R_max, r, dtype=torch.float64), torch.zeros(R_max, r, dtype=torch.float64)
        for g, p, i in self.groups():
            s[p] = x[i].double() @ self.a[g].T
            err[p] = self._sum_err(K) * (x[i].double().abs() @ self.a[g].abs().T)
        return s, err

    def forward(self, x, base, R_max, n_rows):
        """s, its bound; y32, its bound (rows of no position: nan)."""
        s, es = self.s(x, R_max)
        N, r = self.b.shape[1:]
        y = torch.full((n_rows, N), float("nan"), dtype=torch.float64)
        ey = torch.zeros_like(y)
        for g, p, i in self.groups():
            w, bt = self.w[g], self.b[g].T
            add = w * (s[p] @ bt)
            mag = w.abs() * (s[p].abs() @ bt.abs())
            b0 = base[i].double() if base is not None else torch.zeros_like(add)
            y[i] = b0 + add
            ey[i] = w.abs() * (es[p] @ bt.abs()) + (U_SPLIT + self._sum_err(2 * r)) * mag + 4 * U_SUM * (b0.abs() + mag)
        return s, es, y, ey

    def backward(self, x, s, dy, dx_base, n_rows):
        G, r, K = self.a.shape
        N = self.b.shape[1]
        dx, edx = torch.full((n_rows, K), float("nan"), dtype=torch.float64), torch.zeros(n_rows, K, dtype=torch.float64)
        da, eda = torch.zeros(G, r, K, dtype=torch.float64), torch.zeros(G, r, K, dtype=torch.float64)
        db, edb = torch.zeros(G, N, r, dtype=torch.float64), torch.zeros(G, N, r, dtype=torch.float64)
        for g, p, i in self.groups():
            w, d = self.w[g], dy[i].double()
            t = w * (d @ self.b[g])
            et = w.abs() * (self._sum_err(N) + 4 * U_SUM) * (d.abs() @ self.b[g].abs())
            b0 = dx_base[i].double() if dx_base is not None else torch.zeros(len(i), K, dtype=torch.float64)
            dx[i] = b0 + t @ self.a[g]
            mag = t.abs() @ self.a[g].abs()
            edx[i] = et @ self.a[g].abs() + (U_SPLIT + self._sum_err(2 * r)) * mag + 4 * U_SUM * (b0.abs() + mag)
            rel = U_SPLIT + self._sum_err(2 * len(p)) + 2 * U_SUM
            if x is not None:
                da[g] = t.T @ x[i].double()
                eda[g] = et.T @ x[i].double().abs() + rel * (t.abs().T @ x[i].double().abs())
            sw = w * s[p].double()
            db[g] = d.T @ sw
            edb[g] = (rel + U_SUM) * (d.abs().T @ sw.abs())
        return dx, edx, da, eda, db, edb


def off_bf16(got, ref, err):
    """How far got (bf16) is outside |got - ref| <= half a step + err, in units
    of that bound (<= 1: inside)."""
    bound = U_BF16 * (ref.abs() + err) + err + 1e-37
    return float(((got.double() - ref).abs() / bound).max()) if ref.numel() else 0.0


def off_f32(got, ref, err):
    bound = err + U_SUM * ref.abs() + 1e-37
    return float(((got.double() - ref).abs() / bound).max()) if ref.numel() else 0.0
