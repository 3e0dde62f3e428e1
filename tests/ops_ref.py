"""Plain float64 definitions of the grouped products, the adapters and the
orthogonalised update (CPU), and the bounds their GPU results are held to.

Bounds.  A sum of K exact products in fp32 makes at most K roundings, each at
most 2^-23 (a whole step, should the matrix unit truncate) of a partial sum.
With terms of random sign a partial sum stays below about 5 s, s =
sqrt(sum of the squared terms), and the roundings add up like a random walk:
5 sqrt(K) 2^-23 s bounds an element's error, some 1/1000 of what a lost or
doubled term changes at the sizes tested.  A bf16 result adds half a step of its value, 2^-8.
A factor that enters a product as two bf16 parts keeps 2^-16 of its value.
"""
import numpy as np
import torch

U32 = 2.0 ** -23
HALF_BF16 = 2.0 ** -8
TWO_PARTS = 2.0 ** -16


def f64(t):
    return t.detach().cpu().double()


def e4m3_values(codes):
    """E4M3 codes (uint8) to float64: bias 7, no infinities."""
    c = codes.cpu().to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (8 + m) * 2.0 ** (e - 10).double(), m * 2.0 ** -9)
    return torch.where(c >= 128, -mag, mag)


def rows_of(offsets, g, R):
    """The group's rows, clamped as moe.h says."""
    b = min(max(int(offsets[g]), 0), R)
    return b, max(b, min(int(offsets[g + 1]), R))


def grouped(x, offsets, w, transposed=False, w_scale=None):
    """(y, s): rows of no group are NaN; s = sqrt of the sum of squared terms."""
    x = f64(x)
    w = e4m3_values(w) * f64(w_scale)[:, :, None] if w_scale is not None else f64(w)
    if transposed:
        w = w.transpose(1, 2)
    y = torch.full((x.shape[0], w.shape[1]), float("nan"), dtype=torch.float64)
    s = y.clone()
    for g in range(w.shape[0]):
        a, b = rows_of(offsets, g, x.shape[0])
        y[a:b] = x[a:b] @ w[g].T
        s[a:b] = ((x[a:b] ** 2) @ (w[g] ** 2).T).sqrt()
    return y, s


def grouped_wgrad(dy, x, offsets):
    dy, x = f64(dy), f64(x)
    G = len(offsets) - 1
    dw = torch.zeros((G, dy.shape[1], x.shape[1]), dtype=torch.float64)
    s = dw.clone()
    n = []
    for g in range(G):
        a, b = rows_of(offsets, g, x.shape[0])
        dw[g] = dy[a:b].T @ x[a:b]
        s[g] = ((dy[a:b] ** 2).T @ (x[a:b] ** 2)).sqrt()
        n.append(b - a)
    return dw, s, n


def product_bound(s, K, y=None):
    """Elementwise bound of a K-term product; y: the value, when it is rounded to bf16."""
    b = 5 * max(K, 1) ** 0.5 * U32 * s
    return b if y is None else b + HALF_BF16 * (y.abs() + b)


def lora(x, w, a, b, adapter, scale):
    """dict of y, xa and the term sizes of both."""
    x, w, a, b = f64(x), f64(w), f64(a), f64(b)
    L, r, _ = a.shape
    ad = adapter.cpu().long()
    sc = torch.ones(L, dtype=torch.float64) if scale is None else f64(scale)
    y, s2 = x @ w.T, (x ** 2) @ (w ** 2).T
    xa = torch.zeros((x.shape[0], r), dtype=torch.float64)
    sxa = xa.clone()
    parts = torch.zeros_like(y)  # sum of |terms| of the second product
    for l in range(L):
        t = torch.nonzero(ad == l).flatten()
        if not len(t):
            continue
        xa[t] = x[t] @ a[l].T
        sxa[t] = ((x[t] ** 2) @ (a[l] ** 2).T).sqrt()
        y[t] += sc[l] * (xa[t] @ b[l].T)
        s2[t] += sc[l] ** 2 * ((xa[t] ** 2) @ (b[l] ** 2).T)
        parts[t] = sc[l].abs() * (xa[t].abs() @ b[l].abs().T * TWO_PARTS
                                  + product_bound(sxa[t], x.shape[1]) @ b[l].abs().T)
    return dict(y=y, s=s2.sqrt(), xa=xa, sxa=sxa, parts=parts)


def lora_backward(x, w, a, b, adapter, scale, dy, xa):
    """dict of dx, da, db with elementwise bounds (fp32 results) under <name>_bound."""
    x, w, a, b, dy, xa = map(f64, (x, w, a, b, dy, xa))
    L, r, D = a.shape
    N = w.shape[0]
    ad = adapter.cpu().long()
    sc = torch.ones(L, dtype=torch.float64) if scale is None else f64(scale)
    dx, s2, extra = dy @ w, (dy ** 2) @ (w ** 2), torch.zeros_like(x)
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    da_b, db_b = torch.zeros_like(a), torch.zeros_like(b)
    for l in range(L):
        t = torch.nonzero(ad == l).flatten()
        if not len(t):
            continue
        u = sc[l] * (dy[t] @ b[l])
        ub = sc[l].abs() * product_bound(((dy[t] ** 2) @ (b[l] ** 2)).sqrt(), N) + TWO_PARTS * u.abs()
        dx[t] += u @ a[l]
        s2[t] += (u ** 2) @ (a[l] ** 2)
        extra[t] = ub @ a[l].abs()
        da[l] = u.T @ x[t]
        da_b[l] = product_bound(((u ** 2).T @ (x[t] ** 2)).sqrt(), 2 * len(t)) + ub.T @ x[t].abs()
        db[l] = sc[l] * (dy[t].T @ xa[t])
        db_b[l] = (sc[l].abs() * (product_bound(((dy[t] ** 2).T @ (xa[t] ** 2)).sqrt(), 2 * len(t))
                                  + TWO_PARTS * (dy[t].abs().T @ xa[t].abs())) + U32 * db[l].abs())
    return dict(dx=dx, da=da, db=db, dx_bound=product_bound(s2.sqrt(), N + 2 * r) + extra,
                da_bound=da_b, db_bound=db_b)


NS = (3.4445, -4.7750, 2.0315)


def orthogonalize(g, steps=5, eps=1e-7):
    """float64 Newton-Schulz steps of every matrix of a stack."""
    a, b, c = NS
    out = []
    for x in f64(g):
        n = x.norm() + eps
        x = x / n if n > 0 else torch.zeros_like(x)
        for _ in range(steps):
            p = x @ x.T
            x = a * x + (b * p + c * p @ p) @ x
        out.append(x)
    return torch.stack(out) if out else f64(g)


def assert_within(got, ref, bound, what=""):
    got = f64(got)
    err = (got - ref).abs()
    bad = ~(err <= bound + 1e-300)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its bound (at %s: %r, expected %r)" % (
        what, int(bad.sum()), bad.numel(), float((err / (bound + 1e-300)).nan_to_num(np.inf).max()),
        tuple(torch.nonzero(bad)[0].tolist()), float(got[bad][0]), float(ref[bad][0]))
