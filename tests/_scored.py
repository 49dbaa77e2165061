"""64-bit references of scored routing and of the int8 layer, written from the
formulas of include/moe.h (numpy and torch float64; no library code)."""
from __future__ import annotations

import numpy as np
import torch

NINF = float("-inf")


# ------------------------------------------------------------------ routing

def scores(l, score):
    """Scores of one row of float64 logits; 0 where the logit is -inf or NaN."""
    live = l > NINF
    s = np.zeros_like(l)
    if not live.any():
        return s
    if score == "softmax":
        m = l[live].max()
        with np.errstate(invalid="ignore"):
            e = np.where(l[live] == m, 1.0, np.exp(l[live] - m))
        s[live] = e / e.sum()
    else:
        with np.errstate(over="ignore"):
            s[live] = 1.0 / (1.0 + np.exp(-l[live]))
    return s


def _weights(l, sel, score, renorm):
    """Gates before the scale of the selected experts `sel` of one row."""
    v = l[sel]
    if not renorm:
        return scores(l, score)[sel]
    M = v.max()
    with np.errstate(invalid="ignore"):
        if score == "softmax":
            w = np.where(v == M, 1.0, np.exp(v - M))
        else:  # sigmoids relative to exp(min(M, 0)): no underflow
            top = np.where(v >= 0, 1.0, np.exp(np.minimum(v, 0) - min(M, 0.0)))
            w = top / (1.0 + np.exp(-np.abs(v)))
    return w / w.sum()


def route(logits, k, sc, bias=None, mask=None):
    """(idx [T, k], gate [T, k] float64); sc: dict of MoeScoring's arguments."""
    l = logits.detach().double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    T, E = l.shape
    G = sc.get("n_group", 1)
    g = E // G
    idx = np.full((T, k), -1, dtype=np.int64)
    gate = np.zeros((T, k))
    for t in range(T):
        if mask is not None and int(mask[t]) == 0:
            continue
        s = scores(l[t], sc["score"])
        # without a bias the logits order the experts
        choice = l[t].copy() if b is None else s + b
        value_of = s if b is None else choice
        live = (l[t] > NINF) & (choice > NINF)
        if G > 1:
            value = np.full(G, NINF)
            for j in range(G):
                mine = [i for i in range(j * g, (j + 1) * g) if live[i]]
                mine.sort(key=lambda i: (-choice[i], i))
                if mine:
                    if sc.get("group_top", 1) == 1:
                        value[j] = choice[mine[0]]
                    else:
                        value[j] = sum(value_of[i] for i in mine[:2])
            order = sorted(range(G), key=lambda j: (-value[j], j))
            for j in order[sc.get("topk_group", 1):]:
                live[j * g:(j + 1) * g] = False
        sel = sorted(np.nonzero(live)[0], key=lambda i: (-choice[i], i))[:k]
        if len(sel):
            idx[t, :len(sel)] = sel
            gate[t, :len(sel)] = sc.get("scale", 1.0) * _weights(l[t], np.array(sel), sc["score"],
                                                               sc.get("renorm", True))
    return idx, gate


def route_backward(logits, idx, dgate, sc):
    """(dlogits [T, E] float64, bound of a float32 evaluation's error)."""
    l = logits.detach().double().cpu().numpy()
    ix = idx.cpu().numpy()
    dg = dgate.double().cpu().numpy()
    T, E = l.shape
    grad = np.zeros((T, E))
    size = np.zeros((T, E))  # magnitudes of the terms, for the bound
    spread = np.zeros((T, 1))
    for t in range(T):
        slots = [r for r in range(ix.shape[1]) if 0 <= ix[t, r] < E and l[t, ix[t, r]] > NINF]
        if not slots:
            continue
        e = ix[t, slots]
        u = sc.get("scale", 1.0) * dg[t, slots]
        s = scores(l[t], sc["score"])
        fin = l[t][np.isfinite(l[t])]
        spread[t] = np.ptp(fin) if fin.size else 0.0
        if sc["score"] == "softmax" and not sc.get("renorm", True):
            total = (u * s[e]).sum()
            grad[t] = -s * total
            size[t] = s * np.abs(u * s[e]).sum()
            np.add.at(grad[t], e, u * s[e])
            np.add.at(size[t], e, np.abs(u * s[e]))
            continue
        w = _weights(l[t], e, sc["score"], sc.get("renorm", True))
        mean = (u * w).sum() if sc.get("renorm", True) else 0.0
        slope = 1.0
        if sc["score"] == "sigmoid":
            with np.errstate(over="ignore"):
                slope = 1.0 / (1.0 + np.exp(l[t, e]))
        np.add.at(grad[t], e, (u - mean) * w * slope)
        np.add.at(size[t], e, (np.abs(u) + np.abs(u * w).sum()) * w * slope)
    return grad, size * gate_rel(spread, E) * 2


def gate_rel(spread, E):
    """Relative error bound of a float32 gate: expf is within 2 ulps (2^-22), its
    argument l - M is rounded (|l - M| 2^-24), once for the term and once for the
    sum; the sum adds E / 32 + 5 roundings, divisions and products 8 more."""
    return (2.0 * (spread + 4.0) + E / 32.0 + 5.0 + 8.0) * 2.0 ** -24


# ------------------------------------------------------------------ int8

def quantize(v):
    """(q, scale) of the rows of a bf16 tensor, q in float64, scale exactly as float32."""
    f = v.double()
    amax = f.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(f).all(-1, keepdim=True)
    q = torch.round(torch.nan_to_num(f * 127.0 / torch.where(amax > 0, amax, 1.0)))
    # through float64: a quotient by 127 is never half way between two floats, so the
    # second rounding changes nothing (and a float division by a number may be a product)
    scale = (amax / 127.0).float()
    q = torch.where(bad | (amax == 0), 0.0, q)
    scale = torch.where(bad, float("nan"), scale)
    return q, scale.squeeze(-1)


def dispatch(idx, E):
    """offsets, perm_tok, inv of the stable expert order (numpy)."""
    ix = idx.cpu().numpy()
    T, k = ix.shape
    flat = ix.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = np.nonzero(ok)[0][np.argsort(flat[ok], kind="stable")]
    inv = np.full(T * k, -1, dtype=np.int64)
    inv[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))])
    return offsets, order // k, inv.reshape(T, k)


def experts(xq, xs, offsets, W1, W3, W2):
    """(o, tolerance) of the int8 experts in float64.

    The integer products are exact.  h is known up to the float32 evaluation of
    SiLU(a) b (relative error 2^-24 (8 + |a|): conversion, two scalings, the
    exponential's argument, the division and two products), so each bf16 h lies
    between the roundings of the two ends; wherever they agree (nearly
    everywhere) its 8-bit value is known exactly, elsewhere the tolerance holds the
    difference.  On top: float32 scaling (4 2^-24) and one rounding to bf16 (2^-8)."""
    R, d = xq.shape[0], W2[0].shape[1]
    o = torch.zeros(R, d, dtype=torch.float64, device=xq.device)
    tol = torch.zeros_like(o)
    off = [int(v) for v in offsets]
    for e in range(len(off) - 1):
        if off[e + 1] <= off[e]:
            continue
        rows = slice(off[e], off[e + 1])
        x, s = xq[rows].double(), xs[rows].double()[:, None]
        a = (x @ W1[0][e].double().T) * s * W1[1][e].double()
        b = (x @ W3[0][e].double().T) * s * W3[1][e].double()
        h = a * torch.sigmoid(a) * b
        err = h.abs() * (8 + a.abs()) * 2.0 ** -24 + 1e-44
        lo, hi = (h - err).bfloat16(), (h + err).bfloat16()
        small = torch.minimum(lo.double().abs(), hi.double().abs()).amax(1, keepdim=True)
        big = torch.maximum(lo.double().abs(), hi.double().abs()).amax(1, keepdim=True)
        vals = []
        for v in (lo, hi):
            for m in (small, big):
                q = torch.round(v.double() * 127.0 / torch.where(m > 0, m, 1.0)).clamp(-128, 128)
                vals.append(q * (m / 127.0).float().double())
        vals = torch.stack(vals)
        top, bottom = vals.amax(0), vals.amin(0)
        w = W2[0][e].double().T * W2[1][e].double()
        o[rows] = ((top + bottom) / 2) @ w
        # (the last term: this reference's own sum of n = d_ff rounded float64 terms is off
        # by up to n 2^-53 of their magnitudes, where the kernel's integer sum is exact)
        size = torch.maximum(top.abs(), bottom.abs()) @ w.abs()
        tol[rows] = ((top - bottom) / 2) @ w.abs() + size * (w.shape[0] + 4) * 2.0 ** -53
    tol = tol + (o.abs() + tol) * (2.0 ** -8 + 4 * 2.0 ** -24) + 1e-38
    return o, tol


def layer(x, idx, gate, W1, W3, W2, E):
    """(y, tolerance) of the layer on a given routing (gate: the float32 gates)."""
    T, k = idx.shape
    offsets, perm, inv = dispatch(idx, E)
    q, s = quantize(x)
    perm_t = torch.as_tensor(perm, device=x.device)
    o, tol = experts(q[perm_t], s[perm_t], offsets, W1, W3, W2)
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(y)
    for j in range(k):
        row = torch.as_tensor(inv[:, j], device=x.device)
        has = (row >= 0)[:, None]
        g = gate[:, j].double()[:, None]
        y += torch.where(has, g * o[row.clamp_min(0)], 0.0)
        bound += torch.where(has, g.abs() * (tol[row.clamp_min(0)] + o[row.clamp_min(0)].abs()
                                             * (2 * k) * 2.0 ** -24), 0.0)
    return y, bound + (y.abs() + bound) * 2.0 ** -8 + 1e-38


def random_weights(E, d, d_ff, seed, device="cuda"):
    """(int8, scale) pairs W1, W3 [E, d_ff, d], W2 [E, d, d_ff]."""
    gen = torch.Generator(device).manual_seed(seed)

    def one(n, kk):
        q = torch.randint(-127, 128, (E, n, kk), generator=gen, device=device).to(torch.int8)
        s = (0.5 + torch.rand(E, n, generator=gen, device=device)) / (70.0 * kk ** 0.5)
        return q, s
    return one(d_ff, d), one(d_ff, d), one(d, d_ff)
