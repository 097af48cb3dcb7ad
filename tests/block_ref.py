"""Plain references in float64 of linear attention with a decay for each head
and of the norms around a block, with their gradients and with the sums of the
terms' absolute values that error bounds are made of.  Written from the
formulas, token by token, on the CPU."""
from __future__ import annotations

import torch


def f64(x):
    return None if x is None else x.detach().cpu().double()


def _row(q, k, v, g, s0, scale):
    """One row: q, k [n, nv, K] (heads expanded), v [n, nv, V], g [n, nv]."""
    S, o, states = s0.clone(), [], []
    for t in range(q.shape[0]):
        S = torch.exp(g[t])[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
        o.append(scale * (q[t][:, :, None] * S).sum(1))
        states.append(S)
    return (torch.stack(o) if o else v.clone()), S, states


def attention(q, k, v, g, offsets, s0, scale):
    """(o [T, nv, V], last states [B, nv, K, V]) in float64; rows outside the
    offsets stay zero."""
    q, k, v = f64(q), f64(k), f64(v)
    nv, G = v.shape[1], v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    g = torch.zeros(q.shape[:2], dtype=torch.float64) if g is None else f64(g)
    B = len(offsets) - 1
    s0 = torch.zeros(B, nv, q.shape[2], v.shape[2], dtype=torch.float64) if s0 is None else f64(s0)
    o, end = torch.zeros(v.shape, dtype=torch.float64), s0.clone()
    for r in range(B):
        a, b = offsets[r], offsets[r + 1]
        o[a:b], end[r], _ = _row(q[a:b], k[a:b], v[a:b], g[a:b], s0[r], scale)
    return o, end


def attention_grads(do, q, k, v, g, offsets, s0, ds, scale, sign=-1.0):
    """dict of dq, dk, dv, dg, ds0 in float64, from the formulas.  With every
    operand replaced by its absolute value and sign=+1, dg is the sum of the
    absolute terms of sum_{i >= j} (q_i . dq_i - k_i . dk_i) + <S, dS>."""
    do, q, k, v = f64(do), f64(q), f64(k), f64(v)
    nv, nk = v.shape[1], q.shape[1]
    G = nv // nk
    qe, ke = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    g = torch.zeros(qe.shape[:2], dtype=torch.float64) if g is None else f64(g)
    B = len(offsets) - 1
    zero = torch.zeros(B, nv, q.shape[2], v.shape[2], dtype=torch.float64)
    s0 = zero if s0 is None else f64(s0)
    ds = zero if ds is None else f64(ds)
    dq, dk = torch.zeros_like(qe), torch.zeros_like(ke)
    dv, dg, d0 = torch.zeros_like(v), torch.zeros_like(g), ds.clone()
    for r in range(B):
        a, b = offsets[r], offsets[r + 1]
        _, end, states = _row(qe[a:b], ke[a:b], v[a:b], g[a:b], s0[r], scale)
        D = ds[r].clone()
        tail = (end * D).sum((1, 2))
        for t in range(b - a - 1, -1, -1):
            i = a + t
            D = D + scale * qe[i][:, :, None] * do[i][:, None, :]
            dq[i] = scale * (states[t] * do[i][:, None, :]).sum(2)
            dk[i] = (D * v[i][:, None, :]).sum(2)
            dv[i] = (D * ke[i][:, :, None]).sum(1)
            before = states[t - 1] if t else s0[r]
            e = torch.exp(g[i])
            if sign < 0:
                dg[i] = e * (D * before).sum((1, 2))
            else:
                tail = tail + (qe[i] * dq[i]).sum(1) + (ke[i] * dk[i]).sum(1)
                dg[i] = tail
            D = e[:, None, None] * D
        d0[r] = D
    fold = lambda x: x.unflatten(1, (nk, G)).sum(2)  # noqa: E731
    return dict(dq=fold(dq), dk=fold(dk), dv=dv, dg=dg, ds0=d0)


# ------------------------------------------------------------------ norms ---

def _act(z, name):
    if name is None:
        return z
    s = torch.sigmoid(z)
    return s if name == "sigmoid" else z * s


def norm(y, w1, group, gate, act, x, c, w2, eps):
    """(h, n, absolute terms of h, absolute terms of n) in float64."""
    y, w1, gate, x, w2 = (f64(t) for t in (y, w1, gate, x, w2))
    T, D = y.shape
    p = y
    if w1 is not None:
        n = group or D
        w = w1.repeat(D // w1.numel())
        u = y.reshape(T, D // n, n)
        p = (u / torch.sqrt(u.square().mean(2, keepdim=True) + eps)).reshape(T, D) * w
    if gate is not None:
        p = p * _act(gate, act)
    h = c * p
    ah = h.abs()
    if x is not None:
        h, ah = h + x, ah + x.abs()
    if w2 is None:
        return h, None, ah, None
    r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    return h, h * r * w2, ah, ah * r * w2.abs()


def norm_grads(dh, dn, y, h, w1, group, gate, act, x, c, w2, eps):
    """dict of dx, dgate, dy, dw1, dw2 in float64, from the formulas, and the
    same names with a leading 'a' for the sums of the absolute terms."""
    dh, dn, y, h, w1, gate, w2 = (f64(t) for t in (dh, dn, y, h, w1, gate, w2))
    T, D = y.shape
    out, H, aH = {}, dh, dh.abs()
    if w2 is not None:
        r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
        hat, t = h * r, dn * w2
        H = H + r * (t - hat * (t * hat).mean(1, keepdim=True))
        aH = aH + r * (t.abs() + hat.abs() * (t * hat).abs().mean(1, keepdim=True))
        out["dw2"], out["adw2"] = (dn * hat).sum(0), (dn * hat).abs().sum(0)
    out["dx"], out["adx"] = H, aH
    hat, w, rr, n = y, torch.ones(D, dtype=torch.float64), None, group or D
    if w1 is not None:
        w = w1.repeat(D // w1.numel())
        u = y.reshape(T, D // n, n)
        rr = 1 / torch.sqrt(u.square().mean(2, keepdim=True) + eps)
        hat = (u * rr).reshape(T, D)
    dp, adp = c * H, abs(c) * aH
    if gate is not None:
        if act is None:
            d = torch.ones_like(gate)
        else:
            s = torch.sigmoid(gate)
            d = s * (1 - s) if act == "sigmoid" else s * (1 + gate * (1 - s))
        dg, adg = dp * hat * w * d, adp * (hat * w * d).abs()
        if act == "silu":  # the derivative's own terms cancel where it is small
            adg = adg + adp * (hat * w).abs() * torch.sigmoid(gate) * (1 + gate.abs())
        if gate.dim() == 1:
            dg, adg = dg.sum(0), adg.sum(0)
        out["dgate"], out["adgate"] = dg, adg
        a = _act(gate, act)
        dp, adp = dp * a, adp * a.abs()
    if w1 is None:
        out["dy"], out["ady"] = dp, adp
        return out
    fold = lambda x: x.reshape(-1, w1.numel()).sum(0)  # noqa: E731
    out["dw1"], out["adw1"] = fold(dp * hat), fold(adp * hat.abs())
    v = lambda x: x.reshape(T, D // n, n)  # noqa: E731
    t, at, hv = v(dp * w), v(adp * w.abs()), v(hat)
    out["dy"] = (rr * (t - hv * (t * hv).mean(2, keepdim=True))).reshape(T, D)
    out["ady"] = (rr * (at + hv.abs() * (at * hv.abs()).mean(2, keepdim=True))).reshape(T, D)
    return out
