"""Plain references in float64 of the selective scan, of the causal Conv1d's
gradient and of the verification of drafted tokens.  Written from the formulas,
token by token, on the CPU.  With absolute=True every factor but the decays is
replaced by its absolute value, so that the results are the sums of the terms'
absolute values that error bounds are made of."""
from __future__ import annotations

import math

import torch


def f64(x):
    return None if x is None else x.detach().cpu().double()


def softplus(x):
    return x.clamp_min(0) + torch.log1p(torch.exp(-x.abs()))


def _steps(dt, bias, soft):
    raw = f64(dt) if bias is None else f64(dt) + f64(bias)
    return raw, (softplus(raw) if soft else raw)


def _rows(x, A, B, delta, a, b, h0):
    """States behind the tokens a..b-1 of one row, [n, D, N]."""
    h, out = h0, []
    for t in range(a, b):
        h = torch.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * B[t]
        out.append(h)
    return out


def scan(x, dt, A, B, C, off, *, D=None, z=None, bias=None, soft=False, h0=None, absolute=False):
    """(out [T, D], last states [rows, D, N]); tokens outside the rows are zero."""
    mag = (lambda v: v.abs()) if absolute else (lambda v: v)
    _, delta = _steps(dt, bias, soft)
    x, A = mag(f64(x)), f64(A)
    per = x.shape[1] // B.shape[1]
    B, C = (mag(f64(t)).repeat_interleave(per, 1) for t in (B, C))
    rows = len(off) - 1
    h0 = torch.zeros(rows, *A.shape, dtype=torch.float64) if h0 is None else mag(f64(h0))
    out, end = torch.zeros(x.shape, dtype=torch.float64), h0.clone()
    for r in range(rows):
        hs = _rows(x, A, B, delta, off[r], off[r + 1], h0[r])
        for t, h in zip(range(off[r], off[r + 1]), hs):
            out[t] = (C[t] * h).sum(1)
            if D is not None:
                out[t] += mag(f64(D)) * x[t]
            end[r] = h
    if z is not None:
        out = out * mag(f64(z) * torch.sigmoid(f64(z)))
    return out, end


def scan_grads(dout, x, dt, A, B, C, off, *, D=None, z=None, bias=None, soft=False, h0=None,
               dh=None, absolute=False):
    """dict of dx, ddt, dA, dB, dC, dD, dz, dbias, dh0."""
    mag = (lambda v: v.abs()) if absolute else (lambda v: v)
    raw, delta = _steps(dt, bias, soft)
    x, A, dy = mag(f64(x)), f64(A), mag(f64(dout))
    T, Dn = x.shape
    G = B.shape[1]
    B, C = (mag(f64(t)).repeat_interleave(Dn // G, 1) for t in (B, C))
    skip = torch.zeros(Dn, dtype=torch.float64) if D is None else mag(f64(D))
    rows = len(off) - 1
    zero = torch.zeros(rows, *A.shape, dtype=torch.float64)
    h0 = zero if h0 is None else mag(f64(h0))
    dh = zero if dh is None else mag(f64(dh))
    y = torch.zeros_like(x)
    dx, dd, dB, dC = (torch.zeros_like(v) for v in (x, x, B, C))
    dA, d0 = torch.zeros_like(A), dh.clone()
    states = [_rows(x, A, B, delta, off[r], off[r + 1], h0[r]) for r in range(rows)]
    for r in range(rows):
        for i, h in enumerate(states[r]):
            y[off[r] + i] = (C[off[r] + i] * h).sum(1) + skip * x[off[r] + i]
    dz = None
    if z is not None:
        zz = f64(z)
        sig = torch.sigmoid(zz)
        slope = sig * (1 + zz * (1 - sig)) if not absolute else sig * (1 + zz.abs() * (1 - sig))
        dz = dy * y * slope
        dy = dy * mag(zz * sig)
    dD = torch.zeros(Dn, dtype=torch.float64)
    for r in range(rows):
        lam_next = dh[r]
        for i in range(off[r + 1] - off[r] - 1, -1, -1):
            t = off[r] + i
            lam = dy[t][:, None] * C[t] + lam_next
            before = states[r][i - 1] if i else h0[r]
            a = torch.exp(delta[t][:, None] * A)
            w = lam * a * before
            s1 = (lam * B[t]).sum(1)
            dx[t] = skip * dy[t] + mag(delta[t]) * s1
            dd[t] = x[t] * s1 + (mag(A) * w).sum(1)
            dA += mag(delta[t])[:, None] * w
            dB[t] = lam * (mag(delta[t]) * x[t])[:, None]
            dC[t] = dy[t][:, None] * states[r][i]
            dD += dy[t] * x[t]
            lam_next = a * lam
        d0[r] = lam_next
    ddt = dd * torch.sigmoid(raw) if soft else dd
    inside = torch.zeros(T, 1, dtype=torch.float64)
    inside[off[0]:off[-1]] = 1
    fold = lambda v: v.unflatten(1, (G, Dn // G)).sum(2)  # noqa: E731
    return dict(dx=dx, ddt=ddt, dA=dA, dB=fold(dB), dC=fold(dC), dD=dD,
                dz=None if dz is None else dz * inside, dbias=ddt.sum(0), dh0=d0)


# ------------------------------------------------------------------ Conv1d ---

def conv(x, w, off, bias=None, silu=False):
    x, w = f64(x), f64(w)
    W = w.shape[1]
    out = torch.zeros_like(x)
    for a, b in zip(off, off[1:]):
        for t in range(a, b):
            for j in range(W):
                s = t - (W - 1 - j)
                if s >= a:
                    out[t] += w[:, j] * x[s]
            if bias is not None:
                out[t] += f64(bias)
    return out * torch.sigmoid(out) if silu else out


def conv_grads(dout, x, w, off, bias=None, silu=False, absolute=False):
    """(dx, dweight, dbias)."""
    mag = (lambda v: v.abs()) if absolute else (lambda v: v)
    g = mag(f64(dout))
    if silu:
        pre = conv(x, w, off, bias)
        sig = torch.sigmoid(pre)
        g = g * (sig * (1 + pre * (1 - sig)) if not absolute else sig * (1 + pre.abs() * (1 - sig)))
    x, w = mag(f64(x)), mag(f64(w))
    W = w.shape[1]
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(w.shape[0], dtype=torch.float64)
    for a, b in zip(off, off[1:]):
        for t in range(a, b):
            db += g[t]
            for j in range(W):
                s = t - (W - 1 - j)
                if s >= a:
                    dx[s] += w[:, j] * g[t]
                    dw[:, j] += g[t] * x[s]
    return dx, dw, db


# ------------------------------------------------------------------ drafts ---

def _largest(row):
    best = -1
    for j, v in enumerate(row):
        if not math.isnan(v) and (best < 0 or v > row[best]):
            best = j
    return best


def verify(tokens, target, off, draft=None, uniform=None):
    """(accepted, next) as lists, by Python floats (float64)."""
    p = f64(target).tolist()
    q = None if draft is None else f64(draft).tolist()
    u = None if uniform is None else f64(uniform).tolist()
    tok = tokens.cpu().tolist()
    counts, after = [], []
    for a, b in zip(off, off[1:]):
        if a == b:
            counts.append(0)
            after.append(-1)
            continue
        n = 1
        while a + n < b:
            x, row = tok[a + n], p[a + n - 1]
            if u is None:
                best = _largest(row)
                stands = best >= 0 and best == x
            elif not 0 <= x < len(row):
                stands = False
            else:
                stands = u[a + n] * (1.0 if q is None else q[a + n][x]) < row[x]
            if not stands:
                break
            n += 1
        counts.append(n)
        row = p[a + n - 1]
        if u is None:
            after.append(_largest(row))
            continue
        good = lambda v: v if v > 0 and v < math.inf else 0.0  # noqa: E731
        w = list(row)
        if a + n < b:
            if q is None:
                if 0 <= tok[a + n] < len(w):
                    w[tok[a + n]] -= 1.0
            else:
                w = [v - o for v, o in zip(w, q[a + n])]
        w = [good(v) for v in w]
        if math.fsum(w) <= 0:
            w = [good(v) for v in row]
        goal, run, found = u[a] * math.fsum(w), 0.0, -1
        for j, v in enumerate(w):
            if v > 0:
                run += v
                found = j
                if run > goal:
                    break
        after.append(found)
    return counts, after
