"""Measured cases of the operators around a linear-attention block: linear
attention with a decay for each head (prompts, single tokens, gradient) and
the norms before and after a block fused with its gate and residual scale
(forward and gradient).

listed() names the cases, draw() draws more of the same ranges, prepare()
makes what a program has in hand, run() is one pass, work() what a pass cannot
do without, exact() the operators' definitions in 64 bits.  With `own` false
run() computes the plain forms in elementary torch operations in float32
(decay exponents and long sums in float64).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2, "f32": 4}
CHUNK = 64
EPS = 1e-6


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # One sequence generating its next token: latency counts.
        dict(name="step 1 row bf16", op="step", rows=1, slots=64, pad=0, nk=16, nv=32, K=128,
             V=128, work="bf16", state="bf16", decay="token"),
        # The decode step of a full server: 256 sequences of a 512-slot pool.
        dict(name="step 256 rows bf16", op="step", rows=256, slots=512, pad=0, nk=16, nv=32,
             K=128, V=128, work="bf16", state="bf16", decay="token"),
        # A partly filled batch (padding rows) in float32, K != V, an odd group of 3.
        dict(name="step 19 rows f32", op="step", rows=19, slots=40, pad=3, nk=4, nv=12, K=64,
             V=96, work="f32", state="f32", decay="head"),
        # A short prompt (a follow-up turn): one ragged tail of a chunk.
        dict(name="prompt 97 bf16", op="fwd", lens="97", slots=8, nk=16, nv=32, K=128, V=128,
             work="bf16", state="bf16", decay="token"),
        # A ragged batch of prompts in float32, an empty and a one-token row among them.
        dict(name="prompts ragged f32", op="fwd", lens="3665,1,911,2048,0,130,1517,64", slots=64,
             nk=16, nv=32, K=128, V=128, work="f32", state="f32", decay="token"),
        # One long document with fixed decays for the heads.
        dict(name="prompt 32768 bf16", op="fwd", lens="32768", slots=8, nk=16, nv=32, K=128,
             V=128, work="bf16", state="bf16", decay="head"),
        # A training step's micro-batch: gradients of q, k, v and the decays.
        dict(name="train 2x2048 bf16", op="bwd", lens="2048,2048", nk=16, nv=16, K=128, V=128,
             work="bf16", state="none", decay="token"),
        # Ragged packed training in float32 through carried states, shared key heads, K != V.
        dict(name="train ragged f32", op="bwd", lens="700,33,1,256,517", nk=4, nv=8, K=64, V=128,
             work="f32", state="f32", decay="token"),
        # The norms between two blocks while one token is generated: latency counts.
        dict(name="norm 1 token bf16", op="norm", tokens=1, D=4096, group=4096, gate="token",
             act="sigmoid", residual=True, pre=True, work="bf16"),
        # The gated norm of every head's output over a long prompt.
        dict(name="norm heads 16384 bf16", op="norm", tokens=16384, D=4096, group=128,
             gate="token", act="silu", residual=False, pre=False, work="bf16"),
        # Its gradient in training.
        dict(name="norm bwd heads 8192 bf16", op="norm_bwd", tokens=8192, D=4096, group=128,
             gate="token", act="silu", residual=False, pre=False, work="bf16"),
        # Norms around a block with a learned gate for each channel, float32, odd token count.
        dict(name="norm bwd 513 f32", op="norm_bwd", tokens=513, D=2048, group=2048,
             gate="channel", act="none", residual=True, pre=True, work="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "fwd", "bwd", "norm", "norm_bwd"])
    work = rng.choice(["bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        group = rng.choice([64, 96, 128, 256, 0])
        D = group * rng.randint(2, 32) if group else 8 * _log(rng, 24, 1024)
        if D == 3 << 10:
            D += group or 8
        most = (16384 if op == "norm" else 8192) * 4096 // D
        return dict(op=op, tokens=_log(rng, 1, most), D=D, group=group or D,
                    gate=rng.choice(["token", "channel", "none"]),
                    act=rng.choice(["silu", "sigmoid", "none"]), residual=rng.random() < 0.6,
                    pre=rng.random() < 0.6, work=work)
    nk = rng.choice([1, 2, 4, 8, 16])
    nv = nk * rng.choice([1, 2, 3, 4])
    K, V = rng.choice([64, 128, 128, 96, 256]), rng.choice([64, 128, 128, 72, 256])
    c = dict(op=op, nk=nk, nv=nv, K=K, V=V, work=work,
             state="bf16" if work == "bf16" else "f32", decay=rng.choice(["token", "head"]))
    if op == "step":
        rows = _log(rng, 1, min(256, 256 * 32 * 128 * 128 * 2 // (nv * K * V * 4)))
        return dict(c, rows=rows, slots=rows + rng.randint(0, 32),
                    pad=min(rows - 1, rng.randint(0, 3)))
    rows = rng.randint(1, 9)
    most = 16384 if op == "fwd" else 4096
    most = max(256, int(most * min(1.0, 16 * 128 * 128 / (nv * max(K * V, 8192)))))
    total = _log(rng, 40, most)
    cut = sorted(rng.randint(0, total) for _ in range(rows - 1))
    lens = [b - a for a, b in zip([0] + cut, cut + [total])]
    c["lens"] = ",".join(map(str, lens))
    if op == "fwd":
        c["slots"] = rows + rng.randint(0, 8)
    elif rng.random() < 0.5:
        c["state"] = "none"
    return c


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ----------------------------------------------------------------- inputs ---

def _chunks(lens, dev):
    """Where plain forms find a ragged batch's tokens: chunks of one row each."""
    idx, row, last = [], [], [-1] * len(lens)
    pos = [0] * sum(lens)
    base = 0
    for r, n in enumerate(lens):
        for c in range(0, n, CHUNK):
            m = min(CHUNK, n - c)
            for i in range(m):
                pos[base + c + i] = len(idx) * CHUNK + i
            idx.append(list(range(base + c, base + c + m)) + [sum(lens)] * (CHUNK - m))
            last[r] = len(row)
            row.append(r)
        base += n
    t = lambda v: torch.tensor(v, dtype=torch.int64, device=dev)  # noqa: E731
    return dict(idx=t(idx), row=t(row), last=t(last), pos=t(pos), rows=len(lens))


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    work = DTYPES[case["work"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=dev) * std

    s = dict(case)
    if case["op"] in ("norm", "norm_bwd"):
        T, D = case["tokens"], case["D"]
        s["y"] = normal(T, D).to(work)
        s["w1"] = 1 + normal(case["group"], std=0.1)  # one weight that all heads share
        s["gate"] = {"token": lambda: normal(T, D).to(work),
                     "channel": lambda: normal(D, std=0.3), "none": lambda: None}[case["gate"]]()
        s["x"] = normal(T, D, std=2.0).to(work) if case["residual"] else None
        s["w2"] = 1 + normal(D, std=0.1) if case["pre"] else None
        s["c"] = 0.7 if case["residual"] else 1.0
        if case["op"] == "norm_bwd":
            s["h"] = normal(T, D, std=2.0).to(work)
            s["dh"] = normal(T, D).to(work)
            s["dn"] = normal(T, D).to(work) if case["pre"] else None
        return s
    nk, nv, K, V = case["nk"], case["nv"], case["K"], case["V"]
    lens = [1] * case["rows"] if case["op"] == "step" else _lens(case)
    T, B = sum(lens), len(lens)
    # q, k and v as channel ranges of one projection's output, like the packed forward's
    packed = normal(T, 2 * nk * K + nv * V)
    packed[:, :2 * nk * K] *= K ** -0.25
    packed = packed.to(work)
    s["q"] = packed[:, :nk * K].unflatten(1, (nk, K))
    s["k"] = packed[:, nk * K:2 * nk * K].unflatten(1, (nk, K))
    s["v"] = packed[:, 2 * nk * K:].unflatten(1, (nv, V))
    if case["decay"] == "head":  # fixed: memory of 2 to about 200 tokens over the heads
        g = -0.5 * torch.exp(-torch.arange(nv, device=dev) * (4.6 / max(1, nv - 1)))
        s["g"] = g.expand(T, nv)
    else:  # from the input
        s["g"] = -torch.nn.functional.softplus(normal(T, nv) - 2.5).to(work)
    s["scale"] = K ** -0.5
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    s["offsets"] = torch.tensor(off, dtype=torch.int32, device=dev)
    if case["op"] != "bwd":
        pool = (normal(case["slots"], nv, K, V, std=0.2)).to(DTYPES[case["state"]])
        slots = torch.randperm(case["slots"], generator=gen, device=dev)[:B].to(torch.int32)
        if case.get("pad"):
            slots[torch.randperm(B, generator=gen, device=dev)[:case["pad"]]] = -1
        s["pool"], s["slots"] = pool, slots
    else:
        s["do"] = normal(T, nv, V).to(work)
        s["s0"] = s["ds"] = None
        if case["state"] != "none":
            s["s0"] = normal(B, nv, K, V, std=0.2).to(DTYPES[case["state"]])
            s["ds"] = normal(B, nv, K, V, std=0.2).to(DTYPES[case["state"]])
    if case["op"] != "step":
        s["plan"] = _chunks(lens, dev)
    return s


# ------------------------------------------------------------ plain forms ---

def _pad(x, plan):
    """[T, h, d] -> float32 [chunks, h, CHUNK, d], zeros past a row's end."""
    x = torch.cat([x.float(), x.new_zeros((1,) + x.shape[1:], dtype=torch.float32)])
    return x[plan["idx"]].transpose(1, 2).contiguous()


def _unpad(o, plan):
    """[chunks, h, CHUNK, d] -> [T, h, d]."""
    return o.transpose(1, 2).flatten(0, 1)[plan["pos"]]


def _decays(g, plan, T):
    """Cumulative log decays of the chunks, and of the chunks' sums, in float64."""
    g = g.double().clamp_min(-1e4)
    g = torch.cat([g, g.new_zeros((1, g.shape[1]))])
    G = g[plan["idx"]].transpose(1, 2).cumsum(2)
    return G, G[:, :, -1].cumsum(0)


def _lower(G, strict=False):
    """exp(G_i - G_j) at j <= i (j < i), zeros elsewhere, in float32."""
    keep = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=G.device).tril(-1 if strict else 0)
    d = (G[..., :, None] - G[..., None, :]).masked_fill(~keep, -math.inf)
    return torch.exp(d).float()


def _over_chunks(dS, first, Gc, tot, plan, reverse):
    """The state that each chunk finds: decayed sums of the row's chunks before
    it (after it where `reverse`) and of the row's first state, and what is
    left at the row's other end.  dS [chunks, h, K, V]; first [rows, h, K, V]
    or None; Gc, tot: [chunks, h], the cumulative and the chunks' own sums."""
    n, h = tot.shape
    row = plan["row"]
    same = row[:, None] == row[None, :]
    order = torch.arange(n, device=row.device)
    before = same & ((order[:, None] < order[None, :]) if reverse else
                     (order[:, None] > order[None, :]))
    if reverse:  # chunk c' after c: the decays of the chunks between them
        W = (Gc - tot)[None, :, :] - Gc[:, None, :]
    else:
        W = (Gc - tot)[:, None, :] - Gc[None, :, :]
    W = torch.exp(W.masked_fill(~before[:, :, None], -math.inf)).float()
    S = torch.matmul(W.permute(2, 0, 1).contiguous(),
                     dS.transpose(0, 1).flatten(2).contiguous())
    S = S.unflatten(2, dS.shape[2:]).transpose(0, 1)
    if first is not None:
        lo = torch.full((plan["rows"], h), math.inf, dtype=torch.float64, device=row.device)
        start = (Gc - tot)
        head = torch.ones(n, dtype=torch.bool, device=row.device)
        head[1:] = row[1:] != row[:-1]
        lo[row[head]] = start[head]
        hi = torch.zeros_like(lo)
        hi[row] = Gc[plan["last"][row]]
        w = (hi[row] - Gc) if reverse else (start - lo[row])
        S = S + torch.exp(w).float()[:, :, None, None] * first[row].float()
    return S


def _plain_fwd(q, k, v, g, plan, first, scale):
    """o [T, nv, V] and the rows' last states, float32."""
    nv, nk = v.shape[1], q.shape[1]
    share = torch.arange(nv, device=q.device) // (nv // nk)
    Q, Kc, Vc = _pad(q, plan)[:, share], _pad(k, plan)[:, share], _pad(v, plan)
    G, Gc = _decays(g, plan, q.shape[0])
    tot = G[:, :, -1]
    P = torch.matmul(Q, Kc.transpose(2, 3)) * _lower(G)
    Kw = Kc * torch.exp(tot[:, :, None] - G).float()[..., None]
    dS = torch.matmul(Kw.transpose(2, 3), Vc)
    S = _over_chunks(dS, first, Gc, tot, plan, False)
    o = torch.matmul(P, Vc) + torch.matmul(Q * torch.exp(G).float()[..., None], S)
    last = plan["last"]
    end = torch.exp(tot).float()[:, :, None, None] * S + dS
    end = torch.where((last >= 0)[:, None, None, None], end[last],
                      first.float() if first is not None else torch.zeros_like(end[:1]))
    return scale * _unpad(o, plan), end


def _plain_bwd(s):
    q, k, v, do, g, plan, scale = (s[n] for n in ("q", "k", "v", "do", "g", "plan", "scale"))
    nv, nk = v.shape[1], q.shape[1]
    share = torch.arange(nv, device=q.device) // (nv // nk)
    Q, Kc, Vc, O = (_pad(q, plan)[:, share], _pad(k, plan)[:, share], _pad(v, plan),
                    scale * _pad(do, plan))
    G, Gc = _decays(g, plan, q.shape[0])
    tot = G[:, :, -1]
    eG, eR = torch.exp(G).float()[..., None], torch.exp(tot[:, :, None] - G).float()[..., None]
    L = _lower(G)
    P = torch.matmul(Q, Kc.transpose(2, 3)) * L
    dP = torch.matmul(O, Vc.transpose(2, 3)) * L
    dS = torch.matmul((Kc * eR).transpose(2, 3), Vc)
    dD = torch.matmul((Q * eG).transpose(2, 3), O)
    S = _over_chunks(dS, s["s0"], Gc, tot, plan, False)
    D = _over_chunks(dD, s["ds"], Gc, tot, plan, True)
    dq_in = torch.matmul(O, S.transpose(2, 3)) * eG
    dk_in = torch.matmul(Vc, D.transpose(2, 3)) * eR
    dq = torch.matmul(dP, Kc) + dq_in
    dk = torch.matmul(dP.transpose(2, 3), Q) + dk_in
    dv = torch.matmul(P.transpose(2, 3), O) + torch.matmul(Kc, D) * eR
    # dg_j: pairs i >= j > l within the chunk, what enters it at either side, and the states'
    M = torch.matmul(Q, Kc.transpose(2, 3)) * torch.matmul(O, Vc.transpose(2, 3)) * _lower(G, True)
    R = M.sum(3, dtype=torch.float64) + (Q * dq_in).sum(3, dtype=torch.float64)
    C = M.sum(2, dtype=torch.float64) + (Kc * dk_in).sum(3, dtype=torch.float64)
    end = torch.exp(tot).float()[:, :, None, None] * S + dS
    dg = (R - C).flip(2).cumsum(2).flip(2) + (D * end).sum((2, 3), dtype=torch.float64)[..., None]
    fold = lambda x: _unpad(x, plan).unflatten(1, (nk, nv // nk)).sum(2)  # noqa: E731
    work = q.dtype
    out = [fold(dq).to(work), fold(dk).to(work), _unpad(dv, plan).to(work)]
    if s["decay"] == "token":
        out.append(_unpad(dg[..., None], plan)[..., 0].to(g.dtype))
    if s["s0"] is not None:
        head = torch.ones_like(plan["row"], dtype=torch.bool)
        head[1:] = plan["row"][1:] != plan["row"][:-1]
        d0 = s["ds"].float().clone()
        d0[plan["row"][head]] = (torch.exp(tot)[:, :, None, None].float() * D + dD)[head]
        out.append(d0.to(s["s0"].dtype))
    return out


def _plain_step(s):
    q, k, v, g, pool, slots = (s[n] for n in ("q", "k", "v", "g", "pool", "slots"))
    nv, nk = v.shape[1], q.shape[1]
    share = torch.arange(nv, device=q.device) // (nv // nk)
    live = slots >= 0
    at = slots[live].long()
    S = pool[at].float() * torch.exp(g[live].double()).float()[:, :, None, None]
    S = S + k[live].float()[:, share, :, None] * v[live].float()[:, :, None, :]
    o = torch.zeros(v.shape, dtype=q.dtype, device=q.device)
    o[live] = ((q[live].float()[:, share, :, None] * S).sum(2) * s["scale"]).to(q.dtype)
    pool[at] = S.to(pool.dtype)
    return o, pool


def _act(x, name):
    if name == "none":
        return x
    sig = 1 / (1 + torch.exp(-x))
    return x * sig if name == "silu" else sig


def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    y, work, n = s["y"].float(), s["y"].dtype, s["group"]
    y = y.unflatten(1, (-1, n))
    p = (y * _rms(y) * s["w1"]).flatten(1)
    if s["gate"] is not None:
        p = p * _act(s["gate"].float(), s["act"])
    h = s["c"] * p if s["x"] is None else s["x"].float() + s["c"] * p
    if s["w2"] is None:
        return [h.to(work)]
    return [h.to(work), (h * _rms(h) * s["w2"]).to(work)]


def _plain_norm_bwd(s):
    work, n = s["y"].dtype, s["group"]
    dh, out = s["dh"].float(), []
    dw2 = None
    if s["w2"] is not None:
        h, dn = s["h"].float(), s["dn"].float()
        r = _rms(h)
        hat = h * r
        dw2 = (dn * hat).sum(0, dtype=torch.float64).float()
        t = dn * s["w2"]
        dh = dh + r * (t - hat * (t * hat).mean(-1, keepdim=True))
    if s["x"] is not None:
        out.append(dh.to(work))
    y = s["y"].float().unflatten(1, (-1, n))
    r = _rms(y)
    hat = y * r
    du = s["c"] * dh
    dp = du
    if s["gate"] is not None:
        x = s["gate"].float()
        a = _act(x, s["act"])
        dp = du * a
        d = torch.ones_like(x)
        if s["act"] != "none":
            sig = 1 / (1 + torch.exp(-x))
            d = sig * (1 - sig) if s["act"] == "sigmoid" else sig * (1 + x * (1 - sig))
        dgate = du * (hat * s["w1"]).flatten(1) * d
        out.append(dgate.to(work) if x.dim() == 2 else dgate.sum(0, dtype=torch.float64).float())
    dp = dp.unflatten(1, (-1, n))
    t = dp * s["w1"]
    out.append((r * (t - hat * (t * hat).mean(-1, keepdim=True))).flatten(1).to(work))
    out.append((dp * hat).sum((0, 1), dtype=torch.float64).float())
    if dw2 is not None:
        out.append(dw2)
    return out


# -------------------------------------------------------------------- run ---

def run(state):
    s, op = state, state["op"]
    if not own:
        if op == "step":
            return _plain_step(s)
        if op == "fwd":
            at = s["slots"].long()
            o, end = _plain_fwd(s["q"], s["k"], s["v"], s["g"], s["plan"], s["pool"][at],
                                s["scale"])
            s["pool"][at] = end.to(s["pool"].dtype)
            return o.to(s["q"].dtype), s["pool"]
        if op == "bwd":
            return _plain_bwd(s)
        return _plain_norm(s) if op == "norm" else _plain_norm_bwd(s)
    import gated_delta_rule_loop_amd as gdr
    if op == "step":
        o = gdr.gdr_linear_attention_step(s["q"], s["k"], s["v"], s["g"], s["pool"], s["slots"],
                                          scale=s["scale"])
        return o, s["pool"]
    if op == "fwd":
        return gdr.gdr_linear_attention_fwd(s["q"], s["k"], s["v"], s["g"], s["offsets"],
                                            state=s["pool"], slot_idx=s["slots"],
                                            scale=s["scale"])
    if op == "bwd":
        got = gdr.gdr_linear_attention_bwd(s["do"], s["q"], s["k"], s["v"], s["g"], s["offsets"],
                                           initial_state=s["s0"], dfinal_state=s["ds"],
                                           need_dg=s["decay"] == "token", scale=s["scale"])
        return [x for x in got if x is not None]
    act = None if s["act"] == "none" else s["act"]
    if op == "norm":
        got = gdr.gdr_block_norm(s["y"], post_weight=s["w1"], group=s["group"], gate=s["gate"],
                                 activation=act, residual=s["x"], residual_scale=s["c"],
                                 pre_weight=s["w2"], eps=EPS)
    else:
        got = gdr.gdr_block_norm_bwd(s["dh"], s["dn"], s["y"], s["h"], post_weight=s["w1"],
                                     group=s["group"], gate=s["gate"], activation=act,
                                     residual=s["x"] is not None, residual_scale=s["c"],
                                     pre_weight=s["w2"], eps=EPS)
    return [x for x in got if x is not None]


def work(case):
    e = ELEM[case["work"]]
    if case["op"] in ("norm", "norm_bwd"):
        n = case["tokens"] * case["D"]
        gate = n if case["gate"] == "token" else 0
        ins = n + gate + (n if case["residual"] else 0)
        outs = n + (n if case["pre"] else 0)
        flops = 10 * n + (6 * n if case["pre"] else 0)
        if case["op"] == "norm_bwd":
            ins = 2 * n + gate + (2 * n if case["pre"] else 0)
            outs = n + gate + (n if case["residual"] else 0)
            flops *= 3
        return {"bytes": e * (ins + outs) + 8 * case["D"], "flops": flops}
    nk, nv, K, V = case["nk"], case["nv"], case["K"], case["V"]
    g = 0 if case["decay"] == "head" else nv * e  # fixed decays: nothing a token, no gradient
    if case["op"] == "step":
        n = case["rows"] - case["pad"]
        token = (2 * nk * K + 2 * nv * V) * e + g
        return {"bytes": n * (2 * nv * K * V * ELEM[case["state"]] + token),
                "flops": 5 * n * nv * K * V}
    lens = _lens(case)
    T, B = sum(lens), sum(n > 0 for n in lens)
    states = B * nv * K * V * ELEM.get(case["state"], 0)
    if case["op"] == "fwd":
        return {"bytes": T * ((2 * nk * K + 2 * nv * V) * e + g) + 2 * states,
                "flops": 4 * T * nv * K * V}
    return {"bytes": T * ((4 * nk * K + 3 * nv * V) * e + 2 * g) + 3 * states,
            "flops": 10 * T * nv * K * V}


# ------------------------------------------------------------------ exact ---

def _exact_rows(q, k, v, g, lens, first, scale):
    """The recurrence token by token, every row at once, in float64."""
    dev, nv, nk = q.device, v.shape[1], q.shape[1]
    B, most = len(lens), max(lens)
    share = [h // (nv // nk) for h in range(nv)]
    off = [sum(lens[:r]) for r in range(B)]
    S = first.double().clone()
    o = torch.zeros(v.shape, dtype=torch.float64, device=dev)
    q, k, v, g = q.double()[:, share], k.double()[:, share], v.double(), g.double()
    by = sorted(range(B), key=lambda r: -lens[r])
    S = S[by]
    at = torch.tensor([off[r] for r in by], device=dev)
    for t in range(most):
        n = sum(m > t for m in lens)
        i = at[:n] + t
        part = S[:n]
        part *= torch.exp(g[i])[:, :, None, None]
        part += k[i][..., :, None] * v[i][..., None, :]
        o[i] = scale * torch.matmul(q[i][..., None, :], part)[..., 0, :]
    end = torch.empty_like(S)
    end[by] = S
    return o, end


def _exact_grads(s, lens):
    """Gradients by automatic differentiation of the sums over pairs of tokens,
    one row and head at a time, in float64."""
    nv, nk, scale = s["v"].shape[1], s["q"].shape[1], s["scale"]
    dq, dk = (torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
              for _ in range(2))
    dv = torch.zeros(s["v"].shape, dtype=torch.float64, device=dq.device)
    dg = torch.zeros(s["g"].shape, dtype=torch.float64, device=dq.device)
    d0 = None if s["s0"] is None else s["ds"].double().clone()
    a = 0
    for r, n in enumerate(lens):
        for h in range(nv if n else 0):
            hk, b = h // (nv // nk), a + n
            leaf = [x.detach().double().clone().requires_grad_(True) for x in
                    (s["q"][a:b, hk], s["k"][a:b, hk], s["v"][a:b, h], s["g"][a:b, h])]
            q, k, v, g = leaf
            G = g.cumsum(0)
            low = torch.ones(n, n, dtype=torch.bool, device=g.device).tril()
            A = torch.exp((G[:, None] - G[None, :]).masked_fill(~low, -math.inf)) * (q @ k.T)
            o = A @ v
            loss = 0
            if d0 is not None:
                s0 = s["s0"][r, h].double().clone().requires_grad_(True)
                leaf.append(s0)
                o = o + torch.exp(G)[:, None] * (q @ s0)
                end = (torch.exp(G[-1] - G)[:, None] * k).T @ v + torch.exp(G[-1]) * s0
                loss = (end * s["ds"][r, h].double()).sum()
            loss = loss + scale * (o * s["do"][a:b, h].double()).sum()
            got = torch.autograd.grad(loss, leaf)
            dq[a:b, hk] += got[0]
            dk[a:b, hk] += got[1]
            dv[a:b, h], dg[a:b, h] = got[2], got[3]
            if d0 is not None:
                d0[r, h] = got[4]
        a += n
    return ([dq, dk, dv] + ([dg] if s["decay"] == "token" else []) +
            ([] if d0 is None else [d0]))


def _exact_norm(s, y, x, gate, w1, w2):
    """[h, n or None] in y's type, differentiable."""
    T, D = y.shape
    rows = y.reshape(T * D // s["group"], s["group"])
    u = (rows / (rows.square().mean(1) + EPS).sqrt()[:, None] * w1).reshape(T, D)
    if gate is not None:
        a = {"none": lambda z: z, "sigmoid": torch.sigmoid,
             "silu": lambda z: z * torch.sigmoid(z)}[s["act"]](gate)
        u = a * u
    h = s["c"] * u
    if x is not None:
        h = x + h
    return h, None if w2 is None else _exact_rms(h) * w2


def _exact_rms(h):
    return h / (h.square().mean(1) + EPS).sqrt()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    wide = lambda x: None if x is None else x.double()  # noqa: E731
    if case["op"] == "norm":
        h, n = _exact_norm(s, *(wide(s[k]) for k in ("y", "x", "gate", "w1", "w2")))
        return [h] if n is None else [h, n]
    if case["op"] == "norm_bwd":
        leaf = {k: wide(s[k]).requires_grad_(True) for k in ("y", "gate", "w1")
                if s[k] is not None}
        dh = wide(s["dh"])
        out, dw2 = [], []
        if s["w2"] is not None:
            h, w2 = wide(s["h"]).requires_grad_(True), wide(s["w2"]).requires_grad_(True)
            more, dw2 = torch.autograd.grad((_exact_rms(h) * w2 * wide(s["dn"])).sum(), [h, w2])
            dh, dw2 = dh + more, [dw2]
        h, _ = _exact_norm(s, leaf["y"], None, leaf.get("gate"), leaf["w1"], None)
        got = dict(zip(leaf, torch.autograd.grad((h * dh).sum(), list(leaf.values()))))
        if s["x"] is not None:
            out.append(dh)
        return out + ([got["gate"]] if "gate" in got else []) + [got["y"], got["w1"]] + dw2
    if case["op"] == "bwd":
        return _exact_grads(s, _lens(case))
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    pool = s["pool"].double()
    if case["op"] == "step":
        o = torch.zeros(s["v"].shape, dtype=torch.float64, device=s["v"].device)
        o[live], pool[at] = _exact_rows(s["q"][live], s["k"][live], s["v"][live], s["g"][live],
                                        [1] * int(live.sum()), pool[at], s["scale"])
        return o, pool
    o, pool[at] = _exact_rows(s["q"], s["k"], s["v"], s["g"], _lens(case), pool[at], s["scale"])
    return o, pool
