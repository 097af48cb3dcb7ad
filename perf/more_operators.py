"""Measured cases of the operators of a state-space layer and of drafted tokens:
the selective state space scan (prompts, single tokens, gradient), the gradient
of its short causal convolution, and the verification of drafted tokens with
the folds that advance convolution history and scan state over what it
accepted.

listed() names the cases, draw() draws more of the same ranges, prepare()
makes what a program has in hand, run() is one pass, work() what a pass cannot
do without, exact() the operators' definitions in 64 bits.  With `own` false
run() computes the plain forms in elementary torch operations in float32 (long
sums and running sums of probabilities in float64); recurrences are computed
for all tokens at once by doubling.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2, "f32": 4}


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # One sequence generating its next token: latency counts.
        dict(name="scan step 1 row bf16", op="step", rows=1, slots=64, pad=0, D=4096, N=16, G=1,
             z=True, work="bf16", state="f32"),
        # The decode step of a full server: 256 sequences of a 512-slot pool.
        dict(name="scan step 256 rows bf16", op="step", rows=256, slots=512, pad=5, D=4096, N=16,
             G=1, z=True, work="bf16", state="bf16"),
        # A short prompt (a follow-up turn).
        dict(name="scan prompt 97 bf16", op="fwd", lens="97", slots=8, D=4096, N=16, G=1, z=True,
             work="bf16", state="f32"),
        # A ragged batch of prompts in float32, an empty and a one-token row among them.
        dict(name="scan prompts ragged f32", op="fwd", lens="3665,1,911,2048,0,130,1517,64",
             slots=64, D=2048, N=16, G=2, z=True, work="f32", state="f32"),
        # One long document.
        dict(name="scan prompt 16384 bf16", op="fwd", lens="16384", slots=8, D=4096, N=16, G=1,
             z=True, work="bf16", state="bf16"),
        # A training step's micro-batch.
        dict(name="scan bwd 2x2048 bf16", op="bwd", lens="2048,2048", D=4096, N=16, G=1, z=True,
             work="bf16", state="none"),
        # Ragged packed training in float32 through carried states, no gate, more states a channel.
        dict(name="scan bwd ragged f32", op="bwd", lens="700,33,1,256,517", D=1032, N=32, G=1,
             z=False, work="f32", state="f32"),
        # The convolution's gradient in that micro-batch, over a packed projection's channels.
        dict(name="conv bwd 2x2048 bf16", op="conv_bwd", lens="2048,2048", C=8192, W=4, silu=True,
             bias=True, work="bf16"),
        # Ragged rows, a channel count that fills no wave, float32.
        dict(name="conv bwd ragged f32", op="conv_bwd", lens="700,33,1,256,517", C=1036, W=3,
             silu=False, bias=False, work="f32"),
        # Four drafted tokens of one sequence are judged, the state follows: latency counts.
        dict(name="drafts 1 row f32", op="drafts", lens="5", vocab=32000, mode="both", D=4096,
             N=16, W=4, fold=True, slots=8, probs="f32", work="bf16", state="f32"),
        # A server's windows, greedily, from the target's bf16 scores.
        dict(name="drafts 64 rows greedy bf16", op="drafts",
             lens=",".join(str(1 + 7 * i % 12) for i in range(64)), vocab=131072, mode="greedy",
             D=4096, N=16, W=4, fold=True, slots=128, probs="bf16", work="bf16", state="bf16"),
        # Many sequences whose drafts come from a lookup (no probabilities of their own).
        dict(name="drafts 256 rows f32", op="drafts",
             lens=",".join(str(1 + 3 * i % 5) for i in range(256)), vocab=50021, mode="target",
             D=0, N=0, W=0, fold=False, slots=0, probs="f32", work="f32", state="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rows(rng, total, rows):
    cut = sorted(rng.randint(0, total) for _ in range(rows - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cut, cut + [total]))


def draw(rng):
    op = rng.choice(["step", "fwd", "bwd", "conv_bwd", "drafts"])
    work = rng.choice(["bf16", "f32"])
    state = rng.choice(["bf16", "f32"]) if work == "bf16" else "f32"
    if op == "conv_bwd":
        C = 4 * _log(rng, 4, 2048)
        most = max(64, 4096 * 8192 * 2 // (C * ELEM[work]))
        return dict(op=op, lens=_rows(rng, _log(rng, 40, min(most, 16384)), rng.randint(1, 9)),
                    C=C, W=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.6,
                    bias=rng.random() < 0.6, work=work)
    if op == "drafts":
        rows = _log(rng, 1, 256)
        lens = [1 + rng.randint(0, 11)] + [rng.randint(0, 12) for _ in range(rows - 1)]
        probs = rng.choice(["bf16", "f32"])
        most = min(131072, max(200, 109 * 10 ** 6 // (max(1, sum(lens)) * ELEM[probs])))
        fold = rng.random() < 0.6
        return dict(op=op, lens=",".join(map(str, lens)), vocab=_log(rng, 100, most),
                    mode=rng.choice(["both", "target", "greedy"]), fold=fold,
                    D=8 * _log(rng, 8, 512) if fold else 0, N=16 if fold else 0,
                    W=4 if fold else 0, slots=rows + rng.randint(0, 8) if fold else 0,
                    probs=probs, work=work, state=state)
    G = rng.choice([1, 1, 2, 4])
    N = rng.choice([8, 16, 16, 16, 32, 64])
    D = 8 * G * _log(rng, 8, 512 // G)
    c = dict(op=op, D=D, N=N, G=G, z=rng.random() < 0.7, work=work, state=state)
    if op == "step":
        rows = _log(rng, 1, min(256, max(1, 256 * 4096 * 16 * 2 // (D * N * ELEM[state]))))
        return dict(c, rows=rows, slots=rows + rng.randint(0, 32),
                    pad=min(rows - 1, rng.randint(0, 3)))
    rows = rng.randint(1, 9)
    most = 16384 if op == "fwd" else 4096
    most = max(256, int(most * min(1.0, 4096 * 16 / (D * N))))
    c["lens"] = _rows(rng, _log(rng, 40, most), rows)
    if op == "fwd":
        c["slots"] = rows + rng.randint(0, 8)
    elif rng.random() < 0.5:
        c["state"] = "none"
    return c


def _lens(case):
    if case["op"] == "step":
        return [1] * case["rows"]
    return [int(x) for x in case["lens"].split(",")]


# ----------------------------------------------------------------- inputs ---

def _plan(lens, dev):
    """Where plain forms find a ragged batch's rows: the rows with tokens, their
    first and last tokens, every token's row and place in it."""
    t = lambda v: torch.tensor(v, dtype=torch.int64, device=dev)  # noqa: E731
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    live = [r for r, n in enumerate(lens) if n]
    return dict(live=t(live), first=t([off[r] for r in live]), last=t([off[r + 1] - 1 for r in live]),
                row=t([r for r, n in enumerate(lens) for _ in range(n)]),
                place=t([i for n in lens for i in range(n)]), start=t(off[:-1]), len=t(lens),
                most=max(lens, default=0), rows=len(lens))


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    work = DTYPES[case["work"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=dev) * std

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    def slots(n):
        return torch.randperm(case["slots"], generator=gen, device=dev)[:n].to(torch.int32)

    s = dict(case)
    lens = _lens(case)
    T, B = sum(lens), len(lens)
    s["plan"] = _plan(lens, dev)
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    s["offsets"] = torch.tensor(off, dtype=torch.int32, device=dev)
    if case["op"] == "conv_bwd":
        s["x"] = normal(T, case["C"]).to(work)
        s["do"] = normal(T, case["C"]).to(work)
        s["w"] = normal(case["C"], case["W"], std=case["W"] ** -0.5)
        s["bias"] = normal(case["C"], std=0.2) if case["bias"] else None
        return s
    if case["op"] == "drafts":
        V = case["vocab"]
        scores = normal(T, V, std=2.0)
        other = scores.roll(1, 0) + normal(T, V, std=0.5)  # a draft model's, a token ahead
        noise = -torch.log(-torch.log(uniform(T, V).clamp(1e-9, 1 - 1e-7)))
        best = scores.roll(1, 0).argmax(1)
        s["tokens"] = torch.where(uniform(T) < 0.8, best, (other + noise).argmax(1)).to(torch.int32)
        if case["mode"] == "both":
            s["tokens"] = (other + noise).argmax(1).to(torch.int32)
        probs = DTYPES[case["probs"]]
        s["p"] = (scores if case["mode"] == "greedy" else torch.softmax(scores, 1)).to(probs)
        s["q"] = torch.softmax(other, 1).to(probs) if case["mode"] == "both" else None
        s["u"] = None if case["mode"] == "greedy" else uniform(T)
        if not case["fold"]:
            return s
    D, N = case["D"], case["N"]
    G = case.get("G", 1)
    # x and z as halves of one projection's output; dt's, B and C as another's
    if case.get("z", False):
        xz = normal(T, 2 * D).to(work)
        s["x"], s["z"] = xz[:, :D], xz[:, D:]
    else:
        s["x"], s["z"] = normal(T, D).to(work), None
    s["dt"] = normal(T, D, std=0.5).to(work)
    bc = normal(T, 2 * G * N).to(work)
    s["B"] = bc[:, :G * N].unflatten(1, (G, N))
    s["C"] = bc[:, G * N:].unflatten(1, (G, N))
    # step sizes of 0.001 to 0.1, decays of 1 to N a unit
    step = torch.exp(uniform(D) * math.log(100.0) + math.log(1e-3))
    s["bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -(torch.arange(1, N + 1, device=dev) * torch.exp(normal(D, N, std=0.1))).contiguous()
    s["skip"] = 1 + normal(D, std=0.1)
    if case["op"] == "bwd":
        s["do"] = normal(T, D).to(work)
        s["h0"] = s["dh"] = None
        if case["state"] != "none":
            s["h0"] = normal(B, D, N, std=0.3).to(DTYPES[case["state"]])
            s["dh"] = normal(B, D, N, std=0.3).to(DTYPES[case["state"]])
        return s
    s["pool"] = normal(case["slots"], D, N, std=0.3).to(DTYPES[case["state"]])
    s["slots"] = slots(B)
    if case.get("pad"):
        s["slots"][torch.randperm(B, generator=gen, device=dev)[:case["pad"]]] = -1
    if case["op"] == "drafts":
        s["pre"] = normal(T, D).to(work)  # what the convolution read in this window
        s["hist"] = normal(case["slots"], case["W"] - 1, D).to(work)
    return s


# ------------------------------------------------------------ plain forms ---

def _softplus(x):
    return x.clamp_min(0) + torch.log1p(torch.exp(-x.abs()))


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _doubling(a, b, most):
    """Every prefix of h_t = a_t h_{t-1} + b_t, by doubling (a is 0 at a row's
    first token)."""
    s = 1
    while s < most:
        b = torch.cat([b[:s], b[s:] + a[s:] * b[:-s]])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _grouped(x, D):
    """[T, G, N] -> [T, D, N]."""
    return x.float().repeat_interleave(D // x.shape[1], 1)


def _states(x, dt, A, B, bias, plan, h0):
    """(step sizes, decays, states behind every token), float32; h0 [rows with
    tokens, D, N] or None."""
    delta = _softplus(dt.float() + bias)
    a = torch.exp(delta[:, :, None] * A)
    b = (delta * x.float())[:, :, None] * _grouped(B, x.shape[1])
    if h0 is not None:
        b[plan["first"]] += a[plan["first"]] * h0.float()
    cut = a.clone()
    cut[plan["first"]] = 0
    return delta, a, _doubling(cut, b, plan["most"])


def _plain_fwd(s, h0):
    x, plan = s["x"].float(), s["plan"]
    _, _, h = _states(s["x"], s["dt"], s["A"], s["B"], s["bias"], plan, h0)
    y = (h * _grouped(s["C"], x.shape[1])).sum(2) + s["skip"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * _sigmoid(z))
    return y.to(s["x"].dtype), h[plan["last"]]


def _plain_bwd(s):
    plan, A, work = s["plan"], s["A"], s["x"].dtype
    x, D = s["x"].float(), s["x"].shape[1]
    G = s["B"].shape[1]
    first, last = plan["first"], plan["last"]
    h0 = None if s["h0"] is None else s["h0"][plan["live"]].float()
    delta, a, h = _states(s["x"], s["dt"], A, s["B"], s["bias"], plan, h0)
    do, dz = s["do"].float(), None
    C = _grouped(s["C"], D)
    if s["z"] is not None:
        z = s["z"].float()
        sig = _sigmoid(z)
        y = (h * C).sum(2) + s["skip"] * x
        dz = do * y * (sig * (1 + z * (1 - sig)))
        do = do * (z * sig)
    lam = do[:, :, None] * C
    if s["dh"] is not None:
        lam[last] += s["dh"][plan["live"]].float()
    nxt = torch.cat([a[1:], torch.zeros_like(a[:1])])
    nxt[last] = 0
    lam = _doubling(nxt.flip(0), lam.flip(0), plan["most"]).flip(0)
    del nxt
    fold = lambda v: v.unflatten(1, (G, D // G)).sum(2, dtype=torch.float64)  # noqa: E731
    dC = fold(do[:, :, None] * h)
    dB = fold(lam * (delta * x)[:, :, None])
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = 0 if h0 is None else h0
    w = lam * a * before
    S1 = (lam * _grouped(s["B"], D)).sum(2)
    ddelta = x * S1 + (A * w).sum(2)
    ddt = ddelta * _sigmoid(s["dt"].float() + s["bias"])
    total = lambda v: v.sum(0, dtype=torch.float64).float()  # noqa: E731
    out = [(s["skip"] * do + delta * S1).to(work), ddt.to(work),
           total(w * delta[:, :, None]), dB.float().to(work), dC.float().to(work), total(do * x)]
    out += [dz.to(work)] if dz is not None else []
    out.append(total(ddt))
    if h0 is not None:
        d0 = s["dh"].float().clone()
        d0[plan["live"]] = (a * lam)[first]
        out.append(d0.to(s["h0"].dtype))
    return out


def _plain_step(s):
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    x = s["x"][live].float()
    delta = _softplus(s["dt"][live].float() + s["bias"])
    h = torch.exp(delta[:, :, None] * s["A"]) * s["pool"][at].float()
    h = h + (delta * x)[:, :, None] * _grouped(s["B"][live], x.shape[1])
    y = (h * _grouped(s["C"][live], x.shape[1])).sum(2) + s["skip"] * x
    if s["z"] is not None:
        z = s["z"][live].float()
        y = y * (z * _sigmoid(z))
    out = torch.zeros(s["x"].shape, dtype=s["x"].dtype, device=y.device)
    out[live] = y.to(out.dtype)
    s["pool"][at] = h.to(s["pool"].dtype)
    return out, s["pool"]


def _back(x, k, plan):
    """x at k tokens before each token of its row (k < 0: behind), zeros outside."""
    t = torch.arange(x.shape[0], device=x.device) - k
    place = plan["place"] - k
    keep = (place >= 0) & (place < plan["len"][plan["row"]])
    return x[t.clamp(0, max(0, x.shape[0] - 1))] * keep[:, None]


def _plain_conv_bwd(s):
    x, g, w, plan, W = s["x"].float(), s["do"].float(), s["w"], s["plan"], s["W"]
    taps = [_back(x, W - 1 - j, plan) for j in range(W)]
    if s["silu"]:
        pre = sum(taps[j] * w[:, j] for j in range(W))
        pre = pre if s["bias"] is None else pre + s["bias"]
        sig = _sigmoid(pre)
        g = g * (sig * (1 + pre * (1 - sig)))
    dx = sum(_back(g, -(W - 1 - j), plan) * w[:, j] for j in range(W))
    dw = torch.stack([(g * t).sum(0, dtype=torch.float64) for t in taps], 1)
    out = [dx.to(s["x"].dtype), dw.float()]
    return out + ([] if s["bias"] is None else [g.sum(0, dtype=torch.float64).float()])


def _plain_verify(s):
    """(tokens of each row's window that stand, the token to go on with)."""
    plan, p, tok = s["plan"], s["p"], s["tokens"].long()
    T, V = p.shape
    dev = p.device
    draft = plan["place"] > 0
    at = torch.arange(T, device=dev)
    if s["u"] is None:
        index = torch.arange(V, device=dev)
        best = torch.where(p == p.amax(1, keepdim=True), index, V).amin(1)
        stands = best[at - 1] == tok
    else:
        q = 1.0 if s["q"] is None else s["q"][at, tok].double()
        stands = s["u"].double() * q < p[at - 1, tok].double()
    wrong = torch.where(draft & ~stands, plan["place"], plan["most"] + 1)
    n = plan["len"].scatter_reduce(0, plan["row"], wrong, "amin")
    n = torch.minimum(n, plan["len"])
    live = plan["live"]
    end = plan["start"][live] + n[live] - 1           # the target's row that goes on
    go = torch.full((plan["rows"],), -1, dtype=torch.int64, device=dev)
    if s["u"] is None:
        go[live] = best[end]
        return n.int(), go.int()
    w = p[end].double()
    more = (n < plan["len"])[live]                     # a draft was refused there
    nxt = (end + 1).clamp_max(T - 1)
    if s["q"] is None:
        rest = w.clone()
        rest[torch.arange(len(end), device=dev), tok[nxt]] -= 1
    else:
        rest = w - s["q"][nxt].double()
    rest = torch.where(more[:, None], rest, w).clamp_min(0)
    w = torch.where(rest.sum(1, keepdim=True) > 0, rest, w)
    c = w.cumsum(1)
    go[live] = (c > s["u"][plan["start"][live]].double()[:, None] * c[:, -1:]).int().argmax(1)
    return n.int(), go.int()


def _plain_folds(s, n):
    """The states and histories of the rows after the first n tokens of each."""
    plan, live = s["plan"], s["plan"]["live"]
    at = s["slots"][live].long()
    _, _, h = _states(s["x"], s["dt"], s["A"], s["B"], s["bias"], plan, s["pool"][at])
    end = plan["start"][live] + n[live].long() - 1
    s["pool"][at] = h[end].to(s["pool"].dtype)
    H = s["W"] - 1
    place = n[live].long()[:, None] + torch.arange(-H, 0, device=h.device)  # in the row
    new = s["pre"][(plan["start"][live][:, None] + place).clamp_min(0)]
    old = s["hist"][at[:, None], (place + H).clamp_max(H - 1)]
    s["hist"][at] = torch.where((place >= 0)[:, :, None], new, old)


# -------------------------------------------------------------------- run ---

def run(state):
    s, op = state, state["op"]
    if not own:
        if op == "step":
            return _plain_step(s)
        if op == "fwd":
            at = s["slots"][s["plan"]["live"]].long()
            out, end = _plain_fwd(s, s["pool"][at])
            s["pool"][at] = end.to(s["pool"].dtype)
            return out, s["pool"]
        if op == "bwd":
            return _plain_bwd(s)
        if op == "conv_bwd":
            return _plain_conv_bwd(s)
        n, go = _plain_verify(s)
        if not s["fold"]:
            return n, go
        _plain_folds(s, n)
        return n, go, s["pool"], s["hist"]
    import gated_delta_rule_loop_amd as gdr
    if op == "step":
        out = gdr.gdr_selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["pool"],
                                          s["slots"], D=s["skip"], z=s["z"], dt_bias=s["bias"],
                                          softplus=True)
        return out, s["pool"]
    if op == "fwd":
        return gdr.gdr_selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["offsets"],
                                          D=s["skip"], z=s["z"], dt_bias=s["bias"], softplus=True,
                                          state=s["pool"], slot_idx=s["slots"])
    if op == "bwd":
        got = gdr.gdr_selective_scan_bwd(s["do"], s["x"], s["dt"], s["A"], s["B"], s["C"],
                                         s["offsets"], D=s["skip"], z=s["z"], dt_bias=s["bias"],
                                         softplus=True, initial_state=s["h0"],
                                         dfinal_state=s["dh"])
        return [x for x in got if x is not None]
    if op == "conv_bwd":
        got = gdr.gdr_causal_conv1d_bwd(s["do"], s["x"], s["w"], s["offsets"], bias=s["bias"],
                                        silu=s["silu"])
        return [x for x in got if x is not None]
    n, go = gdr.gdr_verify_drafts(s["tokens"], s["p"], s["offsets"], draft=s["q"],
                                  uniform=s["u"])
    if not s["fold"]:
        return n, go
    gdr.gdr_selective_scan_fold(s["pool"], s["x"], s["dt"], s["A"], s["B"], s["offsets"], n,
                                s["slots"], dt_bias=s["bias"], softplus=True)
    gdr.gdr_causal_conv1d_fold(s["hist"], s["pre"], s["offsets"], n, s["slots"])
    return n, go, s["pool"], s["hist"]


def work(case):
    e, lens = ELEM[case["work"]], _lens(case)
    T, B = sum(lens), sum(n > 0 for n in lens)
    if case["op"] == "conv_bwd":
        return {"bytes": 3 * T * case["C"] * e + 8 * case["C"] * case["W"],
                "flops": 6 * T * case["C"] * case["W"]}
    D, N, es = case["D"], case["N"], ELEM.get(case["state"], 0)
    if case["op"] == "drafts":
        V, ep = case["vocab"], ELEM[case["probs"]]
        rows = T if case["mode"] == "greedy" else (2 * B if case["mode"] == "both" else B)
        bytes_, flops = rows * V * ep, 2 * rows * V
        if case["fold"]:  # the accepted prefix is one token at least
            bytes_ += B * (2 * D * N * es + (2 * D + N) * e + 2 * (case["W"] - 1) * D * e)
            flops += 5 * B * D * N
        return {"bytes": bytes_, "flops": flops}
    G, gate = case["G"], 1 if case["z"] else 0
    if case["op"] == "step":
        n = B - case["pad"]
        return {"bytes": n * (2 * D * N * es + ((3 + gate) * D + 2 * G * N) * e) + 4 * D * N,
                "flops": 7 * n * D * N}
    if case["op"] == "fwd":
        return {"bytes": T * ((3 + gate) * D + 2 * G * N) * e + 2 * B * D * N * es + 4 * D * N,
                "flops": 7 * T * D * N}
    return {"bytes": T * ((5 + 2 * gate) * D + 4 * G * N) * e + 3 * B * D * N * es + 8 * D * N,
            "flops": 20 * T * D * N}


# ------------------------------------------------------------------ exact ---

def _walk(x, dt, A, B, bias, lens, first, keep=False, upto=None):
    """The recurrence token by token, every row at once, in float64: (step sizes,
    states behind every token where `keep`, last states)."""
    dev, D = x.device, x.shape[1]
    delta = torch.logaddexp(dt.double() + bias.double(), torch.zeros((), dtype=torch.float64,
                                                                     device=dev))
    A, B, x = A.double(), B.double(), x.double()
    off = [sum(lens[:r]) for r in range(len(lens))]
    upto = lens if upto is None else upto
    by = sorted(range(len(lens)), key=lambda r: -upto[r])
    at = torch.tensor([off[r] for r in by], device=dev)
    S = first.double()[by]
    h = torch.zeros((x.shape[0], D, A.shape[1]), dtype=torch.float64, device=dev) if keep else None
    for t in range(max(upto, default=0)):
        n = sum(m > t for m in upto)
        i = at[:n] + t
        d = delta[i]
        add = B[i].repeat_interleave(D // B.shape[1], dim=1) * (d * x[i]).unsqueeze(-1)
        S[:n] = S[:n] * (d.unsqueeze(-1) * A).exp() + add
        if keep:
            h[i] = S[:n]
    end = torch.empty_like(S)
    end[by] = S
    return delta, h, end


def _exact_out(s, h, sel=slice(None)):
    x = s["x"][sel].double()
    C = s["C"][sel].double().repeat_interleave(x.shape[1] // s["G"], dim=1)
    y = torch.matmul(h.unsqueeze(-2), C.unsqueeze(-1))[..., 0, 0] + x * s["skip"].double()
    if s["z"] is None:
        return y
    z = s["z"][sel].double()
    return y * z * torch.sigmoid(z)


def _exact_bwd(s, lens):
    D, G, A = s["D"], s["G"], s["A"].double()
    none = torch.zeros(len(lens), D, s["N"], dtype=torch.float64, device=A.device)
    h0 = none if s["h0"] is None else s["h0"].double()
    delta, h, _ = _walk(s["x"], s["dt"], s["A"], s["B"], s["bias"], lens, h0, keep=True)
    x, dy, dz = s["x"].double(), s["do"].double(), None
    Bw, Cw = (s[k].double().repeat_interleave(D // G, dim=1) for k in ("B", "C"))
    if s["z"] is not None:
        z = s["z"].double().requires_grad_(True)
        y = torch.einsum("tdn,tdn->td", h, Cw) + x * s["skip"].double()
        dz, = torch.autograd.grad((torch.nn.functional.silu(z) * y * dy).sum(), z)
        dy = dy * torch.nn.functional.silu(z.detach())
    dx, dd = torch.zeros_like(x), torch.zeros_like(x)
    dB, dC = (torch.zeros(x.shape[0], D, s["N"], dtype=torch.float64, device=x.device)
              for _ in range(2))
    dA = torch.zeros_like(A)
    L = (none if s["dh"] is None else s["dh"].double()).clone()
    off = [sum(lens[:r]) for r in range(len(lens))]
    by = sorted(range(len(lens)), key=lambda r: -lens[r])
    for back in range(max(lens)):                      # tokens behind, one of every row at a time
        rows = [r for r in by if lens[r] > back]
        i = torch.tensor([off[r] + lens[r] - 1 - back for r in rows], device=x.device)
        start = torch.tensor([lens[r] - 1 == back for r in rows], device=x.device)
        rows = torch.tensor(rows, device=x.device)
        lam = L[rows] + dy[i].unsqueeze(-1) * Cw[i]
        prev = torch.where(start[:, None, None], h0[rows], h[(i - 1).clamp_min(0)])
        a = (delta[i].unsqueeze(-1) * A).exp()
        dC[i] = dy[i].unsqueeze(-1) * h[i]
        dB[i] = lam * (delta[i] * x[i]).unsqueeze(-1)
        in_ = (lam * Bw[i]).sum(-1)
        dx[i] = dy[i] * s["skip"].double() + delta[i] * in_
        grow = lam * a * prev
        dd[i] = x[i] * in_ + (grow * A).sum(-1)
        dA += (grow * delta[i].unsqueeze(-1)).sum(0)
        L[rows] = a * lam
    ddt = dd * torch.sigmoid(s["dt"].double() + s["bias"].double())
    out = [dx, ddt, dA, dB.reshape(-1, G, D // G, s["N"]).sum(2),
           dC.reshape(-1, G, D // G, s["N"]).sum(2), (dy * x).sum(0)]
    out += [] if dz is None else [dz]
    out.append(ddt.sum(0))
    return out + ([] if s["h0"] is None else [L])


def _exact_conv(s, lens):
    """By automatic differentiation of one row after another, padded to the left."""
    x = s["x"].double().requires_grad_(True)
    w = s["w"].double().requires_grad_(True)
    leaf = [x, w]
    if s["bias"] is not None:
        leaf.append(s["bias"].double().requires_grad_(True))
    loss, a = 0, 0
    for n in lens:
        if n:
            row = torch.nn.functional.pad(x[a:a + n], (0, 0, s["W"] - 1, 0)).unfold(0, s["W"], 1)
            y = torch.einsum("tcw,cw->tc", row, w)
            y = y if s["bias"] is None else y + leaf[2]
            y = torch.nn.functional.silu(y) if s["silu"] else y
            loss = loss + (y * s["do"][a:a + n].double()).sum()
        a += n
    return list(torch.autograd.grad(loss, leaf))


def _exact_verify(s, lens):
    counts, following, a = [], [], 0
    p = s["p"].double()
    u = None if s["u"] is None else s["u"].double().tolist()
    tok = s["tokens"].tolist()
    for n in lens:
        if not n:
            counts.append(0)
            following.append(-1)
            continue
        k = 1
        while k < n:
            row = p[a + k - 1]
            if u is None:
                good = int((row == row.max()).nonzero()[0, 0]) == tok[a + k]
            else:
                q = 1.0 if s["q"] is None else float(s["q"][a + k, tok[a + k]])
                good = u[a + k] * q < float(row[tok[a + k]])
            if not good:
                break
            k += 1
        row = p[a + k - 1]
        counts.append(k)
        if u is None:
            following.append(int((row == row.max()).nonzero()[0, 0]))
        else:
            w = row.clone()
            if k < n and s["q"] is None:
                w[tok[a + k]] = max(0.0, float(w[tok[a + k]]) - 1.0)
            elif k < n:
                w = torch.relu(w - s["q"][a + k].double())
            w = w if float(w.sum()) > 0 else row
            c = torch.cumsum(w, 0)
            following.append(int((c > u[a] * c[-1]).nonzero()[0, 0]))
        a += n
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=p.device)  # noqa: E731
    return t(counts), t(following)


def exact(case, seed):
    s, lens = prepare(case, seed), _lens(case)
    op = case["op"]
    if op == "conv_bwd":
        return _exact_conv(s, lens)
    if op == "bwd":
        return _exact_bwd(s, lens)
    if op == "drafts":
        n, go = _exact_verify(s, lens)
        if not case["fold"]:
            return n, go
        pool, hist, at = s["pool"].double(), s["hist"].double(), s["slots"].long()
        pool[at] = _walk(s["x"], s["dt"], s["A"], s["B"], s["bias"], lens, pool[at],
                         upto=n.tolist())[2]
        H, a = case["W"] - 1, 0
        for r, k in enumerate(n.tolist()):
            hist[at[r]] = torch.cat([hist[at[r]], s["pre"][a:a + k].double()])[-H:]
            a += lens[r]
        return n, go, pool, hist
    pool = s["pool"].double()
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    if op == "step":
        _, h, pool[at] = _walk(s["x"][live], s["dt"][live], s["A"], s["B"][live], s["bias"],
                               [1] * int(live.sum()), pool[at], keep=True)
        out = torch.zeros(s["x"].shape, dtype=torch.float64, device=pool.device)
        out[live] = _exact_out(s, h, live)
        return out, pool
    if sum(lens) * case["D"] * case["N"] > 1 << 31:
        return None
    _, h, pool[at] = _walk(s["x"], s["dt"], s["A"], s["B"], s["bias"], lens, pool[at], keep=True)
    return torch.cat([_exact_out(s, h[i:i + 2048], slice(i, i + 2048))
                      for i in range(0, sum(lens), 2048)]), pool
