"""Linear attention and the fused norms where their calls border on something
else.  Error bounds as in test_block_ops.py."""
import contextlib

import pytest
import torch

import gated_delta_rule_loop_amd as gdr
from gated_delta_rule_loop_amd import _binding as B
from tests import block_ref as ref
from tests.test_block_ops import (BWD, D, DT, FAKE, I32, U32, _call, _fwd, bounds, bwd_inputs,
                                  close, inputs, near)


# ------------------------------------------------- tokens outside the rows ---

@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    BWD[2], BWD[3], BWD[11], BWD[12],
    ([1], 1, 2, 8, 8, "f32", True, "token"),
    ([0], 1, 2, 16, 16, "bf16", True, "token"),
    ([40] * 20, 2, 6, 32, 64, "f32", False, "head"),
], ids=str)
def test_backward_leaves_tokens_outside_the_rows_alone(case):
    """One token before the first row, two after the last; NaN in the workspace."""
    do, q, k, v, g, off, offs, s0, ds = bwd_inputs(case)
    floats = gdr.gdr_linear_attention_workspace(q.shape[0], len(off) - 1, q.shape[1], v.shape[1],
                                                q.shape[2], v.shape[2], True)
    out = {name: torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
           for name, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g))}
    gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs, initial_state=s0, dfinal_state=ds,
                                 workspace=torch.full((max(1, floats),), float("nan"),
                                                      device="cuda"), **out)
    for name, x in out.items():
        assert (x[:off[0]] == 7).all() and (x[off[-1]:] == 7).all(), name
        assert torch.isfinite(x).all(), name


# ---------------------------------------------------------------- outliers ---

@pytest.mark.gpu
@pytest.mark.parametrize("at", ["first", "middle"])
@pytest.mark.parametrize("work", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[180], [700], [64] * 20, [513] + [1] * 70],
                         ids=["uncut", "cut", "rows", "long"])
def test_decay_gradient_after_a_few_large_tokens(lens, work, at):
    """Four tokens a hundred times the others' size, at a row's start or a third of
    the way, with decays that forget them: the later half's gradients carry the
    roundings of their own terms only (test_backward's bound, on that half)."""
    q, k, v, _, off, offs, gen = inputs(lens, 1, 2, 64, 64, DT[work], "none", seed=21)
    g = torch.full((q.shape[0], 2), -0.5, device="cuda")
    do = torch.randn(v.shape, generator=gen).to(DT[work]).cuda()
    late = []
    for a, b in zip(off, off[1:]):
        big = a if at == "first" else a + (b - a) // 3
        for x in (q, k, v):
            x[big:big + 4] *= 100
        late += range((a + b) // 2, b)
    dg = gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs)[3]
    want = ref.attention_grads(do, q, k, v, g, off, None, None, 64 ** -0.5)["dg"]
    n = max(lens)
    near("dg", dg[late], want[late], (40 * U32 + (2.0 ** -16 if work == "bf16" else 0)) * n ** 0.5)


# ----------------------------------------------------- the caller's stream ---

@pytest.mark.parametrize("call", ["conv", "update"])
def test_entry_points_allocate_on_the_callers_stream(call, monkeypatch):
    """The Python functions hand their stream on to what they allocate."""
    class Stop(Exception):
        pass

    def new(like, shape=None, dtype=None, stream=None):
        raise Stop(stream)

    monkeypatch.setattr(B, "_new", new)
    x = torch.ones(4, 2, 2, 8)
    with pytest.raises(Stop, match="side"):
        if call == "conv":
            gdr.gdr_causal_conv1d(x[0, 0], x[0, 0], None, stream="side")
        else:
            gdr.gdr_fused_recurrent_update(x, x, x, stream="side")


def test_buffers_made_for_a_stream_come_from_its_memory(monkeypatch):
    """The allocator hands a block out again in the order of the stream that freed
    it: what a call on another stream writes has to be allocated on that one.  An
    output is also held for the program's current stream."""
    current, made, held = ["main"], [], []

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    def counted(f):
        def g(*a, **kw):
            made.append(current[0])
            return f(*a, **kw)
        return g

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[0])
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, counted(getattr(torch, name)))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: held.append(s))
    x = torch.ones(4, 6)
    B._scratch(10, x, "side")
    assert made == ["side"]
    for like, shape in ((x, None), (x.t(), None), (x, (3, 2))):
        made.clear(), held.clear()
        assert B._new(like, shape, stream="side").shape == (shape or like.shape)
        assert made == ["side"] and held == ["main"]
    made.clear(), held.clear()
    B._scratch(10, x, None)
    B._new(x)
    assert made == ["main"] * 2 and not held and current == ["main"]


def busy_then_fill(floats, value):
    """A block that the current stream has freed and will yet write, after about a
    millisecond of other work; its address."""
    a = torch.ones(4096, 4096, device="cuda")
    x = torch.empty(floats, device="cuda")
    torch.cuda.synchronize()
    for _ in range(4):
        a = a @ a * 1e-4
    x.fill_(value)
    return x.data_ptr()


@pytest.mark.gpu
def test_calls_on_a_stream_do_not_wait_for_the_current_one():
    """Inputs ready, nothing else ordered between the streams: results are those of
    the current stream, whatever it is still writing into memory it has freed."""
    do, q, k, v, g, off, offs, s0, ds = bwd_inputs(BWD[11])
    y = torch.randn(64, 256, generator=torch.Generator().manual_seed(1)).cuda()
    w = torch.ones(256, device="cuda")
    conv, rows = torch.full((256, 4), 0.25, device="cuda"), torch.tensor([0, 64]).int().cuda()
    u = torch.randn(2, 8, 2, 32, generator=torch.Generator().manual_seed(2)).cuda()
    ug, u0 = -u[..., 0].abs().contiguous(), torch.ones(2, 2, 32, 32, device="cuda")
    beta = ug.sigmoid()
    s = slice(off[0], off[-1])
    calls = {
        "fwd": lambda st: gdr.gdr_linear_attention_fwd(
            q, k, v, g, offs, initial_state=s0, output_final_state=True, stream=st),
        "bwd": lambda st: gdr.gdr_linear_attention_bwd(
            do, q, k, v, g, offs, initial_state=s0, dfinal_state=ds, stream=st),
        "norm": lambda st: gdr.gdr_block_norm(y, residual=y, pre_weight=w, stream=st),
        "norm bwd": lambda st: gdr.gdr_block_norm_bwd(y, y, y, y, pre_weight=w, stream=st),
        "conv": lambda st: (gdr.gdr_causal_conv1d(y, conv, rows, stream=st),),
        "update": lambda st: gdr.gdr_fused_recurrent_update(
            u, u, u, ug, beta, initial_state=u0, output_final_state=True, stream=st),
    }
    inside = lambda t: t[s] if t.shape[0] == q.shape[0] else t  # noqa: E731
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = [inside(t).clone() for t in call(None) if t is not None]
        sizes = {t.numel() * t.element_size() // 4 for t in call(None) if t is not None}
        torch.cuda.synchronize()
        freed = [busy_then_fill(n, float("nan")) for n in sizes]
        got = [t for t in call(side) if t is not None]
        assert not {t.data_ptr() for t in got} & set(freed), name
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, inside(b)), name


# -------------------------------------------------- strides and launch sizes ---

@pytest.mark.parametrize("name,shape", [("q", [2000, 2, 64]), ("k", [2000, 2, 64]),
                                        ("v", [2000, 4, 32])])
def test_forward_refuses_tokens_in_falling_order_of_address(name, shape):
    back = D(shape, stride=[-shape[1] * shape[2], shape[2], 1], data=FAKE * 64)
    assert _call("gdr_linear_attention_fwd", _fwd(**{name: back, "ws": None})) == -2
    assert f"{name} has a negative token stride" in B.gdr_last_error_message()


@pytest.mark.parametrize("name", ["do", "q", "k", "v"])
def test_backward_refuses_tokens_in_falling_order_of_address(name):
    a = dict(do=D([100, 4, 32]), q=D([100, 2, 64]), k=D([100, 2, 64]), v=D([100, 4, 32]),
             g=D([100, 4]), off=D([3], I32), scale=-1.0, s0=None, ds=None,
             dq=D([100, 2, 64], data=FAKE * 2), dk=D([100, 2, 64], data=FAKE * 3),
             dv=D([100, 4, 32], data=FAKE * 4), dg=D([100, 4], data=FAKE * 6), d0=None,
             ws=None, stream=None)
    shape = list(a[name].shape[:3])
    a[name] = D(shape, stride=[-shape[1] * shape[2], shape[2], 1], data=FAKE * 64)
    assert _call("gdr_linear_attention_bwd", list(a.values())) == -2
    assert f"{name} has a negative token stride" in B.gdr_last_error_message()


def refused_as_too_large(fn, args):
    assert _call(fn, args) == -1
    assert "too large for one launch" in B.gdr_last_error_message()


@pytest.mark.parametrize("T,R", [(4, 2 ** 26), (9 * 2 ** 25, 2 ** 25)], ids=["step", "walk"])
def test_forward_refuses_what_one_launch_cannot_hold(T, R):
    """Before the first launch: the short rows' states do not move when the long
    rows cannot be walked."""
    x = D([T, 1, 8])
    refused_as_too_large("gdr_linear_attention_fwd", _fwd(
        o=D([T, 1, 8], data=FAKE * 2), q=x, k=x, v=x, g=None, off=D([R + 1], I32),
        state=D([R, 1, 8, 8]), slot=None, ws=D([2 ** 40])))


def test_step_refuses_what_one_launch_cannot_hold():
    x = D([2 ** 26, 1, 8])
    refused_as_too_large("gdr_linear_attention_step", [
        D([2 ** 26, 1, 8], data=FAKE * 2), x, x, x, None, D([2 ** 26, 1, 8, 8]), None, -1.0, None])


@pytest.mark.parametrize("T,nk,nv,K,R,dg", [
    (2 ** 23, 1, 1, 64, 2 ** 23, False),        # three walks of 256 threads a row
    (2 ** 22, 1, 1, 256, 2 ** 22, True),        # scans: 64 workgroups a state
    (2 ** 30, 1, 2, 16, 1, False),              # sums over heads: a thread for 4 values
], ids=["walks", "scans", "sums"])
def test_backward_refuses_what_one_launch_cannot_hold(T, nk, nv, K, R, dg):
    q, v = D([T, nk, K]), D([T, nv, K])
    refused_as_too_large("gdr_linear_attention_bwd", [
        v, q, q, v, D([T, nv]), D([R + 1], I32), -1.0, None, None, D([T, nk, K], data=FAKE * 2),
        D([T, nk, K], data=FAKE * 3), D([T, nv, K], data=FAKE * 4),
        D([T, nv], data=FAKE * 6) if dg else None, None, D([2 ** 50]), None])


def test_norm_refuses_what_one_launch_cannot_hold():
    x = D([2 ** 26, 64])
    refused_as_too_large("gdr_block_norm", [
        D([2 ** 26, 64], data=FAKE * 2), None, x, None, None, None, None, 0, 1.0, 1e-6, 0, None])


# --------------------------------------------------------- what a test can see ---

@pytest.mark.gpu
def test_gradient_of_a_shared_decay_against_differences():
    """The float64 reference's own central differences (2^-17: cubic terms and
    rounding below 1e-6 of the slope).  The kernel's sum over N tokens is off by
    sqrt(N) times test_backward's bound of the whole at most, below a thousandth."""
    case = ([90, 20], 1, 2, 32, 32, "f32", True, "head")
    do, q, k, v, g, off, offs, s0, ds = bwd_inputs(case)
    s = slice(off[0], off[-1])
    dg = gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs, initial_state=s0, dfinal_state=ds)[3]
    got = dg[s].double().sum(0).cpu()
    do, ds, rates = do.cpu().double()[s], ds.cpu().double(), g[0].cpu().double()

    def loss(rates):
        o, end = ref.attention(q, k, v, rates.expand(q.shape[0], 2), off, s0, 32 ** -0.5)
        return float((o[s] * do).sum() + (end * ds).sum())

    most = 110 ** 0.5 * 40 * 90 ** 0.5 * U32 * float(dg[s].double().norm())
    for h in range(2):
        step = torch.zeros(2, dtype=torch.float64)
        step[h] = 2.0 ** -17
        want = (loss(rates + step) - loss(rates - step)) / 2.0 ** -16
        assert most < 1e-3 * abs(want)
        assert abs(float(got[h]) - want) <= most, (h, float(got[h]), want, most)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[150], [700, 300], [1] * 15 + [700]], ids=["uncut", "cut", "many"])
@pytest.mark.parametrize("initial", [False, True])
def test_float32_states_of_bf16_work_hold_float32(lens, initial):
    """A float32 state takes three bf16 terms of each decayed value, in the segments'
    own sums too.  Its error in the 2-norm: about 200 additions that count (64 tokens
    of a chunk, three terms) as a random walk, 14 u / sqrt(3), the exponents' 4 u and
    the terms' 2^-24: below 2^-20.  Two terms would leave 2^-18.9."""
    q, k, v, g, off, offs, gen = inputs(lens, 2, 4, 64, 64, torch.bfloat16, seed=23)
    s0 = (0.3 * torch.randn((len(lens), 4, 64, 64), generator=gen)).cuda() if initial else None
    _, end = gdr.gdr_linear_attention_fwd(q, k, v, g, offs, initial_state=s0,
                                          output_final_state=True)
    want = ref.attention(q, k, v, g, off, s0, 0.125)[1]
    for r, n in enumerate(lens):
        near(f"state of {n}", end[r], want[r], 2.0 ** -20)


def spread(gen, *xs):
    """Tokens of sizes from a hundredth to a hundred times the others'."""
    for x in xs:
        f = 10 ** (4 * torch.rand(x.shape[0], 1, 1, generator=gen) - 2)
        x *= f.to(x.dtype).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("work", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[180], [600, 3, 70]], ids=["uncut", "cut"])
def test_tokens_of_very_different_sizes(lens, work):
    """Every output and gradient within the elementwise bounds of test_block_ops.py,
    which follow the sizes of the terms."""
    case = (lens, 1, 2, 64, 64, work, True, "token")
    do, q, k, v, g, off, offs, s0, ds = bwd_inputs(case)
    spread(torch.Generator().manual_seed(24), do, q, k, v)
    s, n, sc = slice(off[0], off[-1]), max(lens), 0.4
    o, end = gdr.gdr_linear_attention_fwd(q, k, v, g, offs, initial_state=s0, scale=sc,
                                          output_final_state=True)
    got = gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs, initial_state=s0, dfinal_state=ds,
                                       scale=sc)
    mag = lambda *xs: [x.detach().cpu().double().abs() for x in xs]  # noqa: E731
    want, wend = ref.attention(q, k, v, g, off, s0, sc)
    A, Aend = ref.attention(*mag(q, k, v), g.cpu(), off, *mag(s0), sc)
    f = bounds(DT[work], 64, n) + 2 * U32
    close("o", o[s], want[s], A[s], f)
    close("state", end, wend, Aend, f)
    want = ref.attention_grads(do, q, k, v, g, off, s0, ds, sc)
    A = ref.attention_grads(*mag(do, q, k, v), g.cpu(), off, *mag(s0, ds), sc, sign=1.0)
    for name, x in zip(("dq", "dk", "dv", "dg"), got):
        close(name, x[s], want[name][s], A[name][s], f + (64 * U32 if name == "dg" else 0))
    close("ds0", got[4], want["ds0"], A["ds0"], f)
