"""Selective state space scan, gradients and history folds of the causal Conv1d,
verification of drafted tokens: the references' gradients against differences
and the host's refusals (CPU); the kernels against the references in float64
(GPU).

Error bounds.  u(t) = finfo(t).eps / 2 is what one rounding to t is off at most,
relative to the value; every output may be off by u(its type) |ref| plus what its
float32 arithmetic is off.  A term of an output (C_t, decays, delta_s x_s B_s) that
has passed m tokens carries m products and m additions, each off by u(float32),
and m exponentials of 2 u (an ulp of the instruction), its step size's softplus (an
exponential, a reciprocal, seven products and sums: 10 u) in the factor and in the
exponents.  An exponent E is off by 12 u E; beyond E = 30 a term is below 1e-13 of
what entered, so that 12 u 30 covers it.  A gradient's term passes the states' and
the gradient's recurrence: twice the tokens' share.  Gates add a sigmoid (an
exponential, a reciprocal, a sum: 6 u) and products.  Sums over N, over channels and
over tokens add their lengths.  Together, for rows of n tokens, below
(4 n + 500) u A forward and (8 n + N + channels of a group + 600) u A backward, A the
sum of the terms' absolute values (sums over segments and runs are float64)."""
import os
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_loop_amd as gdr
from gated_delta_rule_loop_amd import _binding as B
from tests import scan_ref as ref
from tests.test_block_ops import BF16, D, DT, F32, FAKE, I32, U32, U32T, _call, close, near, u

CU = "cuda"


# ----------------------------------------------------------- the references ---

def _draws(seed):
    gen = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)


def _slopes(loss, x, got, names, draw):
    """Central differences along random directions."""
    for name, grad in names:
        d, e = draw(*x[name].shape), 1e-5
        up, down = loss({**x, name: x[name] + e * d}), loss({**x, name: x[name] - e * d})
        # cubic terms of size e^2 and rounding of size 2^-52 / e: both below 1e-8
        assert abs((up - down) / (2 * e) - float((got[grad] * d).sum())) < 1e-7, name


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("soft", [True, False])
def test_scan_reference_gradients_match_differences(gate, soft):
    r = _draws(1)
    off, Dn, N, G = [0, 0, 5, 6], 4, 3, 2
    x = dict(x=r(6, Dn), dt=0.3 * r(6, Dn), A=-r(Dn, N).abs(), B=r(6, G, N), C=r(6, G, N),
             D=r(Dn), bias=0.2 * r(Dn), h0=r(3, Dn, N))
    if gate:
        x["z"] = r(6, Dn)
    do, dh = r(6, Dn), r(3, Dn, N)
    args = lambda x: dict(D=x["D"], z=x.get("z"), bias=x["bias"], soft=soft, h0=x["h0"])  # noqa: E731

    def loss(x):
        out, end = ref.scan(x["x"], x["dt"], x["A"], x["B"], x["C"], off, **args(x))
        return float((out * do).sum() + (end * dh).sum())

    got = ref.scan_grads(do, x["x"], x["dt"], x["A"], x["B"], x["C"], off, dh=dh, **args(x))
    names = [("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"),
             ("bias", "dbias"), ("h0", "dh0")] + ([("z", "dz")] if gate else [])
    _slopes(loss, x, got, names, r)


@pytest.mark.parametrize("silu", [True, False])
def test_conv_reference_gradients_match_differences(silu):
    r = _draws(2)
    off = [0, 1, 1, 7]
    x = dict(x=r(7, 3), w=r(3, 3), b=r(3))
    do = r(7, 3)
    got = dict(zip(("dx", "dw", "db"), ref.conv_grads(do, x["x"], x["w"], off, x["b"], silu)))
    _slopes(lambda x: float((ref.conv(x["x"], x["w"], off, x["b"], silu) * do).sum()), x, got,
            [("x", "dx"), ("w", "dw"), ("b", "db")], r)


# ---------------------------------------------------------------- refusals ---

def _scan_args(**over):
    T, Dn, N, G, R = 200, 64, 16, 2, 3
    a = dict(out=D([T, Dn], data=FAKE * 2), x=D([T, Dn]), dt=D([T, Dn]), A=D([Dn, N]),
             B=D([T, G, N]), C=D([T, G, N]), skip=D([Dn]), z=D([T, Dn]), bias=D([Dn]),
             off=D([R + 1], I32), s0=None, end=None, state=D([5, Dn, N]), slot=D([R], I32), flags=32,
             ws=D([10 ** 7]), stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code,word", [
    (dict(out=None), -1, "out is null"),
    (dict(x=D([200, 64], U32T)), -2, "dtype"),
    (dict(x=D([200, 60]), dt=D([200, 60])), -2, "multiple of 4"),
    (dict(x=D([200, 63])), -1, "multiple of B's groups"),
    (dict(B=D([200, 0, 16])), -1, "multiple of B's groups"),
    (dict(B=D([200, 2, 12])), -2, "state size 12"),
    (dict(B=D([200, 2, 128])), -2, "state size 128"),
    (dict(dt=D([200, 64], BF16)), -2, "work dtype"),
    (dict(dt=D([199, 64])), -1, "dt dim 0"),
    (dict(A=D([64, 16], BF16)), -2, "dtype"),
    (dict(A=D([64, 8])), -1, "A dim 1"),
    (dict(A=D([64, 16], stride=[32, 1])), -2, "contiguous"),
    (dict(A=D([64, 16], data=FAKE + 4)), -2, "aligned"),
    (dict(C=D([200, 1, 16])), -1, "C dim 1"),
    (dict(C=D([200, 2, 16], stride=[34, 16, 1])), -2, "multiple of 4"),
    (dict(skip=D([64], BF16)), -2, "dtype"),
    (dict(skip=D([64], stride=[2])), -2, "contiguous"),
    (dict(bias=D([63])), -1, "dt_bias dim 0"),
    (dict(z=D([200, 64], stride=[130, 1])), -2, "multiple of 4"),
    (dict(x=D([200, 64], data=FAKE + 8)), -2, "aligned"),
    (dict(x=D([200, 64], stride=[128, 2])), -2, "innermost"),
    (dict(x=D([200, 64], data=FAKE * 64, stride=[-64, 1])), -2, "x has a token stride"),
    (dict(C=D([200, 2, 16], stride=[2 ** 24, 16, 1])), -2, "C has a token stride"),
    (dict(out=D([200, 64], data=FAKE * 2, stride=[32, 1])), -1, "overlap"),
    (dict(out=D([200, 64])), -1, "alias"),
    (dict(off=D([0], I32)), -1, "empty"),
    (dict(off=D([4], F32)), -2, "dtype"),
    (dict(state=D([5, 64, 8])), -1, "state dim 2"),
    (dict(state=D([5, 64, 16], stride=[2048, 32, 1])), -2, "dense"),
    (dict(state=D([5, 64, 16], stride=[0, 16, 1])), -1, "overlap"),
    (dict(state=D([2, 64, 16]), slot=None), -1, "fewer slots"),
    (dict(slot=D([4], I32)), -1, "slot_idx dim 0"),
    (dict(state=None), -1, "slot_idx needs state"),
    (dict(s0=D([3, 64, 16])), -1, "give state, or"),
    (dict(state=None, slot=None, s0=D([2, 64, 16])), -1, "initial_state dim 0"),
    (dict(state=None, slot=None, s0=D([3, 64, 16]), end=D([3, 64, 16], BF16)), -2, "final_state must"),
    (dict(state=None, slot=None, s0=D([3, 64, 16]), end=D([3, 64, 16])), -1, "alias"),
    (dict(state=None, slot=None, flags=16), -1, "KEEP_STATE needs state"),
    (dict(flags=64), -1, "unknown flags"),
    (dict(ws=None), -1, "workspace is null"),
    (dict(ws=D([64])), -1, "needed"),
    (dict(ws=D([10 ** 7], BF16)), -1, "float32"),
    (dict(ws=D([10 ** 7], data=FAKE + 4)), -2, "aligned"),
])
def test_forward_refuses(over, code, word):
    over = {"x": D([2 ** 12, 64]), "dt": D([2 ** 12, 64]), "out": D([2 ** 12, 64], data=FAKE * 2),
            "B": D([2 ** 12, 2, 16]), "C": D([2 ** 12, 2, 16]), "z": D([2 ** 12, 64]),
            **over} if "ws" in over else over
    assert _call("gdr_selective_scan_fwd", _scan_args(**over)) == code
    assert word in B.gdr_last_error_message()


def test_forward_refuses_what_one_launch_cannot_hold():
    for T, R in ((2 ** 30, 2 ** 26), (2 ** 26, 2 ** 26)):
        rows = lambda at: D([T, 64], data=at)  # noqa: E731
        a = _scan_args(out=rows(FAKE * 2), x=rows(FAKE), dt=rows(FAKE), z=None, B=D([T, 1, 16]),
                       C=D([T, 1, 16]), off=D([R + 1], I32), state=D([R, 64, 16]), slot=None,
                       ws=D([2 ** 50]))
        assert _call("gdr_selective_scan_fwd", a) == -1
        assert "too large for one launch" in B.gdr_last_error_message()


@pytest.mark.parametrize("over,code,word", [
    (dict(state=None), -1, "state is null"),
    (dict(state=D([3, 64, 16]), slot=None), -1, "fewer slots"),
    (dict(slot=D([5], I32)), -1, "slot_idx dim 0"),
    (dict(flags=16), -1, "unknown flags"),
    (dict(out=D([4, 64])), -1, "alias"),
])
def test_step_refuses(over, code, word):
    T, Dn, N = 4, 64, 16
    a = dict(out=D([T, Dn], data=FAKE * 2), x=D([T, Dn]), dt=D([T, Dn]), A=D([Dn, N]),
             B=D([T, 1, N]), C=D([T, 1, N]), skip=None, z=None, bias=None, state=D([9, Dn, N]),
             slot=D([T], I32), flags=32, stream=None)
    a.update(over)
    assert _call("gdr_selective_scan_step", list(a.values())) == code
    assert word in B.gdr_last_error_message()


@pytest.mark.parametrize("over,code,word", [
    (dict(state=None), -1, "state is null"),
    (dict(acc=None), -1, "accepted is null"),
    (dict(acc=D([4], I32)), -1, "accepted dim 0"),
    (dict(acc=D([3], F32)), -2, "dtype"),
    (dict(flags=16), -1, "unknown flags"),
])
def test_fold_refuses(over, code, word):
    T, Dn, N, R = 20, 64, 16, 3
    a = dict(state=D([9, Dn, N]), x=D([T, Dn]), dt=D([T, Dn]), A=D([Dn, N]), B=D([T, 1, N]),
             bias=None, off=D([R + 1], I32), acc=D([R], I32), slot=D([R], I32), flags=32, stream=None)
    a.update(over)
    assert _call("gdr_selective_scan_fold", list(a.values())) == code
    assert word in B.gdr_last_error_message()


def _bwd_args(**over):
    T, Dn, N, R = 200, 64, 16, 3
    o = lambda k, *s: D(list(s), data=FAKE * k)  # noqa: E731
    a = dict(do=D([T, Dn]), x=D([T, Dn]), dt=D([T, Dn]), A=D([Dn, N]), B=D([T, 2, N]),
             C=D([T, 2, N]), skip=D([Dn]), z=D([T, Dn]), bias=D([Dn]), off=D([R + 1], I32), h0=None,
             dh=None, dx=o(2, T, Dn), ddt=o(3, T, Dn), dA=o(4, Dn, N), dB=o(5, T, 2, N),
             dC=o(6, T, 2, N), dD=o(7, Dn), dz=o(8, T, Dn), dbias=o(9, Dn), d0=None, flags=32,
             ws=D([10 ** 8]), stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code,word", [
    (dict(do=D([200, 64], BF16)), -2, "work dtype"),
    (dict(dz=None), -1, "dz is given exactly"),
    (dict(z=None), -1, "dz is given exactly"),
    (dict(dD=None), -1, "dD is given exactly"),
    (dict(bias=None), -1, "ddt_bias is given exactly"),
    (dict(dA=None), -1, "dA is null"),
    (dict(dA=D([64, 16], BF16, data=FAKE * 4)), -2, "dtype"),
    (dict(dB=D([200, 1, 16], data=FAKE * 5)), -1, "dB dim 1"),
    (dict(dx=D([200, 64])), -1, "alias"),
    (dict(ddt=D([200, 64], data=FAKE * 2)), -1, "share memory"),
    (dict(dC=D([200, 2, 16], data=FAKE * 5)), -1, "share memory"),
    (dict(dx=D([200, 64], data=FAKE * 2, stride=[0, 1])), -1, "overlap"),
    (dict(h0=D([2, 64, 16])), -1, "initial_state dim 0"),
    (dict(dh=D([3, 64, 16], I32)), -2, "dtype"),
    (dict(d0=D([3, 64, 8], data=FAKE * 11)), -1, "dinitial_state dim 2"),
    (dict(flags=16), -1, "unknown flags"),
    (dict(ws=None), -1, "workspace is null"),
    (dict(ws=D([100])), -1, "needed"),
])
def test_backward_refuses(over, code, word):
    assert _call("gdr_selective_scan_bwd", _bwd_args(**over)) == code
    assert word in B.gdr_last_error_message()


@pytest.mark.parametrize("over,code,word", [
    (dict(x=D([20, 62]), do=D([20, 62])), -2, "multiple of 4"),
    (dict(do=D([20, 64], BF16)), -2, "work dtype"),
    (dict(w=D([64, 5])), -2, "width 5"),
    (dict(dw=D([64, 3], data=FAKE * 3)), -1, "dweight dim 1"),
    (dict(dw=D([64, 4], data=FAKE * 3, stride=[2, 1])), -1, "overlap"),
    (dict(w=D([64, 4], stride=[1, 64])), -2, "unit stride"),
    (dict(dx=D([20, 64])), -1, "alias"),
    (dict(dw=D([64, 4])), -1, "alias"),
    (dict(b=None), -1, "dbias needs bias"),
    (dict(flags=16), -1, "unknown flags"),
    (dict(ws=None), -1, "workspace is null"),
])
def test_conv_backward_refuses(over, code, word):
    a = dict(do=D([20, 64]), x=D([20, 64]), w=D([64, 4]), b=D([64]), off=D([4], I32),
             dx=D([20, 64], data=FAKE * 2), dw=D([64, 4], data=FAKE * 3), db=D([64], data=FAKE * 4),
             flags=2, ws=D([10 ** 6]), stream=None)
    a.update(over)
    assert _call("gdr_causal_conv1d_bwd", list(a.values())) == code
    assert word in B.gdr_last_error_message()


@pytest.mark.parametrize("over,code,word", [
    (dict(st=D([5, 4, 64])), -2, "history of 4"),
    (dict(st=D([5, 3, 64], BF16)), -2, "work dtype"),
    (dict(st=D([5, 3, 64], stride=[0, 64, 1])), -1, "overlap"),
    (dict(st=D([2, 3, 64]), slot=None), -1, "fewer slots"),
    (dict(acc=None), -1, "accepted is null"),
    (dict(x=D([20, 62])), -2, "multiple of 4"),
])
def test_conv_fold_refuses(over, code, word):
    a = dict(st=D([5, 3, 64]), x=D([20, 64]), off=D([4], I32), acc=D([3], I32), slot=D([3], I32),
             stream=None)
    a.update(over)
    assert _call("gdr_causal_conv1d_fold", list(a.values())) == code
    assert word in B.gdr_last_error_message()


@pytest.mark.parametrize("over,code,word", [
    (dict(target=D([20, 0])), -1, "vocabulary"),
    (dict(target=D([20, 100], I32)), -2, "dtype"),
    (dict(target=D([20, 100], stride=[200, 2])), -2, "innermost"),
    (dict(draft=D([20, 100], BF16)), -2, "work dtype"),
    (dict(draft=D([20, 99])), -1, "draft dim 1"),
    (dict(draft=D([20, 100], stride=[200, 2])), -2, "innermost"),
    (dict(u=None), -1, "draft needs uniform"),
    (dict(u=D([19])), -1, "uniform dim 0"),
    (dict(tokens=D([20], F32)), -2, "dtype"),
    (dict(tokens=D([19], I32)), -1, "tokens dim 0"),
    (dict(acc=D([4], I32, data=FAKE * 2)), -1, "accepted dim 0"),
    (dict(nxt=D([3], I32, data=FAKE * 2)), -1, "alias"),
    (dict(ws=None), -1, "workspace is null"),
    (dict(ws=D([10 ** 5], data=FAKE + 8)), -2, "aligned"),
])
def test_verify_refuses(over, code, word):
    a = dict(acc=D([3], I32, data=FAKE * 2), nxt=D([3], I32, data=FAKE * 3), tokens=D([20], I32),
             target=D([20, 100]), draft=D([20, 100]), u=D([20]), off=D([4], I32), ws=D([10 ** 5]),
             stream=None)
    a.update(over)
    assert _call("gdr_verify_drafts", list(a.values())) == code
    assert word in B.gdr_last_error_message()


def test_workspace_sizes():
    L = B.lib()
    assert L.gdr_selective_scan_workspace(1, 1, 4096, 16, 1, 0) == 0
    assert L.gdr_selective_scan_workspace(0, 0, 4096, 16, 1, 0) == 0
    assert L.gdr_selective_scan_workspace(-1, 1, 4096, 16, 1, 0) == -1
    assert L.gdr_selective_scan_workspace(10, 1, 4096, 16, 3, 1) == -1
    assert L.gdr_causal_conv1d_workspace(-1, 4, 4) == -1
    assert L.gdr_verify_drafts_workspace(4, 1, 0) == -1


# --------------------------------------------------------------- the kernels ---

def offsets_of(lens, lead=0):
    off = [lead]
    for n in lens:
        off.append(off[-1] + n)
    return off, torch.tensor(off, dtype=torch.int32, device=CU)


def inputs(lens, Dn, N, G, work, *, z=True, skip=True, bias=True, seed=0, lead=0, tail=0,
           packed=True, step=(1e-3, 0.1)):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    off, offs = offsets_of(lens, lead)
    T = off[-1] + tail
    dt = DT[work]
    if packed and z:  # halves of a projection's output, of another's columns
        xz = r(T, 2 * Dn).to(dt).to(CU)
        x, zz = xz[:, :Dn], xz[:, Dn:]
    else:
        x, zz = r(T, Dn).to(dt).to(CU), (r(T, Dn).to(dt).to(CU) if z else None)
    cols = 2 * G * N + (24 if packed else 0)
    bc = r(T, cols).to(dt).to(CU)
    s = torch.exp(torch.rand(Dn, generator=gen) * (torch.log(torch.tensor(step[1] / step[0]))) +
                  torch.log(torch.tensor(step[0])))
    return dict(x=x, dt=(0.5 * r(T, Dn)).to(dt).to(CU),
                A=(-torch.arange(1, N + 1) * torch.exp(0.1 * r(Dn, N))).contiguous().to(CU),
                B=bc[:, cols - 2 * G * N:cols - G * N].unflatten(1, (G, N)),
                C=bc[:, cols - G * N:].unflatten(1, (G, N)),
                D=(1 + 0.1 * r(Dn)).to(CU) if skip else None, z=zz,
                bias=(s + torch.log(-torch.expm1(-s))).to(CU) if bias else None), off, offs, r


def kernel_args(a):
    return dict(D=a["D"], z=a["z"], dt_bias=a["bias"])


def ref_args(a):
    return dict(D=a["D"], z=a["z"], bias=a["bias"])


OPS = ("x", "dt", "A", "B", "C")


def forward_bound(lens):
    return (4 * max(lens, default=0) + 500) * U32


def check_forward(a, off, out, end, soft, h0, got_rows=None):
    want, last = ref.scan(*(a[k] for k in OPS), off, soft=soft, h0=h0, **ref_args(a))
    A, Aend = ref.scan(*(a[k] for k in OPS), off, soft=soft, h0=h0, absolute=True, **ref_args(a))
    f = forward_bound([b - c for b, c in zip(off[1:], off)])
    rows = slice(off[0], off[-1])
    close("out", out[rows], want[rows], A[rows], f)
    if end is not None:
        close("state", end, last, Aend, f)
    return want, last


FWD = [  # rows, channels, states, groups, work, states' type
    ([1], 8, 8, 1, "f32", "f32"),
    ([3], 64, 16, 1, "bf16", "bf16"),
    ([16, 17, 0, 1], 72, 16, 1, "f32", "f32"),
    ([64], 136, 16, 1, "bf16", "f32"),
    ([65], 136, 16, 1, "bf16", "f32"),
    ([200, 1, 0, 130, 64], 80, 16, 2, "f32", "bf16"),
    ([333], 40, 8, 1, "bf16", "bf16"),
    ([129, 64, 300], 48, 32, 2, "bf16", "f32"),
    ([70, 5], 24, 64, 1, "f32", "f32"),
    ([30, 20], 16, 64, 2, "bf16", "bf16"),
    ([1] * 9 + [150, 0, 16, 17], 32, 16, 4, "f32", "f32"),   # both walks in one call
    ([700], 4096, 16, 1, "bf16", "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("soft", [True, False])
@pytest.mark.parametrize("case", FWD, ids=str)
def test_forward(case, soft):
    """On a pool (one row of more than four is padding), tokens before and behind the
    rows, projections' columns in place."""
    lens, Dn, N, G, work, st = case
    a, off, offs, r = inputs(lens, Dn, N, G, work, lead=1, tail=2, bias=soft)
    if not soft:  # step sizes as they come, positive
        a["dt"] = (a["dt"].abs() * 0.1 + 1e-3).to(a["dt"].dtype)
    rows = len(lens)
    pool = (0.3 * r(rows + 3, Dn, N)).to(DT[st]).to(CU)
    slots = torch.randperm(rows + 3, generator=torch.Generator().manual_seed(5))[:rows].int()
    pad = rows > 4
    if pad:
        slots[1] = -1
    before, h0 = pool.clone(), pool.cpu()[slots.long()]
    out = torch.full(a["x"].shape, 7.0, dtype=a["x"].dtype, device=CU)
    floats = gdr.gdr_selective_scan_workspace(out.shape[0], rows, Dn, N, G)
    got, end = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=soft, state=pool,
                                          slot_idx=slots.to(CU), out=out,
                                          workspace=torch.full((max(1, floats),), float("nan"),
                                                               device=CU), **kernel_args(a))
    assert got is out and end is pool
    want, last = ref.scan(*(a[k] for k in OPS), off, soft=soft, h0=h0, **ref_args(a))
    A, Aend = ref.scan(*(a[k] for k in OPS), off, soft=soft, h0=h0, absolute=True, **ref_args(a))
    keep = torch.ones(out.shape[0], dtype=torch.bool)
    keep[:off[0]] = keep[off[-1]:] = False
    assert (out.cpu()[~keep] == 7).all()
    live = torch.tensor([i for i, n in enumerate(lens) if n and not (pad and i == 1)])
    if pad:
        assert (out[off[1]:off[2]] == 0).all()
        keep[off[1]:off[2]] = False
    f = forward_bound(lens)
    close("out", out.cpu()[keep], want[keep], A[keep], f)
    close("state", pool.cpu()[slots[live].long()], last[live], Aend[live], f)
    same = torch.ones(rows + 3, dtype=torch.bool)
    same[slots[live].long()] = False
    assert torch.equal(pool.cpu()[same], before.cpu()[same])


WALKS = [  # rows, channels, states, groups, work, states' type
    ([600], 40, 16, 1, "f32", "f32"), ([530, 0, 90, 17, 16, 1], 72, 16, 2, "bf16", "bf16"),
    ([600], 24, 32, 1, "bf16", "f32"), ([33, 0, 570, 5], 24, 32, 2, "f32", "bf16"),
    ([600], 24, 64, 1, "bf16", "f32"), ([580, 64, 0, 1], 40, 64, 2, "f32", "f32"),
    ([65], 4, 16, 1, "f32", "f32"), ([79, 0, 1, 80, 15, 16], 24, 16, 6, "bf16", "bf16"),
    ([81], 12, 32, 1, "f32", "f32"), ([31, 0, 48, 1, 2, 0], 40, 32, 1, "bf16", "bf16"),
    ([66], 12, 64, 1, "f32", "bf16"), ([70, 3, 0, 17, 1], 24, 64, 1, "bf16", "f32"),
    ([17, 1, 0, 33, 16, 18, 49, 2, 5, 64], 536, 16, 1, "f32", "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", WALKS, ids=str)
def test_forward_of_every_walk(case):
    """Calls on either side of the rule between the lane walk and segments, blocks of
    16 tokens that end early, channels that end inside a wave and a workgroup."""
    test_forward(case, True)


MIXED = [  # single tokens and short rows beside cut ones: rows, channels, states, groups, work, states
    ([1] * 250 + [40, 80], 4096, 16, 1, "bf16", "f32"),
    ([80] + [1] * 250 + [40], 4096, 16, 1, "f32", "bf16"),
    ([1] * 511 + [48, 200], 2048, 16, 2, "bf16", "bf16"),
    ([1] * 300 + [40, 80], 64, 8, 1, "f32", "f32"),
    ([1] * 400 + [80, 0] + [1] * 150 + [17, 64, 90], 40, 8, 1, "f32", "f32"),
    ([1] * 260 + [100, 63, 33] + [1] * 360 + [65, 20], 72, 8, 3, "f32", "bf16"),
    ([1] * 300 + [40, 70, 33], 2048, 64, 1, "bf16", "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", MIXED, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1]}-{c[2]}")
def test_forward_of_short_rows_beside_cut_ones(case):
    """Rows longer than a segment that the narrow walk takes have no segment of their
    own: before, between and behind rows that have some, those start from their own
    states."""
    test_forward(case, True)


@pytest.mark.gpu
def test_mixed_batch_on_dense_states():
    """The same beside rows without tokens, which hand on their state; a cut row's
    outputs have the bits that the rows beside it leave in a call of other values."""
    lens = [1] * 150 + [0, 40, 0, 80] + [1] * 500 + [64, 130, 0, 17]
    a, off, offs, r = inputs(lens, 64, 8, 1, "f32", packed=False)
    h0 = (0.3 * r(len(lens), 64, 8)).to(CU)
    call = lambda: gdr.gdr_selective_scan_fwd(  # noqa: E731
        *(a[k] for k in OPS), offs, softplus=True, initial_state=h0, output_final_state=True,
        **kernel_args(a))
    out, end = call()
    check_forward(a, off, out, end, True, h0)
    a["x"][off[151]:off[152]] *= 100  # the row of 40, before the one of 80
    other, _ = call()
    rows = torch.ones(off[-1], dtype=torch.bool, device=CU)
    rows[off[151]:off[152]] = False
    assert torch.equal(out[rows], other[rows])
    assert not torch.equal(out[~rows], other[~rows])


@pytest.mark.gpu
@pytest.mark.parametrize("N", [8, 16, 64])
@pytest.mark.parametrize("lens", [[1], [13], [70], [90, 7], [700, 1]], ids=str)
def test_decays_of_minus_infinity_forget(lens, N):
    """exp(delta A) is 0 there, also in the last tokens of a row; delta is positive."""
    a, off, offs, r = inputs(lens, 24, N, 1, "f32")
    a["A"][:, 0] = float("-inf")
    a["A"][5] = float("-inf")
    h0 = (0.3 * r(len(lens), 24, N)).to(CU)
    out, end = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=True,
                                          initial_state=h0, output_final_state=True,
                                          **kernel_args(a))
    check_forward(a, off, out, end, True, h0)


@pytest.mark.gpu
@pytest.mark.parametrize("work", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[5, 0, 9], [100, 0, 3], [0, 0], [0, 500, 0]], ids=str)
@pytest.mark.parametrize("initial", [True, False])
def test_forward_with_dense_states(lens, work, initial):
    """Rows without tokens hand on their state."""
    a, off, offs, r = inputs(lens, 40, 16, 1, work, packed=False)
    h0 = (0.3 * r(len(lens), 40, 16)).to(CU) if initial else None
    out, end = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=True,
                                          initial_state=h0, output_final_state=True,
                                          **kernel_args(a))
    check_forward(a, off, out, end, True, h0)


@pytest.mark.gpu
def test_forward_without_gate_skip_and_bias():
    for lens in ([7], [90, 41]):
        a, off, offs, _ = inputs(lens, 24, 8, 1, "f32", z=False, skip=False, bias=False)
        out, none = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=True)
        assert none is None
        check_forward(a, off, out, None, True, None)


STEP = [
    (1, 64, 16, 1, "bf16", "f32", 0), (5, 4096, 16, 1, "bf16", "bf16", 1),
    (19, 136, 16, 2, "f32", "f32", 3), (3, 24, 8, 1, "f32", "bf16", 0),
    (7, 40, 32, 1, "bf16", "f32", 1), (4, 72, 64, 1, "f32", "f32", 0),
    (4, 16, 64, 2, "bf16", "bf16", 1), (2, 8, 8, 1, "bf16", "f32", 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", STEP, ids=str)
def test_step(case):
    rows, Dn, N, G, work, st, pad = case
    a, off, offs, r = inputs([1] * rows, Dn, N, G, work, seed=3)
    pool = (0.3 * r(rows + 4, Dn, N)).to(DT[st]).to(CU)
    slots = torch.randperm(rows + 4, generator=torch.Generator().manual_seed(6))[:rows].int()
    slots[rows - pad:] = -1
    before, h0 = pool.clone(), pool.cpu()[slots.long().clamp_min(0)]
    out = gdr.gdr_selective_scan_step(*(a[k] for k in OPS), pool, slots.to(CU), softplus=True,
                                      **kernel_args(a))
    want, last = ref.scan(*(a[k] for k in OPS), off, soft=True, h0=h0, **ref_args(a))
    A, Aend = ref.scan(*(a[k] for k in OPS), off, soft=True, h0=h0, absolute=True, **ref_args(a))
    n, f = rows - pad, forward_bound([1])
    close("out", out[:n], want[:n], A[:n], f)
    assert (out[n:] == 0).all()
    close("state", pool.cpu()[slots[:n].long()], last[:n], Aend[:n], f)
    same = torch.ones(rows + 4, dtype=torch.bool)
    same[slots[:n].long()] = False
    assert torch.equal(pool.cpu()[same], before.cpu()[same])
    # a forward over one-token rows gives the same bits
    again = before.clone()
    fwd, _ = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=True, state=again,
                                        slot_idx=slots.to(CU), **kernel_args(a))
    assert torch.equal(fwd, out) and torch.equal(again, pool)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[12], [20, 7, 0, 64], [3, 70, 200]], ids=str)
@pytest.mark.parametrize("work,st", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_window_then_fold(lens, work, st):
    """A window that keeps the states, then a fold over a prefix of every row: the
    outputs are the forward's, the states those of a forward over the prefix."""
    a, off, offs, r = inputs(lens, 72, 16, 1, work, seed=8)
    rows = len(lens)
    pool = (0.3 * r(rows + 1, 72, 16)).to(DT[st]).to(CU)
    slots = torch.arange(rows, 0, -1, dtype=torch.int32, device=CU)
    before = pool.clone()
    kw = dict(softplus=True, slot_idx=slots, **kernel_args(a))
    out, _ = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, state=pool, keep_state=True, **kw)
    assert torch.equal(pool, before)
    moved = before.clone()
    full, _ = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, state=moved, **kw)
    assert torch.equal(out, full)
    for share in (0.0, 0.4, 1.0, 2.0):
        n = [min(k + 1, int(k * share)) for k in lens]  # the last: above the row's length
        acc = torch.tensor(n, dtype=torch.int32, device=CU)
        folded = gdr.gdr_selective_scan_fold(before.clone(), a["x"], a["dt"], a["A"], a["B"], offs,
                                             acc, slots, dt_bias=a["bias"], softplus=True)
        cut = [k if k <= m else 0 for k, m in zip(n, lens)]
        keep = torch.cat([torch.arange(o, o + k) for o, k in zip(off, cut)]).to(CU)
        short = {k: (v if k in ("A", "D", "bias") or v is None else v[keep].contiguous())
                 for k, v in a.items()}
        _, offs2 = offsets_of(cut)
        want = before.clone()
        gdr.gdr_selective_scan_fwd(*(short[k] for k in OPS), offs2, state=want, slot_idx=slots,
                                   softplus=True, **kernel_args(short))
        if sum(cut) <= 64:  # token by token in one piece: the same bits
            assert torch.equal(folded, want)
        else:
            h0 = before.cpu()[slots.cpu().long()]
            o2 = [0]
            for k in cut:
                o2.append(o2[-1] + k)
            kw2 = dict(soft=True, h0=h0, **ref_args(short))
            _, last = ref.scan(*(short[k] for k in OPS), o2, **kw2)
            _, Aend = ref.scan(*(short[k] for k in OPS), o2, absolute=True, **kw2)
            close("state", folded[slots.long()], last, Aend, forward_bound(cut))


@pytest.mark.gpu
@pytest.mark.parametrize("Dn,N,work,st", [
    (2048, 16, "bf16", "bf16"), (2048, 8, "f32", "f32"), (40, 16, "f32", "f32"),
    (40, 8, "bf16", "f32"), (24, 64, "bf16", "bf16"), (2048, 32, "bf16", "f32"),
], ids=str)
def test_folds_leave_the_bits_of_every_walk(Dn, N, work, st):
    """70 windows of up to 16 tokens, enough rows to fill the chip and few channels: a fold
    of whole rows leaves what the forward leaves, bit for bit."""
    lens = [1 + 5 * i % 16 for i in range(68)] + [0, 16]
    a, off, offs, r = inputs(lens, Dn, N, 1, work, seed=12)
    pool = (0.3 * r(len(lens), Dn, N)).to(DT[st]).to(CU)
    moved, kept = pool.clone(), pool.clone()
    out, _ = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, state=moved, softplus=True,
                                        **kernel_args(a))
    again, _ = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, state=kept, softplus=True,
                                          keep_state=True, **kernel_args(a))
    assert torch.equal(kept, pool) and torch.equal(again, out)
    acc = torch.tensor(lens, dtype=torch.int32, device=CU)
    folded = gdr.gdr_selective_scan_fold(pool.clone(), a["x"], a["dt"], a["A"], a["B"], offs, acc,
                                         dt_bias=a["bias"], softplus=True)
    assert torch.equal(folded, moved)
    check_forward(a, off, out, moved if st == "f32" else None, True, pool)


@pytest.mark.gpu
def test_prompt_then_tokens_continue_one_row():
    a, off, offs, r = inputs([300], 136, 16, 1, "f32")
    want, _ = ref.scan(*(a[k] for k in OPS), off, soft=True, **ref_args(a))
    A, _ = ref.scan(*(a[k] for k in OPS), off, soft=True, absolute=True, **ref_args(a))
    state = torch.zeros(1, 136, 16, device=CU)
    part = lambda i, j: {k: (v if k in ("A", "D", "bias") else v[i:j]) for k, v in a.items()}  # noqa: E731
    first = part(0, 290)
    out = [gdr.gdr_selective_scan_fwd(*(first[k] for k in OPS), offsets_of([290])[1], state=state,
                                      softplus=True, **kernel_args(first))[0]]
    for t in range(290, 300):
        tok = part(t, t + 1)
        out.append(gdr.gdr_selective_scan_step(*(tok[k] for k in OPS), state, softplus=True,
                                               **kernel_args(tok)))
    close("out", torch.cat(out), want, A, forward_bound([300]))


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[10, 20, 12], [100, 300, 70]], ids=str)
def test_rows_do_not_touch_their_neighbours(lens):
    a, off, offs, _ = inputs(lens, 40, 16, 1, "f32")
    clean, _ = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=True, **kernel_args(a))
    for k in ("x", "dt", "B", "C", "z"):
        a[k][off[1]:off[2]] = float("nan")
    out, _ = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=True, **kernel_args(a))
    assert torch.equal(out[:off[1]], clean[:off[1]]) and torch.equal(out[off[2]:], clean[off[2]:])
    assert torch.isnan(out[off[1]:off[2]]).all()


@pytest.mark.gpu
def test_large_and_small_steps():
    """Steps that forget everything at once and steps of almost nothing; a row's
    softplus at both ends of its range."""
    a, off, offs, _ = inputs([90], 64, 16, 1, "f32", bias=False)
    a["dt"] = torch.linspace(-60, 60, 90 * 64, device=CU).reshape(90, 64)
    out, end = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=True,
                                          output_final_state=True, **kernel_args(a))
    check_forward(a, off, out, end, True, None)


def wide_sweep(*shape, seed=0, least=-1e30):
    """-200 to 200, half of it within -130 to -85, where e^-x passes float32's
    largest value, in any order."""
    n = 1
    for s in shape:
        n *= s
    v = torch.cat([torch.linspace(-200, 200, n - n // 2), torch.linspace(-130, -85, n // 2)])
    v = v[torch.randperm(n, generator=torch.Generator().manual_seed(seed))]
    v[3] = least
    return v.reshape(shape)


# A sigmoid below 2^-126 is 0 in the kernels: an output is off by |z| 2^-126 times a
# number of ordinary size, below the 1e-30 that close() lets through.
@pytest.mark.gpu
@pytest.mark.parametrize("work", ["f32", "bf16"])
@pytest.mark.parametrize("lens,N", [([60], 8), ([50, 0, 43], 16), ([90], 64), ([90, 30], 8)], ids=str)
def test_gates_of_every_size(lens, N, work):
    """Narrow, lane and wide walk."""
    a, off, offs, _ = inputs(lens, 64, N, 1, work, packed=False)
    a["z"] = wide_sweep(off[-1], 64).to(DT[work]).to(CU)
    out, end = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=True,
                                          output_final_state=True, **kernel_args(a))
    check_forward(a, off, out, end, True, None)


@pytest.mark.gpu
@pytest.mark.parametrize("work", ["f32", "bf16"])
def test_step_gates_of_every_size(work):
    a, off, offs, r = inputs([1] * 60, 64, 16, 1, work, packed=False)
    a["z"] = wide_sweep(60, 64).to(DT[work]).to(CU)
    pool = (0.3 * r(60, 64, 16)).to(CU)
    h0 = pool.clone()
    out = gdr.gdr_selective_scan_step(*(a[k] for k in OPS), pool, softplus=True, **kernel_args(a))
    check_forward(a, off, out, pool, True, h0)


@pytest.mark.gpu
@pytest.mark.parametrize("work", ["f32", "bf16"])
@pytest.mark.parametrize("N", [8, 16, 64])
def test_backward_gates_of_every_size(N, work):
    case = ([70, 1, 20], 64, N, 1, work, True, True, True)
    a, off, offs, do, h0, dh = bwd_inputs(case, lead=0, tail=0)
    a["z"] = wide_sweep(*do.shape).to(DT[work]).to(CU)
    got = dict(zip(GRADS, gdr.gdr_selective_scan_bwd(do, *(a[k] for k in OPS), offs, softplus=True,
                                                     initial_state=h0, dfinal_state=dh,
                                                     **kernel_args(a))))
    kw = dict(soft=True, h0=h0, dh=dh, **ref_args(a))
    want = ref.scan_grads(do, *(a[k] for k in OPS), off, **kw)
    A = ref.scan_grads(do, *(a[k] for k in OPS), off, absolute=True, **kw)
    for k in GRADS:
        close(k, got[k], want[k], A[k], (8 * 70 + N + 64 + 600) * U32)


@pytest.mark.gpu
@pytest.mark.parametrize("work", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_backward_of_every_size(W, work):
    """SiLU's slope s(p) = sig (1 + p (1 - sig)) changes by at most sig (1 - sig) (2 + |p|),
    twice S = sig (1 + |p| (1 - sig)), which A holds; p is off by (W + 2) u of its terms'
    size P.  Beside it 40 u, and a run's sums, as above."""
    lens, C = [33, 0, 40, 1], 64
    gen = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    off, offs = offsets_of(lens)
    x, do = wide_sweep(off[-1], C, least=-200).to(DT[work]).to(CU), r(off[-1], C).to(DT[work]).to(CU)
    w = 0.02 * r(C, W)
    w[:, -1] = 1
    w, b = w.to(CU), r(C).to(CU)
    got = gdr.gdr_causal_conv1d_bwd(do, x, w, offs, bias=b, silu=True)
    P = float(ref.conv(x.abs(), w.abs(), off, b.abs()).max())
    f = (2 * P * (W + 2) + 40) * U32
    want = ref.conv_grads(do, x, w, off, b, True)
    A = ref.conv_grads(do, x, w, off, b, True, absolute=True)
    for name, g, e, size, more in zip(("dx", "dw", "db"), got, want, A, (0, 140, 140)):
        close(name, g, e, size, f + more * U32)


# ---------------------------------------------------------------- gradients ---

BWD = [  # rows, channels, states, groups, work, states, gate, skip and bias
    ([1], 8, 8, 1, "f32", False, True, True),
    ([16], 64, 16, 1, "f32", True, True, True),
    ([17, 0, 1], 72, 16, 1, "f32", True, False, True),
    ([40, 33], 80, 16, 2, "bf16", True, True, True),
    ([130, 64, 5], 40, 8, 1, "f32", False, True, False),
    ([200], 264, 16, 1, "bf16", False, True, True),
    ([90, 0, 20], 48, 32, 2, "f32", True, True, True),
    ([70], 24, 64, 1, "f32", True, False, False),
    ([100, 3], 144, 64, 1, "bf16", True, True, True),
    ([700, 90], 32, 16, 1, "f32", True, True, True),
    ([1] * 20 + [150], 16, 16, 1, "f32", True, True, True),
]
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")


def bwd_inputs(case, seed=11, lead=1, tail=2):
    lens, Dn, N, G, work, states, gate, extra = case
    a, off, offs, r = inputs(lens, Dn, N, G, work, z=gate, skip=extra, bias=extra, seed=seed,
                             lead=lead, tail=tail)
    do = r(*a["x"].shape).to(DT[work]).to(CU)
    rows = len(lens)
    h0 = (0.3 * r(rows, Dn, N)).to(DT[work]).to(CU) if states else None
    dh = (0.3 * r(rows, Dn, N)).to(DT[work]).to(CU) if states else None
    return a, off, offs, do, h0, dh


@pytest.mark.gpu
@pytest.mark.parametrize("soft", [True, False])
@pytest.mark.parametrize("case", BWD, ids=str)
def test_backward(case, soft):
    lens, Dn, N, G, work, *_ = case
    a, off, offs, do, h0, dh = bwd_inputs(case)
    if not soft:
        a["dt"] = (a["dt"].abs() * 0.1 + 1e-3).to(a["dt"].dtype)
        a["bias"] = None
    floats = gdr.gdr_selective_scan_workspace(do.shape[0], len(lens), Dn, N, G, True)
    fill = {k: torch.full(a[k2].shape, 7.0, dtype=a[k2].dtype, device=CU)
            for k, k2 in (("dx", "x"), ("ddt", "dt"), ("dB", "B"), ("dC", "C"), ("dz", "z"))
            if a[k2] is not None}
    got = dict(zip(GRADS, gdr.gdr_selective_scan_bwd(
        do, *(a[k] for k in OPS), offs, softplus=soft, initial_state=h0, dfinal_state=dh,
        workspace=torch.full((max(1, floats),), float("nan"), device=CU), **kernel_args(a), **fill)))
    kw = dict(soft=soft, h0=h0, dh=dh, **ref_args(a))
    want = ref.scan_grads(do, *(a[k] for k in OPS), off, **kw)
    A = ref.scan_grads(do, *(a[k] for k in OPS), off, absolute=True, **kw)
    n = max(lens)
    f = (8 * n + N + Dn // G + 600) * U32
    rows = slice(off[0], off[-1])
    for k in GRADS:
        if got[k] is None:
            continue
        g, w, b = got[k].cpu(), want[k], A[k]
        if k in fill:
            assert (g[:off[0]] == 7).all() and (g[off[-1]:] == 7).all(), k
            g, w, b = g[rows], w[rows], b[rows]
        close(k, g, w, b, f)
    assert (got["dh0"] is None) == (h0 is None) and (got["dz"] is None) == (a["z"] is None)
    # and as a whole: errors of independent roundings grow as the root of their number
    for k in ("dx", "ddt", "dA"):
        g, w = got[k].cpu(), want[k]
        if k in fill:
            g, w = g[rows], w[rows]
        near(k, g, w, (40 * U32 + (u(torch.bfloat16) if g.dtype == torch.bfloat16 else 0)) * n ** 0.5)


UNCUT = [  # 520 groups are workgroups enough for whole rows: none is cut into segments
    ([40] + [0] * 8 + [20], 2080, 8, 520, "f32", True, True, True),
    ([50, 3] + [0] * 15 + [20, 33], 2080, 16, 520, "f32", False, True, True),
    ([40] + [0] * 32 + [33, 17], 2080, 32, 520, "bf16", True, False, True),
    ([40, 70] + [0] * 63 + [20, 1, 18], 2080, 64, 520, "bf16", True, True, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", UNCUT, ids=lambda c: f"{len(c[0])}-{c[2]}")
def test_backward_of_uncut_rows(case):
    """Rows of several parts in a call that cuts none: the states before their parts are
    their own, whatever the rows behind them are."""
    test_backward(case, True)


@pytest.mark.gpu
def test_backward_against_the_forwards_differences():
    """The kernels' own forward in float32: a step of 2^-7 along a direction, the
    slope's cubic term and the forward's roundings (2^-24 of about 10^3 terms over
    2^-6) below 2e-3 of the directions' size."""
    case = ([60, 33], 16, 8, 1, "f32", False, True, True)
    a, off, offs, do, _, _ = bwd_inputs(case, lead=0, tail=0)
    got = dict(zip(GRADS, gdr.gdr_selective_scan_bwd(do, *(a[k] for k in OPS), offs, softplus=True,
                                                     **kernel_args(a))))
    gen = torch.Generator().manual_seed(3)

    def loss(b):
        out, _ = gdr.gdr_selective_scan_fwd(*(b[k] for k in OPS), offs, softplus=True, **kernel_args(b))
        return float((out.double() * do.double()).sum())

    for name, grad in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"),
                       ("z", "dz"), ("bias", "dbias")):
        d = torch.randn(a[name].shape, generator=gen).to(CU)
        d = d * (a[name].abs().mean() / d.abs().mean())
        e = 2.0 ** -7
        slope = (loss({**a, name: a[name] + e * d}) - loss({**a, name: a[name] - e * d})) / (2 * e)
        size = float((got[grad].double().abs() * d.double().abs()).sum())
        assert abs(slope - float((got[grad].double() * d.double()).sum())) < 2e-3 * size, name


@pytest.mark.gpu
@pytest.mark.parametrize("case", [BWD[3], BWD[9]], ids=str)
def test_same_call_same_bits(case):
    a, off, offs, do, h0, dh = bwd_inputs(case)
    runs = []
    for _ in range(2):
        out, end = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=True,
                                              initial_state=h0, output_final_state=True,
                                              **kernel_args(a))
        g = gdr.gdr_selective_scan_bwd(do, *(a[k] for k in OPS), offs, softplus=True,
                                       initial_state=h0, dfinal_state=dh, **kernel_args(a))
        rows = slice(off[0], off[-1])
        runs.append([out[rows], end] + [x[rows] if x.shape[0] == do.shape[0] else x for x in g])
    assert all(torch.equal(p, q) for p, q in zip(*runs))


@pytest.mark.gpu
def test_empty_batches():
    for lens in ([], [0], [0, 0, 0]):
        a, off, offs, r = inputs(lens, 16, 16, 1, "f32")
        out, end = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, softplus=True,
                                              state=torch.ones(3, 16, 16, device=CU), **kernel_args(a))
        assert (end == 1).all() and out.shape == (0, 16)
        dh = torch.full((len(lens), 16, 16), 2.0, device=CU)
        g = gdr.gdr_selective_scan_bwd(a["x"], *(a[k] for k in OPS), offs, softplus=True,
                                       initial_state=torch.ones_like(dh), dfinal_state=dh,
                                       **kernel_args(a))
        assert (g[2] == 0).all() and (g[5] == 0).all() and (g[7] == 0).all() and (g[8] == 2).all()
        conv = gdr.gdr_causal_conv1d_bwd(a["x"], a["x"], torch.ones(16, 4, device=CU), offs,
                                         bias=torch.ones(16, device=CU))
        assert (conv[1] == 0).all() and (conv[2] == 0).all()
        n, go = gdr.gdr_verify_drafts(torch.zeros(0, dtype=torch.int32, device=CU),
                                      torch.zeros(0, 10, device=CU), offs)
        assert n.tolist() == [0] * len(lens) and go.tolist() == [-1] * len(lens)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[40, 0, 3, 25], [150]], ids=str)
def test_a_layer_trains(lens):
    """Conv1d with SiLU, the scan of its output, and both gradients back to the
    convolution's input and weights, in float32, against the formulas in float64 of
    the same chain.

    The convolution's output x carries 2 (W + 9) u of its terms' sizes (W + 1 products
    and sums, a sigmoid of 6 u), here |x| <= A_x; dx does not depend on x, dA, ddt and
    dB are linear in it.  Bounds are linear too: a gradient of the scan is off by f A
    (A of |x| replaced by A_x), and the convolution's gradient carries the error f A of
    its dout on through absolute weights, besides its own."""
    Dn, N, W = 24, 16, 4
    a, off, offs, r = inputs(lens, Dn, N, 1, "f32")
    T = off[-1]
    w, b = (0.5 * r(Dn, W)).to(CU), (0.1 * r(Dn)).to(CU)
    raw, do = r(T, Dn).to(CU), r(T, Dn).to(CU)
    a["x"] = gdr.gdr_causal_conv1d(raw, w, offs, bias=b, silu=True)
    g = dict(zip(GRADS, gdr.gdr_selective_scan_bwd(do, *(a[k] for k in OPS), offs, softplus=True,
                                                   **kernel_args(a))))
    dx, dw, db = gdr.gdr_causal_conv1d_bwd(g["dx"], raw, w, offs, bias=b, silu=True)
    exact = ref.conv(raw, w, off, b, True)
    size = ref.conv(raw.abs(), w.abs(), off, b.abs(), False)  # |silu(s)| <= |s|
    full = [exact if k == "x" else a[k] for k in OPS]
    kw = dict(soft=True, **ref_args(a))
    want = ref.scan_grads(do, *full, off, **kw)
    A = ref.scan_grads(do, *(size if k == "x" else a[k] for k in OPS), off, absolute=True, **kw)
    f = (8 * max(lens) + N + Dn + 600 + 2 * (W + 9)) * U32
    for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz"):
        close(k, g[k], want[k], A[k], f)
    ends = ref.conv_grads(want["dx"], raw, w, off, b, True)
    E = ref.conv_grads(A["dx"], raw, w, off, b, True, absolute=True)
    fc = f + (8 * 8 * (W + 2) + 180) * U32  # the convolution's own, as it is tested alone
    for name, p, q, e in zip(("dx", "dw", "db"), (dx, dw, db), ends, E):
        close(name, p, q, e, fc)


# ------------------------------------------------------------------- Conv1d ---

CONV = [
    ([1], 4, 2, "f32", False, False), ([5, 0, 1, 2], 12, 4, "f32", True, True),
    ([16, 17], 260, 3, "bf16", True, False), ([300, 2, 41], 1036, 4, "bf16", True, True),
    ([129], 64, 4, "f32", False, True), ([1, 1, 1, 70, 1], 20, 3, "f32", True, True),
    ([3000], 8, 4, "f32", True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_backward(case):
    lens, C, W, work, silu, bias = case
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    off, offs = offsets_of(lens, 1)
    T = off[-1] + 2
    x = r(T, C + 8).to(DT[work]).to(CU)[:, :C]
    do, w = r(T, C).to(DT[work]).to(CU), (r(C, W) * W ** -0.5).to(CU)
    b = r(C).to(CU) if bias else None
    dx = torch.full((T, C), 7.0, dtype=x.dtype, device=CU)
    got = gdr.gdr_causal_conv1d_bwd(do, x, w, offs, bias=b, silu=silu, dx=dx)
    want = ref.conv_grads(do, x, w, off, b, silu)
    A = ref.conv_grads(do, x, w, off, b, silu, absolute=True)
    assert (dx[:off[0]] == 7).all() and (dx[off[-1]:] == 7).all()
    rows = slice(off[0], off[-1])
    # the slope of SiLU: a sigmoid of a sum of W + 1 terms whose size is at most 8 here,
    # off by 8 (W + 2) u, and 10 u of its own; a run's sums of up to 128 tokens
    f = (8 * 8 * (W + 2) + 40) * U32
    close("dx", dx[rows], want[0][rows], A[0][rows], f)
    close("dw", got[1], want[1], A[1], f + 140 * U32)
    if bias:
        close("db", got[2], want[2], A[2], f + 140 * U32)
    again = gdr.gdr_causal_conv1d_bwd(do, x, w, offs, bias=b, silu=silu)
    assert torch.equal(again[1], got[1]) and torch.equal(again[0][rows], dx[rows])


@pytest.mark.gpu
@pytest.mark.parametrize("work", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_window_then_fold(W, work):
    """A window leaves the histories alone; folding a prefix gives the history of a
    call over the prefix, bit for bit."""
    lens = [1, 0, 2, 3, 12, 5]
    gen = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    off, offs = offsets_of(lens)
    C = 36
    x, w = r(off[-1], C).to(DT[work]).to(CU), r(C, W).to(CU)
    hist = r(8, W - 1, C).to(DT[work]).to(CU)
    slots = torch.tensor([4, 0, 7, 2, 5, -1], dtype=torch.int32, device=CU)
    kept, moved = hist.clone(), hist.clone()
    out = gdr.gdr_causal_conv1d(x, w, offs, conv_state=kept, slot_idx=slots, silu=True,
                                keep_state=True)
    full = gdr.gdr_causal_conv1d(x, w, offs, conv_state=moved, slot_idx=slots, silu=True)
    assert torch.equal(out, full) and torch.equal(kept, hist) and not torch.equal(moved, hist)
    for n in ([1, 0, 2, 3, 12, 5], [0, 0, 1, 1, 2, 5], [1, 0, 2, 2, 1, 0], [2, 1, 3, 3, 7, 1]):
        acc = torch.tensor(n, dtype=torch.int32, device=CU)
        folded = gdr.gdr_causal_conv1d_fold(hist.clone(), x, offs, acc, slots)
        cut = [k if k <= m else 0 for k, m in zip(n, lens)]
        keep = torch.cat([torch.arange(o, o + k) for o, k in zip(off, cut)]).to(CU)
        want = hist.clone()
        gdr.gdr_causal_conv1d(x[keep].contiguous(), w, offsets_of(cut)[1], conv_state=want,
                              slot_idx=slots, silu=True)
        assert torch.equal(folded, want)


# ------------------------------------------------------------------- drafts ---

def draft_inputs(lens, V, dtype, mode, seed=0, lead=0, tail=0, pad=0):
    gen = torch.Generator().manual_seed(seed)
    off, offs = offsets_of(lens, lead)
    T = off[-1] + tail
    scores = 2 * torch.randn(T, V, generator=gen)
    other = scores.roll(1, 0) + 0.5 * torch.randn(T, V, generator=gen)
    best = scores.roll(1, 0).argmax(1)
    pick = torch.multinomial(torch.softmax(other, 1), 1, generator=gen)[:, 0] if T else best
    tokens = torch.where(torch.rand(T, generator=gen) < 0.6, best, pick).int()
    p = scores if mode == "greedy" else torch.softmax(scores, 1)
    wide = torch.zeros(T, V + pad)
    wide[:, :V] = p
    p = wide.to(dtype).to(CU)[:, :V]
    q = torch.softmax(other, 1).to(dtype).to(CU) if mode == "both" else None
    uu = None if mode == "greedy" else torch.rand(T, generator=gen).to(CU)
    return tokens.to(CU), p, q, uu, off, offs


DRAFTS = [
    ([1], 1), ([5], 7), ([3, 0, 1, 12], 100), ([8, 8], 2048), ([6, 1, 9], 2049), ([70, 3], 333),
    ([4] * 30, 50), ([2, 7], 5000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["both", "target", "greedy"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", DRAFTS, ids=str)
def test_verify_drafts(case, dtype, mode):
    lens, V = case
    for seed in range(4):
        tok, p, q, uu, off, offs = draft_inputs(lens, V, dtype, mode, seed, lead=1, tail=1,
                                                pad=seed)
        n, go = gdr.gdr_verify_drafts(tok, p, offs, draft=q, uniform=uu)
        want = ref.verify(tok, p, off, q, uu)
        assert (n.tolist(), go.tolist()) == want


@pytest.mark.gpu
def test_verify_drafts_of_many_slices():
    """A vocabulary of more values than 256 slices of the least length hold."""
    V = 600_011
    gen = torch.Generator().manual_seed(2)
    tok = torch.randint(0, V, (3,), generator=gen).int().to(CU)
    p = torch.rand(3, V, generator=gen).to(CU)
    offs = offsets_of([3])[1]
    for uniform in (0.0, 0.25, 0.9999):
        uu = torch.tensor([uniform, 0.0, 0.999], device=CU)
        n, go = gdr.gdr_verify_drafts(tok, p, offs, uniform=uu)
        c = p[int(n) - 1].double()
        if int(n) < 3:
            c[tok[int(n)].long()] = 0
        c = c.cumsum(0)
        assert int(go) == int((c > uu[0].double() * c[-1]).nonzero()[0, 0])
        best, go = gdr.gdr_verify_drafts(tok, p, offs)
        assert int(best) == 1 and int(go) == int(p[0].argmax())


@pytest.mark.gpu
def test_verify_drafts_at_the_edges():
    """Ties, equal and empty distributions, values that are no numbers, drafts outside
    the vocabulary, random numbers at the ends."""
    inf, nan = float("inf"), float("nan")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=CU)  # noqa: E731
    f = lambda *v: torch.tensor(v, device=CU)  # noqa: E731
    run = lambda tok, p, **kw: tuple(  # noqa: E731
        int(v) for v in gdr.gdr_verify_drafts(i32(*tok), p, i32(0, len(tok)), **kw))
    half = f([0.5, 0.5, 0.0], [0.5, 0.5, 0.0])
    # equal distributions: every draft with a probability stands, whatever its number
    assert run((0, 1), half, draft=half, uniform=f(0.0, 0.9999)) == (2, 0)
    # not standing needs uniform q >= p: nothing is left of p - q, so p itself is drawn from
    assert run((0, 2), half, draft=half, uniform=f(0.6, 0.0)) == (1, 1)
    assert run((0, 1), f([0.5, 0.5], [1.0, 0.0]), uniform=f(0.0, 0.5)) == (1, 0)  # 0.5 < 0.5 is false
    assert run((0, 1), f([0.0, 2.0], [1.0, 0.0]), uniform=f(0.0, 0.9)) == (2, 0)
    assert run((0,), f([0.0, 0.0, 0.0]).reshape(1, 3), uniform=f(0.5)) == (1, -1)
    assert run((0,), f([nan, inf, 0.0, 0.25]).reshape(1, 4), uniform=f(0.0)) == (1, 3)
    assert run((0,), f([0.25, 0.5, 0.0]).reshape(1, 3), uniform=f(1.0)) == (1, 1)   # the last weight
    assert run((0,), f([0.25, 0.5, 0.0]).reshape(1, 3), uniform=f(nan)) == (1, 1)
    assert run((0, 7), half, uniform=f(0.0, 0.0)) == (1, 0)
    assert run((0, -3), half, uniform=f(0.7, 0.0)) == (1, 1)
    # greedily
    assert run((0, 1, 1), f([1.0, 3.0, 3.0], [0.0, 1.0, 0.5], [-inf, -inf, -2.0])) == (3, 2)
    assert run((0, 2), f([1.0, 3.0, 3.0], [0.0, 1.0, 0.5])) == (1, 1)               # ties: the lowest
    assert run((0, 0), f([-0.0, 0.0], [1.0, 0.0])) == (2, 0)
    assert run((0, 0), f([nan, nan], [1.0, 0.0])) == (1, -1)
    assert run((0, 1), f([nan, -inf], [nan, 0.0])) == (2, 1)


# ---------------------------------------------------------- together, elsewhere ---

@pytest.mark.gpu
def test_a_drafted_window_from_verification_to_folds():
    """What a server does with a window: convolution and scan that keep their states,
    the verdict, both folds; then the next window starts where the accepted tokens end."""
    lens, Dn, N, V = [5, 1, 0, 7], 72, 16, 300
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    tok, p, q, uu, off, offs = draft_inputs(lens, V, torch.float32, "both", 3)
    pre, w = r(off[-1], Dn).to(CU), r(Dn, 4).to(CU)
    slots = torch.tensor([3, 0, 1, 2], dtype=torch.int32, device=CU)
    hist, state = r(4, 3, Dn).to(CU), (0.3 * r(4, Dn, N)).to(CU)
    a, *_ = inputs(lens, Dn, N, 1, "f32", seed=9)
    hist0, state0 = hist.clone(), state.clone()

    def layer(rows, offs, hist, state, keep):
        x = gdr.gdr_causal_conv1d(pre[rows], w, offs, conv_state=hist, slot_idx=slots, silu=True,
                                  keep_state=keep)
        t = {k: v if k in ("A", "D", "bias") else v[rows] for k, v in a.items()}
        out, _ = gdr.gdr_selective_scan_fwd(x, t["dt"], t["A"], t["B"].contiguous(),
                                            t["C"].contiguous(), offs, softplus=True, state=state,
                                            slot_idx=slots, keep_state=keep, **kernel_args(t))
        return x, out

    every = torch.arange(off[-1], device=CU)
    x, out = layer(every, offs, hist, state, True)
    assert torch.equal(hist, hist0) and torch.equal(state, state0)
    n, go = gdr.gdr_verify_drafts(tok, p, offs, draft=q, uniform=uu)
    want = ref.verify(tok, p, off, q, uu)
    assert (n.tolist(), go.tolist()) == want
    gdr.gdr_selective_scan_fold(state, x, a["dt"], a["A"], a["B"], offs, n, slots,
                                dt_bias=a["bias"], softplus=True)
    gdr.gdr_causal_conv1d_fold(hist, pre, offs, n, slots)
    kept = torch.cat([torch.arange(o, o + k) for o, k in zip(off, want[0])]).to(CU)
    _, again = layer(kept, offsets_of(want[0])[1], hist0, state0, False)
    assert torch.equal(again, out[kept])
    assert torch.equal(hist, hist0) and torch.equal(state, state0)


@pytest.mark.gpu
def test_verified_counts_roll_snapshots_back():
    """The verdict goes into gdr_snapshot_rollback as it is."""
    lens = [4, 4, 4]
    tok, p, q, uu, off, offs = draft_inputs(lens, 64, torch.float32, "both", 5)
    n, _ = gdr.gdr_verify_drafts(tok, p, offs, draft=q, uniform=uu)
    snaps = torch.randn(3, 4, 2, 16, 16, device=CU)
    state = torch.randn(3, 2, 16, 16, device=CU)
    gdr.gdr_snapshot_rollback(state, torch.arange(3, dtype=torch.int32, device=CU), snaps, n)
    want = ref.verify(tok, p, off, q, uu)[0]
    assert all(torch.equal(state[b], snaps[b, k - 1]) for b, k in enumerate(want))


def _all_calls():
    a, off, offs, do, h0, dh = bwd_inputs(BWD[9])
    tok, p, q, uu, _, doffs = draft_inputs([5, 3], 5000, torch.float32, "both")
    w, b = torch.full((32, 4), 0.25, device=CU), torch.ones(32, device=CU)
    pool = torch.zeros(2, 32, 16, device=CU)
    hist = torch.zeros(2, 3, 32, device=CU)
    acc = torch.tensor([9, 4], dtype=torch.int32, device=CU)

    def call(stream=None):
        kw = dict(softplus=True, stream=stream, **kernel_args(a))
        ops = [a[k] for k in OPS]
        res = list(gdr.gdr_selective_scan_fwd(*ops, offs, initial_state=h0, output_final_state=True, **kw))
        res += gdr.gdr_selective_scan_bwd(do, *ops, offs, initial_state=h0, dfinal_state=dh, **kw)
        res += gdr.gdr_causal_conv1d_bwd(do, a["x"], w, offs, bias=b, silu=True, stream=stream)
        res += gdr.gdr_verify_drafts(tok, p, doffs, draft=q, uniform=uu, stream=stream)
        res += gdr.gdr_verify_drafts(tok, p, doffs, stream=stream)
        one = [t if k == "A" else t[off[0]:off[0] + 2] for k, t in zip(OPS, ops)]
        kw["z"] = kw["z"][off[0]:off[0] + 2]
        res.append(gdr.gdr_selective_scan_step(*one, pool, **kw))
        res.append(gdr.gdr_selective_scan_fold(pool, *ops[:4], offs, acc, dt_bias=a["bias"],
                                               softplus=True, stream=stream))
        res.append(gdr.gdr_causal_conv1d_fold(hist, a["x"], offs, acc, stream=stream))
        return res

    rows = slice(off[0], off[-1])
    inside = lambda ts: [t[rows] if t.shape[0] == do.shape[0] else t for t in ts]  # noqa: E731
    return call, inside, (pool, hist), a["x"]


@pytest.mark.gpu
def test_other_streams():
    call, inside, bufs, _ = _all_calls()
    want = [t.clone() for t in inside(call())]
    for t in bufs:
        t.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(side)
    side.synchronize()
    for p, q in zip(want, inside(got)):
        assert torch.equal(p, q)


@pytest.mark.gpu
def test_graphs_replay_to_the_eager_results():
    call, inside, bufs, x = _all_calls()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(4):
        x.mul_(0.5 if i % 2 else 1.5)
        for t in bufs:
            t.zero_()
        want = [t.clone() for t in inside(call())]
        for t in got:
            t.fill_(3)
        for t in bufs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(want, inside(got)):
            assert torch.equal(p, q)
        torch.ones(1000, device=CU).sum().item()


def _of_walk(lens, Dn, N, seed, ws=None):
    """A forward and a gradient as one call, into buffers of its own."""
    a, off, offs, r = inputs(lens, Dn, N, 1, "f32", seed=seed)
    state = (0.3 * r(len(lens), Dn, N)).to(CU)
    do = r(*a["x"].shape).to(CU)
    T = do.shape[0]
    floats = max(gdr.gdr_selective_scan_workspace(T, len(lens), Dn, N, 1),
                 gdr.gdr_selective_scan_workspace(T, len(lens), Dn, N, 1, True))
    if ws is None:
        ws = torch.full((floats,), float("nan"), device=CU)
    out, end = torch.empty(T, Dn, device=CU), torch.empty_like(state)

    def call(stream=None):
        gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, initial_state=state, final_state=end,
                                   softplus=True, out=out, workspace=ws, stream=stream,
                                   **kernel_args(a))
        g = gdr.gdr_selective_scan_bwd(do, *(a[k] for k in OPS), offs, initial_state=state,
                                       dfinal_state=state, softplus=True, workspace=ws,
                                       stream=stream, **kernel_args(a))
        return [out, end, *g]

    return call, floats


WALK_CALLS = [([600, 20], 40, 16), ([90, 0, 17], 72, 16), ([1] * 9, 64, 16), ([40, 600], 24, 64)]


@pytest.mark.gpu
def test_calls_on_two_streams_at_once():
    calls = [_of_walk(*w, seed=i)[0] for i, w in enumerate(WALK_CALLS)]
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [c(streams[i % 2]) for i, c in enumerate(calls)]
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(p, q))


@pytest.mark.gpu
def test_graphs_that_share_a_workspace():
    """Nothing in it is expected to be what an earlier call left."""
    floats = max(_of_walk(*w, seed=i)[1] for i, w in enumerate(WALK_CALLS))
    ws = torch.full((floats,), float("nan"), device=CU)
    calls = [_of_walk(*w, seed=i, ws=ws)[0] for i, w in enumerate(WALK_CALLS)]
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = c()
        graphs.append((g, got))
    for turn in range(3):
        for i in (range(4), reversed(range(4)), (2, 0, 3, 1))[turn]:
            g, got = graphs[i]
            for t in got:
                t.fill_(3)
            ws.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(want[i], got))


# ------------------------------------------------- offsets that pass 32 bits ---

def _spread(a, stride, columns=()):
    """The operands, and outputs of x's shape named in `columns`, as columns of one
    buffer with `stride` elements from token to token."""
    T = a["x"].shape[0]
    buf, at, wide = torch.empty(T * stride, dtype=a["x"].dtype, device=CU), 0, dict(a)
    for k in ("x", "dt", "z", "B", "C", *columns):
        like = a[k] if k in a else a["x"]
        n = like[0].numel()
        view = buf[at:].as_strided((T, n), (stride, 1)).unflatten(1, like.shape[1:])
        if k in a:
            view.copy_(like)
        wide[k], at = view, at + n
    return wide


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Dn,stride", [
    ([65000, 0, 1000], 64, 65536),      # segments, the last rows behind 2^32 elements
    ([300, 900], 16, 1 << 22),          # the lane walk
    ([1] * 40 + [10] * 110, 16, 3 << 20),   # short rows
], ids=["long", "short", "rows"])
def test_far_tokens_scan_as_near_ones(lens, Dn, stride):
    a, off, offs, r = inputs(lens, Dn, 16, 1, "bf16", packed=False)
    if off[-1] * stride < 2 ** 32:
        stride = 2 ** 32 // off[-1] // 8 * 8 + 8
    assert stride < 2 ** 24 and off[-1] * stride >= 2 ** 32
    far = _spread(a, stride, ("out", "dx", "ddt", "dz", "do"))
    far["do"].copy_(r(*a["x"].shape).to(torch.bfloat16))
    kw = dict(softplus=True)
    near, end = gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, output_final_state=True,
                                           **kw, **kernel_args(a))
    out, last = gdr.gdr_selective_scan_fwd(*(far[k] for k in OPS), offs, output_final_state=True,
                                           out=far["out"], **kw, **kernel_args(far))
    assert torch.isfinite(near).all() and torch.equal(out, near) and torch.equal(last, end)
    g = gdr.gdr_selective_scan_bwd(far["do"].contiguous(), *(a[k] for k in OPS), offs, **kw,
                                   **kernel_args(a))
    f = gdr.gdr_selective_scan_bwd(far["do"], *(far[k] for k in OPS), offs, dx=far["dx"],
                                   ddt=far["ddt"], dz=far["dz"], **kw, **kernel_args(far))
    assert all(torch.equal(p, q) for p, q in zip(g[:8], f[:8]))
    w = torch.full((Dn, 4), 0.5, device=CU)
    c = gdr.gdr_causal_conv1d_bwd(far["do"].contiguous(), a["x"], w, offs, silu=True)
    d = gdr.gdr_causal_conv1d_bwd(far["do"], far["x"], w, offs, silu=True, dx=far["dx"])
    assert torch.equal(c[0], d[0]) and torch.equal(c[1], d[1])


@pytest.mark.gpu
def test_far_slots_and_vocabulary_rows():
    Dn, N, slots = 4096, 16, 65600  # 2^32 elements and some
    a, off, offs, r = inputs([1, 1, 1], Dn, N, 1, "bf16")
    pool = torch.empty(slots, Dn, N, dtype=torch.bfloat16, device=CU)
    at = torch.tensor([slots - 1, 7, slots - 30], dtype=torch.int32, device=CU)
    small = (0.3 * r(3, Dn, N)).to(torch.bfloat16).to(CU)
    for step in (True, False):
        pool[at.long()] = small
        near = small.clone()
        if step:
            args = [a[k] for k in OPS]
            o = gdr.gdr_selective_scan_step(*args, near, softplus=True, **kernel_args(a))
            p = gdr.gdr_selective_scan_step(*args, pool, at, softplus=True, **kernel_args(a))
        else:
            b, _, offs, _ = inputs([20, 30, 70], Dn, N, 1, "bf16")
            args = [b[k] for k in OPS]
            o = gdr.gdr_selective_scan_fwd(*args, offs, state=near, softplus=True, **kernel_args(b))[0]
            p = gdr.gdr_selective_scan_fwd(*args, offs, state=pool, slot_idx=at, softplus=True,
                                           **kernel_args(b))[0]
        assert torch.equal(o, p) and torch.equal(pool[at.long()], near)
    del pool
    T, V, stride = 5, 5003, 2 ** 30 + 17
    probs = torch.rand(T, V, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(CU)
    buf = torch.empty((T - 1) * stride + V, dtype=torch.bfloat16, device=CU)
    far = buf.as_strided((T, V), (stride, 1))
    far.copy_(probs)
    tok = probs.float().argmax(1).int().roll(1).contiguous()
    _, offs = offsets_of([5])
    for u01 in (None, torch.tensor([0.7, 0.1, 0.2, 0.3, 0.999], device=CU)):
        n, go = gdr.gdr_verify_drafts(tok, probs, offs, uniform=u01)
        m, gm = gdr.gdr_verify_drafts(tok, far, offs, uniform=u01)
        assert torch.equal(n, m) and torch.equal(go, gm) and go[0] >= 0


@pytest.mark.gpu
def test_index_checks_cover_the_new_entries():
    a, off, offs, _ = inputs([3, 2], 16, 16, 1, "f32")
    pool = torch.zeros(2, 16, 16, device=CU)
    twice = torch.tensor([1, 1], dtype=torch.int32, device=CU)
    far = torch.tensor([0, 3, 99], dtype=torch.int32, device=CU)
    was = gdr.gdr_set_debug_checks(True)
    try:
        with pytest.raises(gdr.GdrError, match="slot 1 is used"):
            gdr.gdr_selective_scan_fwd(*(a[k] for k in OPS), offs, state=pool, slot_idx=twice)
        with pytest.raises(gdr.GdrError, match="past the 5 tokens"):
            gdr.gdr_selective_scan_bwd(a["x"].contiguous(), *(a[k] for k in OPS), far)
        with pytest.raises(gdr.GdrError, match="past the 5 tokens"):
            gdr.gdr_verify_drafts(torch.zeros(5, dtype=torch.int32, device=CU),
                                  torch.zeros(5, 9, device=CU), far)
        with pytest.raises(gdr.GdrError, match="slot 1 is used"):
            gdr.gdr_causal_conv1d_fold(torch.zeros(2, 3, 16, device=CU), a["x"], offs, twice, twice)
    finally:
        gdr.gdr_set_debug_checks(was)
