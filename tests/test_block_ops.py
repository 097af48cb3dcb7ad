"""Linear attention with a decay for each head and the norms around a block:
the references' gradients against differences, and the host's refusals (CPU);
the kernels against the references in float64 (GPU).

Error bounds.  u(t) = finfo(t).eps / 2 is what one rounding to t is off at
most, relative to the value; every output may be off by u(its type) |ref| plus
what its float32 sums are off.  That is at most (number of terms added one after
another) u(float32) times the sum of the terms' absolute values, A, which the
references compute as the same formula on absolute values.  In bf16 work the
factors that are multiplied again are held in two bf16 terms, each within u(bf16)
of what it stands for: u(bf16)^2 = 2^-16 of the value; an output has three such
factors (the products of a chunk, the state, and the state's own sums).  The
decays' exponents are exact to u(float32) of themselves (|g| sums below 2^5 where
the result counts): 2^-19.  Together below 2^-13 A."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_loop_amd as gdr
from gated_delta_rule_loop_amd import _binding as B
from tests import block_ref as ref

U32 = torch.finfo(torch.float32).eps / 2


def u(dtype):
    return torch.finfo(dtype).eps / 2


# ----------------------------------------------------------- the references ---

def test_attention_reference_gradients_match_differences():
    gen = torch.Generator().manual_seed(1)
    off, nk, nv, K, V, s = [0, 0, 5, 6], 1, 2, 3, 4, 0.6
    r = lambda *n: torch.randn(n, generator=gen, dtype=torch.float64)  # noqa: E731
    x = dict(q=r(6, nk, K), k=r(6, nk, K), v=r(6, nv, V), g=-r(6, nv).abs(), s0=r(3, nv, K, V))
    do, ds = r(6, nv, V), r(3, nv, K, V)

    def loss(x):
        o, end = ref.attention(x["q"], x["k"], x["v"], x["g"], off, x["s0"], s)
        return float((o * do).sum() + (end * ds).sum())

    got = ref.attention_grads(do, x["q"], x["k"], x["v"], x["g"], off, x["s0"], ds, s)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("s0", "ds0")):
        d = r(*x[name].shape)
        e = 1e-5
        up = loss({**x, name: x[name] + e * d})
        down = loss({**x, name: x[name] - e * d})
        # cubic terms of size e^2 and rounding of size 2^-52 / e: both below 1e-8
        assert abs((up - down) / (2 * e) - float((got[grad] * d).sum())) < 1e-7, name


@pytest.mark.parametrize("act", [None, "sigmoid", "silu"])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_norm_reference_gradients_match_differences(gate, act):
    if gate == "none" and act:
        pytest.skip("an activation needs a gate")
    gen = torch.Generator().manual_seed(2)
    T, D, n = 3, 16, 8
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x = dict(y=r(T, D), x=r(T, D), w1=r(n), w2=r(D))
    if gate != "none":
        x["gate"] = r(T, D) if gate == "token" else r(D)
    dh, dn = r(T, D), r(T, D)

    def loss(x):
        h, m, _, _ = ref.norm(x["y"], x["w1"], n, x.get("gate"), act, x["x"], 0.3, x["w2"], 1e-6)
        return float((h * dh).sum() + (m * dn).sum())

    h = ref.norm(x["y"], x["w1"], n, x.get("gate"), act, x["x"], 0.3, x["w2"], 1e-6)[0]
    got = ref.norm_grads(dh, dn, x["y"], h, x["w1"], n, x.get("gate"), act, x["x"], 0.3, x["w2"],
                         1e-6)
    for name, grad in (("y", "dy"), ("x", "dx"), ("w1", "dw1"), ("w2", "dw2"), ("gate", "dgate")):
        if name in x:
            d, e = r(*x[name].shape), 1e-5
            up, down = loss({**x, name: x[name] + e * d}), loss({**x, name: x[name] - e * d})
            assert abs((up - down) / (2 * e) - float((got[grad] * d).sum())) < 1e-7, name


# ---------------------------------------------------------------- refusals ---

FAKE = 0x10000  # never dereferenced: validation fails first
F32, BF16, U32T, I32 = B.GDR_DTYPE_F32, B.GDR_DTYPE_BF16, B.GDR_DTYPE_U32, B.GDR_DTYPE_I32


def D(shape, dtype=F32, stride=None, data=FAKE):
    d = B.GdrTensor()
    d.data, d.dtype, d.ndim = data, dtype, len(shape)
    if stride is None:
        stride, acc = [], 1
        for s in reversed(shape):
            stride.insert(0, acc)
            acc *= s
    for i, (s, st) in enumerate(zip(shape, stride)):
        d.shape[i], d.stride[i] = s, st
    return d


def _call(fn, args):
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libgdr.so not built")
    r = [ctypes.byref(a) if isinstance(a, B.GdrTensor) else a for a in args]
    return getattr(B.lib(), fn)(*r)


def _fwd(**over):
    T, nk, nv, K, V, R = 2000, 2, 4, 64, 32, 3
    a = dict(o=D([T, nv, V], data=FAKE * 2), q=D([T, nk, K]), k=D([T, nk, K]), v=D([T, nv, V]),
             g=D([T, nv]), off=D([R + 1], I32), scale=-1.0, s0=None, end=None,
             state=D([5, nv, K, V]), slot=D([R], I32), ws=D([10 ** 7]), stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code,word", [
    (dict(o=None), -1, "o is null"),
    (dict(q=D([2000, 2, 60]), k=D([2000, 2, 60])), -2, "multiples of 8"),
    (dict(q=D([2000, 2, 264]), k=D([2000, 2, 264])), -2, "multiples of 8"),
    (dict(q=D([2000, 3, 64]), k=D([2000, 3, 64])), -1, "multiple"),
    (dict(k=D([2000, 2, 32])), -1, "k dim 2"),
    (dict(v=D([2000, 4, 32], BF16)), -2, "work dtype"),
    (dict(q=D([2000, 2, 64], U32T)), -2, "dtype"),
    (dict(q=D([2000, 2, 64], stride=[128, 64, 2])), -2, "innermost"),
    (dict(q=D([2000, 2, 64], stride=[130, 64, 1])), -2, "multiple of 4"),
    (dict(q=D([2000, 2, 64], data=FAKE + 8)), -2, "aligned"),
    (dict(o=D([2000, 4, 32], data=FAKE * 2, stride=[0, 32, 1])), -1, "overlap"),
    (dict(o=D([2000, 4, 32], data=FAKE * 2, stride=[64, 32, 1])), -1, "overlap"),
    (dict(o=D([2000, 4, 32])), -1, "alias"),
    (dict(g=D([2000, 2])), -1, "g dim 1"),
    (dict(g=D([2000, 4], I32)), -2, "dtype"),
    (dict(off=D([0], I32)), -1, "empty"),
    (dict(off=D([4], F32)), -2, "dtype"),
    (dict(state=D([5, 4, 32, 64])), -1, "state dim 2"),
    (dict(state=D([5, 4, 64, 32], stride=[8192, 2048, 33, 1])), -2, "dense"),
    (dict(state=D([2, 4, 64, 32]), slot=None), -1, "fewer slots"),
    (dict(state=None), -1, "slot_idx needs state"),
    (dict(s0=D([3, 4, 64, 32])), -1, "give state, or"),
    (dict(state=None, slot=None, s0=D([2, 4, 64, 32])), -1, "initial_state dim 0"),
    (dict(state=None, slot=None, s0=D([3, 4, 64, 32], BF16), end=D([3, 4, 64, 32])), -2, "dtype"),
    (dict(ws=None), -1, "workspace is null"),
    (dict(ws=D([16])), -1, "needed"),
    (dict(ws=D([10 ** 7], BF16)), -1, "float32 vector"),
    (dict(ws=D([10 ** 7], data=FAKE + 4)), -2, "aligned"),
])
def test_forward_refuses(over, code, word):
    assert _call("gdr_linear_attention_fwd", _fwd(**over)) == code
    assert word in B.gdr_last_error_message()


@pytest.mark.parametrize("over,code,word", [
    (dict(state=None), -1, "state is null"),
    (dict(state=D([2, 4, 64, 32]), slot=None), -1, "fewer slots"),
    (dict(slot=D([2], I32)), -1, "slot_idx dim 0"),
    (dict(q=D([3, 2, 4]), k=D([3, 2, 4])), -2, "multiples of 8"),
    (dict(o=D([3, 4, 32])), -1, "alias"),
])
def test_step_refuses(over, code, word):
    a = dict(o=D([3, 4, 32], data=FAKE * 2), q=D([3, 2, 64]), k=D([3, 2, 64]), v=D([3, 4, 32]),
             g=D([3, 4]), state=D([5, 4, 64, 32]), slot=D([3], I32), scale=-1.0, stream=None)
    a.update(over)
    assert _call("gdr_linear_attention_step", list(a.values())) == code
    assert word in B.gdr_last_error_message()


@pytest.mark.parametrize("over,code,word", [
    (dict(do=D([100, 4, 64])), -1, "do dim 2"),
    (dict(dq=None), -1, "dq is null"),
    (dict(dk=D([100, 2, 64], data=FAKE * 2)), -1, "alias"),
    (dict(dv=D([100, 4, 32], data=FAKE * 4, stride=[128, 0, 1])), -1, "overlap"),
    (dict(dg=D([100, 4], data=FAKE * 6, stride=[0, 1])), -1, "overlap"),
    (dict(g=None), -1, "dg needs g"),
    (dict(ds=D([1, 4, 64, 32])), -1, "dfinal_state dim 0"),
    (dict(d0=D([2, 4, 32, 64], data=FAKE * 7)), -1, "dinitial_state dim 2"),
    (dict(ws=None), -1, "workspace is null"),
])
def test_backward_refuses(over, code, word):
    a = dict(do=D([100, 4, 32]), q=D([100, 2, 64]), k=D([100, 2, 64]), v=D([100, 4, 32]),
             g=D([100, 4]), off=D([3], I32), scale=-1.0, s0=None, ds=None,
             dq=D([100, 2, 64], data=FAKE * 2), dk=D([100, 2, 64], data=FAKE * 3),
             dv=D([100, 4, 32], data=FAKE * 4), dg=D([100, 4], data=FAKE * 6), d0=None,
             ws=D([10 ** 8]), stream=None)
    a.update(over)
    assert _call("gdr_linear_attention_bwd", list(a.values())) == code
    assert word in B.gdr_last_error_message()


def _norm_args(over):
    a = dict(h=D([5, 64], data=FAKE * 2), n=D([5, 64], data=FAKE * 3), y=D([5, 64]),
             x=D([5, 64]), gate=D([5, 64]), w1=D([16]), w2=D([64]), group=16, c=1.0, eps=1e-6,
             flags=B.GDR_FLAG_GATE_SILU, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code,word", [
    (dict(y=D([5, 60])), -2, "multiples of 8"),
    (dict(y=D([5, 16392])), -2, "multiples of 8"),
    (dict(group=24), -1, "groups of 24"),
    (dict(group=12), -1, "groups of 12"),
    (dict(w1=None), -1, "groups need post_weight"),
    (dict(w1=D([32])), -1, "post_weight dim 0"),
    (dict(w1=D([16], BF16)), -2, "post_weight must be"),
    (dict(gate=D([4, 64])), -1, "gate dim 0"),
    (dict(gate=D([32])), -1, "gate dim 0"),
    (dict(flags=12), -1, "one activation"),
    (dict(flags=16), -1, "unknown flags"),
    (dict(n=None), -1, "go together"),
    (dict(w2=None), -1, "go together"),
    (dict(n=D([5, 64], data=FAKE * 2)), -1, "must not alias h"),
    (dict(h=D([5, 64], data=FAKE * 2, stride=[32, 1])), -1, "overlap"),
    (dict(x=D([5, 64], BF16)), -2, "work dtype"),
    (dict(eps=-1.0), -1, "eps"),
    (dict(eps=float("nan")), -1, "eps"),
])
def test_norm_refuses(over, code, word):
    assert _call("gdr_block_norm", _norm_args(over)) == code
    assert word in B.gdr_last_error_message()


@pytest.mark.parametrize("over,code,word", [
    (dict(dy=None), -1, "dy is null"),
    (dict(dn=None), -1, "dn is null"),
    (dict(h=None), -1, "h is null"),
    (dict(w2=None, dw2=None), -1, "dn needs pre_weight"),
    (dict(dgate=None), -1, "dgate is null"),
    (dict(dw1=None), -1, "dpost_weight is null"),
    (dict(dw2=None), -1, "dpre_weight is null"),
    (dict(dx=D([5, 64], data=FAKE * 3)), -1, "share memory"),
    (dict(ws=None), -1, "workspace is null"),
    (dict(ws=D([3])), -1, "needed"),
])
def test_norm_backward_refuses(over, code, word):
    a = dict(dx=D([5, 64], data=FAKE * 2), dy=D([5, 64], data=FAKE * 3),
             dgate=D([5, 64], data=FAKE * 4), dw1=D([16], data=FAKE * 5),
             dw2=D([64], data=FAKE * 6), dh=D([5, 64]), dn=D([5, 64]), y=D([5, 64]),
             h=D([5, 64]), gate=D([5, 64]), w1=D([16]), w2=D([64]), group=16, c=1.0, eps=1e-6,
             flags=B.GDR_FLAG_GATE_SILU, ws=D([10 ** 6]), stream=None)
    a.update(over)
    assert _call("gdr_block_norm_bwd", list(a.values())) == code
    assert word in B.gdr_last_error_message()


def test_workspace_sizes():
    f = gdr.gdr_linear_attention_workspace
    assert f(0, 0, 1, 1, 64, 64) == 0 and f(100, 1, 2, 2, 64, 64) == 0
    assert f(-1, 1, 1, 1, 64, 64) == -1
    # a long row is cut into segments: a state for each at least
    assert f(32768, 1, 16, 32, 128, 128) >= 2 * 32 * 128 * 128
    assert f(100, 1, 1, 2, 64, 64, True) >= 2 * 100 * 2 * 64
    assert gdr.gdr_block_norm_workspace(4, 64) >= 4 * 64
    assert gdr.gdr_block_norm_workspace(1, 16392) == -1


# --------------------------------------------------------------------- GPU ---

def bounds(work, K, T, chunk=32):
    """Factor of the absolute sums A that float32 sums and split factors are off."""
    adds = (K + 2 * 64 + T / chunk + 64) * U32
    return adds + (2.0 ** -13 if work == torch.bfloat16 else 0.0)


def close(what, got, want, A, factor):
    """|got - want| <= u |want| + factor A for every element."""
    own = torch.finfo(got.dtype).eps / 2
    got, want, A = got.detach().cpu().double(), want.double(), A.double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    most = own * want.abs() + factor * A + 1e-30
    worst = float(((got - want).abs() / most).max()) if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def near(what, got, want, most):
    """The 2-norm of the difference against that of the values."""
    d = float((got.detach().cpu().double() - want).norm())
    n = float(want.norm())
    assert d <= most * n + 1e-30, f"{what}: {d / max(n, 1e-300):.3g} relative, {most:.3g} allowed"


def inputs(lens, nk, nv, K, V, work, decay="token", seed=0, lead=0, tail=0, packed=True):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens) + lead + tail
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    qkv = n(T, 2 * nk * K + nv * V)
    qkv[:, :2 * nk * K] *= K ** -0.25
    qkv = qkv.to(work).cuda()
    q = qkv[:, :nk * K].unflatten(1, (nk, K))
    k = qkv[:, nk * K:2 * nk * K].unflatten(1, (nk, K))
    v = qkv[:, 2 * nk * K:].unflatten(1, (nv, V))
    if not packed:  # heads outermost: other strides
        q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    if decay == "token":
        g = -torch.nn.functional.softplus(n(T, nv) - 2).to(work).cuda()
    elif decay == "head":
        g = (-0.7 * 2.0 ** -torch.arange(nv).float()).cuda().expand(T, nv)
    elif decay == "zeros":  # some tokens forget everything, some nothing
        g = -torch.nn.functional.softplus(n(T, nv) - 1)
        g[torch.rand((T, nv), generator=gen) < 0.05] = -float("inf")
        g[torch.rand((T, nv), generator=gen) < 0.2] = 0.0
        g = g.cuda()
    else:
        g = None
    off = [lead]
    for m in lens:
        off.append(off[-1] + m)
    return q, k, v, g, off, torch.tensor(off, dtype=torch.int32, device="cuda"), gen


FWD = [
    # lens, nk, nv, K, V, work, state dtype, decay
    ([1], 1, 1, 8, 8, "f32", "f32", "token"),
    ([2, 1, 3], 1, 2, 16, 16, "bf16", "bf16", "token"),
    ([5, 5], 2, 2, 24, 40, "f32", "f32", "token"),
    ([63], 2, 4, 64, 64, "bf16", "bf16", "head"),
    ([64], 2, 4, 64, 128, "bf16", "f32", "token"),
    ([65, 0, 31, 33], 1, 3, 128, 64, "bf16", "bf16", "token"),
    ([65, 0, 31, 33], 1, 3, 128, 64, "f32", "f32", "token"),
    ([129, 128, 1], 2, 4, 128, 128, "bf16", "bf16", "zeros"),
    ([129, 128, 1], 2, 4, 128, 128, "f32", "bf16", "zeros"),
    ([100, 17], 1, 2, 256, 256, "bf16", "f32", "token"),
    ([100, 17], 1, 2, 256, 256, "f32", "f32", "none"),
    ([90], 1, 2, 96, 72, "bf16", "bf16", "head"),
    ([90], 1, 2, 200, 136, "f32", "f32", "token"),
    ([700, 3, 0, 257], 1, 2, 64, 64, "bf16", "f32", "token"),   # cut into segments
    ([700, 3, 0, 257], 1, 2, 64, 64, "f32", "f32", "zeros"),
    ([513], 2, 2, 128, 128, "bf16", "bf16", "head"),
    ([1100], 1, 1, 32, 256, "f32", "f32", "head"),
]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def absolute(*xs):
    return [None if x is None else x.detach().cpu().double().abs() for x in xs]


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("case", FWD, ids=str)
def test_forward(case, packed):
    lens, nk, nv, K, V, work, st, decay = case
    work, st = DT[work], DT[st]
    q, k, v, g, off, offs, gen = inputs(lens, nk, nv, K, V, work, decay, 3, 2, 5, packed)
    T, R = q.shape[0], len(lens)
    pool = (0.3 * torch.randn((R + 3, nv, K, V), generator=gen)).to(st).cuda()
    before = pool.clone()
    slots = torch.randperm(R + 3, generator=gen)[:R].to(torch.int32)
    if R > 2:
        slots[1] = -1
    o = torch.full((T, nv, V), 7.0, dtype=work, device="cuda")
    gdr.gdr_linear_attention_fwd(q, k, v, g, offs, state=pool, slot_idx=slots.cuda(), o=o,
                                 scale=0.3)
    torch.cuda.synchronize()
    live = slots >= 0
    s0 = torch.zeros(R, nv, K, V, dtype=torch.float64)
    s0[live] = before.cpu()[slots[live].long()].double()
    want, end = ref.attention(q, k, v, g, off, s0, 0.3)
    A, Aend = ref.attention(*absolute(q, k, v), None if g is None else g.cpu(), off, s0.abs(), 0.3)
    f = bounds(work, K, max(lens))
    for r in range(R):
        a, b = off[r], off[r + 1]
        if live[r]:
            close("o", o[a:b], want[a:b], A[a:b], f)
            fs = bounds(torch.float32, 64, max(lens)) + (
                2.0 ** -22 if st == torch.float32 else 2.0 ** -13 if work == torch.bfloat16 else 0)
            if len(lens) and work == torch.bfloat16 and T > 256:
                fs += 2.0 ** -13     # segments' own sums come in with their states
            close("state", pool[slots[r]], end[r], Aend[r], fs)
            if a == b:
                assert torch.equal(pool[slots[r]], before[slots[r]])
        else:
            assert (o[a:b] == 0).all() and not torch.signbit(o[a:b]).any()
    # nothing else is written
    assert (o[:off[0]] == 7).all() and (o[off[-1]:] == 7).all()
    used = set(slots[live].tolist())
    for s in range(R + 3):
        if s not in used:
            assert torch.equal(pool[s], before[s])


# Sixteen rows and more: those of up to eight tokens and the longer ones take
# different ways, whatever stands beside them.
MANY = [
    ([1] * 15 + [40] + [8, 9, 0, 1], 1, 2, 64, 64, "bf16", "bf16", "token"),
    ([1] * 16 + [700] + [3] * 4 + [150, 0, 7, 10], 1, 2, 64, 96, "f32", "f32", "token"),
    ([2] * 18 + [600, 64, 65, 1], 2, 2, 128, 128, "bf16", "f32", "head"),
    ([1] * 17, 2, 6, 64, 40, "f32", "bf16", "token"),
    ([20] * 16, 1, 1, 128, 128, "bf16", "bf16", "none"),
    ([0] * 20, 1, 2, 8, 16, "f32", "f32", "token"),
    ([0] * 70 + [300] + [1] * 70 + [9, 8], 1, 3, 16, 24, "bf16", "bf16", "token"),
    # heads enough to fill the chip: only what is longer than its share is cut
    ([1] * 14 + [1300, 5, 0, 900, 64, 130], 2, 32, 16, 24, "bf16", "bf16", "token"),
    ([1] * 70 + [321, 5, 0, 1200, 9] + [3] * 70 + [320], 2, 32, 16, 24, "f32", "f32", "zeros"),
    ([70] * 16, 4, 32, 8, 16, "f32", "bf16", "head"),
    ([64] * 15 + [65, 66, 130, 1], 2, 32, 16, 24, "f32", "f32", "token"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", MANY, ids=lambda c: "%d-rows-%s" % (len(c[0]), c[1:]))
def test_forward_of_many_rows(case):
    test_forward(case, True)


@pytest.mark.gpu
@pytest.mark.parametrize("initial", [True, False])
def test_dense_states_of_many_rows(initial):
    lens = [1] * 14 + [33, 0, 8, 9, 700, 0, 2]
    q, k, v, g, off, offs, gen = inputs(lens, 1, 2, 64, 64, torch.float32, seed=15)
    s0 = (0.3 * torch.randn((len(lens), 2, 64, 64), generator=gen)).cuda()
    start = s0 if initial else torch.zeros_like(s0)
    pool = start.clone()
    o1, end = gdr.gdr_linear_attention_fwd(q, k, v, g, offs, initial_state=s0 if initial else None,
                                           output_final_state=True)
    o2, _ = gdr.gdr_linear_attention_fwd(q, k, v, g, offs, state=pool)
    assert torch.equal(o1, o2) and torch.equal(end, pool)
    assert torch.equal(end[15], start[15]) and torch.equal(end[19], start[19])


@pytest.mark.gpu
@pytest.mark.parametrize("work", ["bf16", "f32"])
def test_forward_dense_states_equal_the_pool(work):
    q, k, v, g, off, offs, gen = inputs([130, 0, 40], 1, 2, 64, 64, DT[work], seed=5)
    s0 = (0.3 * torch.randn((3, 2, 64, 64), generator=gen)).cuda()
    pool = s0.clone()
    o1, end = gdr.gdr_linear_attention_fwd(q, k, v, g, offs, initial_state=s0,
                                           output_final_state=True)
    o2, _ = gdr.gdr_linear_attention_fwd(q, k, v, g, offs, state=pool)
    assert torch.equal(o1, o2) and torch.equal(end, pool) and torch.equal(end[1], s0[1])


@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    (1, 1, 1, 8, 8, "f32", "f32", "token"), (7, 2, 6, 64, 96, "f32", "f32", "head"),
    (19, 4, 8, 128, 128, "bf16", "bf16", "token"), (5, 1, 2, 256, 256, "bf16", "f32", "zeros"),
    (33, 2, 2, 96, 72, "bf16", "bf16", "none"), (3, 1, 4, 16, 256, "f32", "bf16", "token")], ids=str)
def test_step(case):
    R, nk, nv, K, V, work, st, decay = case
    work, st = DT[work], DT[st]
    q, k, v, g, off, offs, gen = inputs([1] * R, nk, nv, K, V, work, decay, 11)
    pool = (0.3 * torch.randn((R + 2, nv, K, V), generator=gen)).to(st).cuda()
    before = pool.clone()
    slots = torch.randperm(R + 2, generator=gen)[:R].to(torch.int32)
    if R > 4:
        slots[2] = -1
    o = gdr.gdr_linear_attention_step(q, k, v, g, pool, slots.cuda())
    live = slots >= 0
    s0 = before.cpu()[slots.long().clamp_min(0)].double()
    sc = K ** -0.5
    want, end = ref.attention(q, k, v, g, off, s0, sc)
    A, Aend = ref.attention(*absolute(q, k, v), None if g is None else g.cpu(), off, s0.abs(), sc)
    f = (K + 8) * U32
    close("o", o[live.cuda()], want[live], A[live], f)
    close("state", pool[slots[live].long().cuda()], end[live], Aend[live], 4 * U32)
    assert (o[(~live).cuda()] == 0).all()
    rest = [s for s in range(R + 2) if s not in slots.tolist()]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.gpu
def test_prompt_then_tokens_continue_one_row():
    q, k, v, g, off, offs, gen = inputs([150], 2, 4, 64, 64, torch.float32, seed=6)
    whole, end = gdr.gdr_linear_attention_fwd(q, k, v, g, offs, output_final_state=True)
    pool = torch.zeros(1, 4, 64, 64, device="cuda")
    cut = torch.tensor([0, 140], dtype=torch.int32, device="cuda")
    parts = [gdr.gdr_linear_attention_fwd(q[:140], k[:140], v[:140], g[:140], cut, state=pool)[0]]
    for t in range(140, 150):
        s = slice(t, t + 1)
        parts.append(gdr.gdr_linear_attention_step(q[s], k[s], v[s], g[s], pool))
    want, _ = ref.attention(q, k, v, g, off, None, 64 ** -0.5)
    A, Aend = ref.attention(*absolute(q, k, v), g.cpu(), off, None, 64 ** -0.5)
    close("o", torch.cat(parts), want, A, bounds(torch.float32, 64, 150))
    close("whole", whole, want, A, bounds(torch.float32, 64, 150))


@pytest.mark.gpu
@pytest.mark.parametrize("work", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[40, 70, 30], [400, 300]])
def test_rows_do_not_touch_their_neighbours(work, lens):
    q, k, v, g, off, offs, gen = inputs(lens, 1, 2, 64, 64, DT[work], seed=8)
    good, _ = gdr.gdr_linear_attention_fwd(q, k, v, g, offs)
    a, b = off[1], off[2]
    for x in (q, k, v):
        x[a:b] = float("nan")
    bad, _ = gdr.gdr_linear_attention_fwd(q, k, v, g, offs)
    assert torch.equal(bad[:a], good[:a]) and torch.equal(bad[b:], good[b:])


BWD = [
    # lens, nk, nv, K, V, work, states, decay
    ([1], 1, 1, 8, 8, "f32", True, "token"),
    ([3, 0, 2], 1, 2, 16, 32, "f32", True, "token"),
    ([64], 2, 2, 64, 64, "bf16", False, "token"),
    ([65, 31], 1, 3, 64, 128, "bf16", True, "token"),
    ([65, 31], 1, 3, 128, 64, "f32", True, "zeros"),
    ([129, 1], 2, 2, 128, 128, "bf16", True, "token"),
    ([129, 1], 2, 2, 128, 128, "f32", False, "token"),
    ([80], 1, 1, 256, 256, "bf16", True, "token"),
    ([80], 1, 1, 256, 256, "f32", True, "token"),
    ([70], 1, 2, 96, 72, "bf16", False, "head"),
    ([40], 1, 2, 64, 64, "f32", True, "none"),
    ([600, 3, 0, 257], 1, 2, 64, 64, "bf16", True, "token"),    # cut into segments
    ([600, 3, 0, 257], 2, 2, 64, 64, "f32", True, "zeros"),
    ([300], 1, 2, 256, 64, "f32", False, "token"),
]


def bwd_inputs(case, seed=4):
    lens, nk, nv, K, V, work, states, decay = case
    work = DT[work]
    q, k, v, g, off, offs, gen = inputs(lens, nk, nv, K, V, work, decay, seed, 1, 2)
    do = torch.randn(v.shape, generator=gen).to(work).cuda()
    s0 = ds = None
    if states:
        s0 = (0.3 * torch.randn((len(lens), nv, K, V), generator=gen)).cuda()
        ds = (0.3 * torch.randn((len(lens), nv, K, V), generator=gen)).cuda()
    return do, q, k, v, g, off, offs, s0, ds


@pytest.mark.gpu
@pytest.mark.parametrize("case", BWD, ids=str)
def test_backward(case):
    lens, nk, nv, K, V, work, states, decay = case
    do, q, k, v, g, off, offs, s0, ds = bwd_inputs(case)
    sc = 0.4
    dq, dk, dv, dg, d0 = gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs, initial_state=s0,
                                                      dfinal_state=ds, scale=sc)
    want = ref.attention_grads(do, q, k, v, g, off, s0, ds, sc)
    gc = None if g is None else g.cpu()
    A = ref.attention_grads(*absolute(do, q, k, v), gc, off, *absolute(s0, ds), sc, sign=1.0)
    n = max(lens)
    s = slice(off[0], off[-1])
    f = bounds(DT[work], max(K, V), n) + nv // nk * U32
    close("dq", dq[s], want["dq"][s], A["dq"][s], f)
    close("dk", dk[s], want["dk"][s], A["dk"][s], f)
    close("dv", dv[s], want["dv"][s], A["dv"][s], f)
    if g is None:
        assert dg is None
    else:
        close("dg", dg[s], want["dg"][s], A["dg"][s], f + K * U32)
        # differences of a segment's sums: far below one rounding in bf16, and
        # in float32 about sqrt(tokens) roundings of their terms
        near("dg", dg[s], want["dg"][s], u(dg.dtype) + 40 * n ** 0.5 * U32 +
             (2.0 ** -16 * n ** 0.5 if work == "bf16" else 0))
    if states:
        close("ds0", d0, want["ds0"], A["ds0"], f)
    else:
        assert d0 is None


@pytest.mark.gpu
def test_backward_of_more_rows_and_heads_than_a_grid_dimension_holds():
    """Every row gets what it gets in a call of its own rows alone, the last ones too."""
    lens = [1] * 2097 + [600, 0, 3]
    q, k, v, g, off, offs, gen = inputs(lens, 16, 32, 8, 8, torch.float32, seed=16)
    s0 = (0.3 * torch.randn((len(lens), 32, 8, 8), generator=gen)).cuda()
    do = torch.randn(v.shape, generator=gen).cuda()
    whole = gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs, initial_state=s0,
                                         dfinal_state=s0)
    at = off[2090]
    part = [x[at:] for x in (do, q, k, v, g)]
    few = gdr.gdr_linear_attention_bwd(*part, offs[2090:] - at, initial_state=s0[2090:],
                                       dfinal_state=s0[2090:])
    for i, (x, y) in enumerate(zip(whole, few)):
        y = y.double().cpu()
        near(i, x[2090:] if i == 4 else x[at:], y, 1e-5)


@pytest.mark.gpu
def test_backward_with_a_shared_decay_and_differences():
    """<grad, d> against the forward's own central differences, float32."""
    do, q, k, v, g, off, offs, s0, ds = bwd_inputs(([90, 20], 1, 2, 32, 32, "f32", True, "head"))
    got = gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs, initial_state=s0, dfinal_state=ds)
    slopes = got[3].sum(0)                      # the tokens share their head's decay

    def loss(q, k, v, slope, s0):
        o, end = gdr.gdr_linear_attention_fwd(q, k, v, slope.expand(q.shape[0], 2), offs,
                                              initial_state=s0, output_final_state=True)
        s = slice(off[0], off[-1])
        return float((o[s].double() * do[s].double()).sum() + (end.double() * ds.double()).sum())

    x = [q.contiguous(), k.contiguous(), v.contiguous(), g[0].clone(), s0]
    size = sum(float(t.double().abs().sum()) for t in (do, ds))
    for i, grad in enumerate([got[0], got[1], got[2], slopes, got[4]]):
        d = torch.randn(x[i].shape, generator=torch.Generator().manual_seed(i)).cuda()
        e = 2.0 ** -7 if i != 3 else 2.0 ** -12
        up, down = (loss(*[t + sgn * e * d if j == i else t for j, t in enumerate(x)])
                    for sgn in (1, -1))
        rows = slice(off[0], off[-1]) if i < 3 else slice(None)
        want = float((grad[rows].double() * d[rows].double()).sum())
        scale = float((grad[rows].double() * d[rows].double()).abs().sum())
        # linear in q, k, v and S_0 (rounding only); quadratic terms in the decays
        most = 40 * size * U32 / e + (1e-3 * scale if i == 3 else 0)
        assert abs((up - down) / (2 * e) - want) <= most, (i, (up - down) / (2 * e), want, most)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [BWD[5], BWD[11]], ids=str)
def test_same_call_same_bits(case):
    do, q, k, v, g, off, offs, s0, ds = bwd_inputs(case)
    call = lambda: gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs, initial_state=s0,  # noqa: E731
                                                dfinal_state=ds)
    s = slice(off[0], off[-1])
    first, second = call(), call()
    for a, b in zip(first[:4], second[:4]):
        assert torch.equal(a[s], b[s])
    assert torch.equal(first[4], second[4])


@pytest.mark.gpu
def test_other_streams():
    do, q, k, v, g, off, offs, s0, ds = bwd_inputs(BWD[11])
    s = slice(off[0], off[-1])
    want = gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs, initial_state=s0, dfinal_state=ds)
    o, end = gdr.gdr_linear_attention_fwd(q, k, v, g, offs, initial_state=s0,
                                          output_final_state=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs, initial_state=s0, dfinal_state=ds,
                                       stream=side)
    o2, end2 = gdr.gdr_linear_attention_fwd(q, k, v, g, offs, initial_state=s0,
                                            output_final_state=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want[:4], got[:4]):
        assert torch.equal(a[s], b[s])
    assert torch.equal(o[s], o2[s]) and torch.equal(end, end2)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [BWD[3], BWD[11]], ids=str)
def test_graphs_replay_to_the_eager_results(case):
    do, q, k, v, g, off, offs, s0, ds = bwd_inputs(case)
    nv, K, V = v.shape[1], q.shape[2], v.shape[2]
    s = slice(off[0], off[-1])
    floats = gdr.gdr_linear_attention_workspace(q.shape[0], len(off) - 1, q.shape[1], nv, K, V, True)
    ws = torch.empty(max(1, floats), device="cuda")
    o, end = torch.empty_like(v).contiguous(), torch.empty_like(s0)
    out = dict(dq=torch.empty(q.shape, dtype=q.dtype, device="cuda"),
               dk=torch.empty(q.shape, dtype=q.dtype, device="cuda"),
               dv=torch.empty(v.shape, dtype=q.dtype, device="cuda"),
               dg=torch.empty(g.shape, dtype=g.dtype, device="cuda"),
               dinitial_state=torch.empty_like(s0))

    def run(stream=None):
        gdr.gdr_linear_attention_fwd(q, k, v, g, offs, initial_state=s0, final_state=end, o=o,
                                     workspace=ws)
        gdr.gdr_linear_attention_bwd(do, q, k, v, g, offs, initial_state=s0, dfinal_state=ds,
                                     workspace=ws, **out)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        v.mul_(0.5 if i % 2 else 1.5)
        run()
        torch.cuda.synchronize()
        want = [x.clone() for x in (o, end, *out.values())]
        for x in (o, end, *out.values()):
            x.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (o, end, *out.values())):
            a, b = (a[s], b[s]) if a.shape[0] == q.shape[0] else (a, b)
            assert torch.equal(a, b)
        torch.ones(1000, device="cuda").sum().item()


@pytest.mark.gpu
def test_index_checks_cover_the_new_entries():
    q, k, v, g, off, offs, gen = inputs([40, 40], 1, 1, 16, 16, torch.float32)
    pool = torch.zeros(2, 1, 16, 16, device="cuda")
    bad = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    was = gdr.gdr_set_debug_checks(True)
    try:
        with pytest.raises(gdr.GdrError, match="used by rows"):
            gdr.gdr_linear_attention_fwd(q, k, v, g, offs, state=pool, slot_idx=bad)
        with pytest.raises(gdr.GdrError, match="used by rows"):
            gdr.gdr_linear_attention_step(q[:2], k[:2], v[:2], g[:2], pool, bad)
        wrong = torch.tensor([0, 90], dtype=torch.int32, device="cuda")
        with pytest.raises(gdr.GdrError, match="past the 80 tokens"):
            gdr.gdr_linear_attention_bwd(q, q, k, v, g, wrong)
    finally:
        gdr.gdr_set_debug_checks(was)


@pytest.mark.gpu
def test_empty_batches():
    z = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    offs = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, end = gdr.gdr_linear_attention_fwd(z(0, 1, 16), z(0, 1, 16), z(0, 2, 16), z(0, 2), offs,
                                          output_final_state=True)
    assert o.shape == (0, 2, 16) and end.shape == (0, 2, 16, 16)
    offs = torch.zeros(3, dtype=torch.int32, device="cuda")  # two rows of no tokens
    s0 = torch.randn(2, 2, 16, 16, device="cuda")
    o, end = gdr.gdr_linear_attention_fwd(z(0, 1, 16), z(0, 1, 16), z(0, 2, 16), z(0, 2), offs,
                                          initial_state=s0, output_final_state=True)
    assert torch.equal(end, s0)
    got = gdr.gdr_linear_attention_bwd(z(0, 2, 16), z(0, 1, 16), z(0, 1, 16), z(0, 2, 16), z(0, 2),
                                       offs, initial_state=s0, dfinal_state=s0)
    near("ds0", got[4], s0.cpu().double(), 4 * U32)
    h, n = gdr.gdr_block_norm(z(0, 64), post_weight=torch.ones(64, device="cuda"))
    assert h.shape == (0, 64) and n is None
    got = gdr.gdr_block_norm_bwd(z(0, 64), None, z(0, 64), None,
                                 post_weight=torch.ones(64, device="cuda"), residual=False)
    assert (got[3] == 0).all()


NORM = [
    # T, D, group, weight length, gate, act, residual, pre, work, weights
    (1, 8, 8, 8, "none", None, True, True, "f32", "f32"),
    (1, 4096, 4096, 4096, "token", "sigmoid", True, True, "bf16", "f32"),
    (3, 64, 16, 16, "token", "silu", False, False, "bf16", "bf16"),
    (5, 768, 96, 96, "token", "silu", False, False, "f32", "f32"),
    (5, 768, 96, 768, "channel", None, True, True, "bf16", "f32"),
    (130, 520, 520, 520, "channel", "sigmoid", True, False, "f32", "f32"),
    (7, 2048, 128, 128, "token", None, True, True, "f32", "f32"),
    (2, 1024, 512, 512, "token", "silu", False, True, "bf16", "bf16"),
    (9, 5120, 5120, 5120, "none", None, True, True, "bf16", "bf16"),
    (2, 16384, 128, 128, "token", "silu", True, True, "bf16", "f32"),
    (2, 10248, 10248, 10248, "token", "silu", True, True, "f32", "f32"),
    (4, 256, 0, 0, "token", "silu", True, True, "bf16", "f32"),       # no post-norm
    (4, 256, 0, 0, "none", None, True, False, "f32", "f32"),
    (1500, 64, 64, 64, "channel", "silu", True, True, "bf16", "f32"),
    (3, 9216, 4608, 4608, "token", "silu", True, True, "f32", "f32"),
]


def norm_inputs(case, seed=9):
    T, D, group, wl, gate, act, res, pre, work, wt = case
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    work, wt = DT[work], DT[wt]
    wide = torch.zeros(T, D + 24, dtype=work, device="cuda")   # rows at another stride
    wide[:, 8:8 + D] = n(T, D).to(work).cuda()
    a = dict(post_weight=(1 + 0.2 * n(wl)).to(wt).cuda() if wl else None, group=group,
             gate={"none": None, "token": n(T, D).to(work).cuda(),
                   "channel": n(D).to(wt).cuda()}[gate], activation=act,
             residual_scale=0.8, pre_weight=(1 + 0.2 * n(D)).to(wt).cuda() if pre else None,
             eps=1e-6)
    x = n(T, D).mul(2).to(work).cuda() if res else None
    return wide[:, 8:8 + D], x, a, n


@pytest.mark.gpu
@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm(case):
    y, x, a, n = norm_inputs(case)
    h, m = gdr.gdr_block_norm(y, residual=x, **a)
    args = (y, a["post_weight"], a["group"], a["gate"], a["activation"], x, 0.8, a["pre_weight"],
            1e-6)
    wh, wn, Ah, An = ref.norm(*args)
    # squares are added along a thread (16) and over a tree, or group / 8 units
    f = (64 + (a["group"] or 0) / 8) * U32
    close("h", h, wh, Ah, f)
    if wn is None:
        assert m is None
    else:
        close("n", m, wn, An, 2 * f)
    if x is not None:                                   # in place on the residual stream
        h2, m2 = gdr.gdr_block_norm(y, residual=x, h=x, **a)
        assert h2 is x and torch.equal(x, h) and (m is None or torch.equal(m, m2))


@pytest.mark.gpu
@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm_backward(case):
    T, D, group, wl, gate, act, res, pre, work, wt = case
    y, x, a, n = norm_inputs(case)
    work = DT[work]
    h = n(T, D).mul(2).to(work).cuda()
    dh, dn = n(T, D).to(work).cuda(), (n(T, D).to(work).cuda() if pre else None)
    got = gdr.gdr_block_norm_bwd(dh, dn, y, h, residual=res, **a)
    again = gdr.gdr_block_norm_bwd(dh, dn, y, h, residual=res, **a)
    want = ref.norm_grads(dh, dn, y, h, a["post_weight"], group, a["gate"], act, x, 0.8,
                          a["pre_weight"], 1e-6)
    f = 2 * (64 + group / 8) * U32
    for name, v, v2 in zip(("dx", "dgate", "dy", "dw1", "dw2"), got, again):
        if v is None:
            assert name == "dx" and not res or name not in want
            continue
        sums = T + D // 8 if v.dim() == 1 else 0
        close(name, v, want[name], want["a" + name], f + sums * U32)
        assert torch.equal(v, v2)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_an_activation_without_a_gate_says_nothing(act):
    y, x, a, n = norm_inputs(NORM[8])
    h, m = gdr.gdr_block_norm(y, residual=x, **a)
    h2, m2 = gdr.gdr_block_norm(y, residual=x, **{**a, "activation": act})
    assert torch.equal(h, h2) and torch.equal(m, m2)
    dh, dn = n(*y.shape).to(y.dtype).cuda(), n(*y.shape).to(y.dtype).cuda()
    got = gdr.gdr_block_norm_bwd(dh, dn, y, h, **a)
    again = gdr.gdr_block_norm_bwd(dh, dn, y, h, **{**a, "activation": act})
    for p, q in zip(got, again):
        assert (p is None and q is None) or torch.equal(p, q)


@pytest.mark.gpu
def test_norm_in_a_graph():
    y, x, a, n = norm_inputs(NORM[6])
    T, D = y.shape
    dh, dn = n(T, D).cuda(), n(T, D).cuda()
    new = lambda t: torch.empty(t.shape, dtype=t.dtype, device="cuda")  # noqa: E731
    h, m = new(y), new(y)
    out = dict(dresidual=new(y), dy=new(y), dgate=new(a["gate"]),
               dpost_weight=new(a["post_weight"]), dpre_weight=new(a["pre_weight"]))
    ws = torch.empty(gdr.gdr_block_norm_workspace(T, D), device="cuda")

    def run():
        gdr.gdr_block_norm(y, residual=x, h=h, n=m, **a)
        gdr.gdr_block_norm_bwd(dh, dn, y, h, workspace=ws, **out, **a)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    every = (h, m, *out.values())
    for i in range(3):
        y.mul_(1.1)
        run()
        torch.cuda.synchronize()
        want = [t.clone() for t in every]
        for t in every:
            t.fill_(2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, every))


@pytest.mark.gpu
def test_example_runs_the_operators_together():
    """examples/linear_attention_block.py: prompt, single tokens and a training
    step.  Two float32 layers whose rows are cut differently: differences of a
    few hundred roundings, 100 u(float32) (K + 64) at most."""
    import importlib.util
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "linear_attention_block.py")
    spec = importlib.util.spec_from_file_location("linear_attention_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    worst, finite = mod.main(["--prompt", "150", "--tokens", "3"])
    assert worst <= 100 * U32 * (64 + 64) and finite
