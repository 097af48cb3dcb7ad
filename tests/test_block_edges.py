"""Linear attention and the fused norms where their calls border on something
else.  Error bounds as in test_block_ops.py."""
import pytest
import torch

import gated_delta_rule_loop_amd as gdr
from tests import block_ref as ref
from tests.test_block_ops import BWD, DT, U32, bwd_inputs, inputs, near


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
