"""Linear attention and the fused norms where their calls border on something
else."""
import pytest
import torch

import gated_delta_rule_loop_amd as gdr
from tests.test_block_ops import BWD, bwd_inputs


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
