"""Host-side checks of the operators of a block's mixer half at the edges of what may be passed (no GPU needed)."""
import pytest
import torch

from int4_grouped_gemm_router_amd import binding as B


# ------------------------------------------------------------------ linear attention

@pytest.mark.parametrize("step", [False, True], ids=["sequences", "step"])
@pytest.mark.parametrize("which", ["in", "out"])
def test_linear_states_without_slots_have_one_for_each_sequence(step, which):
    """A pool of fewer states than sequences needs slots: without them the last sequences' states would be lost."""
    l, n = B.linear_attention(2, 4, 64, 32), 3
    q, k = (torch.zeros(n, 2, 64, dtype=torch.bfloat16) for _ in range(2))
    v, o = (torch.zeros(n, 4, 32, dtype=torch.bfloat16) for _ in range(2))
    g, cu = torch.zeros(n, 4), torch.arange(n + 1, dtype=torch.int32)

    def call(states, slots=None):
        kw = {f"state_{which}": torch.zeros(states, 4, 64, 32), f"slots_{which}": slots}
        if step:
            B.moe_linear_attention_step(l, q, k, v, g, o, n, **kw)
        else:
            B.moe_linear_attention(l, q, k, v, g, o, cu, n, **kw)
    with pytest.raises(ValueError, match=f"state_{which}: .* slots"):
        call(n - 1)
    slots = torch.zeros(n, dtype=torch.int32)
    for ok in (dict(states=n), dict(states=n + 4), dict(states=1, slots=slots)):
        with pytest.raises(ValueError, match="tensors on a GPU"):    # every check passes; there is no CPU path
            call(**ok)
