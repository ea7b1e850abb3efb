"""Host-side checks of the operators of a block's mixer half at the edges of what may be passed (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from int4_grouped_gemm_router_amd import binding as B


# ------------------------------------------------------------------ int8 projection

def test_int8_needs_no_workspace():
    """0 bytes at every size, from one token and one output to the largest; the binding has none to hand out."""
    n = ctypes.c_size_t(7)
    for N in (1, 64, 2000, 12288, 1 << 18):
        for K in (64, 2048, 65536):
            for T in (0, 1, 4, 5, 64, 500, 4096, 1 << 18, 1 << 30):
                n.value = 7
                assert B.lib().moe_project_int8_workspace_bytes(N, K, T, ctypes.byref(n)) == B.MOE_OK
                assert n.value == 0, (N, K, T)
    assert B.project_int8_workspace(12288, 2048, 4096, device="cpu") is None


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


# ------------------------------------------------------------------ rotary positions

def _inverse_two_pi(bits):
    """2^bits / (2 pi) to the nearest whole number but one, by Machin's formula in whole numbers."""
    one = 1 << (bits + 40)

    def arctan_inverse(n):  # of 1 / n
        term, total, k = one // n, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    return (one << bits) // (2 * pi)


def test_rope_turns_of_fast_pairs_keep_all_their_bits():
    """Frequencies of many turns a position: within one step of 2^-64 turns of the exact fraction, as slow ones are."""
    bits = 256
    inverse = _inverse_two_pi(bits)
    values = [1e-9, 0.1, 0.5, 1.0, -1.0, 3.0, 7.5, -12.25, 100.0, 1e3, -4321.1, 1e6 / 3, 1e9 + 0.7, -2.0 ** 40 - 0.375, 1e15 / 7,
              2.0 ** 60 + 4096, -2.0 ** 61]
    rad = np.array(values)
    out = np.empty(len(values), np.uint64)
    assert B.lib().moe_rope_turns(rad.ctypes.data, len(values), out.ctypes.data) == B.MOE_OK
    for value, got in zip(values, out.tolist()):
        num, den = value.as_integer_ratio()
        # round(value / (2 pi) * 2^64) modulo 2^64
        want = ((num * inverse) // (den << (bits - 65)) + 1) // 2 % (1 << 64)
        off = (got - want) % (1 << 64)
        assert min(off, (1 << 64) - off) <= 1, (value, off)


def test_rope_turns_refuse_what_has_no_fraction_left():
    out = np.empty(2, np.uint64)
    for bad in (2.0 ** 61 * 1.0001, -2.0 ** 62, 1e300):
        rad = np.array([1.0, bad])
        assert B.lib().moe_rope_turns(rad.ctypes.data, 2, out.ctypes.data) == B.MOE_EUNSUPPORTED
        with pytest.raises(B.MoeError):
            B.rope(4, radians=rad, device="cpu")
