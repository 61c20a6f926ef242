"""What the binding hands to the library, on the CPU: a call's log-sum-exp output, integers past 32 bits,
frequencies."""
import math

import pytest
import torch

from block_sparse_attention_27_b200 import build, dsa


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dsa.load()


def test_log_sum_exp_output_is_the_calls_own():
    """Without the argument none is written, whatever address the caller's dims still hold."""
    dims = dsa.make_dims(1, 2, 2, 1, 64, 16, 4, 1, 4)
    assert dsa._with_lse_out(dims, None, 0) is dims
    dims.lse_out = 1 << 20
    assert dsa._with_lse_out(dims, None, 0).lse_out is None and dims.lse_out == 1 << 20
    with pytest.raises(TypeError):
        dsa._with_lse_out(dims, torch.zeros(1, 2, 2), 0)


@pytest.mark.parametrize("window,sinks", [(-(2 ** 32) + 64, 0), (-(2 ** 40), 0), (64, -(2 ** 32)), (64, -(2 ** 32) + 4), (0, 0), (-1, 0),
                                          (64, -1)])
def test_integers_below_32_bits_are_refused(lib, window, sinks):
    dims = dsa.make_dims(1, 2, 2, 1, 64, 16, 4, 1, 4)
    with pytest.raises(dsa.DsaError) as e:
        dsa.window_launches(dims, window, sinks)
    assert e.value.code == dsa.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("rot,base,n0", [(128, 1e4, 131072), (64, 1e4, 262144), (128, 1e4, 4096), (128, 1e6, 32768), (64, 5e5, 8192),
                                         (8, 100.0, 4096)])
def test_yarn_ramp(rot, base, n0):
    """Against the method's definition, also where every pair turns more than once within n0: there the
    ramp ends behind the last pair, which is stretched in part only."""
    f = 4.0
    got, scale = dsa.rope_inv_freq(rot, base, scaling=("yarn", f, n0), device="cpu")
    turns = [n0 * base ** (-2 * i / rot) / (2 * math.pi) for i in range(rot // 2)]

    def at(t):  # the pair index, not whole, that turns t times
        return rot / 2 * math.log(n0 / (2 * math.pi * t)) / math.log(base)

    lo, hi = max(0, math.floor(at(32))), min(rot - 1, math.ceil(at(1)))
    for i, x in enumerate(got.tolist()):
        ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
        want = base ** (-2 * i / rot) * (1 - ramp + ramp / f)
        assert abs(x - want) <= 2.0 ** -23 * want, (i, x, want)  # one rounding to fp32, and 64-bit arithmetic
        if turns[i] > 32 and hi > lo:
            assert ramp == 0
        if 1 < turns[i]:
            assert ramp < 1 or hi - lo < 1
    assert scale == 0.1 * math.log(f) + 1
