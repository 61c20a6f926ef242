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
