"""How a call over the paged cache is cut, on the CPU."""
import pytest

from block_sparse_attention_27_b200 import build, dsa


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dsa.load()


@pytest.mark.parametrize("B", [1, 32])
def test_tiles_past_32_bits_are_not_shared_out(lib, B):
    """Equal shares are cut out of the units' tiles in a row, counted in 32 bits: a batch over
    prefixes that could hold more (page tables may name one page many times) takes whole units."""
    def dims(S, pages):
        return dsa.make_dims(S, B, 8, 8, 64, 64, pages, 1, 1 << 20)

    far = 1 << 24  # pages of a prefix of 2^30 tokens, 2^23 tiles
    assert dsa.kv4_launches(dims(1, far), sparse=False) == 2  # 2^26 tiles: shares, and pieces to join
    assert dsa.kv4_launches(dims(31, far), sparse=False) == 2
    assert dsa.kv4_launches(dims(32, far), sparse=False) == 1  # 2^31 tiles
    assert dsa.kv4_launches(dims(140, far), sparse=False) == 1
    assert dsa.kv4_launches(dims(140, 1 << 10), sparse=False) == 2
    assert dsa.window_launches(dims(140, far), 1 << 30, 0) == 1
    assert dsa.window_launches(dims(140, far), 4096, 4) == 2  # a window bounds a unit's tiles
