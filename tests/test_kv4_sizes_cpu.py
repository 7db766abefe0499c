"""Attention over a 4-bit cache: what the host works out for sizes at their ends."""
import pytest

from structured_rotations_amd import kv4


@pytest.mark.parametrize("sequences", [5, 1 << 23, (1 << 24) - 1000, (1 << 24) - 1, 1 << 24])
@pytest.mark.parametrize("heads", [1, 64])
@pytest.mark.parametrize("tokens", [1, 40])
def test_workspace_of_tables_of_any_width(tokens, heads, sequences):
    """Few rows are cut into as many parts as the chip has room for, and no more
    however long the sequences may be."""
    if sequences * heads > 1 << 30:
        pytest.skip("beyond what a call may have")
    need = [kv4.harp_kv4_attention_workspace(tokens, 2 * heads, heads, 128, 1 << 20, sequences, 1 << w) for w in range(5, 25)]
    assert need[0] > 0 and need == need[:1] * len(need)
    # a tile's rows of two slots for each of 256 compute units' three workgroups
    rows = 16 if 2 * tokens <= 16 * sequences else 32
    assert need[0] == 4 * (2 * 768 * rows * (128 + 2) + 2 * tokens * 2 * heads)
