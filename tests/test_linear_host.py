"""Host side of the linear operators: the descriptor's range."""

import pytest

import moe_expert_layer_sigmoid_amd as mx


@pytest.mark.parametrize("name", ["rows", "N", "K", "groups"])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 3, -2 ** 31 - 1, 2 ** 64])
def test_descriptor_refuses_what_32_bits_do_not_hold(name, value):
    """2^32 + 3 rows would otherwise be 3 rows without a word."""
    with pytest.raises(ValueError, match=name):
        mx.Linear(**{**dict(rows=4, N=16, K=16, groups=1), name: value})


def test_descriptor_keeps_32_bit_values():
    d = mx.Linear(2 ** 31 - 1, -1, -2 ** 31, groups=7)
    assert (d.rows, d.N, d.K, d.groups) == (2 ** 31 - 1, -1, -2 ** 31, 7)
