"""What the Python binding takes for pointers and streams (no GPU)."""

import enum

import pytest

from quantized_rank_fine_amd import qlora as q


class Address(int):
    """A device address with a type of its own."""


class Place(enum.IntEnum):
    START = 4096


@pytest.mark.parametrize("p", [4096, Address(4096), Place.START])
def test_pointers_as_integers(p):
    """Any int is an address, of a subclass too."""
    assert q._ptr(p) == 4096
    assert q._ptr(None) is None
    with pytest.raises(q.QloraError) as e:               # refused by the library itself
        q.qlora_dropout(p, 64, None, 0, 4, 64, q.BF16, 1.0, 0, 0, p, 64, stream=0)
    assert e.value.status == 7
