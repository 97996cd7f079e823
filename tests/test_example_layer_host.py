"""The example's decoder layer: its bookkeeping of sequences (no GPU)."""

import pytest

from examples.decode_layer import Layer
from synthetic import CONFIGS


def test_sequences_longer_than_their_pages_are_refused():
    layer = Layer(CONFIGS["c1"], 4, 4, 20, 2, device="cpu")   # two pages of 16 a sequence
    b = layer.batch([32, 5])
    assert b["ctx"].tolist() == [32, 5] and b["table"].tolist() == [[0, 1], [2, 3]]
    with pytest.raises(ValueError):
        layer.batch([1, 1])
    assert layer.lengths == [32, 5]
    assert layer.batch([0, 27])["ctx"].tolist() == [32, 32]
