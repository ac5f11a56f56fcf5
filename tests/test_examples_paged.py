"""The example's pages: the same logits as on its contiguous cache."""
import pytest

from tests.test_examples import load


@pytest.mark.gpu
def test_hybrid_layers_on_pages():
    """16-bit pages hold the same keys and values as the contiguous cache; attention
    on them differs by the rounding of its weights and output, as generation
    and the whole text's pass do (about 16 stored activations, half a step of 2^-8
    each).  4 bits are off by up to half a step, a 14th of the largest of 32 values:
    finite, and of the logits' own size at most."""
    r = load("hybrid_layers").main(30)
    assert r["paged"] <= 16 * 2 ** -8 * r["largest"], r
    assert r["paged_4_bits"] <= r["largest"], r
