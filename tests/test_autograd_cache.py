"""Caches of a caller's own, without a GPU: what the differentiable products ask
of them."""

import pytest

from mxfp8_block_scaled_06_amd import autograd


class Kept(autograd.WeightCache):
    """A cache written for MXFP8 weights alone."""

    def get(self, W, as_experts=None):
        return ("kept", W)


class Both(autograd.WeightCache):
    def get(self, W, as_experts=None, weight_format="mxfp8"):
        return (weight_format, W)


def test_a_cache_of_mxfp8_weights_is_asked_as_it_always_was():
    W = object()
    assert autograd._weights_for(W, None, Kept(), "mxfp8") == ("kept", W)
    assert autograd._weights_for(W, None, Both(), "mxfp8") == ("mxfp8", W)
    assert autograd._weights_for(W, None, Both(), "mxfp4") == ("mxfp4", W)
    with pytest.raises(TypeError):
        autograd._weights_for(W, None, Kept(), "mxfp4")
    with pytest.raises(ValueError, match="weight_format"):
        autograd._weights_for(W, None, Kept(), "mxfp6")
