"""Scalings of rotary frequencies that have no meaning are refused."""

import math

import pytest

import bwd_packed_varlen_gb300 as ta


@pytest.mark.parametrize("bad", [dict(beta_fast=1.0, beta_slow=32.0), dict(beta_fast=2.0, beta_slow=2.0),
                                 dict(beta_fast=math.nan), dict(original_length=0), dict(original_length=-4096),
                                 dict(factor=math.inf), dict(factor=math.nan), dict(base=math.inf), dict(base=0.0)])
def test_refused(bad):
    """A ramp that runs backwards (it divided what it should keep) or over nothing, and values
    that make angles of zero or NaN."""
    with pytest.raises(ValueError):
        ta.rope_frequencies(64, scaling="yarn", **{"factor": 8.0, **bad}, device="cpu")
