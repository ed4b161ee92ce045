"""Frequency forms outside their range are refused (no GPU)."""
import pytest

import scaled_dot_product_fwd_gb300 as S


@pytest.mark.parametrize("base", [0.5, 1.0])
def test_blended_frequencies_want_a_base_above_one(base):
    """Below 1 the pairs turn faster and faster: those that are to stay would be stretched and the
    others kept."""
    with pytest.raises(ValueError):
        S.rope_frequencies(64, base=base, scaling="yarn", factor=4.0, original_length=4096)
    freq, gain = S.rope_frequencies(64, base=0.5)  # (without it any positive base is one)
    assert freq[0] == 1.0 and gain == 1.0 and freq == sorted(freq)


def test_blended_frequencies_just_above_one():
    own, _ = S.rope_frequencies(64, base=1.5)
    freq, _ = S.rope_frequencies(64, base=1.5, scaling="yarn", factor=4.0, original_length=4096)
    assert freq == own  # every pair turns more than beta_fast times
