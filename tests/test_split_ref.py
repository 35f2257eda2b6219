"""The bounds of the tests of joined splits tell a plain form that loses a stretch of keys, or counts one twice, from
one that does not (64 bits, on the CPU)."""
import pytest
import torch

from tests.split_ref import STRETCH, bound, keys_and_values, off, result


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("even", [True, False])
@pytest.mark.parametrize("length", [700, 5000, 20011, 40000])
def test_a_lost_or_doubled_stretch_is_told(dt, even, length):
    gen = torch.Generator().manual_seed(length)
    scores, channel = keys_and_values(length, gen, even)
    for factor in (1.0, -0.5):
        one = torch.ones(length, dtype=torch.float64)
        want, rel = result(scores, channel, factor, one), bound(length, dt, even)
        assert want.min() >= 0 and torch.isfinite(want).all()
        # rounded as the kernel rounds it, the right result is told right
        assert not off(want.to(dt).double(), want, rel)
        for count in (0.0, 2.0):
            for first in range(0, length - STRETCH + 1, STRETCH * (1 + length // 3000)):
                planted = one.clone()
                planted[first:first + STRETCH] = count
                assert off(result(scores, channel, factor, planted), want, rel), (factor, count, first)
        # a split is several stretches; one that takes part with the weights of another maximum
        planted = one.clone()
        planted[length // 2:length // 2 + 160] *= 0.5
        assert off(result(scores, channel, factor, planted), want, rel)
