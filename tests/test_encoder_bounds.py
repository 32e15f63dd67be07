"""Bounds of distances that the binding refuses (no GPU needed): what does not fit the C configuration's 32 bits must not be
cut to what does."""
import pytest

import catalogue_cross_entropy_amd as rece


@pytest.mark.parametrize("bounds", [[(1 << 32) + 1], [1, (1 << 32) + 2], [-(1 << 32) + 5], [0, 1], [1, 1], [5, 4], [1, 4097]])
def test_bounds_out_of_range(bounds):
    for make in (lambda: rece.SequenceAttention(10, 2, 4, 32, bounds=bounds),
                 lambda: rece.LastAttention(2, 10, 4, 32, 5, bounds=bounds)):
        with pytest.raises((ValueError, rece.ReceError)):
            make()


def test_bounds_in_range():
    for bounds in ([], [1], [4096], [1, 2, 4096], list(range(1, 128))):
        assert rece.SequenceAttention(10, 2, 4, 32, bounds=bounds).bounds == bounds
