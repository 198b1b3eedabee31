"""Sizes at the ends of what the token operators take; refusals come before any device work (the addresses are never touched)."""
import ctypes

import pytest
import torch

import exact_bpe_tokenization_amd as tt

INVALID, HIP = 1, 6


def _area(i):   # addresses 4 TiB apart
    return ctypes.c_void_p((i + 1) << 42)


def _sample(rows, mask_stride, out):
    return tt.lib().toktier_sample(_area(0), 1, rows, 40, 40, _area(1), mask_stride, None, None, None, None, _area(2), out, None,
                                   _area(6), 256, None)


@pytest.mark.parametrize("rows,stride", [((1 << 24) + 1, 1 << 40), (1 << 20, 1 << 30), ((1 << 31) - 1, 1 << 33), (2, 1 << 62)])
def test_masks_beyond_the_address_space_are_refused(rows, stride):
    assert _sample(rows, stride, _area(4)) == INVALID
    assert _sample(rows, stride, ctypes.c_void_p(_area(1).value + 4096)) == INVALID


def test_masks_of_many_rows_are_taken():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the call would touch its addresses")
    for rows, stride in ((1 << 24, 2), (1 << 20, 1 << 16), (1, 1 << 40)):
        assert _sample(rows, stride, _area(4)) == HIP
