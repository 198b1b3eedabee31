"""Distillation's workspaces for rows that are split, without a GPU: one sized for the largest call holds every smaller one of
every type."""
import ctypes

import pytest
import torch

import exact_bpe_tokenization_amd as tt

HIP = 6


def _area(i):   # addresses 4 TiB apart: no argument lies on another
    return ctypes.c_void_p((i + 1) << 42)


@pytest.mark.parametrize("n,v,k", [(64, 65536, 20), (128, 131328, 8), (200, 524288, 64), (160, 1 << 21, 1024)])
def test_a_workspace_for_the_largest_call_is_enough(n, v, k):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the calls would touch their addresses")
    given = tt.toktier_distill_workspace_bytes(n, v, k)
    for kind in (1, 2, 3):
        for a in sorted({1, 63, 64, 65, 96, 127, 128, 129, 158, 159, 160, n}):
            for b in sorted({65535, 65536, 131328, 262143, 262144, 524287, 524288, 1 << 20, v}):
                if a <= n and b <= v:
                    for grad in (None, _area(6)):
                        args = (_area(0), kind, a, b, b, _area(1), k, _area(2), k, k, None, 1.0, _area(3), _area(4), None, 1.0, grad, b,
                                _area(5), given, None)
                        assert tt.lib().toktier_distill(*args) == HIP, (kind, a, b)


def test_sizes_never_fall_where_rules_change():
    rows = [1, 63, 64, 65, 128, 129, 159, 160, 1000]
    vocabs = [65535, 65536, 131328, 262143, 262144, 524287, 524288, 786432, 1 << 20, 1 << 21]
    size = {(n, v): tt.toktier_distill_workspace_bytes(n, v, 64) for n in rows for v in vocabs}
    for n in rows:
        line = [size[n, v] for v in vocabs]
        assert line == sorted(line)
    for v in vocabs:
        line = [size[n, v] for n in rows]
        assert line == sorted(line)
