"""Workspaces of the token operators: one that was sized for the largest call is enough for every smaller one.

The calls go to addresses that nothing may touch; without a GPU they pass all checks and then fail in the launch
(E_HIP), or with E_CAPACITY where the workspace is too small."""
import ctypes

import pytest
import torch

import exact_bpe_tokenization_amd as tt

CAPACITY, HIP = 5, 6
V1, V2, V3 = 1256, 33024, 131328
MOST = 1 << 21


def _area(i):   # addresses 4 TiB apart: no argument lies on another
    return ctypes.c_void_p((i + 1) << 42)


def _no_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the calls would touch their addresses")


def _never_falls(sizes):
    return all(a <= b for a, b in zip(sizes, sizes[1:]))


LOSS_ROWS = [1, 2, 127, 128, 129, 158, 159, 160, 161, 192, 256, 8192, 1 << 20, (1 << 31) - 1]
LOSS_VOCABS = [1, V1, V2, 65535, 65536, 65537, V3, 200019, MOST]


def test_cross_entropy_sizes_never_fall():
    f = tt.toktier_cross_entropy_workspace_bytes
    for vocab in LOSS_VOCABS:
        assert f(0, vocab) >= 256
        assert _never_falls([f(rows, vocab) for rows in [0] + LOSS_ROWS]), vocab
    for rows in LOSS_ROWS:
        assert _never_falls([f(rows, vocab) for vocab in LOSS_VOCABS]), rows


@pytest.mark.parametrize("most,vocab", [(8192, V3), (160, 65536), (192, MOST), (1 << 20, V3)])
def test_cross_entropy_takes_the_workspace_of_a_larger_call(most, vocab):
    _no_gpu()
    given = tt.toktier_cross_entropy_workspace_bytes(most, vocab)
    for rows in LOSS_ROWS:
        for v in LOSS_VOCABS:
            if rows <= most and v <= vocab:
                assert tt.lib().toktier_cross_entropy(_area(0), 3, rows, v, v, _area(1), _area(2), _area(3), None, 1.0, None, 0,
                                                      _area(4), given, None) == HIP, (rows, v)


TOKENS = [1, 4096, 4097, 5000, 8191, 8192, 16383, 16384, 32767, 32768, 65535, 65536, 131071, 131072, 262143, 262144, 262145,
          524288, 524289, 1 << 20, (1 << 20) + 1, 1 << 26]
VOCABS = [1, 3, 1023, 1024, V1, 2047, 2048, V2, V3, MOST]
DIMS = [1, 7, 8, 64, 512, 513, 1024, 1025, 2048, 4096, 4097]


def test_gradient_sizes_never_fall():
    f = tt.toktier_embed_backward_workspace_bytes
    for dim in DIMS:
        for vocab in VOCABS:
            assert _never_falls([f(n, vocab, dim) for n in TOKENS]), (vocab, dim)
        for n in TOKENS:
            assert _never_falls([f(n, vocab, dim) for vocab in VOCABS]), (n, dim)
    for n in TOKENS:
        assert _never_falls([f(n, V3, dim) for dim in DIMS]), n


def test_gradient_sizes_stay_near_the_tokens():
    """IDs and positions twice, the histograms, partial sums of a chunk of 64 tokens or of 4,096 wavefronts."""
    f = tt.toktier_embed_backward_workspace_bytes
    for n in TOKENS:
        for dim in DIMS:
            assert f(n, V3, dim) <= 16 * n + n * (dim + 8) // 8 + 40_000_000


@pytest.mark.parametrize("most,vocab,dim", [(65536, V3, 64), (32768, V3, 4096), (262145, V3, 512), (1 << 20, MOST, 1025),
                                            (65536, 2048, 513), (4097, V3, 4097)])
def test_gradient_takes_the_workspace_of_a_larger_call(most, vocab, dim):
    _no_gpu()
    given = tt.toktier_embed_backward_workspace_bytes(most, vocab, dim)
    for n in TOKENS + [most - 1, most]:
        for v in VOCABS:
            for d in DIMS:
                if n <= most and v <= vocab and d <= dim:
                    assert tt.lib().toktier_embed_backward(_area(0), 3, d, _area(1), n, 1.0, _area(2), 1, v, d, d, 1, _area(3),
                                                           given, None) == HIP, (n, v, d)
