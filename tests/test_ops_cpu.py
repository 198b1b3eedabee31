"""Token operators without a GPU: every refusal that toktier.h documents comes back as its status before any
device call (the addresses passed here are host memory that nothing may touch), workspace sizes, the
binding's own checks, and a loud failure where there is no device."""
import ctypes

import numpy as np
import pytest
import torch

import exact_bpe_tokenization_amd as tt

INVALID, CAPACITY = 1, 5
BUF = np.zeros(1 << 20, dtype=np.uint8)
BASE = (BUF.ctypes.data + 255) & ~255


def at(offset):
    return ctypes.c_void_p(BASE + offset)


EMBED = dict(table=at(0), table_type=1, n_vocab=10, dim=8, table_stride=8, ids=at(4096), n_tokens=4, scale=1.0,
             out=at(8192), out_type=1, out_stride=8, stream=None)
EMBED_BACKWARD = dict(grad=at(0), grad_type=3, grad_stride=8, ids=at(4096), n_tokens=4, scale=1.0, table=at(8192),
                      table_type=1, n_vocab=10, dim=8, table_stride=8, accumulate=0, workspace=at(65536),
                      workspace_bytes=1 << 16, stream=None)
LOSS = dict(logits=at(0), type=3, n_rows=4, n_vocab=10, stride=16, targets=at(4096), loss=at(8192), lse=at(12288),
            grad_loss=at(16384), grad_scale=1.0, grad=at(20480), grad_stride=10, workspace=at(65536),
            workspace_bytes=1 << 16, stream=None)
LOSS_BACKWARD = dict(logits=at(0), type=2, n_rows=4, n_vocab=10, stride=10, targets=at(4096), lse=at(12288),
                     grad_loss=None, grad_scale=1.0, grad=at(0), grad_stride=10, stream=None)
SAMPLE = dict(logits=at(0), type=1, n_rows=4, n_vocab=40, stride=40, mask=at(4096), mask_stride=2,
              temperature=at(8192), top_k=at(8448), top_p=at(8704), min_p=at(8960), uniform=at(9216),
              out_ids=at(9472), out_logprobs=at(9728), workspace=at(65536), workspace_bytes=1 << 16, stream=None)

BIG = (1 << 21) + 1
REFUSALS = [
    ("toktier_embed", EMBED, INVALID, [
        dict(table=None), dict(ids=None), dict(out=None), dict(table_type=0), dict(out_type=4), dict(n_vocab=0),
        dict(n_vocab=BIG), dict(dim=0), dict(table_stride=7), dict(out_stride=7), dict(table=at(2)), dict(out=at(8193)),
        dict(ids=at(4097)), dict(n_tokens=0xFFFFFFFF), dict(out=at(0)), dict(out=at(256)), dict(out=at(4096)),
        dict(table_stride=1 << 62), dict(out_stride=1 << 62)]),
    ("toktier_embed_backward", EMBED_BACKWARD, INVALID, [
        dict(grad=None), dict(ids=None), dict(table=None), dict(workspace=None), dict(workspace=at(65537)),
        dict(grad_type=7), dict(table_type=0), dict(n_vocab=0), dict(n_vocab=BIG), dict(dim=0), dict(grad_stride=7),
        dict(table_stride=7), dict(grad=at(1)), dict(table=at(8194)), dict(ids=at(4098)), dict(table=at(0)),
        dict(workspace=at(4096)), dict(workspace=at(8192)), dict(n_tokens=0xFFFFFFFF), dict(table=at(4096))]),
    ("toktier_embed_backward", EMBED_BACKWARD, CAPACITY, [dict(workspace_bytes=255), dict(workspace_bytes=0)]),
    ("toktier_cross_entropy", LOSS, INVALID, [
        dict(logits=None), dict(targets=None), dict(loss=None), dict(lse=None), dict(workspace=None),
        dict(workspace=at(65537)), dict(type=0), dict(type=4), dict(n_vocab=0), dict(n_vocab=BIG), dict(stride=9),
        dict(grad_stride=9), dict(logits=at(1)), dict(grad=at(20481)), dict(targets=at(4097)), dict(loss=at(8194)),
        dict(lse=at(12289)), dict(grad_loss=at(16386)), dict(grad=at(0)), dict(grad=at(32), grad_stride=16),
        dict(grad=at(4096)), dict(grad=at(12288)), dict(grad=at(16384)), dict(n_rows=1 << 31), dict(stride=1 << 62)]),
    ("toktier_cross_entropy", LOSS, CAPACITY, [dict(workspace_bytes=255)]),
    ("toktier_cross_entropy_backward", LOSS_BACKWARD, INVALID, [
        dict(logits=None), dict(targets=None), dict(lse=None), dict(grad=None), dict(type=9), dict(n_vocab=0),
        dict(stride=9), dict(grad_stride=11), dict(grad=at(2)), dict(grad=at(12288)), dict(targets=at(2))]),
    ("toktier_sample", SAMPLE, INVALID, [
        dict(logits=None), dict(uniform=None), dict(out_ids=None), dict(workspace=None), dict(workspace=at(65540)),
        dict(type=0), dict(n_vocab=0), dict(n_vocab=BIG), dict(stride=39), dict(mask_stride=1), dict(mask=at(4097)),
        dict(temperature=at(8193)), dict(top_k=at(8449)), dict(top_p=at(8706)), dict(min_p=at(8961)),
        dict(uniform=at(9217)), dict(out_ids=at(9473)), dict(out_logprobs=at(9730)), dict(out_ids=at(0)),
        dict(out_logprobs=at(4)), dict(out_logprobs=at(9472)), dict(n_rows=1 << 31)]),
    ("toktier_sample", SAMPLE, CAPACITY, [dict(workspace_bytes=255)]),
]


def call(name, base, **changes):
    return getattr(tt.lib(), name)(*{**base, **changes}.values())


@pytest.mark.parametrize("name,base,status,change", [
    pytest.param(n, b, s, c, id=f"{n}-{s}-" + ",".join(f"{k}={getattr(v, 'value', v)}" for k, v in c.items()).replace(str(BASE), ""))
    for n, b, s, cs in REFUSALS for c in cs])
def test_refusals(name, base, status, change):
    assert call(name, base, **change) == status


@pytest.mark.parametrize("name,base,empty", [
    ("toktier_embed", EMBED, dict(n_tokens=0, ids=None, out=None)),
    ("toktier_cross_entropy", LOSS, dict(n_rows=0, logits=None, targets=None, loss=None, lse=None, grad=None)),
    ("toktier_cross_entropy_backward", LOSS_BACKWARD, dict(n_rows=0, logits=None, targets=None, lse=None, grad=None)),
    ("toktier_sample", SAMPLE, dict(n_rows=0, logits=None, uniform=None, out_ids=None)),
    ("toktier_embed_backward", EMBED_BACKWARD, dict(n_tokens=0, grad=None, ids=None, workspace=None, accumulate=1)),
])
def test_nothing_to_do_is_ok(name, base, empty):
    assert call(name, base, **empty) == 0


@pytest.mark.parametrize("name,base", [("toktier_embed", EMBED), ("toktier_embed_backward", EMBED_BACKWARD),
                                       ("toktier_cross_entropy", LOSS), ("toktier_sample", SAMPLE),
                                       ("toktier_cross_entropy_backward", LOSS_BACKWARD)])
def test_fails_loudly_without_gpu(name, base):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert call(name, base) == 6
    assert tt.lib().toktier_last_hip_error() != b""


def test_workspace_bytes():
    f = tt.toktier_embed_backward_workspace_bytes
    assert 0 < f(0, 1, 1) <= f(1, 256, 8) < f(10000, 131328, 1024) < f(1 << 20, 131328, 1024)
    assert tt.toktier_cross_entropy_workspace_bytes(0, 1) > 0
    assert tt.toktier_sample_workspace_bytes(0, 1) > 0
    for bad in (lambda: f(1, 0, 8), lambda: f(1, 10, 0), lambda: f(0xFFFFFFFF, 10, 8), lambda: f(1, BIG, 8),
                lambda: tt.toktier_cross_entropy_workspace_bytes(1, 0),
                lambda: tt.toktier_cross_entropy_workspace_bytes(1 << 31, 8),
                lambda: tt.toktier_sample_workspace_bytes(1, BIG)):
        with pytest.raises(tt.ToktierError) as e:
            bad()
        assert e.value.status == INVALID


def test_binding_refuses_host_tensors():
    x, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    v, ws = torch.zeros(4), torch.zeros(4096, dtype=torch.uint8)
    for f in (lambda: tt.toktier_embed(x, i, x), lambda: tt.toktier_embed_backward(x, i, x, ws),
              lambda: tt.toktier_cross_entropy(x, i, v, v, ws), lambda: tt.toktier_sample(x, v, i, v, ws),
              lambda: tt.toktier_cross_entropy_backward(x, i, v, x)):
        with pytest.raises(tt.ToktierError) as e:
            f()
        assert e.value.status == INVALID


@pytest.mark.parametrize("name,base,change", [
    ("toktier_sample", SAMPLE, dict(out_ids=at(9216))), ("toktier_sample", SAMPLE, dict(out_ids=at(8192))),
    ("toktier_sample", SAMPLE, dict(out_logprobs=at(8448))), ("toktier_sample", SAMPLE, dict(out_logprobs=at(8712))),
    ("toktier_sample", SAMPLE, dict(out_ids=at(8964))), ("toktier_sample", SAMPLE, dict(out_logprobs=at(4096 + 24))),
    ("toktier_cross_entropy", LOSS, dict(loss=at(4096))), ("toktier_cross_entropy", LOSS, dict(lse=at(4104))),
    ("toktier_cross_entropy", LOSS, dict(loss=at(16384))), ("toktier_cross_entropy", LOSS, dict(lse=at(16380))),
    ("toktier_cross_entropy", LOSS, dict(workspace=at(4096))), ("toktier_cross_entropy", LOSS, dict(workspace=at(16384)))])
def test_outputs_on_inputs_are_refused(name, base, change):
    args = {**base, **change}
    assert getattr(tt.lib(), name)(*args.values()) == INVALID
