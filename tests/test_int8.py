"""Products in 8-bit integers without a GPU: what the C entry points and the binding refuse."""
import pytest
import torch

import attention_relation_kl_b200 as rk
from attention_relation_kl_b200 import _abi

FAKE = 1 << 24    # never dereferenced: every case fails its checks or has no work
INV, OK, WS = _abi.RELKL_ERR_INVALID, _abi.RELKL_OK, _abi.RELKL_ERR_WORKSPACE


def _quantize(**kw):
    a = dict(rows=4, K=100, x=FAKE, dtype=0, stride=100, q=2 * FAKE, q_stride=112, scale=3 * FAKE) | kw
    return _abi.lib().relkl_quantize_rows(*a.values(), None)


def _matmul(**kw):
    a = dict(rows=4, cols=8, K=100, q=FAKE, q_stride=112, q_scale=FAKE, w=FAKE, w_stride=112,
             w_scale=FAKE, bias=None, y=2 * FAKE, dtype=0, y_stride=8, ws=FAKE, ws_bytes=256) | kw
    return _abi.lib().relkl_matmul_i8(*a.values(), None)


def _linear(**kw):
    a = dict(rows=40, cols=8, K=100, x=FAKE, x_dtype=0, x_stride=100, w=FAKE, w_stride=112,
             w_scale=FAKE, bias=None, y=2 * FAKE, dtype=0, y_stride=8, scratch=FAKE, nbytes=1 << 20,
             ws=FAKE, ws_bytes=256) | kw
    return _abi.lib().relkl_linear_i8(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(K=0), dict(K=131072), dict(x=None), dict(x=FAKE + 1), dict(dtype=3),
    dict(dtype=1, x=FAKE + 2), dict(stride=99), dict(stride=1 << 60), dict(q=None), dict(q=FAKE + 8),
    dict(q_stride=104), dict(q_stride=96), dict(scale=None), dict(scale=FAKE + 2),
])
def test_quantize_refusals(bad):
    assert _quantize(**bad) == INV


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(cols=-1), dict(K=0), dict(K=131072), dict(q=None), dict(q=FAKE + 4),
    dict(q_stride=100), dict(q_stride=96), dict(w=None), dict(w=FAKE + 1), dict(w_stride=101),
    dict(q_scale=None), dict(w_scale=None), dict(q_scale=FAKE + 1), dict(bias=FAKE + 2), dict(y=None),
    dict(y=FAKE + 1), dict(dtype=2), dict(dtype=1, y=FAKE + 2), dict(y_stride=7),
])
def test_product_refusals(bad):
    assert _matmul(**bad) == INV
    for theirs in ("q", "q_stride", "q_scale"):
        bad.pop(theirs, None)
    if bad:
        assert _linear(**bad) == INV


def test_linear_refusals():
    for bad in (dict(x=None), dict(x=FAKE + 1), dict(x_dtype=9), dict(x_dtype=1, x=FAKE + 2), dict(x_stride=99)):
        assert _linear(**bad) == INV
    for bad in (dict(ws=None), dict(ws_bytes=10), dict(ws=FAKE + 16), dict(scratch=None),
                dict(scratch=FAKE + 8), dict(nbytes=40 * 112 + 40 * 4 - 1)):
        assert _linear(**bad) == WS
    assert _matmul(ws=None) == WS


def test_no_rows_or_channels_are_no_ops():
    assert _quantize(rows=0, x=None, q=None, scale=None) == OK
    for empty in (dict(rows=0), dict(cols=0)):
        assert _matmul(q=None, w=None, y=None, ws=None, **empty) == OK
        assert _linear(x=None, w=None, y=None, scratch=None, ws=None, **empty) == OK


def test_scratch_sizes():
    b = _abi.lib().relkl_linear_i8_bytes
    assert b(1, 4096) == 0 and b(4, 4096) == 0          # one kernel, no scratch
    assert b(5, 4096) == 5 * 4096 + 20 and b(40, 100) == 40 * 112 + 160
    assert b(2, 131071) == 2 * 131072 + 8               # codes too large for shared memory
    assert b(-1, 10) == 0 and b(100, 0) == 0


def test_binding_checks_before_the_call():
    x, q = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8)
    s = torch.ones(4)
    for call in (lambda: rk.relkl_quantize_rows(x), lambda: rk.relkl_linear_i8(x, q, s),
                 lambda: rk.relkl_matmul_i8(q, s, q, s)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
