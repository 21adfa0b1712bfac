"""Rotary positions without a GPU: argument checks of the C entry point and of the
binding, and the scaled frequencies against their formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_relation_kl_b200 as rk
from attention_relation_kl_b200 import _abi, ops

FAKE = 0x100000   # never dereferenced: every case fails its checks or has no work


def _plan(**kw):
    p = _abi.relkl_rotary_plan()
    p.B, p.N, p.d, p.rot = 2, 8, 64, 64
    p.x_dtype = p.y_dtype = _abi.RELKL_BF16
    p.mscale, p.pos_scale, p.inv_freq = 1.0, 1.0, FAKE
    for k, v in kw.items():
        if k == "pos_stride":
            p.pos_stride[:] = v
        else:
            setattr(p, k, v)
    return p


def _tensor(x=FAKE, y=16 * FAKE, H=2, apply=1, xs=(1024, 512, 64), ys=(1024, 512, 64)):
    t = _abi.relkl_rotary_tensor()
    t.x, t.y, t.H, t.apply = x, y, H, apply
    t.x_stride[:], t.y_stride[:] = xs, ys
    return t


def _call(plan, *tensors, n=None):
    arr = (_abi.relkl_rotary_tensor * max(len(tensors), 1))(*tensors)
    return _abi.lib().relkl_rotary(len(tensors) if n is None else n, arr, ctypes.byref(plan), None)


@pytest.mark.parametrize("plan", [
    dict(rot=63), dict(rot=66), dict(rot=-2), dict(d=0), dict(d=514), dict(B=-1), dict(N=-1),
    dict(x_dtype=2), dict(y_dtype=-1), dict(interleaved=2), dict(inverse=-1),
    dict(mscale=float("nan")), dict(mscale=float("inf")), dict(pos_scale=float("inf")),
    dict(pos_offset=float("nan")), dict(inv_freq=None), dict(inv_freq=FAKE + 4),
    dict(pos_bytes=4), dict(positions=FAKE, pos_bytes=0), dict(positions=FAKE, pos_bytes=2),
    dict(positions=FAKE + 2, pos_bytes=4), dict(positions=FAKE + 4, pos_bytes=8),
    dict(positions=FAKE, pos_bytes=4, pos_stride=(-1, 1)),
])
def test_bad_plans_are_refused(plan):
    assert _call(_plan(**plan), _tensor()) == _abi.RELKL_ERR_INVALID


@pytest.mark.parametrize("tensor", [
    dict(x=None), dict(y=None), dict(x=FAKE + 1), dict(y=FAKE + 1), dict(H=-1), dict(apply=2),
    dict(xs=(-1024, 512, 64)), dict(ys=(1024, 512, -64)),
    dict(ys=(0, 512, 64)),            # the batches of y overlap
    dict(ys=(1024, 512, 63)),         # the tokens of y overlap
    dict(ys=(512, 512, 64)),
    dict(xs=(1 << 60, 512, 64)),      # offsets past any address
    dict(y=FAKE + 64),                # y begins inside x
    dict(y=FAKE, ys=(1024, 64, 128)),  # x and y are one buffer, in another layout
])
def test_bad_tensors_are_refused(tensor):
    assert _call(_plan(), _tensor(**tensor)) == _abi.RELKL_ERR_INVALID


def test_counts_null_arguments_and_crossing_tensors_are_refused():
    inv = _abi.RELKL_ERR_INVALID
    lib = _abi.lib()
    plan = _plan()
    assert _call(plan, n=0) == inv
    assert _call(plan, *[_tensor()] * 4) == inv
    assert lib.relkl_rotary(1, None, ctypes.byref(plan), None) == inv
    assert lib.relkl_rotary(1, (_abi.relkl_rotary_tensor * 1)(_tensor()), None, None) == inv
    # one tensor's output begins inside another's input
    assert _call(plan, _tensor(), _tensor(x=2 * FAKE, y=FAKE + 512)) == inv


X, Y, ST = FAKE, 16 * FAKE, (1024, 512, 64)


@pytest.mark.parametrize("tensors", [
    [dict(y=X), dict(y=X)],                              # one tensor in place twice
    [dict(y=X), dict(y=X, apply=0)],                     # turned, and moved onto itself
    [dict(y=X), dict(x=X + 128, y=X + 128)],             # in place, a row further
    [dict(y=X), dict(x=X + 2 * 1024, y=X + 2 * 1024)],   # in place, a head further
    [dict(), dict(x=2 * X)],                             # two inputs, one output
    [dict(), dict(x=2 * X, y=Y + 2)],                    # ... an element further
    [dict(), dict(x=2 * X, y=Y + 2 * 2047)],             # the last element of the one, the first of the other
    [dict(), dict(x=2 * X, y=3 * Y), dict(x=4 * X)],     # the first and the third
    [dict(ys=(4096, 64, 512)), dict(x=2 * X, ys=(4096, 64, 512), y=Y + 2 * 63)],   # beside, one short
    [dict(), dict(x=2 * X, H=1, ys=(2048, 0, 256), y=Y + 2 * 64)],    # at other strides
])
def test_outputs_with_an_element_in_common_are_refused(tensors):
    assert _call(_plan(), *[_tensor(**t) for t in tensors]) == _abi.RELKL_ERR_INVALID


def test_no_work_is_a_no_op():
    assert _call(_plan(B=0), _tensor(x=None, y=None)) == _abi.RELKL_OK
    assert _call(_plan(N=0), _tensor(x=None, y=None)) == _abi.RELKL_OK
    assert _call(_plan(), _tensor(x=None, y=None, H=0)) == _abi.RELKL_OK


def test_binding_checks_before_the_call():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rk.relkl_rotary(x, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="1 to 3"):
        rk.relkl_rotary_qkv([], torch.zeros(32, dtype=torch.float64))
    with pytest.raises(TypeError, match="tensors"):
        rk.relkl_rotary_qkv([1], torch.zeros(32, dtype=torch.float64))
    with pytest.raises(TypeError):
        rk.relkl_rotary_qkv(x, None)


def test_frequencies_follow_their_formulas():
    r, base, s, L = 64, 1e4, 8.0, 4096
    i = np.arange(r // 2)
    f = base ** (-2.0 * i / r)
    get = lambda *a, **k: rk.rotary_freqs(r, base, *a, device="cpu", **k)  # noqa: E731
    assert np.allclose(get().inv_freq.numpy(), f, rtol=1e-15)
    assert np.allclose(get("linear", s).inv_freq.numpy(), f / s, rtol=1e-15)
    # the slowest pair of the enlarged base is exactly factor times slower, the fastest unchanged
    ntk = get("ntk", s).inv_freq.numpy()
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], f[-1] / s, rel_tol=1e-12)
    yarn = get("yarn", s, original_length=L)
    turns = L * f / (2 * np.pi)
    y = yarn.inv_freq.numpy()
    # numpy's and torch's powers are each within an ulp, so never more than 2^-51 apart
    assert np.allclose(y[turns > 40], f[turns > 40], rtol=2.0 ** -51, atol=0)
    assert np.allclose(y[turns < 0.5], f[turns < 0.5] / s, rtol=1e-15)
    assert np.all(np.diff(y) < 0) and math.isclose(yarn.mscale, 0.1 * math.log(s) + 1.0)
    bands = get("bands", s, original_length=L, high_turns=4.0)
    b = bands.inv_freq.numpy()
    assert bands.mscale == 1.0
    assert np.allclose(b[turns >= 4], f[turns >= 4], rtol=2.0 ** -51, atol=0)
    assert np.allclose(b[turns <= 1], f[turns <= 1] / s, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    keep = (turns[mid] - 1) / 3
    assert np.allclose(b[mid], f[mid] * (keep + (1 - keep) / s), rtol=1e-14)
    assert rk.rotary_freqs(0, device="cpu").inv_freq.numel() == 0


@pytest.mark.parametrize("args", [(63,), (-2,), (64, 1.0), (64, 1e4, "linear", 0.0),
                                  (64, float("nan")), (64, 1e4, "other"), (2, 1e4, "ntk", 2.0)])
def test_bad_frequencies_are_refused(args):
    with pytest.raises(ValueError):
        rk.rotary_freqs(*args, device="cpu")


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0

    with pytest.raises(ValueError, match="stream is on cuda:1"):
        ops._on(torch.device("cuda", 0), Stream())
    ops._on(torch.device("cuda", 1), Stream())       # entered by no one


def test_turns_that_bands_and_yarn_take_without_being_given():
    get = lambda *a, **k: rk.rotary_freqs(128, 5e5, *a, original_length=8192, device="cpu", **k)  # noqa: E731
    for kind, usual in (("bands", 4.0), ("yarn", 32.0)):
        assert torch.equal(get(kind, 8.0).inv_freq, get(kind, 8.0, high_turns=usual).inv_freq)
    # the published frequencies for bands: wavelengths from a quarter of the length to all of it
    f = 5e5 ** (-2.0 * np.arange(64) / 128)
    wave = 2 * np.pi / f
    smooth = (8192 / wave - 1.0) / (4.0 - 1.0)
    want = np.where(wave < 8192 / 4, f, np.where(wave > 8192, f / 8, (1 - smooth) * f / 8 + smooth * f))
    assert np.allclose(get("bands", 8.0).inv_freq.numpy(), want, rtol=1e-14, atol=0)
