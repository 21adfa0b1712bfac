"""AdamW and the gradient norm without a GPU: what the C entry points and the binding refuse."""
import ctypes

import pytest
import torch

import attention_relation_kl_b200 as rk
from attention_relation_kl_b200 import _abi, optim

FAKE = 1 << 24    # never dereferenced: every case fails its checks or has no work
INV = _abi.RELKL_ERR_INVALID


def _tensor(bits=32, at=FAKE, **kw):
    t = _abi.relkl_adamw_tensor()
    t.grad, t.param, t.copy, t.m, t.v = (at + k * FAKE for k in range(5))
    if bits == 8:
        t.m_scale, t.v_scale = at + 5 * FAKE, at + 6 * FAKE
    t.n, t.grad_dtype, t.param_dtype = 1000, _abi.RELKL_FP32, _abi.RELKL_FP32
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _plan(bits=32, **kw):
    p = _abi.relkl_adamw_plan()
    p.state_bits, p.lr, p.beta1, p.beta2, p.eps, p.step = bits, 1e-3, 0.9, 0.999, 1e-8, 1
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _call(plan, *tensors):
    arr = (_abi.relkl_adamw_tensor * max(1, len(tensors)))(*tensors)
    return _abi.lib().relkl_adamw(len(tensors), arr, ctypes.byref(plan), None)


@pytest.mark.parametrize("plan", [
    dict(state_bits=16), dict(reserved=1), dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0),
    dict(beta1=-0.1), dict(beta2=float("nan")), dict(eps=-1e-8), dict(eps=float("inf")),
    dict(step=0), dict(lr_dev=FAKE + 2), dict(step_dev=FAKE + 4), dict(grad_scale=FAKE + 1),
])
def test_bad_plans_are_refused(plan):
    assert _call(_plan(**plan), _tensor()) == INV


@pytest.mark.parametrize("bits,tensor", [
    (32, dict(grad=None)), (32, dict(param=None)), (32, dict(m=None)), (32, dict(v=None)),
    (32, dict(n=-1)), (32, dict(reserved=1)), (32, dict(grad_dtype=2)), (32, dict(param_dtype=-1)),
    (32, dict(weight_decay=-0.1)), (32, dict(weight_decay=float("nan"))),
    (32, dict(grad=FAKE + 2)), (32, dict(m=3 * FAKE + 2)), (32, dict(copy=3 * FAKE + 1)),
    (32, dict(m_scale=9 * FAKE)), (32, dict(v_scale=9 * FAKE)),
    (8, dict(m_scale=None)), (8, dict(v_scale=None)), (8, dict(v_scale=FAKE * 7 + 2)),
    # arrays that overlap one that is written
    (32, dict(param=FAKE)), (32, dict(m=FAKE + 3996)), (32, dict(v=4 * FAKE)),
    (32, dict(copy=2 * FAKE)), (8, dict(v=4 * FAKE + 999)), (8, dict(m_scale=6 * FAKE + 12, v_scale=6 * FAKE)),
])
def test_bad_tensors_are_refused(bits, tensor):
    assert _call(_plan(bits), _tensor(bits, **tensor)) == INV


@pytest.mark.parametrize("bits,eps", [(8, 2.0 ** -127), (8, 1e-40), (8, 1e-45), (8, 1e-60), (32, 1e-60)])
def test_an_eps_that_the_kernel_would_take_for_zero_is_refused(bits, eps):
    assert _call(_plan(bits, eps=eps), _tensor(bits)) == INV


def test_the_same_tensor_twice_is_refused():
    t, u = _tensor(), _tensor(at=16 * FAKE)
    assert _call(_plan(), t, u, t) == INV
    u.param = t.param
    assert _call(_plan(), t, u) == INV
    u.param = t.param + 4 * t.n - 4          # one element in common
    assert _call(_plan(), t, u) == INV


def test_checks_by_themselves():
    lib = _abi.lib()

    def refused(plan, *tensors):
        return lib.relkl_adamw_check(len(tensors), (_abi.relkl_adamw_tensor * max(1, len(tensors)))(*tensors),
                                     ctypes.byref(plan))

    # taken, on the host: nothing is launched
    assert refused(_plan(), _tensor(), _tensor(at=16 * FAKE)) == _abi.RELKL_OK
    assert refused(_plan(8), _tensor(8), _tensor(8, at=16 * FAKE, grad=FAKE)) == _abi.RELKL_OK
    assert refused(_plan()) == _abi.RELKL_OK
    for plan, tensors in [(_plan(step=0), [_tensor()]), (_plan(), [_tensor(), _tensor()]),
                          (_plan(8, eps=1e-40), [_tensor(8)]), (_plan(8), [_tensor()]),
                          (_plan(), [_tensor(), _tensor(at=16 * FAKE, weight_decay=-1.0)])]:
        assert refused(plan, *tensors) == INV
    assert lib.relkl_adamw_check(1, None, ctypes.byref(_plan())) == INV
    assert lib.relkl_adamw_check(0, None, None) == INV


def test_nothing_to_do():
    assert _call(_plan()) == _abi.RELKL_OK
    assert _call(_plan(), _tensor(n=0, grad=None, param=None, m=None, v=None)) == _abi.RELKL_OK
    assert _abi.lib().relkl_adamw(-1, None, ctypes.byref(_plan()), None) == INV
    assert _abi.lib().relkl_adamw(1, None, ctypes.byref(_plan()), None) == INV
    assert _abi.lib().relkl_adamw(0, None, None, None) == INV


def test_norm_refusals():
    lib = _abi.lib()
    need = lib.relkl_grad_norm_bytes(3)

    def call(n=1, max_norm=1.0, out=FAKE, scratch=FAKE, nbytes=need, **kw):
        t = _abi.relkl_norm_tensor()
        t.grad, t.n, t.dtype = FAKE, 100, _abi.RELKL_FP32
        for k, v in kw.items():
            setattr(t, k, v)
        return lib.relkl_grad_norm(n, (_abi.relkl_norm_tensor * 3)(t, t, t), max_norm, out, scratch,
                                   nbytes, None)

    for bad in (dict(n=-1), dict(max_norm=0.0), dict(max_norm=float("nan")), dict(out=None),
                dict(out=FAKE + 2), dict(grad=None), dict(grad=FAKE + 2), dict(dtype=5),
                dict(reserved=1)):
        assert call(**bad) == INV, bad
    for bad in (dict(scratch=None), dict(scratch=FAKE + 4), dict(nbytes=need - 1)):
        assert call(**bad) == _abi.RELKL_ERR_WORKSPACE, bad
    assert lib.relkl_grad_norm_bytes(1000) > need >= 8


def test_binding_packs_the_plan():
    assert optim._PLAN.size == ctypes.sizeof(_abi.relkl_adamw_plan)
    p = _abi.relkl_adamw_plan.from_buffer_copy(optim._PLAN.pack(8, 0, 1.0, 2.0, 3.0, 4.0, 5, 6, 7, 8))
    assert (p.lr, p.eps, p.step, p.lr_dev, p.grad_scale) == (1.0, 4.0, 5, 6, 8)


def test_binding_checks_before_the_call():
    p = [torch.zeros(4)]
    s = [rk.adamw_state(p[0])]
    with pytest.raises(ValueError, match="CUDA"):
        rk.relkl_adamw(p, p, s, lr=1e-3, step=1)
    with pytest.raises(ValueError, match="one entry"):
        rk.relkl_adamw(p, [], s, lr=1e-3, step=1)
    with pytest.raises(ValueError, match="weight_decay"):
        rk.relkl_adamw(p, p, s, lr=1e-3, step=1, weight_decay=[0.1, 0.1])
    for bad in ((1, p, s), (p, [None], s), (p, p, [None]), (p, p, [(p[0], p[0])])):
        with pytest.raises((TypeError, ValueError)):
            rk.relkl_adamw(*bad, lr=1e-3, step=1)
    with pytest.raises(ValueError, match="CUDA"):
        rk.relkl_grad_norm(p)
    with pytest.raises(ValueError, match="bits"):
        rk.adamw_state(p[0], 16)
    rk.relkl_adamw([], [], [], lr=1e-3, step=1)
    s8 = rk.adamw_state(torch.zeros(3, 100), 8)
    assert s8.m.dtype == torch.float8_e4m3fn and s8.m.shape == (3, 100) and s8.m_scale.shape == (2,)


def test_optimizer_state_round_trip_on_the_host():
    p = [torch.zeros(300), torch.zeros(2, 2)]
    a, b = (rk.AdamW(p, state_bits=8) for _ in range(2))
    for x in a.state:
        x.m.view(torch.uint8).random_(0, 100)
        x.v_scale.normal_()
    a.steps = 7
    b.load_state_dict(a.state_dict())
    assert b.steps == 7
    for x, y in zip(a.state, b.state):
        assert torch.equal(x.m.view(torch.uint8), y.m.view(torch.uint8))
        assert torch.equal(x.v_scale, y.v_scale)
    with pytest.raises(ValueError):
        b.load_state_dict(rk.AdamW(p, state_bits=32).state_dict())
    with pytest.raises(ValueError):
        b.load_state_dict(rk.AdamW(p[:1], state_bits=8).state_dict())
    with pytest.raises(ValueError):
        a.step([None])
    assert a.step() is None and a.steps == 7      # no gradient, no step


def test_counts_of_each_parameter():
    p = [torch.zeros(300), torch.zeros(2, 2)]
    a, b = rk.AdamW(p), rk.AdamW(p)
    assert a.counts == [0, 0]
    a.steps = 5                                   # of all of them
    assert a.counts == [5, 5] and a.steps == 5
    a.counts[1] = 3
    b.load_state_dict(a.state_dict())
    assert b.steps == 5 and b.counts == [5, 3]
    b.counts[0] = 9
    assert a.counts == [5, 3]
    old = {k: v for k, v in a.state_dict().items() if k != "counts"}
    b.load_state_dict(old)                        # saved without counts
    assert b.counts == [5, 5]
    with pytest.raises(ValueError):
        b.load_state_dict({**a.state_dict(), "counts": [1]})
    s = [rk.adamw_state(x) for x in p]
    for bad in ([1], [1, 2, 3], [1, "a"], 1.0, None):
        with pytest.raises((TypeError, ValueError)):
            rk.relkl_adamw(p, p, s, lr=1e-3, step=bad)
