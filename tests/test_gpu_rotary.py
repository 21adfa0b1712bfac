"""Rotary positions on the GPU against the rotation in float64, element by element.

Tolerance.  cos and sin come with at most 1 ulp of sincospif (2^-24 below 1), half an
ulp each of the residual's fma and of the factor's product, and the factor's own rounding:
m (2^-23 + 2^-24).  The two products and their sum round three times at 2^-24 of at most
m (|a| + |b|), so a float32 result is off by at most 2.5 * 2^-23 m (|a| + |b|), and the
angle, a double, adds 4 * 2^-53 of itself.  A bf16 result adds half a step, 2^-8.
"""
import numpy as np
import pytest
import torch

import attention_relation_kl_b200 as rk

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _reference(x, inv_freq, pos, m, interleaved, inverse):
    """(y, bound of the float32 error) of x [B, H, N, d] at positions [B, N]."""
    x = x.detach().cpu().double().numpy()
    f = inv_freq.cpu().numpy()
    r = 2 * f.size
    ang = pos[:, None, :, None] * f
    c, s = m * np.cos(ang), m * np.sin(ang) * (-1.0 if inverse else 1.0)
    ia, ib = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    a, b = x[..., ia], x[..., ib]
    y, err = x.copy(), np.zeros_like(x)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    e = abs(m) * (np.abs(a) + np.abs(b)) * (2.5 * 2.0 ** -23 + 4 * 2.0 ** -53 * np.abs(ang))
    err[..., ia] = err[..., ib] = e
    return y, err


def _check(got, want, err):
    g = got.detach().cpu().double().numpy()
    tol = err if got.dtype == F32 else err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    assert g.shape == want.shape
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.abs(g - want).max()))


def _positions(pos, B, N, scale=1.0, offset=0.0):
    p = np.arange(N, dtype=np.float64) if pos is None else pos.cpu().numpy().astype(np.float64)
    return offset + scale * np.broadcast_to(p, (B, N))


def _randn(shape, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=gen).to(dtype).cuda()


# head sizes whose rotated part, half or rest cannot be read in wide accesses among them
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32), (80, 40), (96, 20), (33, 18), (7, 2),
                                   (64, 0), (2, 2), (512, 510)])
def test_heads_types_and_pairings(d, rot, xt, yt, interleaved):
    B, N = 2, 37
    xs = [_randn((B, h, N, d), xt, h) for h in (5, 2, 3)]
    f, m = rk.rotary_freqs(rot, 1e4, "yarn", 4.0) if rot else rk.rotary_freqs(0)
    pos = _positions(None, B, N, 0.25, 3.0)
    for inverse in (False, True):
        got = rk.relkl_rotary_qkv(xs, f, apply=(True, True, False), pos_scale=0.25, pos_offset=3.0,
                                  mscale=m, interleaved=interleaved, inverse=inverse, out_dtype=yt)
        for x, y in zip(xs[:2], got):
            _check(y, *_reference(x, f, pos, m, interleaved, inverse))
        assert torch.equal(got[2], xs[2].to(yt))     # moved, rounded once


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [1, 2, 255, 1000])
def test_views_of_one_projection_to_heads_and_back(N, dtype):
    # q, k, v side by side in one buffer whose rows are longer than their parts
    B, d, heads = 2, 64, (6, 2, 2)
    buf = _randn((B, N, sum(heads) * d + 24), dtype, N)
    parts = buf[..., :sum(heads) * d].split([h * d for h in heads], -1)
    xs = [p.unflatten(-1, (h, d)).transpose(1, 2) for p, h in zip(parts, heads)]
    f, _ = rk.rotary_freqs(d)
    got = rk.relkl_rotary_qkv(xs, f, apply=(True, True, False))
    pos = _positions(None, B, N)
    for x, y in zip(xs[:2], got):
        assert y.is_contiguous()
        _check(y, *_reference(x, f, pos, 1.0, False, False))
    assert torch.equal(got[2], xs[2])
    # back into views of a second buffer; what lies between them stays as it was
    dst = torch.full_like(buf, 7.0)
    outs = [p.unflatten(-1, (h, d)).transpose(1, 2)
            for p, h in zip(dst[..., :sum(heads) * d].split([h * d for h in heads], -1), heads)]
    rk.relkl_rotary_qkv(got, f, apply=(True, True, False), inverse=True, out=outs)
    for x, y in zip(got[:2], outs):
        _check(y, *_reference(x, f, pos, 1.0, False, True))
    assert torch.equal(dst[..., sum(heads) * d:], torch.full_like(dst[..., sum(heads) * d:], 7.0))


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_any_alignment(dtype, offset, interleaved):
    B, H, N, d = 1, 3, 21, 64
    raw = _randn((B * H * N * d + offset,), dtype, 5)
    x = raw[offset:].view(B, H, N, d)
    out = torch.empty(B * H * N * (d + 1) + offset, dtype=dtype, device="cuda")
    y = out[offset:].view(B, H, N, d + 1)[..., :d]
    f, _ = rk.rotary_freqs(d)
    rk.relkl_rotary(x, f, out=y, interleaved=interleaved)
    _check(y, *_reference(x, f, _positions(None, B, N), 1.0, interleaved, False))


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_given_positions_far_negative_and_shared(kind):
    B, H, N, d = 3, 2, 40, 64
    x = _randn((B, H, N, d), F32, 1)
    f, _ = rk.rotary_freqs(d, 5e5)
    gen = torch.Generator().manual_seed(2)
    pos = torch.randint(-1000, 10_000_000, (B, N), generator=gen).to(kind).cuda()
    pos[0, 0], pos[1, 1] = 0, 2 ** 31 - 1
    y = rk.relkl_rotary(x, f, positions=pos)
    _check(y, *_reference(x, f, _positions(pos, B, N), 1.0, False, False))
    one = pos[0].contiguous()                       # [N], for every batch element
    assert torch.equal(rk.relkl_rotary(x, f, positions=one),
                       rk.relkl_rotary(x, f, positions=one.expand(B, N)))
    every = torch.stack((pos, pos), -1)[..., 0]     # a strided view
    assert not every.is_contiguous()
    assert torch.equal(rk.relkl_rotary(x, f, positions=every), y)


def test_in_place_and_broadcast_input():
    B, H, N, d = 2, 4, 19, 64
    f, _ = rk.rotary_freqs(d)
    buf = _randn((B, N, 3 * H * d), BF16, 3)
    views = [p.unflatten(-1, (H, d)).transpose(1, 2) for p in buf.split(H * d, -1)]
    want = rk.relkl_rotary_qkv(views, f)
    got = rk.relkl_rotary_qkv(views, f, out=views)   # parts of one buffer, each on itself
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and got[0] is views[0]
    x = _randn((1, 1, N, d), F32, 4).expand(B, H, N, d)
    assert torch.equal(rk.relkl_rotary(x, f), rk.relkl_rotary(x.contiguous(), f))
    with pytest.raises(RuntimeError):                # another layout of the same memory
        rk.relkl_rotary(views[0], f, out=buf.view(-1)[:B * H * N * d].view(B, H, N, d))


def test_many_heads_and_no_tokens():
    f, _ = rk.rotary_freqs(8)
    x = _randn((1, 70000, 1, 8), BF16, 6)            # more heads than a grid has rows
    _check(rk.relkl_rotary(x, f, pos_offset=5.0),
           *_reference(x, f, _positions(None, 1, 1, offset=5.0), 1.0, False, False))
    assert rk.relkl_rotary(torch.empty(2, 3, 0, 8, device="cuda"), f).shape == (2, 3, 0, 8)
    empty = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    assert rk.relkl_rotary(torch.empty(0, 3, 4, 8, device="cuda"), f, positions=empty).numel() == 0


def test_offsets_past_32_bits():
    far = 2 ** 31 + 64                               # elements between the two batch elements
    f, _ = rk.rotary_freqs(64)
    buf = torch.zeros(far + 3 * 5 * 64, dtype=BF16, device="cuda")
    x = buf.as_strided((2, 3, 5, 64), (far, 5 * 64, 64, 1))
    small = _randn((2, 3, 5, 64), BF16, 21)
    x.copy_(small)
    want = rk.relkl_rotary(small, f)
    assert torch.equal(rk.relkl_rotary(x, f), want)
    rk.relkl_rotary(x, f, out=x)
    assert torch.equal(x, want)


def test_special_values_stay_in_their_pair():
    f, _ = rk.rotary_freqs(8)
    x = _randn((1, 1, 3, 16), F32, 7)
    x[0, 0, 1, 2], x[0, 0, 1, 12] = float("nan"), float("inf")
    y = rk.relkl_rotary(x, f)
    clean = x.clone()
    clean[0, 0, 1, 2], clean[0, 0, 1, 12] = 1.0, 1.0
    want = rk.relkl_rotary(clean, f)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 0, 1, [2, 6, 12]] = True                  # the pair (2, 6), and the entry behind the rotation
    assert torch.equal(y[~hit], want[~hit]) and y[0, 0, 1, 12] == float("inf")
    assert torch.isnan(y[0, 0, 1, [2, 6]]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_the_formula_and_differences(interleaved):
    B, H, N, d, rot = 2, 3, 11, 20, 12
    f, m = rk.rotary_freqs(rot, 1e4, "yarn", 4.0)
    pos = torch.randint(0, 500, (B, N), generator=torch.Generator().manual_seed(1)).cuda()
    x = _randn((B, N, H, d), F32, 8).transpose(1, 2).requires_grad_()
    w = _randn((B, H, N, d), F32, 9)
    args = dict(positions=pos, mscale=m, interleaved=interleaved, pos_scale=0.5)
    y = rk.rotary(x, f, **args)
    (g,) = torch.autograd.grad((y * w).sum(), x, create_graph=False)
    _check(g, *_reference(w, f, _positions(pos, B, N, 0.5), m, interleaved, True))
    # y is linear in x: a difference along u is w . y(u), exactly up to rounding
    u = _randn((B, H, N, d), F32, 10)
    with torch.no_grad():
        dy = rk.relkl_rotary(x + u, f, **args).double() - rk.relkl_rotary(x - u, f, **args).double()
    slope = float((dy * w.double()).sum() / 2)
    # float32 errors of the two rotations and of x +- u: at most 4 * 2^-22 of each product
    room = 4 * 2.0 ** -22 * m * float(((x.abs() + u.abs()).double().sum(-1, keepdim=True) * w.abs().double()).sum())
    assert abs(slope - float((g.double() * u.double()).sum())) <= room
    # a broadcast gradient, and a second derivative
    z = _randn((1, 2, 3, 8), F32, 11).requires_grad_()
    f8, _ = rk.rotary_freqs(8)
    (gz,) = torch.autograd.grad(rk.rotary(z, f8).sum(), z)
    assert torch.equal(gz, rk.relkl_rotary(torch.ones_like(z), f8, inverse=True))
    v = torch.ones(1, 2, 3, 8, device="cuda", requires_grad=True)
    (g1,) = torch.autograd.grad(rk.rotary(z, f8), z, v, create_graph=True)
    (g2,) = torch.autograd.grad(g1, v, torch.ones_like(g1))
    assert torch.equal(g2, rk.relkl_rotary(torch.ones_like(z), f8))


def test_bf16_gradient_keeps_the_input_type():
    f, _ = rk.rotary_freqs(64)
    x = _randn((1, 2, 5, 64), BF16, 12).requires_grad_()
    rk.rotary(x, f, out_dtype=F32).square().sum().backward()
    assert x.grad.dtype == BF16
    _check(x.grad, *_reference(2 * rk.relkl_rotary(x.detach(), f, out_dtype=F32), f,
                               _positions(None, 1, 5), 1.0, False, True))


def test_other_stream_and_captured_graph():
    f, _ = rk.rotary_freqs(64)
    x = _randn((2, 4, 300, 64), BF16, 13)
    want = rk.relkl_rotary(x, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = rk.relkl_rotary(x, f, stream=side)
    z = rk.relkl_rotary(x, f, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want) and torch.equal(z, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rk.relkl_rotary(x, f, out=out)
    x.copy_(_randn(x.shape, BF16, 14))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, rk.relkl_rotary(x, f))


def test_bad_calls_are_refused():
    f, _ = rk.rotary_freqs(64)
    x = torch.zeros(1, 2, 4, 64, device="cuda")
    for bad in (dict(positions=torch.zeros(1, 4, device="cuda")),
                dict(positions=torch.zeros(1, 5, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(1, 4, dtype=torch.int32)),
                dict(out=torch.zeros(1, 2, 4, 64)), dict(out=torch.zeros(1, 2, 5, 64, device="cuda")),
                dict(out=torch.zeros(1, 2, 4, 128, device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            rk.relkl_rotary(x, f, **bad)
    with pytest.raises(ValueError):
        rk.relkl_rotary(x, f.float())
    with pytest.raises(ValueError):
        rk.relkl_rotary(x[..., :32], f)
    with pytest.raises(ValueError):
        rk.relkl_rotary(x.transpose(2, 3), f)
    with pytest.raises(TypeError):
        rk.relkl_rotary(x.half(), f)
    with pytest.raises(TypeError):
        rk.relkl_rotary(x, f, out_dtype=torch.float16)
    with pytest.raises(RuntimeError):
        rk.relkl_rotary(x, f, out=x[:, :, :1].expand(1, 2, 4, 64))


# each tensor of a launch is read in accesses of its own width: a rotated or a moved one
# whose rows start anywhere leaves the others', and the rest of a head, as they should be
@pytest.mark.parametrize("odd", [0, 1, 2])
@pytest.mark.parametrize("apply", [(True, False, True), (False, False, False)])
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("d,rot", [(64, 4), (64, 62), (48, 16), (128, 20)])
def test_tensors_of_different_alignment_in_one_launch(d, rot, xt, yt, apply, odd):
    B, N = 2, 19
    xs, outs = [], []
    for i, h in enumerate((5, 1, 3)):
        shift = 1 if i == odd else 0
        xs.append(_randn((B * h * N * d + shift,), xt, i)[shift:].view(B, h, N, d))
        outs.append(torch.full((B * h * N * d + shift,), 7.0, dtype=yt, device="cuda")[shift:].view(B, h, N, d))
    f, _ = rk.rotary_freqs(rot)
    pos = _positions(None, B, N)
    for interleaved in (False, True):
        rk.relkl_rotary_qkv(xs, f, apply=apply, interleaved=interleaved, out=outs)
        for x, y, turns in zip(xs, outs, apply):
            if turns:
                want, err = _reference(x, f, pos, 1.0, interleaved, False)
                _check(y[..., :rot], want[..., :rot], err[..., :rot])
                assert torch.equal(y[..., rot:], x[..., rot:].to(yt))
            else:
                assert torch.equal(y, x.to(yt))


def test_captured_backward_pass():
    x = _randn((1, 3, 17, 64), F32, 1).requires_grad_()
    w = _randn((1, 3, 17, 64), F32, 2)
    f, _ = rk.rotary_freqs(64)
    eager = rk.rotary(x, f)
    # x's gradient node belongs to the eager graph's stream: refused, and nothing is lost
    with pytest.raises(RuntimeError, match="eager graph"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            z = rk.rotary(x * 1.0, f)
            torch.autograd.grad(z, x, w)
    del z
    (want,) = torch.autograd.grad(eager, x, w)
    del eager
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = rk.rotary(x * 1.0, f)
        (got,) = torch.autograd.grad(z, x, w)
    for _ in range(2):
        got.zero_()
        graph.replay()
        assert torch.equal(got, want)


def test_given_outputs_are_seen_as_changed_in_place():
    x, f = _randn((1, 2, 5, 64), F32), rk.rotary_freqs(64).inv_freq
    a = torch.zeros_like(x, requires_grad=True)
    y = (a * x).sum()                     # x is saved for a's gradient
    rk.relkl_rotary(x, f, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_outputs_are_written_once():
    # any two outputs in one buffer: taken exactly where no element is in both
    f, gen = rk.rotary_freqs(4).inv_freq, np.random.default_rng(5)
    counts = {True: 0, False: 0}
    for case in range(400):
        B, N, d = int(gen.integers(1, 4)), int(gen.integers(1, 5)), int(gen.integers(4, 7))
        buf = torch.zeros(6000, device="cuda")
        outs, places = [], []
        inner = int(gen.integers(1, 4)) * d            # the heads' distance in interleaved parts
        for r in range(int(gen.integers(2, 4))):
            H = int(gen.integers(1, 4))
            order = gen.permutation(3) if case % 2 else np.array([1, 2, 0])
            stride, reach = [0, 0, 0], d if case % 2 else inner
            for o in order:                            # each step passes what the smaller ones reach
                stride[o] = reach + (int(gen.integers(0, 9)) if case % 2 else 0)
                reach = stride[o] * (B, 3 if case % 2 == 0 else H, N)[o]
            at = int(gen.integers(0, 60 * d))
            y = buf.as_strided((B, H, N, d), (*stride, 1), at)
            outs.append(y)
            places.append(set(torch.arange(6000).as_strided(y.shape, y.stride(), at).flatten().tolist()))
        free = all(not (a & b) for i, a in enumerate(places) for b in places[:i])
        counts[free] += 1
        xs = [_randn(y.shape, F32, case) for y in outs]
        if free:
            rk.relkl_rotary_qkv(xs, f, out=outs)
            for x, y in zip(xs, outs):
                assert torch.equal(y, rk.relkl_rotary(x, f))
        else:
            with pytest.raises(RuntimeError, match="INVALID"):
                rk.relkl_rotary_qkv(xs, f, out=outs)
            assert not buf.any()
    assert min(counts.values()) > 40
    x, f = _randn((1, 2, 9, 64), F32, 1), rk.rotary_freqs(64).inv_freq
    q = _randn((1, 4, 9, 64), F32, 2)
    with pytest.raises(RuntimeError, match="INVALID"):     # a layer that shares K and V
        rk.relkl_rotary_qkv([q, x, x], f, apply=(True, True, False), out=[q, x, x])


def test_transforms_without_a_rule_are_refused():
    x, f = _randn((1, 2, 5, 64), F32), rk.rotary_freqs(64).inv_freq
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda z: rk.rotary(z, f))(x[None])
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda z: rk.rotary(z, f).sum())(x)
    with pytest.raises(RuntimeError), torch.autograd.forward_ad.dual_level():
        rk.rotary(torch.autograd.forward_ad.make_dual(x, torch.ones_like(x)), f)
