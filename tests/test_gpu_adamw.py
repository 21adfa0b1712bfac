"""AdamW over many tensors and the gradient norm on the GPU against the formulas in float64.

Tolerances, u = 2^-24.  m: the two coefficients, the scaled gradient and the two operations
round, each once: 5 u (|b1 m| + |c1 g|).  v: 6 u v'.  The step's quotient takes the root
(4 u), three scalars, a sum, a quotient and a product: 12 u |step| next to m's own error
over the same denominator.  The weight: its factor, and the last sum.  bf16 adds half a
step, 2^-8; an e4m3 number is off by half a step, 2^-4 of itself or 2^-10 of its scale, a
tiny root by 2^-9 of its scale.
"""
import math

import numpy as np
import pytest
import torch

import attention_relation_kl_b200 as rk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
SIZES = (1, 2, 3, 5, 7, 255, 256, 257, 1000, 4095, 4096, 4097, 8193, 20001)


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _f64(x):
    return x.detach().cpu().double().numpy().reshape(-1)


def _decoded(codes, scale):
    return _f64(codes.float()) * np.repeat(_f64(scale), 256)[:codes.numel()]


def _moments(s):
    if s.m_scale is None:
        return _f64(s.m), _f64(s.v)
    return _decoded(s.m, s.m_scale), _decoded(s.v, s.v_scale) ** 2


class Expected:
    """One step from the current values of a tensor and its state, and the bounds."""

    def __init__(self, p, g, s, t, lr, b1, b2, eps, wd, coef=1.0, ecoef=0.0):
        # ecoef: relative error of the factor on the gradients
        p, g, (m, v) = _f64(p), coef * _f64(g), _moments(s)
        c1, c2 = 1 - b1, 1 - b2
        self.m, self.v = b1 * m + c1 * g, b2 * v + c2 * g * g
        self.em = 5 * U * (np.abs(b1 * m) + np.abs(c1 * g)) + ecoef * np.abs(c1 * g)
        # a decoded moment is itself a rounded product (and v a square of one)
        if s.m_scale is not None:
            self.em += U * np.abs(b1 * m)
        self.ev = (6 if s.m_scale is None else 9) * U * self.v + 2 * ecoef * c2 * g * g
        self.root = np.sqrt(self.v)
        den = self.root / math.sqrt(1 - b2 ** t) + eps
        size = lr / (1 - b1 ** t)
        step = size * self.m / den
        self.p = p * (1 - lr * wd) - step
        self.ep = 2.5 * U * np.abs(p) + (14 * U + ecoef) * np.abs(step) + size * self.em / den

    def check(self, p, s, copy=None):
        got = _f64(p)
        tol = self.ep + (2.0 ** -8 * (np.abs(self.p) + self.ep) if p.dtype == BF16 else 0)
        assert np.all(np.abs(got - self.p) <= tol), np.max(np.abs(got - self.p) - tol)
        if copy is not None:
            assert np.all(np.abs(_f64(copy) - self.p) <= self.ep + 2.0 ** -8 * (np.abs(self.p) + self.ep))
            if p.dtype == F32:
                assert torch.equal(copy, p.to(BF16))
        if s.m_scale is None:
            assert np.all(np.abs(_f64(s.m) - self.m) <= self.em)
            assert np.all(np.abs(_f64(s.v) - self.v) <= self.ev)
            return
        for codes, scale, x, e, root in ((s.m, s.m_scale, self.m, self.em, False),
                                         (s.v, s.v_scale, self.root, 6 * U * self.root, True)):
            n = x.size
            rows = np.zeros((-(-n // 256), 256))
            rows.reshape(-1)[:n] = np.abs(x)
            most = rows.max(1)
            err = np.zeros_like(rows)
            err.reshape(-1)[:n] = e
            assert np.all(np.abs(_f64(scale) - most / 448) <= (err.max(1) + 2 * U * most) / 448)
            each = np.repeat(most / 448, 256)[:n]
            least = 2.0 ** -9 if root else 2.0 ** -10
            tol = np.maximum(2.0 ** -4 * np.abs(x), least * each) * (1 + 2.0 ** -20) + e * 2
            got = _decoded(codes, scale)
            assert np.all(np.abs(got - x) <= tol)
            if root:
                assert np.all((got > 0) == (x > 0)) and np.all(got >= 0)


def _make(sizes, bits, pt, gt, seed, offset=0, copies=False):
    gen = torch.Generator().manual_seed(seed)

    def place(x):       # `offset` elements behind an aligned address
        raw = torch.zeros(x.numel() + offset, dtype=x.dtype).cuda()
        raw[offset:].copy_(x)
        return raw[offset:]

    params, grads, states, cs = [], [], [], []
    for n in sizes:
        params.append(place((0.02 * torch.randn(n, generator=gen)).to(pt)))
        size = torch.randn(n, generator=gen).exp() * 1e-3
        grads.append(place((size * torch.randn(n, generator=gen)).to(gt)))
        m, v = 0.3 * size * torch.randn(n, generator=gen), size ** 2 * torch.rand(n, generator=gen)
        if bits == 32:
            states.append(rk.AdamWState(place(m), place(v)))
        else:
            out = []
            for x in (m, v.sqrt()):
                rows = torch.nn.functional.pad(x, (0, -n % 256)).view(-1, 256)
                scale = rows.abs().amax(1) / 448
                codes = (rows / scale.clamp(min=1e-30)[:, None]).reshape(-1)[:n].to(E4M3)
                out += [place(codes.view(torch.uint8)).view(E4M3), scale.cuda()]
            states.append(rk.AdamWState(out[0], out[2], out[1], out[3]))
        cs.append(place(torch.zeros(n, dtype=BF16)))
    return params, grads, states, cs if copies else None


HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8)


def _expect(params, grads, states, step, wd, coef=1.0):
    wd = wd if isinstance(wd, (list, tuple)) else [wd] * len(params)
    return [Expected(p, g, s, step, HYPER["lr"], *HYPER["betas"], HYPER["eps"], w, coef)
            for p, g, s, w in zip(params, grads, states, wd)]


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("pt,gt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("bits", [32, 8])
def test_sizes_types_and_alignment(bits, pt, gt, offset):
    params, grads, states, copies = _make(SIZES, bits, pt, gt, 1, offset, copies=True)
    want = _expect(params, grads, states, 7, 0.1)
    rk.relkl_adamw(params, grads, states, step=7, weight_decay=0.1, copies=copies, **HYPER)
    for w, p, s, c in zip(want, params, states, copies):
        w.check(p, s, c)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_steps_from_a_fresh_state(bits):
    params, grads, _, _ = _make((513, 64), bits, F32, F32, 2)
    grads[0][5] = 0.0
    states = [rk.adamw_state(p, bits) for p in params]
    for t in range(1, 6):
        want = _expect(params, grads, states, t, 0.01)
        rk.relkl_adamw(params, grads, states, step=t, weight_decay=0.01, **HYPER)
        for w, p, s in zip(want, params, states):
            w.check(p, s)
    assert float(states[0].m.float()[5]) == 0.0 and float(states[0].v.float()[5]) == 0.0


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_table_holds(bits):
    sizes = [1 + (7 * k) % 600 for k in range(801)] + [0, 0]
    params, grads, states, copies = _make(sizes, bits, BF16, F32, 3, copies=True)
    decay = [0.1 * (k % 3) for k in range(len(sizes))]
    want = _expect(params, grads, states, 2, decay)
    rk.relkl_adamw(params, grads, states, step=2, weight_decay=decay, copies=copies, **HYPER)
    for w, p, s, c in zip(want, params, states, copies):
        if p.numel():
            w.check(p, s, c)
    assert rk.relkl_adamw([params[-1]], [grads[-1]], [states[-1]], step=1, lr=1e-3) is None


def test_states_of_both_kinds_in_one_call():
    a = _make((300, 4000), 8, F32, F32, 4)
    b = _make((17, 900), 32, BF16, BF16, 5)
    params, grads, states = (list(x) + list(y) for x, y in zip(a[:3], b[:3]))
    order = [0, 2, 1, 3]
    params, grads, states = ([x[k] for k in order] for x in (params, grads, states))
    want = _expect(params, grads, states, 3, [0.1, 0.0, 0.2, 0.3])
    rk.relkl_adamw(params, grads, states, step=3, weight_decay=[0.1, 0.0, 0.2, 0.3], **HYPER)
    for w, p, s in zip(want, params, states):
        w.check(p, s)


@pytest.mark.parametrize("bits", [32, 8])
def test_clipping_and_a_step_left_out(bits):
    params, grads, states, copies = _make((700, 4100), bits, F32, F32, 6, copies=True)
    for limit in (1e-3, 1e9):
        clip = rk.relkl_grad_norm(grads, limit)
        norm = math.sqrt(sum(float((_f64(g) ** 2).sum()) for g in grads))
        assert abs(float(clip[0]) - norm) <= 6 * U * norm
        coef = float(clip[1])
        assert abs(coef - min(1.0, limit / (norm + 1e-6))) <= 8 * U * coef
        want = _expect(params, grads, states, 9, 0.1, coef)
        rk.relkl_adamw(params, grads, states, step=9, weight_decay=0.1, copies=copies,
                       grad_scale=clip[1:], **HYPER)
        for w, p, s, c in zip(want, params, states, copies):
            w.check(p, s, c)
    # a norm that is no finite number: nothing is written
    for bad in (float("nan"), float("inf"), 1e30):
        grads[1][3] = bad
        clip = rk.relkl_grad_norm(grads, 1.0)
        assert not math.isfinite(float(clip[0])) and math.isnan(float(clip[1]))
        before = [x.clone() for x in params + copies] + [y.clone() for s in states for y in s if y is not None]
        rk.relkl_adamw(params, grads, states, step=10, copies=copies, grad_scale=clip[1:], **HYPER)
        after = params + copies + [y for s in states for y in s if y is not None]
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(before, after))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_nan_gradient_without_a_scale_stays_in_its_block(bits):
    params, grads, states, _ = _make((1000,), bits, F32, F32, 7)
    clean = [x.clone() for x in (params[0], *[y for y in states[0] if y is not None])]
    other = rk.AdamWState(*clean[1:])
    good = grads[0].clone()
    grads[0][300] = float("nan")
    rk.relkl_adamw(params, grads, states, step=5, **HYPER)
    rk.relkl_adamw([clean[0]], [good], [other], step=5, **HYPER)
    hit = torch.zeros(1000, dtype=torch.bool, device="cuda")
    hit[300] = True
    assert torch.equal(params[0][~hit], clean[0][~hit]) and torch.isnan(params[0][300])
    if bits == 32:
        assert torch.equal(states[0].v[~hit], other.v[~hit]) and torch.isnan(states[0].v[300])
    else:
        assert torch.isnan(states[0].v_scale[1]) and torch.isnan(states[0].m_scale[1])
        at = [0, 2, 3]
        assert torch.equal(states[0].v_scale[at], other.v_scale[at])
        keep = torch.cat((torch.arange(256), torch.arange(512, 1000)))
        assert torch.equal(states[0].m.view(torch.uint8)[keep.cuda()], other.m.view(torch.uint8)[keep.cuda()])


def test_wide_ranges_in_one_8_bit_block():
    # roots 2^-30 .. 1 in a block: those below the smallest code keep a positive one, so
    # no step is divided by eps alone, and the largest value of a block decays exactly
    n = 256
    p = torch.zeros(n, device="cuda")
    g = (2.0 ** -torch.linspace(0, 30, n)).cuda()
    s = rk.adamw_state(p, 8)
    rk.relkl_adamw([p], [g], [s], lr=1e-3, step=1, eps=1e-12, weight_decay=0.0)
    root = _decoded(s.v, s.v_scale)
    # the first step is lr g / (g + eps), each of its twelve operations rounded
    assert np.all(root > 0) and np.allclose(_f64(p), -1e-3 * _f64(g) / (_f64(g) + 1e-12), rtol=14 * U, atol=0)
    g.zero_()
    before = p.clone()
    top = float(s.v_scale[0])
    for t in range(2, 12):
        rk.relkl_adamw([p], [g], [s], lr=1e-3, step=t, eps=1e-12, weight_decay=0.0)
    # ten steps of sqrt(b2), each rounding a few times
    assert abs(float(s.v_scale[0]) / (top * 0.999 ** 5) - 1) <= 10 * 8 * U
    assert float((p - before).abs().max()) < 0.05
    # a block of zeros, and one whose scale would be no normal number
    z = torch.full((300,), 1e-22, device="cuda")
    s = rk.adamw_state(z, 8)
    rk.relkl_adamw([torch.zeros_like(z)], [z], [s], lr=1e-3, step=1)
    assert torch.count_nonzero(s.v.view(torch.uint8)) == 0 and torch.count_nonzero(s.v_scale) == 0
    assert torch.count_nonzero(s.m_scale) == 2


def test_no_learning_rate_and_no_moments():
    params, grads, states, _ = _make((777,), 32, F32, F32, 8)
    want = _expect(params, grads, states, 1, 0.0)
    before = params[0].clone()
    rk.relkl_adamw(params, grads, states, lr=0.0, step=1, betas=HYPER["betas"], weight_decay=0.5)
    assert torch.equal(params[0], before)
    assert np.all(np.abs(_f64(states[0].m) - want[0].m) <= want[0].em)
    rk.relkl_adamw(params, grads, states, lr=1e-3, step=1, betas=(0.0, 0.0), weight_decay=0.0)
    assert torch.equal(states[0].m, grads[0])
    # the step is lr g / (|g| + eps), with the roundings of any step (14 u) and of the weight
    g = _f64(grads[0])
    off = np.abs(_f64(params[0]) - (_f64(before) - 1e-3 * g / (np.abs(g) + 1e-8)))
    assert np.all(off <= 14 * U * 1e-3 + 2.5 * U * np.abs(_f64(before)))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_take_lr_and_step_from_the_device(bits):
    params, grads, states, copies = _make((5000, 33), bits, F32, F32, 9, copies=True)
    lr = torch.tensor([3e-3], device="cuda")
    step = torch.ones(1, dtype=torch.int64, device="cuda")

    def one():
        clip = rk.relkl_grad_norm(grads, 0.05)
        rk.relkl_adamw(params, grads, states, lr=lr, step=step, betas=HYPER["betas"], eps=HYPER["eps"],
                       weight_decay=0.1, copies=copies, grad_scale=clip[1:])
        step.add_(1)

    first = [x.clone() for x in params] + [y.clone() for s in states for y in s if y is not None]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    for t, rate in ((1, 3e-3), (2, 1e-3), (3, 0.02)):
        lr.fill_(rate)
        for g in grads:
            g.mul_(1.5)
        norm = math.sqrt(sum(float((_f64(g) ** 2).sum()) for g in grads))
        rate = float(lr)      # as the device holds it
        # the factor is a rounded quotient by a rounded norm: 8 u
        want = [Expected(p, g, s, t, rate, *HYPER["betas"], HYPER["eps"], 0.1,
                         min(1.0, 0.05 / (norm + 1e-6)), 8 * U) for p, g, s in zip(params, grads, states)]
        graph.replay()
        torch.cuda.synchronize()
        for w, p, s, c in zip(want, params, states, copies):
            w.check(p, s, c)
    assert int(step) == 4 and not torch.equal(first[0], params[0])


def test_norm_of_many_sizes_is_the_same_each_time():
    gen = torch.Generator().manual_seed(10)
    for sizes in ((1,), (8191,), (8193, 3), (32768,), (40000, 1, 100000), tuple(range(1, 500))):
        for dtype in (F32, BF16):
            for offset in (0, 1):
                grads = [torch.randn(n + offset, generator=gen).to(dtype).cuda()[offset:] for n in sizes]
                a, b = rk.relkl_grad_norm(grads), rk.relkl_grad_norm(grads)
                want = math.sqrt(sum(float((_f64(g) ** 2).sum()) for g in grads))
                # eight squares in float32: 8 u; the root halves it; the result rounds
                assert abs(float(a[0]) - want) <= 6 * U * want, (sizes, dtype)
                assert torch.equal(a, b) and float(a[1]) == 1.0
    zero = [torch.zeros(10, device="cuda"), torch.zeros(0, device="cuda")]
    assert rk.relkl_grad_norm(zero, 1.0).tolist() == [0.0, 1.0]
    out = torch.empty(2, device="cuda")
    assert rk.relkl_grad_norm(zero, 1.0, out=out) is out


def test_optimizer_over_steps_and_missing_gradients():
    params, grads, _, copies = _make((400, 64, 3000), 8, F32, F32, 11, copies=True)
    opt = rk.AdamW(params, lr=3e-3, betas=HYPER["betas"], weight_decay=[0.1, 0.0, 0.2], state_bits=8,
                   max_norm=1e9, copies=copies)
    for t in (1, 2):
        want = _expect(params, grads, opt.state, t, [0.1, 0.0, 0.2])
        still = params[1].clone()
        norm = opt.step([grads[0], None, grads[2]])
        for k in (0, 2):
            want[k].check(params[k], opt.state[k], copies[k])
        assert torch.equal(params[1], still) and float(norm) > 0
    twin = [p.clone() for p in params]
    other = rk.AdamW(twin, lr=3e-3, betas=HYPER["betas"], weight_decay=[0.1, 0.0, 0.2], state_bits=8,
                     max_norm=1e9)
    other.load_state_dict(opt.state_dict())
    opt.step(grads)
    for p, g in zip(twin, grads):
        p.grad = g
    other.step()
    assert all(torch.equal(a, b) for a, b in zip(params, twin)) and other.steps == 3
    with pytest.raises(RuntimeError, match="captur"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            opt.step(grads)


def test_updated_leaves_are_known_to_autograd():
    w = torch.ones(8, device="cuda", requires_grad=True)
    y = (w * w).sum()
    s = rk.adamw_state(w.detach())
    rk.relkl_adamw([w], [torch.ones(8, device="cuda")], [s], lr=1e-3, step=1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.backward()


@pytest.mark.parametrize("bits", [32, 8])
def test_offsets_past_32_bits(bits):
    n, tail = 2 ** 31 + 2 ** 20 + 77, 2 ** 20 + 77
    params, grads, states, _ = _make((tail,), bits, BF16, BF16, 14)

    def big(x):          # zeros up to a block's start, then x
        raw = torch.uint8 if x.dtype == E4M3 else x.dtype
        y = torch.zeros(n, dtype=raw, device="cuda")
        y[n - tail:] = x.view(raw)
        return y.view(x.dtype)

    p, g = big(params[0]), big(grads[0])
    m, v = big(states[0].m), big(states[0].v)
    if bits == 8:
        skip = (n - tail) // 256
        scales = [torch.cat((torch.zeros(skip, device="cuda"), s)) for s in states[0][2:]]
        s = rk.AdamWState(m, v, *scales)
    else:
        s = rk.AdamWState(m, v)
    clip, clip_small = rk.relkl_grad_norm([g], 0.1), rk.relkl_grad_norm(grads, 0.1)
    # the same squares in other partial sums: two roundings
    assert abs(float(clip[0]) / float(clip_small[0]) - 1) <= 2 * U
    rk.relkl_adamw([p], [g], [s], step=3, **HYPER)
    rk.relkl_adamw(params, grads, states, step=3, **HYPER)
    assert torch.equal(p[n - tail:], params[0]) and not p[:1000].any()
    assert torch.equal(s.m.view(torch.uint8)[-tail * m.element_size():], states[0].m.view(torch.uint8))


def test_other_stream():
    params, grads, states, _ = _make((50000,), 8, F32, F32, 12)
    want = _expect(params, grads, states, 2, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    clip = rk.relkl_grad_norm(grads, 1e9, stream=side)
    rk.relkl_adamw(params, grads, states, step=2, weight_decay=0.1, grad_scale=clip[1:], stream=side, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    want[0].check(params[0], states[0])


def test_bad_calls_are_refused():
    p, g, s, c = _make((100,), 32, F32, F32, 13, copies=True)
    q, _, s8, _ = _make((100,), 8, F32, F32, 13)
    ok = dict(lr=1e-3, step=1)
    for error, args, kw in [
        (ValueError, (p, [g[0][:50]], s), {}),
        (ValueError, (p, [g[0].cpu()], s), {}),
        (ValueError, ([p[0].view(10, 10).t()], [g[0].view(10, 10)], [rk.AdamWState(s[0].m.view(10, 10), s[0].v.view(10, 10))]), {}),
        (TypeError, (p, [g[0].half()], s), {}),
        (TypeError, ([p[0].double()], g, s), {}),
        (TypeError, (p, g, [rk.AdamWState(s[0].m, s8[0].v)]), {}),
        (ValueError, (p, g, [rk.AdamWState(s8[0].m, s8[0].v)]), {}),
        (ValueError, (p, g, [rk.AdamWState(s8[0].m, s8[0].v, s8[0].m_scale, s8[0].v_scale.repeat(2))]), {}),
        (ValueError, (p, g, [rk.AdamWState(s[0].m, s[0].v, s8[0].m_scale, s8[0].v_scale)]), {}),
        (TypeError, (p, g, s), dict(copies=[p[0].clone()])),
        (ValueError, (p, g, s), dict(grad_scale=torch.ones(2, device="cuda"))),
        (ValueError, (p, g, s), dict(lr=torch.ones(1))),
        (ValueError, (p, g, s), dict(step=torch.ones(1, device="cuda"))),
        (RuntimeError, (p, g, s), dict(step=0)),
        (RuntimeError, (p, g, s), dict(betas=(1.0, 0.9))),
        (RuntimeError, (p, p, s), {}),
        (RuntimeError, (p * 2, g * 2, s * 2), {}),
        (RuntimeError, (p, g, [rk.AdamWState(s[0].m, s[0].m)]), {}),
    ]:
        with pytest.raises(error):
            rk.relkl_adamw(*args, **{**ok, **kw})
    with pytest.raises(RuntimeError):
        rk.relkl_grad_norm(g, 0.0)
    with pytest.raises(ValueError):
        rk.relkl_grad_norm([])
    with pytest.raises(ValueError):
        rk.relkl_grad_norm(g, out=torch.empty(3, device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", [(37,), (8192, 100), (300000, 5)])
def test_norm_whose_squares_leave_float32(sizes, dtype):
    gen = torch.Generator().manual_seed(12)
    for powers in ((18,), (-24,), (-35, -20), (18, -30), (0, -24)):
        for offset in (0, 1):
            grads = []
            for k, n in enumerate(sizes):
                g = torch.randn(n + offset, generator=gen) * 10.0 ** powers[k % len(powers)]
                g[offset::3] = 0.0
                grads.append(g.to(dtype).cuda()[offset:])
            got = rk.relkl_grad_norm(grads)
            want = math.sqrt(sum(float((_f64(g) ** 2).sum()) for g in grads))
            # as in range: 8 u of eight squares, halved by the root, and the result's rounding
            assert abs(float(got[0]) - want) <= 6 * U * want and float(got[1]) == 1.0
        # an element from 2^64 on counts as infinite, wherever it stands
        for at in (0, sizes[0] - 1):
            for x in (2.0 ** 64, -2.0 ** 64):
                grads[0][at] = x
                assert float(rk.relkl_grad_norm(grads)[0]) == math.inf
            grads[0][at] = 2.0 ** 63
        got, want = rk.relkl_grad_norm(grads), math.sqrt(sum(float((_f64(g) ** 2).sum()) for g in grads))
        assert abs(float(got[0]) - want) <= 6 * U * want


# many elements: a warp holds two blocks of 256, and pieces of the same tensors one at a time
# give the same bits
@pytest.mark.parametrize("pt,gt,copies", [(F32, BF16, True), (BF16, BF16, False), (F32, F32, False),
                                          (BF16, F32, True)])
def test_many_elements_and_their_pieces(pt, gt, copies):
    sizes = [(1 << 25) - 256, 256 * 7, 3, 512 * 9 + 1, 256, 70000, 511]
    params, grads, states, cs = _make([2 ** 20 + 256 * 3], 8, pt, gt, 13, copies=copies)
    tile = lambda x, n: x.repeat(-(-n // x.numel()))[:n].clone()  # noqa: E731
    first = [params[0], grads[0], *states[0][:2]]
    whole = []
    for k, n in enumerate(sizes):
        raw = [tile(x.view(torch.uint8) if x.dtype == E4M3 else x, n + 1)[int(k == 5):][:n] for x in first]
        blocks = -(-n // 256)
        whole.append([raw[0], raw[1], rk.AdamWState(raw[2].view(E4M3), raw[3].view(E4M3),
                                                   tile(states[0][2], blocks), tile(states[0][3], blocks)),
                      torch.zeros(n, dtype=BF16, device="cuda")])
    twin = [[p.clone(), g, rk.AdamWState(*(x.clone() for x in s)), c.clone()] for p, g, s, c in whole]

    def step(rows):
        rk.relkl_adamw([r[0] for r in rows], [r[1] for r in rows], [r[2] for r in rows], step=4,
                       weight_decay=0.1, copies=[r[3] for r in rows] if copies else None, **HYPER)

    step(whole)
    for p, g, s, c in twin:
        for a in range(0, p.numel(), 1 << 23):
            b = min(a + (1 << 23), p.numel())
            step([[p[a:b], g[a:b], rk.AdamWState(s.m[a:b], s.v[a:b], s.m_scale[a // 256:-(-b // 256)],
                                                 s.v_scale[a // 256:-(-b // 256)]), c[a:b]]])
    for x, y in zip(whole, twin):
        assert torch.equal(x[0], y[0]) and torch.equal(x[3], y[3])
        for a, b in zip(x[2], y[2]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits,eps", [(32, 1e-40), (32, 2.0 ** -126), (8, 2.0 ** -126)])
def test_the_smallest_eps_leaves_elements_without_moments(bits, eps):
    p = torch.ones(300, device="cuda")
    g = torch.zeros(300, device="cuda")
    g[7] = 1e-3
    rk.relkl_adamw([p], [g], [rk.adamw_state(p, bits)], lr=1e-3, step=1, eps=eps, weight_decay=0.0)
    # lr g / (|g| + eps): fourteen roundings of the step, and the weight's own
    assert abs(float(p[7]) - (1 - 1e-3)) <= 14 * U * 1e-3 + 2.5 * U
    p[7] = 1.0
    assert torch.equal(p, torch.ones_like(p))
    with pytest.raises(RuntimeError):
        rk.relkl_adamw([p], [g], [rk.adamw_state(p, 8)], lr=1e-3, step=1, eps=1e-40)


def test_a_refused_call_of_both_kinds_of_states_changes_nothing():
    a = _make((300, 4000), 32, F32, F32, 15)
    b = _make((700, 90), 8, F32, F32, 16)
    params, grads, states = (list(x) + list(y) for x, y in zip(a[:3], b[:3]))
    ok = dict(step=3, weight_decay=[0.1] * 4)
    twice = lambda xs, k: xs + [xs[k]]  # noqa: E731
    other = rk.AdamWState(*(x.clone() for x in states[0][:2]))
    whole = params + [y for s in states for y in s if y is not None]
    before = [x.clone() for x in whole]
    versions = [p._version for p in params]
    for args, kw in [
        ((twice(params, 3), twice(grads, 3), twice(states, 3)), dict(weight_decay=0.1)),
        ((params, grads, states), dict(weight_decay=[0.1, 0.1, 0.1, -0.1])),
        ((params, grads, states), dict(eps=1e-40)),      # the 8-bit states' limit
        # a parameter with a state of each kind, and one tensor's gradient that another writes
        ((params + [params[3]], grads + [grads[3]], states + [rk.AdamWState(*(
            torch.zeros(90, device="cuda") for _ in range(2)))]), dict(weight_decay=0.1)),
        ((params, [params[2][:300], *grads[1:]], states), {}),
    ]:
        with pytest.raises(RuntimeError):
            rk.relkl_adamw(*args, **{**HYPER, **ok, **kw})
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(whole, before))
        assert [p._version for p in params] == versions
    # the same gradient twice is read twice
    rk.relkl_adamw([params[0], params[3]], [grads[0], grads[0][:90]], [other, states[3]], step=3, **HYPER)
    assert params[0]._version == versions[0] + 1


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_are_corrected_by_each_parameters_own_steps(bits):
    params, grads, _, copies = _make((400, 64, 3000), bits, F32, F32, 17, copies=True)
    decay = [0.1, 0.0, 0.2]
    opt = rk.AdamW(params, weight_decay=decay, state_bits=bits, copies=copies, **HYPER)
    for t, with_gradient in enumerate([(0, 2), (0, 2), (0, 1, 2), (1,), (0, 1, 2)]):
        want = {k: Expected(params[k], grads[k], opt.state[k], opt.counts[k] + 1, HYPER["lr"], *HYPER["betas"],
                            HYPER["eps"], decay[k]) for k in with_gradient}
        opt.step([g if k in with_gradient else None for k, g in enumerate(grads)])
        for k, w in want.items():
            w.check(params[k], opt.state[k], copies[k])
        assert opt.steps == t + 1
    assert opt.counts == [4, 3, 4]
    # the first step of a parameter goes lr along its gradient's sign, whenever it comes
    p = [torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda")]
    late = rk.AdamW(p, weight_decay=0.0, state_bits=bits, **HYPER)
    one = torch.ones(8, device="cuda")
    for _ in range(10):
        late.step([one, None])
    late.step([one, one])
    assert np.all(np.abs(_f64(p[1]) + HYPER["lr"]) <= HYPER["lr"] * (14 * U + HYPER["eps"]))


def test_steps_given_for_each_tensor():
    a = _make((300, 4000, 17), 32, F32, F32, 18)
    b = _make((700, 90), 8, F32, F32, 19)
    params, grads, states = (list(x) + list(y) for x, y in zip(a[:3], b[:3]))
    steps = [7, 1, 7, np.int64(1), 12]
    want = [Expected(p, g, s, int(t), HYPER["lr"], *HYPER["betas"], HYPER["eps"], 0.1)
            for p, g, s, t in zip(params, grads, states, steps)]
    rk.relkl_adamw(params, grads, states, step=steps, weight_decay=0.1, **HYPER)
    for w, p, s in zip(want, params, states):
        w.check(p, s)
    whole = params + [y for s in states for y in s if y is not None]
    before = [x.clone() for x in whole]
    for bad in (dict(step=[7, 1, 7, 1, 0]), dict(step=[1, 2, 1, 1, 1], weight_decay=[0, 0, 0, 0, -1.0])):
        with pytest.raises(RuntimeError):
            rk.relkl_adamw(params, grads, states, **{"weight_decay": 0.1, **HYPER, **bad})
    # one tensor at two numbers of steps
    with pytest.raises(RuntimeError, match="overlaps"):
        rk.relkl_adamw(params[:1] * 2, grads[:1] * 2, states[:1] * 2, step=[1, 2], **HYPER)
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(whole, before))
