"""The operators together, as one layer's distillation step uses them: 8-bit teacher
projections and their rotation, the relation loss, its gradient turned back to the weights,
clipping and the update."""
import math

import numpy as np
import pytest
import torch

import attention_relation_kl_b200 as rk
import workload
from oracle import chain, dense
from parity import DX_TOL_BF16, to_np

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _rotated(x, freqs, pos, interleaved=False):
    """x [B, heads, N, d] in float64, rotated at pos [N]."""
    f = freqs.inv_freq.cpu().numpy()
    r, a = 2 * f.size, pos[:, None] * f
    c, s = freqs.mscale * np.cos(a), freqs.mscale * np.sin(a)
    lo, hi = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y = x.copy()
    y[..., lo], y[..., hi] = x[..., lo] * c - x[..., hi] * s, x[..., hi] * c + x[..., lo] * s
    return y


def _heads(y, d):
    B, N, cols = y.shape
    return y.reshape(B, N, cols // d, d).transpose(0, 2, 1, 3)


@pytest.mark.parametrize("N", [1, 45, 300])
def test_teacher_relations(N):
    B, D, d, heads = 2, 136, 64, dict(q=4, k=2, v=2)
    gen = torch.Generator().manual_seed(N)
    h = torch.randn(B, N, D, generator=gen).to(BF16).cuda()
    freqs = rk.rotary_freqs(32, 1e4, "yarn", 4.0)
    weights, bias = {}, torch.randn(heads["q"] * d, generator=gen).cuda()
    for r, n in heads.items():
        weights[r] = rk.relkl_quantize_rows(torch.randn(n * d, D, generator=gen).cuda() / D ** 0.5)
    weights["q"] = (*weights["q"], bias)
    got = rk.teacher_relations_i8(h, weights, d, freqs, pos_scale=0.5, interleaved=True)
    x = to_np(h).reshape(B * N, D)
    most = np.abs(x).max(1, keepdims=True)
    codes, scale = np.rint(127 * x / most), most / 127
    for r, n in heads.items():
        w, sw = to_np(weights[r][0]), to_np(weights[r][1])
        y = (codes @ w.T) * scale * sw + (to_np(bias) if r == "q" else 0)
        y = _heads(y.reshape(B, N, -1), d)
        want = y if r == "v" else _rotated(y, freqs, 0.5 * np.arange(N), True)
        assert got[r].shape == (B, n, N, d) and got[r].is_contiguous()
        # bf16 twice: the projection's rounding passes through the rotation as a vector of its
        # length, at most mscale (|a| + |b|), and the result rounds
        size = np.abs(y).max() if r == "v" else freqs.mscale * 2 * np.abs(y).max()
        assert np.abs(to_np(got[r]) - want).max() <= 2.0 ** -8 * (size + np.abs(want).max()) * 1.01


def test_distillation_step_of_one_layer():
    cw = workload.CHAIN_CONFIGS["chain_small"]
    c = workload.generate_chain(cw)
    hs, ht = c["h_s"].cuda(), c["h_t"].cuda()
    rels = ("q", "k", "v")
    freqs_t = rk.rotary_freqs(cw.d, cw.rope_base)
    freqs_s = rk.rotary_freqs(cw.d, cw.rope_base, "ntk", cw.pi_factor)
    weights = {r: rk.relkl_quantize_rows(c["w"][r].t().contiguous().cuda()) for r in rels}
    teacher = rk.teacher_relations_i8(ht, weights, cw.d, freqs_t)
    masters = [c["w"][r].float().cuda() for r in rels]
    copies = [w.to(BF16) for w in masters]
    opt = rk.AdamW(masters, lr=1e-3, betas=(0.9, 0.95), weight_decay=0.1, max_norm=1e-3, copies=copies)
    for step in (1, 2):
        before = [to_np(w) for w in masters]
        m0 = [(to_np(s.m), to_np(s.v)) for s in opt.state]
        xs = [(hs @ w).unflatten(-1, (-1, cw.d)).transpose(1, 2) for w in copies]
        student = dict(zip(rels, rk.relkl_rotary_qkv(xs, freqs_s.inv_freq, apply=(True, True, False),
                                                     mscale=freqs_s.mscale)))
        pairs = {r: (teacher[r], student[r]) for r in rels}
        grads, norm = rk.student_step(pairs, hs, opt, freqs=freqs_s)
        assert rk.relkl_get_device_error() == (0, 0)
        # the gradients against the float64 oracle on the same relation inputs
        for r in rels:
            dx = dense.bwd(to_np(pairs[r][0]), to_np(pairs[r][1]))
            if r != "v":
                turned = rk.RotaryFreqs(-freqs_s.inv_freq, freqs_s.mscale)
                dx = _rotated(dx, turned, np.arange(cw.N, dtype=np.float64))
            want = chain.weight_grad(to_np(hs), chain.heads_to_tokens(dx))
            got = to_np(grads[r])
            assert np.abs(got - want).max() <= DX_TOL_BF16 * np.abs(want).max(), r
        # clipping and update from these gradients
        size = math.sqrt(sum(float((to_np(g) ** 2).sum()) for g in grads.values()))
        assert abs(float(norm) - size) <= 1e-6 * size
        coef = min(1.0, 1e-3 / (size + 1e-6))
        for k, r in enumerate(rels):
            g = coef * to_np(grads[r])
            m, v = 0.9 * m0[k][0] + 0.1 * g, 0.95 * m0[k][1] + 0.05 * g * g
            move = 1e-3 * (m / (1 - 0.9 ** step)) / (np.sqrt(v / (1 - 0.95 ** step)) + 1e-8)
            want = before[k] * (1 - 1e-4) - move
            # the step rounds some twenty times at 2^-24 of itself, m against its larger terms
            room = 30 * 2.0 ** -24 * (np.abs(before[k]) + 1e-3 * (1 + (np.abs(g) + np.abs(m0[k][0])) /
                                                                    (np.sqrt(v) + 1e-8)))
            assert np.all(np.abs(to_np(masters[k]) - want) <= room)
            assert torch.equal(copies[k], masters[k].to(BF16))
    assert opt.steps == 2
    with pytest.raises(ValueError):
        rk.student_step({"q": pairs["q"]}, hs, opt)
    with pytest.raises(ValueError):
        rk.student_weight_grads(pairs, hs, 1e4, 1.0, interleaved=True)


def test_given_frequencies_equal_the_base():
    # the powers of the base as frequencies: the older backward's gradients, up to its rounding
    cw = workload.CHAIN_CONFIGS["chain_small"]
    c = workload.generate_chain(cw)
    pairs = {r: (c["x"][r][0].cuda(), c["x"][r][1].cuda()) for r in "qkv"}
    hs = c["h_s"].cuda()
    a = rk.student_weight_grads(pairs, hs, cw.rope_base, 1.0 / cw.pi_factor)
    b = rk.student_weight_grads(pairs, hs, cw.rope_base, 1.0 / cw.pi_factor,
                                freqs=rk.rotary_freqs(cw.d, cw.rope_base))
    for r in "qkv":
        # both round the same gradient to bf16 (2^-8), its float32 sums add in another order
        assert float((a[r] - b[r]).abs().max()) <= 2.0 ** -7 * float(a[r].abs().max())


# the tokens are coded once for all relations, or by each one's product: the same bits
@pytest.mark.parametrize("B,N", [(2, 0), (1, 1), (4, 1), (5, 1), (2, 150)])
def test_teacher_relations_equal_one_after_the_other(B, N):
    gen, freqs = torch.Generator().manual_seed(3), rk.rotary_freqs(64)
    h = torch.randn(B, N, 136, generator=gen).to(BF16).cuda()
    weights = {r: rk.relkl_quantize_rows(torch.randn(n * 64, 136, generator=gen).cuda())
               for r, n in dict(q=3, k=1, v=1).items()}
    got = rk.teacher_relations_i8(h, weights, 64, freqs)
    for r in weights:
        (one,) = rk.teacher_relations_i8(h, {r: weights[r]}, 64, freqs).values()
        assert torch.equal(got[r], one)
