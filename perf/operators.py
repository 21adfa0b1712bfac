"""Measured cases of the operators around the relation-KL loss: rotary positions, AdamW over many
tensors and the 8-bit integer product of the frozen teacher's projections.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, with ``own``
set, through the package's entry points; ``exact`` gives the definition's result in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
DTYPES = {"bf16": BF16, "fp32": F32}
BLOCK = 256            # elements that share one scale of an 8-bit optimizer state
E4M3_MAX = 448.0
TINY = 2.0 ** -126     # a block scale below the smallest normal number is held as zero


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token for each of 16 sequences that are at different positions: launch latency
        dict(name="rotary one token", op="rotary", B=16, H=32, H_kv=8, N=1, d=128, rot=128,
             pairs="half", scaling="bands", factor=8.0, base=5e5, way="forward", dtype="bf16",
             out="bf16", positions="given", with_v=False, fused=True),
        # student inputs of the 32K workload: projections token by token to rotated heads
        dict(name="rotary student 32K", op="rotary", B=1, H=32, H_kv=32, N=32768, d=128, rot=128,
             pairs="half", scaling="linear", factor=8.0, base=1e4, way="forward", dtype="bf16",
             out="bf16", positions="counted", with_v=True, fused=False),
        # gradients of the grouped-head 16K workload on their way to the weight gradient
        dict(name="rotary gradient 16K", op="rotary", B=2, H=32, H_kv=8, N=16384, d=128, rot=128,
             pairs="half", scaling="yarn", factor=4.0, base=5e5, way="gradient", dtype="fp32",
             out="bf16", positions="counted", with_v=True, fused=False),
        # packed sequences, neighbouring pairs, half of an odd-sized head rotated, all in fp32
        dict(name="rotary packed part", op="rotary", B=1, H=12, H_kv=4, N=5003, d=80, rot=40,
             pairs="neighbours", scaling="ntk", factor=4.0, base=1e4, way="forward", dtype="fp32",
             out="fp32", positions="given", with_v=True, fused=True),
        # the three projections of one small layer: launch latency
        dict(name="adamw small layer", op="adamw", layers=1, D=256, H=4, H_kv=2, d=64, bits=32,
             param="fp32", grad="fp32", copy=True, clip=True, extra=0, packed=False),
        # four layers of 4096 x 4096 projections, master weights in fp32 and their bf16 copies
        dict(name="adamw 4 layers", op="adamw", layers=4, D=4096, H=32, H_kv=32, d=128, bits=32,
             param="fp32", grad="fp32", copy=True, clip=True, extra=0, packed=False),
        # eight layers of grouped-head projections with 8-bit states
        dict(name="adamw 8 layers 8 bit", op="adamw", layers=8, D=4096, H=32, H_kv=8, d=128,
             bits=8, param="fp32", grad="fp32", copy=True, clip=False, extra=0, packed=False),
        # many tensors of odd sizes laid end to end in one buffer, all in bf16, 8-bit states
        dict(name="adamw ragged 8 bit", op="adamw", layers=2, D=1000, H=6, H_kv=2, d=80, bits=8,
             param="bf16", grad="bf16", copy=False, clip=True, extra=60, packed=True),
        # one new token through a teacher projection: the weights' bytes
        dict(name="int8 one token", op="int8", rows=1, K=4096, cols=4096, dtype="bf16",
             out="bf16", bias=False),
        # a few ragged sequences through a grouped key projection
        dict(name="int8 77 tokens", op="int8", rows=77, K=4096, cols=1024, dtype="bf16",
             out="fp32", bias=True),
        # the teacher at the 4K workload
        dict(name="int8 4K tokens", op="int8", rows=4096, K=4096, cols=4096, dtype="bf16",
             out="bf16", bias=False),
        # the teacher at the 32K workload
        dict(name="int8 32K tokens", op="int8", rows=32768, K=4096, cols=4096, dtype="bf16",
             out="bf16", bias=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "adamw", "int8"))
    if op == "rotary":
        d = rng.choice((64, 80, 96, 128))
        H_kv = rng.choice((1, 2, 4, 8))
        H, B = H_kv * rng.choice((1, 2, 4)), rng.randint(1, 4)
        most = 32768 * 96 * 128 // 2
        N = min(_log_int(rng, 1, 32768), max(1, most // (B * (H + 2 * H_kv) * d)))
        way = rng.choice(("forward", "gradient"))
        return dict(op=op, B=B, H=H, H_kv=H_kv, N=N, d=d,
                    rot=rng.choice((d, d // 2, d // 4 * 2, d // 8 * 2)),
                    pairs=rng.choice(("half", "neighbours")),
                    scaling=rng.choice(("none", "linear", "ntk", "yarn", "bands")),
                    factor=rng.choice((2.0, 4.0, 8.0)), base=rng.choice((1e4, 5e5)), way=way,
                    dtype=rng.choice(("bf16", "fp32")), out=rng.choice(("bf16", "fp32")),
                    positions=rng.choice(("counted", "given")), with_v=rng.random() < 0.5,
                    fused=way == "forward" and rng.random() < 0.5)
    if op == "adamw":
        param = rng.choice(("fp32", "bf16"))
        d = rng.choice((64, 80, 128))
        H_kv = rng.choice((1, 2, 4, 8))
        return dict(op=op, layers=rng.randint(1, 4), D=_log_int(rng, 64, 4096),
                    H=H_kv * rng.choice((1, 2, 4)), H_kv=H_kv, d=d, bits=rng.choice((8, 32)),
                    param=param, grad=rng.choice(("fp32", "bf16")),
                    copy=param == "fp32" and rng.random() < 0.5, clip=rng.random() < 0.5,
                    extra=rng.randint(0, 40), packed=rng.random() < 0.5)
    K = _log_int(rng, 64, 8192)
    cols = _log_int(rng, 64, 8192)
    rows = min(_log_int(rng, 1, 32768), max(1, 32768 * 4096 * 4096 // (K * cols)))
    return dict(op=op, rows=rows, K=K, cols=cols, dtype=rng.choice(("bf16", "fp32")),
                out=rng.choice(("bf16", "fp32")), bias=rng.random() < 0.5)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"rotary": _rotary_inputs, "adamw": _adamw_inputs, "int8": _int8_inputs}[case["op"]](case, gen)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotary": _rotary_own, "adamw": _adamw_own, "int8": _int8_own}[op](state)
    return {"rotary": _rotary_plain, "adamw": _adamw_plain, "int8": _int8_plain}[op](state)


def work(case):
    return {"rotary": _rotary_work, "adamw": _adamw_work, "int8": _int8_work}[case["op"]](case)


def exact(case, seed):
    state = prepare(case, seed)
    return {"rotary": _rotary_exact, "adamw": _adamw_exact, "int8": _int8_exact}[case["op"]](state)


def _size(name):
    return {"bf16": 2, "fp32": 4}[name]


# ------------------------------------------------------------------------------ rotary positions
# y = m R(pos f) x on the first `rot` entries of a head, the others as they are; the gradient is
# the transposed rotation.  q and k rotate, v is only moved to the layout of the others.

def _frequencies(c):
    """Pair frequencies in 64 bits and the factor on the rotated part."""
    r, factor, base = c["rot"], c["factor"], c["base"]
    i = np.arange(r // 2, dtype=np.float64)
    f, m = base ** (-2.0 * i / r), 1.0
    first = 4096.0     # length of the sequences before the extension
    if c["scaling"] == "linear":
        f = f / factor
    elif c["scaling"] == "ntk":
        f = (base * factor ** (r / max(r - 2, 1))) ** (-2.0 * i / r)
    elif c["scaling"] == "yarn":
        at = lambda turns: r * math.log(first / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        ramp = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        f, m = f / factor * ramp + f * (1.0 - ramp), 0.1 * math.log(factor) + 1.0
    elif c["scaling"] == "bands":
        turns = first * f / (2 * math.pi)
        smooth = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = (1.0 - smooth) * f / factor + smooth * f
    return f, m


def _heads(c):
    return [c["H"], c["H_kv"]] + ([c["H_kv"]] if c["with_v"] else [])


def _rotary_inputs(c, gen):
    B, N, d, heads = c["B"], c["N"], c["d"], _heads(c)
    dtype = DTYPES[c["dtype"]]
    if c["way"] == "gradient":     # [B, H, N, d], as the loss's backward leaves them
        xs = [torch.randn(B, h, N, d, generator=gen, device="cuda").mul_(1e-3).to(dtype) for h in heads]
    elif c["fused"]:               # one projection's output, its heads side by side
        x = torch.randn(B, N, sum(heads) * d, generator=gen, device="cuda").to(dtype)
        xs = [p.view(B, N, h, d).transpose(1, 2) for p, h in zip(x.split([h * d for h in heads], -1), heads)]
    else:                          # three projections' outputs
        xs = [torch.randn(B, N, h, d, generator=gen, device="cuda").to(dtype).transpose(1, 2) for h in heads]
    positions = None
    if c["positions"] == "given":
        if N == 1:                 # each sequence at a place of its own
            positions = torch.randint(0, 131072, (B, 1), generator=gen, device="cuda")
        else:                      # packed sequences: each counts from zero again
            first = torch.rand(B, N, generator=gen, device="cuda") < 4.0 / N
            at = torch.arange(N, device="cuda").expand(B, N)
            positions = at - torch.where(first, at, 0).cummax(1).values
        positions = positions.to(torch.int32)
    f, m = _frequencies(c)
    return dict(case=c, xs=xs, positions=positions, mscale=m, inv_freq=torch.from_numpy(f).cuda())


def _rotary_out(c, x):
    """A new output in the layout that the next step reads: heads for the loss, tokens for a weight gradient."""
    B, H, N, d = x.shape
    if c["way"] == "gradient":
        return torch.empty(B, N, H, d, dtype=DTYPES[c["out"]], device=x.device).transpose(1, 2)
    return torch.empty(B, H, N, d, dtype=DTYPES[c["out"]], device=x.device)


def _rotary_own(state):
    import attention_relation_kl_b200 as rk
    c = state["case"]
    outs = [_rotary_out(c, x) for x in state["xs"]]
    return rk.relkl_rotary_qkv(state["xs"], state["inv_freq"], apply=(True, True, False)[:len(outs)],
                               positions=state["positions"], mscale=state["mscale"],
                               interleaved=c["pairs"] == "neighbours",
                               inverse=c["way"] == "gradient", out=outs)


def _rotate(c, x, cos, sin, out):
    r = c["rot"]
    x = x.float()
    if c["pairs"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.cat((ya, yb), -1) if c["pairs"] == "half" else torch.stack((ya, yb), -1).flatten(-2)
    return out.copy_(torch.cat((y, x[..., r:]), -1))


def _rotary_plain(state):
    c, xs = state["case"], state["xs"]
    pos = state["positions"]
    if pos is None:
        pos = torch.arange(c["N"], device="cuda").expand(c["B"], c["N"])
    angle = pos.double()[:, None, :, None] * state["inv_freq"]
    cos, sin = (state["mscale"] * angle.cos()).float(), (state["mscale"] * angle.sin()).float()
    if c["way"] == "gradient":
        sin = -sin
    outs = [_rotate(c, x, cos, sin, _rotary_out(c, x)) for x in xs[:2]]
    return outs + [_rotary_out(c, x).copy_(x.float()) for x in xs[2:]]


def _rotary_exact(state):
    c, r = state["case"], state["case"]["rot"]
    pos = state["positions"]
    if pos is None:
        pos = torch.arange(c["N"], device="cuda").repeat(c["B"], 1)
    # as a product of complex numbers; the gradient multiplies by the conjugate
    theta = torch.einsum("bn,p->bnp", pos.to(F64), state["inv_freq"])[:, None]
    turn = torch.polar(torch.full_like(theta, state["mscale"]), -theta if c["way"] == "gradient" else theta)
    outs = []
    for k, x in enumerate(state["xs"]):
        y = x.to(F64).clone()
        if k < 2:
            lo = slice(0, r // 2) if c["pairs"] == "half" else slice(0, r, 2)
            hi = slice(r // 2, r) if c["pairs"] == "half" else slice(1, r, 2)
            z = torch.complex(y[..., lo], y[..., hi]) * turn
            y[..., lo], y[..., hi] = z.real, z.imag
        outs.append(y)
    return outs


def _rotary_work(c):
    n = c["B"] * c["N"] * c["d"] * sum(_heads(c))
    turned = c["B"] * c["N"] * c["rot"] * (c["H"] + c["H_kv"])
    return {"bytes": n * (_size(c["dtype"]) + _size(c["out"])) + 4 * c["B"] * c["N"] * (c["positions"] == "given"),
            "flops": 3 * turned}


# ------------------------------------------------------------------- AdamW over many tensors
# g = coef g;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
# p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
# With 8-bit states m and sqrt(v) are e4m3 numbers times one fp32 scale for each 256 elements.

HYPER = dict(lr=2e-4, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
MAX_NORM = 1.0


def _shapes(c):
    layer = [(c["D"], c["H"] * c["d"]), (c["D"], c["H_kv"] * c["d"]), (c["D"], c["H_kv"] * c["d"])]
    # biases, norms and other small tensors of odd sizes, from one element on
    return layer * c["layers"] + [(1 + (k * k * 37) % (5 * c["D"]),) for k in range(c["extra"])]


def _cut(shapes, dtype, packed, count=lambda n: n):
    """Tensors of the shapes in one buffer: end to end, or each from a 256-element boundary."""
    sizes = [count(math.prod(s)) for s in shapes]
    steps = sizes if packed else [-(-n // 256) * 256 for n in sizes]
    buffer = torch.zeros(sum(steps), dtype=dtype, device="cuda")
    at = np.concatenate(([0], np.cumsum(steps)))
    parts = [buffer[int(a):int(a) + n] for a, n in zip(at, sizes)]
    return buffer, [p.view(s) if p.numel() == math.prod(s) else p for p, s in zip(parts, shapes)]


def _blocks(x):
    """x as rows of one block each, the last filled up with zeros."""
    x = x.reshape(-1)
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def _encode(x, root):
    """e4m3 codes of x by blocks, and the blocks' scales.  A positive root never becomes zero."""
    rows = _blocks(x)
    scale = rows.abs().amax(1, keepdim=True) / torch.full((), E4M3_MAX, device=x.device)
    scale = torch.where(scale < TINY, 0.0, scale)
    y = torch.where(scale > 0, rows / scale, 0.0)
    if root:
        y = torch.where(y > 0, y.clamp(min=2.0 ** -9), y)
    return y.reshape(-1)[:x.numel()].view(x.shape).to(E4M3), scale.view(-1)


def _join(xs):
    """All tensors' blocks one below the other, in fp32."""
    return torch.cat([_blocks(x.float()) for x in xs])


def _part(rows, like):
    """The tensors of which _join made these rows."""
    parts = rows.split([-(-x.numel() // BLOCK) for x in like])
    return [r.reshape(-1)[:x.numel()].view(x.shape) for r, x in zip(parts, like)]


def _adamw_inputs(c, gen):
    shapes, packed = _shapes(c), c["packed"]
    P, params = _cut(shapes, DTYPES[c["param"]], packed)
    G, grads = _cut(shapes, DTYPES[c["grad"]], packed)
    P.copy_(torch.randn(P.shape, generator=gen, device="cuda").mul_(0.02))
    # gradients whose size differs from place to place, as rows of a weight's gradient do
    size = torch.randn(-(-G.numel() // 512), generator=gen, device="cuda").exp_().mul_(1e-4).repeat_interleave(512)[:G.numel()]
    G.copy_(torch.randn(G.shape, generator=gen, device="cuda").mul_(size))
    copies, C = None, None
    if c["copy"]:
        C, copies = _cut(shapes, BF16, packed)
        C.copy_(P)
    m = torch.randn(G.shape, generator=gen, device="cuda").mul_(size).mul_(0.3)
    v = torch.rand(G.shape, generator=gen, device="cuda").add_(0.1).mul_(size).mul_(size)
    state = dict(case=c, params=params, grads=grads, copies=copies, P=P, C=C, step=100)
    if c["bits"] == 32:
        M, ms = _cut(shapes, F32, packed)
        V, vs = _cut(shapes, F32, packed)
        M.copy_(m)
        V.copy_(v)
        return state | dict(M=M, V=V, m=ms, v=vs)
    M, ms = _cut(shapes, E4M3, packed)
    V, vs = _cut(shapes, E4M3, packed)
    blocks = lambda n: -(-n // BLOCK)  # noqa: E731
    MS, m_scale = _cut(shapes, F32, packed, blocks)
    VS, v_scale = _cut(shapes, F32, packed, blocks)
    for x, codes, scales, root in ((m, ms, m_scale, False), (v.sqrt(), vs, v_scale, True)):
        for g, code, scale in zip(grads, codes, scales):
            at = g.storage_offset()
            a, b = _encode(x[at:at + g.numel()].view(g.shape), root)
            code.copy_(a)
            scale.view(-1).copy_(b)
    return state | dict(M=M, V=V, MS=MS, VS=VS, m=ms, v=vs, m_scale=[x.view(-1) for x in m_scale],
                        v_scale=[x.view(-1) for x in v_scale])


def _adamw_outputs(state, norm):
    return {k: state[k] for k in ("P", "C", "M", "V", "MS", "VS") if state.get(k) is not None} | {"norm": norm}


def _adamw_own(state):
    import attention_relation_kl_b200 as rk
    c = state["case"]
    state["step"] += 1
    clip = rk.relkl_grad_norm(state["grads"], MAX_NORM) if c["clip"] else None
    if c["bits"] == 32:
        states = [rk.AdamWState(m, v) for m, v in zip(state["m"], state["v"])]
    else:
        states = [rk.AdamWState(*s) for s in zip(state["m"], state["v"], state["m_scale"], state["v_scale"])]
    rk.relkl_adamw(state["params"], state["grads"], states, step=state["step"], copies=state["copies"],
                   grad_scale=None if clip is None else clip[1:], **HYPER)
    return _adamw_outputs(state, None if clip is None else clip[0])


def _adamw_plain(state):
    c = state["case"]
    state["step"] += 1
    grads, params, norm = [g.float() for g in state["grads"]], state["params"], None
    if c["clip"]:
        norm = torch.stack([g.square().sum(dtype=F64) for g in grads]).sum().sqrt()
        grads = torch._foreach_mul(grads, (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float())
        norm = norm.float()
    (b1, b2), lr = HYPER["betas"], HYPER["lr"]
    if c["bits"] == 32:
        m, v, p = state["m"], state["v"], [x.float() for x in params]
    else:
        grads, p = [_join(grads)], [_join(params)]
        m = [_join(state["m"]) * torch.cat(state["m_scale"])[:, None]]
        v = [(_join(state["v"]) * torch.cat(state["v_scale"])[:, None]).square_()]
    torch._foreach_mul_(m, b1)
    torch._foreach_add_(m, grads, alpha=1 - b1)
    torch._foreach_mul_(v, b2)
    torch._foreach_addcmul_(v, grads, grads, value=1 - b2)
    root = torch._foreach_sqrt(v)
    below = torch._foreach_div(root, math.sqrt(1 - b2 ** state["step"]))
    torch._foreach_add_(below, HYPER["eps"])
    p = torch._foreach_mul(p, 1 - lr * HYPER["weight_decay"])
    torch._foreach_addcdiv_(p, m, below, value=-lr / (1 - b1 ** state["step"]))
    if c["bits"] == 8:
        p = _part(p[0], params)
        (m, m_scale), (v, v_scale) = _encode(m[0], False), _encode(root[0], True)
        torch._foreach_copy_(state["m"] + state["v"], _part(m, params) + _part(v, params))
        blocks = [s.numel() for s in state["m_scale"]]
        torch._foreach_copy_(state["m_scale"] + state["v_scale"], [*m_scale.split(blocks), *v_scale.split(blocks)])
    torch._foreach_copy_(params, p)
    if state["copies"] is not None:
        torch._foreach_copy_(state["copies"], p)
    return _adamw_outputs(state, norm)


def _adamw_exact(state):
    c, t = state["case"], state["step"] + 1
    (b1, b2), lr, eps, wd = HYPER["betas"], HYPER["lr"], HYPER["eps"], HYPER["weight_decay"]
    norm, coef = None, 1.0
    if c["clip"]:
        norm = math.sqrt(sum(float(g.to(F64).pow(2).sum()) for g in state["grads"]))
        coef = min(1.0, MAX_NORM / (norm + 1e-6))
    new = {k: state[k].to(F64) for k in ("P", "C", "M", "V", "MS", "VS") if state.get(k) is not None}

    def place(key, like, x):
        at = like.storage_offset()
        new[key][at:at + x.numel()] = x.reshape(-1)

    def whole(codes, scale):
        each = scale.to(F64).repeat_interleave(BLOCK)[:codes.numel()]
        return codes.to(F64).reshape(-1) * each

    for k, (p, g) in enumerate(zip(state["params"], state["grads"])):
        g = coef * g.to(F64).reshape(-1)
        if c["bits"] == 32:
            m, v = state["m"][k].to(F64).reshape(-1), state["v"][k].to(F64).reshape(-1)
        else:
            m, v = whole(state["m"][k], state["m_scale"][k]), whole(state["v"][k], state["v_scale"][k]) ** 2
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        step = (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)) ** 0.5 + eps) + wd * p.to(F64).reshape(-1)
        q = p.to(F64).reshape(-1) - lr * step
        place("P", p, q)
        if state["copies"] is not None:
            place("C", state["copies"][k], q)
        for key, skey, x, root in (("M", "MS", m, False), ("V", "VS", v if c["bits"] == 32 else v ** 0.5, True)):
            if c["bits"] == 8:
                n = x.numel()
                rows = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=F64, device=x.device)
                rows[:n] = x
                scale = rows.view(-1, BLOCK).abs().max(1).values / E4M3_MAX
                place(skey, state["m_scale" if key == "M" else "v_scale"][k], scale)
                y = x / scale.repeat_interleave(BLOCK)[:n]
                y = torch.nan_to_num(torch.where((y > 0) & (y < 2.0 ** -9) & root, 2.0 ** -9, y))
                x = y.float().to(E4M3).to(F64)
            place(key, state["m" if key == "M" else "v"][k], x)
    return new | {"norm": norm}


def _adamw_work(c):
    n = sum(math.prod(s) for s in _shapes(c))
    each = _size(c["grad"]) + 2 * _size(c["param"]) + (2 if c["copy"] else 0)
    each += 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * each, "flops": 14 * n + (2 * n if c["clip"] else 0)}


# ------------------------------------------------------- products in 8-bit integers
# y = (sx qx) (sw qw)^T + bias with qx = rint(127 x / max|x|), sx = max|x| / 127 for each token;
# the weights' codes and their scales for each output channel are made once, before the call.

def _quantize(x):
    """Codes as fp32 numbers, and scales.  The quotient is taken in 64 bits: many lie at a half."""
    most = x.float().abs().amax(-1)
    q = x.double().mul_(127.0).div_(most[..., None]).nan_to_num_(0.0).round_()
    return q.float(), most / torch.full((), 127.0, device=x.device)


def _int8_inputs(c, gen):
    rows, K, cols = c["rows"], c["K"], c["cols"]
    # hidden states: a few channels are much larger than the others
    size = torch.where(torch.rand(K, generator=gen, device="cuda") < 0.01, 8.0, 1.0)
    x = torch.randn(rows, K, generator=gen, device="cuda").mul_(size).to(DTYPES[c["dtype"]])
    w, w_scale = _quantize(torch.randn(cols, K, generator=gen, device="cuda").mul_(K ** -0.5))
    pitch = -(-K // 16) * 16      # rows of the codes start at 16-byte boundaries
    codes = torch.zeros(cols, pitch, dtype=torch.int8, device="cuda")[:, :K]
    codes.copy_(w)
    bias = torch.randn(cols, generator=gen, device="cuda").mul_(0.1) if c["bias"] else None
    return dict(case=c, x=x, w=codes, w_scale=w_scale, bias=bias)


def _int8_own(state):
    import attention_relation_kl_b200 as rk
    return rk.relkl_linear_i8(state["x"], state["w"], state["w_scale"], bias=state["bias"],
                              out_dtype=DTYPES[state["case"]["out"]])


def _int8_plain(state):
    q, scale = _quantize(state["x"])
    y = torch.matmul(q, state["w"].float().t()) * (scale[:, None] * state["w_scale"])
    if state["bias"] is not None:
        y = y + state["bias"]
    return y.to(DTYPES[state["case"]["out"]])


def _int8_exact(state):
    w = state["w"].to(F64) * state["w_scale"].to(F64)[:, None]
    outs = []
    for x in state["x"].split(4096):
        x = x.to(F64)
        most = x.abs().max(1, keepdim=True).values
        y = torch.einsum("rk,ck->rc", torch.round(127.0 * x / most) * (most / 127.0), w)
        outs.append(y if state["bias"] is None else y + state["bias"].to(F64))
    return torch.cat(outs)


def _int8_work(c):
    rows, K, cols = c["rows"], c["K"], c["cols"]
    nbytes = rows * K * _size(c["dtype"]) + cols * (K + 4) + rows * cols * _size(c["out"]) + 4 * cols * c["bias"]
    return {"bytes": nbytes, "flops": 2 * rows * K * cols}
