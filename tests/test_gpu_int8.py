"""Products in 8-bit integers on the GPU.

Codes are compared exactly: rint(127 x / m) in float64 is the exact one, as a quotient of
a 31-bit and a 24-bit number that is no half differs from every half by 2^-26 of itself.
Sums are exact integers; with u = 2^-24 a result rounds the sum, the token's scale, the
product of the scales and the last sum: 4 u |sum sx sw| + u |bias|, plus 2^-8 in bf16.
"""
import threading

import numpy as np
import pytest
import torch

import attention_relation_kl_b200 as rk
from attention_relation_kl_b200 import _abi

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    assert rk.relkl_get_device_error() == (0, 0)     # no wait ran out


def _np(x):
    return x.detach().cpu().double().numpy()


def _codes(x):
    """(codes, scales) in float64 by the definition."""
    x = _np(x).reshape(-1, x.shape[-1])
    most = np.abs(x).max(1)
    with np.errstate(all="ignore"):
        q = np.rint(127.0 * x / most[:, None])
    q[~(most > 0) | ~np.isfinite(most)] = 0
    return q, np.where(np.isfinite(most), most / 127.0, np.nan)


def _check(y, q, sx, w, sw, bias=None):
    acc = q @ _np(w).T                                   # below 2^53: exact
    scale = sx[:, None] * _np(sw)
    want = acc * scale + (0 if bias is None else _np(bias))
    tol = 4 * U * np.abs(acc * scale) + (0 if bias is None else U * np.abs(_np(bias))) + U * np.abs(want)
    if y.dtype == BF16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    got = _np(y).reshape(want.shape)
    bad = ~((np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3])


def _randn(shape, dtype=F32, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=gen).to(dtype).cuda()


def _weights(cols, K, seed=1):
    return rk.relkl_quantize_rows(_randn((cols, K), F32, seed))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 15), (9, 16), (2, 100), (33, 129), (5, 2048), (4, 2056),
                                    (3, 5000), (1000, 64)])
def test_codes_are_exact(rows, K, dtype):
    x = _randn((rows, K), dtype, rows + K)
    q, s = rk.relkl_quantize_rows(x)
    want, scale = _codes(x)
    assert q.shape == (rows, K) and q.stride(0) % 16 == 0
    assert np.array_equal(_np(q), want)
    assert np.all(np.abs(_np(s) - scale) <= U * scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_codes_of_ties_extremes_and_rows_without_a_scale(dtype):
    K = 40
    x = torch.zeros(12, K)
    x[0] = (torch.arange(K) - 20) + 0.5                      # with 127 as the largest: exact halves
    x[0, 0] = 127.0
    x[1, :3] = torch.tensor([3e38, -3e38, 1.5e38])
    x[2, :3] = torch.tensor([1e-40, -1e-40, 5e-41])          # subnormal
    x[3, :2] = torch.tensor([float("inf"), 1.0])
    x[4, :2] = torch.tensor([float("nan"), 1.0])
    x[5, :2] = torch.tensor([float("-inf"), float("nan")])
    x[7] = -1.0
    x[8, 5] = 1e-30
    x[9] = torch.linspace(-1, 1, K)
    x[10, :2] = torch.tensor([2.0 ** -149, -(2.0 ** -149)])
    x[11] = torch.nextafter(torch.full((K,), 0.5), torch.tensor(1.0)) * 63.0 / 64
    x = x.to(dtype).cuda()
    q, s = rk.relkl_quantize_rows(x)
    want, scale = _codes(x)
    assert np.array_equal(_np(q), want)
    got = _np(s)
    assert np.array_equal(np.isnan(got), np.isnan(scale)) and np.isnan(got[3:6]).all()
    ok = ~np.isnan(scale)
    assert np.all(np.abs(got[ok] - scale[ok]) <= U * scale[ok] + 2.0 ** -150)
    # products of such rows: NaN for the whole row, the bias for a row of zeros
    w, sw = _weights(9, K)
    bias = _randn((9,), F32, 3)
    z = rk.relkl_linear_i8(x, w, sw, bias=bias, out_dtype=F32)
    y = torch.cat([rk.relkl_linear_i8(x[k:k + 4], w, sw, bias=bias, out_dtype=F32) for k in (0, 4)])
    for t in (y, z[:8]):
        assert torch.isnan(t[3:6]).all() and torch.equal(t[6], bias)
        assert torch.isfinite(t[[0, 7]]).all()
    assert torch.equal(y.view(torch.int32), z[:8].view(torch.int32))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_codes_of_every_pair_of_bf16_mantissas(dtype):
    # a row for each mantissa of its largest element, with every bf16 number down to 2^-12
    # of it: every half that bf16 numbers can make is there
    b = torch.arange(128, 256, dtype=torch.float32)
    x = torch.cat([b * 2.0 ** -e for e in range(13)])
    rows = torch.where(x[None, :] <= b[:, None], x[None, :], 0.0)
    rows = torch.cat((rows, -rows), 1)
    for scale in (1.0, 2.0 ** -60, 2.0 ** 90, 2.0 ** -120):
        y = (rows * scale).to(dtype).cuda()
        q, _ = rk.relkl_quantize_rows(y)
        assert np.array_equal(_np(q), _codes(y)[0])


ROWS = [1, 2, 4, 5, 6, 7, 8, 9, 16, 77, 128, 129, 300]


@pytest.mark.parametrize("cols,K", [(1, 1), (7, 17), (64, 128), (65, 100), (200, 129), (1000, 64), (33, 4096),
                                    (136, 5000), (520, 1040)])
@pytest.mark.parametrize("rows", ROWS)
def test_products(rows, cols, K):
    xt, yt = (BF16, F32) if (rows + cols) % 2 else (F32, BF16)
    x = _randn((rows, K), xt, rows)
    w, sw = _weights(cols, K)
    bias = _randn((cols,), F32, 2) if rows % 3 else None
    q, sx = _codes(x)
    y = rk.relkl_linear_i8(x, w, sw, bias=bias, out_dtype=yt)
    _check(y, q, sx, w, sw, bias)
    # the same bits from the codes by themselves
    z = rk.relkl_matmul_i8(*rk.relkl_quantize_rows(x), w, sw, bias=bias, out_dtype=yt)
    assert torch.equal(y, z)


@pytest.mark.parametrize("rows,cols,K", [(2500, 1000, 300), (5121, 1000, 136), (700, 4096, 256), (4100, 2056, 520),
                                         (20000, 264, 144)])
@pytest.mark.parametrize("yt", [BF16, F32])
def test_many_tiles(rows, cols, K, yt):
    x = _randn((rows, K), BF16, 4)
    w, sw = _weights(cols, K)
    q, sx = _codes(x)
    _check(rk.relkl_linear_i8(x, w, sw, out_dtype=yt), q, sx, w, sw)


def test_longest_sums_and_lowest_codes():
    K = 131071
    q = torch.full((3, K + 1), 127, dtype=torch.int8, device="cuda")[:, :K]
    w = torch.full((5, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
    w[1] = 127
    one3, one5 = torch.ones(3, device="cuda"), torch.ones(5, device="cuda")
    y = rk.relkl_matmul_i8(q, one3, w, one5, out_dtype=F32)
    _check(y, _np(q), np.ones(3), w, one5)
    q[0] = -128
    y = rk.relkl_matmul_i8(q, one3, w, one5, out_dtype=F32)
    _check(y, _np(q), np.ones(3), w, one5)
    x = torch.full((1, K), 2.0, dtype=BF16, device="cuda")
    _check(rk.relkl_linear_i8(x, w, one5), *_codes(x), w, one5)


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_views_strides_and_alignment(rows, dtype, offset):
    K, cols = 96, 72
    x = _randn((rows, K + 37), dtype, 5)[:, offset:offset + K]
    w, sw = _weights(cols, K)
    q, sx = _codes(x)
    buf = torch.full((rows, cols + 11), 7.0, dtype=dtype, device="cuda")
    y = buf[:, offset:offset + cols]
    assert rk.relkl_linear_i8(x, w, sw, out_dtype=dtype, out=y) is y
    _check(y, q, sx, w, sw)
    rest = torch.cat((buf[:, :offset], buf[:, offset + cols:]), 1)
    assert torch.equal(rest, torch.full_like(rest, 7.0))      # beside the output: as it was
    # leading dimensions, and codes cut out of wider rows
    x3 = _randn((2, rows, K), dtype, 6)
    y3 = rk.relkl_linear_i8(x3, w, sw)
    assert y3.shape == (2, rows, cols) and y3.dtype == dtype
    _check(y3, *_codes(x3), w, sw)
    wide = torch.zeros(cols, 128, dtype=torch.int8, device="cuda")
    wide.fill_(99)
    wide[:, 16:16 + K] = w
    assert torch.equal(rk.relkl_linear_i8(x3, wide[:, 16:16 + K], sw), y3)
    one = rk.relkl_linear_i8(x3[0, 0], w, sw)
    assert one.shape == (cols,) and torch.equal(one, y3[0, 0])


# rows of y that start at 16-byte boundaries and end anywhere, in every kernel
@pytest.mark.parametrize("yt", [BF16, F32])
@pytest.mark.parametrize("rows", [3, 40, 300, 600, 5000])
@pytest.mark.parametrize("cols", [3, 993, 1001, 1002, 1004, 1007, 1008])
def test_nothing_is_written_beside_a_wide_output(cols, rows, yt):
    x = _randn((rows, 64), BF16, 16)
    w, sw = _weights(cols, 64)
    buf = torch.full((rows + 2, (cols + 15) // 8 * 8), 7.0, dtype=yt, device="cuda")
    rk.relkl_linear_i8(x, w, sw, out_dtype=yt, out=buf[1:-1, :cols])
    assert torch.equal(buf[1:-1, :cols], rk.relkl_linear_i8(x, w, sw, out_dtype=yt))
    _check(buf[1:-1, :cols], *_codes(x), w, sw)
    buf[1:-1, :cols] = 7.0
    assert (buf == 7.0).all()


@pytest.mark.parametrize("rows", [2, 40, 300, 600, 5000])
@pytest.mark.parametrize("K", [1, 5, 15, 17, 31, 100, 130, 1001])
def test_what_lies_behind_the_rows_of_codes_is_not_read(K, rows):
    cols, pitch = 1000, (K + 31) // 16 * 16

    def padded(q):
        wide = torch.full((q.shape[0], pitch), 99, dtype=torch.int8, device="cuda")
        wide[:, :K] = q
        return wide[:, :K]

    x = _randn((rows, K), BF16, 17)
    w, sw = _weights(cols, K)
    q, s = rk.relkl_quantize_rows(x)
    want = rk.relkl_matmul_i8(padded(q), s, padded(w), sw, out_dtype=F32)
    _check(want, *_codes(x), w, sw)
    assert torch.equal(rk.relkl_linear_i8(x, padded(w), sw, out_dtype=F32), want)


@pytest.mark.parametrize("cols", [4096, 4097])
def test_offsets_past_32_bits(cols):
    rows, K = 2 ** 31 // 4096 + 300, 16              # more than 2^31 results
    w, sw = _weights(cols, K)
    x = _randn((rows, K), BF16, 15)
    y = rk.relkl_linear_i8(x, w, sw)
    for at in (0, rows - 259):
        assert torch.equal(y[at:at + 259], rk.relkl_linear_i8(x[at:at + 259], w, sw))


def test_no_rows_and_no_channels():
    w, sw = _weights(8, 32)
    assert rk.relkl_linear_i8(torch.empty(0, 32, device="cuda"), w, sw).shape == (0, 8)
    assert rk.relkl_linear_i8(_randn((5, 32)), w[:0], sw[:0]).shape == (5, 0)
    q, s = rk.relkl_quantize_rows(torch.empty(0, 32, device="cuda"))
    assert q.shape == (0, 32) and rk.relkl_matmul_i8(q, s, w, sw).shape == (0, 8)


@pytest.mark.parametrize("rows", [2, 300])
def test_streams_and_captured_graphs(rows):
    K, cols = 512, 384
    w, sw = _weights(cols, K)
    x = _randn((rows, K), BF16, 7)
    want = rk.relkl_linear_i8(x, w, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = rk.relkl_linear_i8(x, w, sw, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    # two graphs of the same call, replayed at the same time on two streams
    xs, outs, graphs = [x.clone(), x.clone()], [], []
    for t in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(rk.relkl_linear_i8(t, w, sw))
        graphs.append(g)
    for k, t in enumerate(xs):
        t.copy_(_randn((rows, K), BF16, 20 + k))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for t, o in zip(xs, outs):
        assert torch.equal(o, rk.relkl_linear_i8(t, w, sw))


# The two pair kernels.  A wait is tried for a hundred microseconds or so before its limit is
# looked at, so the sums are as long as they may be: 300 us and more.
@pytest.mark.parametrize("rows,cols,K", [(500, 4096, 131071), (5000, 1024, 131071)])
def test_wait_that_runs_out_is_reported_and_the_context_survives(rows, cols, K):
    gen = torch.Generator(device="cuda").manual_seed(8)
    q, s = rk.relkl_quantize_rows(torch.randn(rows, K, generator=gen, device="cuda").to(BF16))
    w, sw = rk.relkl_quantize_rows(torch.randn(cols, K, generator=gen, device="cuda"))
    ws = torch.empty(rk.relkl_workspace_bytes(), dtype=torch.uint8, device="cuda")
    rk.relkl_workspace_init(ws)
    want = rk.relkl_matmul_i8(q, s, w, sw, ws=ws)
    assert rk.relkl_get_device_error(ws) == (0, 0)
    old = rk.relkl_set_wait_timeout_ns(0)
    try:
        rk.relkl_matmul_i8(q, s, w, sw, ws=ws)
        code, where = rk.relkl_get_device_error(ws)
    finally:
        rk.relkl_set_wait_timeout_ns(old)
    assert code == _abi.RELKL_ERR_TIMEOUT and where != 0
    rk.relkl_workspace_init(ws)
    assert torch.equal(rk.relkl_matmul_i8(q, s, w, sw, ws=ws), want)
    assert rk.relkl_get_device_error(ws) == (0, 0)


def test_bad_calls_are_refused():
    x = _randn((4, 64))
    w, sw = _weights(8, 64)
    q, s = rk.relkl_quantize_rows(x)
    for call in (lambda: rk.relkl_linear_i8(x[:, :63], w, sw),
                 lambda: rk.relkl_linear_i8(x, w, sw[:7]),
                 lambda: rk.relkl_linear_i8(x, w, sw.half()),
                 lambda: rk.relkl_linear_i8(x, w.float(), sw),
                 lambda: rk.relkl_linear_i8(x, w[:, 1:33], sw),
                 lambda: rk.relkl_linear_i8(x, w, sw, bias=torch.zeros(9, device="cuda")),
                 lambda: rk.relkl_linear_i8(x, w.cpu(), sw),
                 lambda: rk.relkl_linear_i8(x, w, sw.cpu()),
                 lambda: rk.relkl_linear_i8(x, w, sw, out=torch.empty(4, 9, device="cuda")),
                 lambda: rk.relkl_linear_i8(x, w, sw, out=x[:, :8]),
                 lambda: rk.relkl_linear_i8(x.t(), w, sw),
                 lambda: rk.relkl_linear_i8(_randn((2, 3, 4, 64)).transpose(0, 1), w, sw),
                 lambda: rk.relkl_matmul_i8(q, s[:3], w, sw),
                 lambda: rk.relkl_matmul_i8(q[:, :48], s, w, sw)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rk.relkl_linear_i8(x.half(), w, sw), lambda: rk.relkl_quantize_rows(x.half()),
                 lambda: rk.relkl_linear_i8(x, w, sw, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(RuntimeError):
        rk.relkl_quantize_rows(torch.zeros(2, 131072, device="cuda"))


def test_given_outputs_are_seen_as_changed_in_place():
    x, w = torch.randn(5, 64, device="cuda"), torch.randn(48, 64, device="cuda")
    (q, s), (qw, sw) = rk.relkl_quantize_rows(x), rk.relkl_quantize_rows(w)
    for call in (lambda out: rk.relkl_linear_i8(x, qw, sw, out=out),
                 lambda out: rk.relkl_matmul_i8(q, s, qw, sw, out=out, out_dtype=torch.float32)):
        out = torch.ones(5, 48, device="cuda")
        a = torch.zeros_like(out, requires_grad=True)
        y = (a * out).sum()
        call(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()


def test_few_long_rows_from_two_threads():
    # codes of 48 to 96 KB in shared memory, of other sizes in each thread
    work = []
    for k, (rows, K) in enumerate([(4, 24000), (4, 13000)]):
        w, sw = _weights(8, K, k)
        x = _randn((rows, K), BF16, 10 + k)
        work.append((x, w, sw, rk.relkl_linear_i8(x, w, sw)))
    go, failed = threading.Barrier(2), []

    def calls(x, w, sw, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                go.wait(60)
                for _ in range(3000):
                    y = rk.relkl_linear_i8(x, w, sw)
                torch.cuda.current_stream().synchronize()
                assert torch.equal(y, want)
        except Exception as e:      # seen by the test's own thread
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=calls, args=a) for a in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


# codes just below, at and above 48 KB, where a block's own shared memory counts too
@pytest.mark.parametrize("rows,K", [(4, 12288), (4, 12272), (4, 12208), (4, 12304), (3, 16384), (3, 16320), (2, 24576),
                                    (2, 24500), (1, 49152), (1, 49088), (1, 49100), (1, 98304)])
def test_few_rows_around_the_default_limit_of_shared_memory(rows, K):
    w, sw = _weights(24, K, 3)
    x = _randn((rows, K), BF16, 4)
    q, sx = _codes(x)
    _check(rk.relkl_linear_i8(x, w, sw, out_dtype=F32), q, sx, w, sw)


# sums by one, two and four CTAs of a cluster: the limits' both sides, shares of unequal length,
# and tiles at the rows' and the channels' end
@pytest.mark.parametrize("rows,cols,K", [(77, 1000, 2432), (77, 1000, 2433), (9, 2370, 3968), (9, 2370, 4100),
                                         (300, 900, 3968), (300, 900, 4500), (129, 2300, 8000),
                                         (77, 1000, 2560), (77, 1000, 2561), (9, 2370, 3585), (9, 2370, 3584),
                                         (8, 64, 1540), (5, 64, 1537), (5, 130, 1536), (300, 900, 5600)])
@pytest.mark.parametrize("yt", [BF16, F32])
def test_shares_of_a_split_sum(rows, cols, K, yt):
    x = _randn((rows, K), BF16, 6)
    w, sw = _weights(cols, K)
    q, sx = _codes(x)
    _check(rk.relkl_linear_i8(x, w, sw, out_dtype=yt), q, sx, w, sw)
