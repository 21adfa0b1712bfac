"""Calls of the loss from two threads at once, each on a stream of its own."""
import ctypes
import threading

import pytest
import torch

import attention_relation_kl_b200 as rk
from attention_relation_kl_b200 import _abi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def test_fp32_heads_of_two_sizes():
    # the CUDA-core path, whose blocks take 17 and 66 KB of shared memory (21 and 70 KB backward);
    # through the C ABI, so that little but the launches is between two calls
    lib, ws = _abi.lib(), rk.workspace("cuda")
    work = []
    for d in (32, 128):
        gen = torch.Generator().manual_seed(d)
        xt, xs = (torch.randn(1, 1, 40, d, generator=gen).cuda() for _ in range(2))
        kl, stats = rk.relkl_fwd(xt, xs)
        work.append((xt, xs, kl, stats, rk.relkl_bwd(xt, xs, stats)))
    go, failed = threading.Barrier(2), []

    def calls(xt, xs, want, want_stats, want_dx):
        try:
            stream = torch.cuda.Stream()
            kl, stats, dx = (torch.empty_like(t) for t in (want, want_stats, want_dx))
            stream.wait_stream(torch.cuda.current_stream())
            desc = ctypes.byref(rk.make_desc(xt))
            at = [t.data_ptr() for t in (xt, xs, kl, stats, dx)]
            tail = (ws.data_ptr(), ws.numel(), stream.cuda_stream)
            go.wait(60)
            for _ in range(10000):
                code = lib.relkl_fwd(desc, *at[:4], *tail) or lib.relkl_bwd(desc, at[0], at[1], at[3], None, at[4], *tail)
                assert code == 0, code
            stream.synchronize()
            assert torch.equal(kl, want) and torch.equal(stats, want_stats)
            # dx is added up by atomics: an element has at most four addends (two row blocks, on
            # both sides of G), and two orders of their sum differ by 2 * 3 * 2^-24 of their
            # magnitudes' sum.  |G| <= 1 / (N sqrt(d)), its rows' sums 2 / (N sqrt(d)).
            N, d = xs.shape[2:]
            room = 6 * 2.0 ** -24 * (1 + 2 / N) / d ** 0.5 * float(xs.abs().max())
            assert float((dx - want_dx).abs().max()) <= room
        except Exception as e:      # seen by the test's own thread
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=calls, args=a) for a in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
