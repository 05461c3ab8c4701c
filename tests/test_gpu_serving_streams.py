"""Serving calls that overlap: one on the current stream, the next on an
explicit one, nothing waited for between them and nothing allocated by the
caller."""
import numpy as np
import pytest
import torch

from _serving import Batch, bf16_from

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("dual_scale_solver_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dual_scale_solver_b200 import build
    build.build()


def _work():
    """(name, call of a stream) of calls that cut their work into pieces, and
    of ones with several results."""
    calls = []
    for seqs, group in (([(1, 3000), (1, 700)], 4), ([(90, 1500)], 4), ([(1, 2500), (120, 1300), (3, 900)], 2)):
        b = Batch(seqs, 16, 2, 64, "mxfp4", 32)
        cache, _ = b.fill()
        q, meta = bf16_from(b.rng, (b.tokens, 2 * group, 64)).cuda(), b.device()
        calls.append(lambda s, q=q, c=cache, m=meta, f=b.fmt: (dq.kv_attention(q, c, *m, f, stream=s),))
        calls.append(lambda s, c=cache, m=meta, f=b.fmt, n=b.tokens: dq.kv_read(c, *m, f, n, stream=s))
    rng = np.random.default_rng(21)
    x, r, w = (bf16_from(rng, shape).cuda() for shape in ((300, 4096), (300, 4096), (4096,)))
    f8 = dq.format_preset("mxfp8_e4m3")
    calls.append(lambda s: dq.add_rmsnorm_quant(x, w, f8, residual=r, stream=s))
    return calls


def test_current_and_explicit_stream_back_to_back():
    calls = _work()
    want = [[t.clone() for t in c(None)] for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for i in range(60):
        j, k = i % len(calls), (i * 3 + 1) % len(calls)
        got.append((j, calls[j](None)))
        got.append((k, calls[k](side)))
        if i % 4 == 3:                               # results dropped while either stream may be at work
            del got[-6:-2]
    torch.cuda.synchronize()
    for i, result in got:
        assert all(torch.equal(a, b) for a, b in zip(result, want[i]))
    assert dq.last_device_status() == 0


def test_results_are_read_on_the_current_stream_and_dropped():
    calls = _work()
    want = [[t.clone() for t in c(None)] for c in calls]
    torch.cuda.synchronize()
    side, sums = torch.cuda.Stream(), []
    for i in range(40):
        j = i % len(calls)
        result = calls[j](side)
        torch.cuda.current_stream().wait_stream(side)
        sums.append((j, [t.clone() for t in result]))
        del result                                   # (the next call may take its memory)
    torch.cuda.synchronize()
    for j, copies in sums:
        assert all(torch.equal(a, b) for a, b in zip(copies, want[j]))


def test_a_captured_step_that_forks():
    """Two attention calls of one graph on two streams, each with the
    workspace that it allocates."""
    calls = _work()
    picked = [calls[0], calls[2]]
    want = [[t.clone() for t in c(None)] for c in picked]
    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        a = picked[0](None)
        b = picked[1](side)
        main.wait_stream(side)
    for _ in range(5):
        for t in (*a, *b):
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for result, w in zip((a, b), want):
        assert all(torch.equal(x, y) for x, y in zip(result, w))
    assert dq.last_device_status() == 0
