"""The norm, recurrence and epilogue calls as a serving loop uses them: they allocate
nothing on the device, run in a captured graph, and from two host threads on two
streams at once; and the recurrence's wait between CTAs gives up in bounded time."""
import threading

import numpy as np
import pytest

import oracle
import t3_synth
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _block(seed, rows, d, length):
    """Buffers of norm, product, recurrence and their gradients over `rows` tokens of d channels, and the
    calls in order; every output, workspace and scratch is here already."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    def room(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")
    f32, i8 = torch.float32, torch.int8
    b, n = rows // length, 2 * d
    w = t3_synth.ternary(t3_synth.rng(seed), (d, n))
    x, res, gamma = rand(rows, d), rand(rows, d), 1 + 0.1 * rand(d, dtype=f32)
    wp = torch.from_numpy(oracle.pack(w)).cuda()
    q, s, rstd, total = room(rows, d, dtype=i8), room(rows, dtype=f32), room(rows, dtype=f32), room(rows, d)
    both, pre, bias = room(rows, n), room(rows, n), rand(n, dtype=f32)
    h0, last = rand(b, d, dtype=f32), room(b, d, dtype=f32)
    resets = (torch.rand((b, length), generator=g, device="cuda") < 0.1).to(torch.uint8)
    h, dh, dl, dboth, dh0 = room(b, length, d), rand(b, length, d), rand(b, d, dtype=f32), room(b, length, n), room(b, d, dtype=f32)
    dz, dbias, dx, dgamma = room(rows, n), room(n, dtype=f32), room(rows, d), room(d, dtype=f32)
    ws, cols = room(rows, n, dtype=torch.int32), room(t3.load().t3_colsum_workspace(rows, n), dtype=f32)
    scratch = room(max(t3.load().t3_gemm_fwd_act_scratch(rows, n, d), 16), dtype=torch.uint8)

    def run(stream=None):
        t3.t3_rmsnorm_quant(x, gamma, res, q=q, row_scale=s, rstd=rstd, sum_out=total, stream=stream)
        t3.t3_gemm_fwd_act(q, wp, K=d, row_scale=s, bias=bias, act=t3.T3_ACT_SILU, kind=t3.T3_OUT_BF16, C=both, pre=pre,
                           workspace=ws, scratch=scratch, stream=stream)
        view = both.view(b, length, n)
        t3.t3_gated_scan_fwd(view[..., :d], view[..., d:], h0, resets, h=h, h_last=last, stream=stream)
        t3.t3_gated_scan_bwd(view[..., :d], view[..., d:], h, dh, h0, resets, dl, dgate=dboth[..., :d], dcand=dboth[..., d:],
                             dh0=dh0, stream=stream)
        t3.t3_act_bwd(dboth.view(rows, n), pre, t3.T3_ACT_SILU, dz=dz, dbias=dbias, workspace=cols, stream=stream)
        t3.t3_rmsnorm_bwd(dh.view(rows, d), total, rstd, gamma, dx=dx, dgamma=dgamma, workspace=cols, stream=stream)
    outs = [q, s, rstd, total, both, pre, h, last, dboth, dh0, dz, dbias, dx, dgamma]
    return run, outs


# single tokens; a few rows; odd widths laid out in scratch; many rows (CTA pairs, clusters)
SIZES = [(4, 512, 1), (24, 264, 12), (600, 243, 300), (2048, 640, 1024)]


@pytest.mark.parametrize("rows,d,length", SIZES)
def test_calls_allocate_nothing_and_replay(rows, d, length):
    run, outs = _block(rows, rows, d, length)
    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    torch.cuda.synchronize()
    before, free = torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]
    run()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    assert torch.cuda.mem_get_info()[0] == free
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    for _ in range(3):
        for t in outs:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(outs, want):
            assert torch.equal(t, w)
    assert t3.t3_last_device_error()[0] == t3.T3_OK


def test_two_threads_on_two_streams():
    blocks = [_block(7, 2048, 640, 1024), _block(8, 600, 243, 300)]
    want = []
    for run, outs in blocks:
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.fill_(3)
    torch.cuda.synchronize()
    errors = []

    def work(run):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                run(stream)
            stream.synchronize()
        except Exception as e:  # reported by the assertion below
            errors.append(e)
    threads = [threading.Thread(target=work, args=(run,)) for run, _ in blocks]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for (_, outs), ws in zip(blocks, want):
        for t, w in zip(outs, ws):
            assert torch.equal(t, w)
    assert t3.t3_last_device_error()[0] == t3.T3_OK


def test_the_recurrences_wait_gives_up():
    """The wait on a cluster's other CTAs, on a barrier that nothing completes: it ends within its limit, the
    error word says so once, and the next recurrence is right."""
    gate = torch.randn((1, 3000, 64), device="cuda")
    cand = torch.randn((1, 3000, 64), device="cuda")
    want = t3.t3_gated_scan_fwd(gate, cand)
    assert t3.t3_last_device_error()[0] == t3.T3_OK
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    t3.t3_selftest_scan_wait_timeout(5_000_000)
    end.record()
    got = t3.t3_gated_scan_fwd(gate, cand)
    assert t3.t3_last_device_error() == (t3.T3_ETIMEOUT, (11 << 8) | 7)
    assert 4.5 <= begin.elapsed_time(end) < 500
    assert t3.t3_last_device_error() == (t3.T3_OK, 0)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    for limit in (0, 999, 2_000_000_001):
        with pytest.raises(t3.T3Error):
            t3.t3_selftest_scan_wait_timeout(limit)
