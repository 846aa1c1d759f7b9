"""What t3_gemm_fwd_act takes besides its operands: scratch by the library's own
limit of small products, and an int32 workspace only where a product does not end
in its epilogue."""
import numpy as np
import pytest

import oracle
import t3_synth
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.fixture
def allocations(monkeypatch):
    """(elements, type) of every tensor the binding allocates."""
    seen, empty = [], t3._empty

    def watch(shape, dtype, dev, stream):
        t = empty(shape, dtype, dev, stream)
        seen.append((t.numel(), dtype))
        return t
    monkeypatch.setattr(t3, "_empty", watch)
    return seen


def test_scratch_follows_the_limit_of_small_products():
    lib = t3.load()
    f, now = lib.t3_gemm_fwd_act_scratch, lib.t3_gemm_fwd_act_scratch_now
    sizes = [(100, 243, 731), (1500, 1001, 129), (64, 729, 243), (33, 8192, 4001)]
    prev = t3.t3_set_small_product_limit(0)
    try:
        for m, n, k in sizes:
            assert now(m, n, k) == f(m, n, k) > 0
        t3.t3_set_small_product_limit(1 << 40)
        for m, n, k in sizes:
            assert now(m, n, k) == 0
        macs = 100 * 243 * 731
        t3.t3_set_small_product_limit(8 * macs)  # aligned operands: an eighth of the limit
        assert now(100, 243, 731) == 0 and now(100, 243, 732) > 0
    finally:
        t3.t3_set_small_product_limit(prev)
    assert now(32, 729, 243) == now(64, 728, 256) == now(64, 0, 3) == now(-1, 3, 3) == 0


def test_scratch_of_sizes_past_64_bits():
    """Sizes that the checks of arguments let through, whose bytes pass 64 bits: the largest count there is, not a
    negative one that any scratch would satisfy."""
    big = (1 << 31) - 1
    for m, n, k in [(big, big, 3), (big, big, big), (big, big - 4, 61)]:
        assert t3.load().t3_gemm_fwd_act_scratch(m, n, k) == (1 << 63) - 1
    assert t3.load().t3_gemm_fwd_act_scratch(big, 3, 61) == big * 64 + 4 * 16 + big * 16


@pytest.mark.gpu
@pytest.mark.parametrize("limit", [0, 8 * 100 * 243 * 731, 1 << 40])
def test_binding_gives_scratch_where_the_library_takes_it(limit, allocations):
    t3.t3_set_small_product_limit(limit)  # the suite's fixture puts it back
    g = t3_synth.rng(1)
    for m, n, k in [(100, 243, 731), (100, 243, 732), (300, 1001, 513)]:
        a, w = t3_synth.int8_uniform(g, (m, k)), t3_synth.ternary(g, (k, n))
        want = a.astype(np.int64) @ w.astype(np.int64)
        del allocations[:]
        out = t3.t3_gemm_fwd_act(_dev(a), _dev(oracle.pack(w)))
        np.testing.assert_array_equal(out.cpu().numpy(), want.astype(np.float32))
        got = [n for n, dtype in allocations if dtype == torch.uint8]
        need = t3.load().t3_gemm_fwd_act_scratch(m, n, k)
        assert got == ([need] if 8 * m * n * k > limit else []), (m, n, k)


# every route: one and a few rows, tiles that are few and many, CTA pairs, odd rows laid out, and what is
# left for the int32 product and a kernel behind it (decode batches, long reductions, empty ones)
SHAPES = [(1, 512, 256), (2, 8192, 33_000), (5, 640, 640), (16, 512, 256), (27, 8192, 2048), (27, 729, 243), (33, 192, 128),
          (300, 384, 256), (300, 273, 96), (777, 2304, 640), (129, 260, 4001), (200, 8, 16), (64, 72, 66_048), (40, 100, 66_001),
          (3, 5, 0), (64, 5, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("limit", [0, 1 << 29])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_a_workspace_is_asked_for_exactly_where_it_is_needed(m, n, k, limit, allocations):
    t3.t3_set_small_product_limit(limit)
    g = t3_synth.rng(m + n + k)
    a, w = t3_synth.int8_uniform(g, (m, k)), t3_synth.ternary(g, (k, n))
    rs = _dev((g.random(m) * 0.02 + 0.01).astype(np.float32))
    z = (a.astype(np.int64) @ w.astype(np.int64)).astype(np.float32) * rs.cpu().numpy()[:, None]
    packed = oracle.pack(w) if k else np.zeros((n, 0), np.uint8)
    R = _dev(g.standard_normal((m, n)).astype(np.float32)).bfloat16()
    want = (torch.from_numpy(z).cuda() + R.float()).bfloat16()
    lib = t3.load()

    def off(t, by):
        buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
        v = buf[by:].view(t.shape)
        v.copy_(t)
        return v
    need = lib.t3_gemm_fwd_act_scratch(m, n, k)
    for odd in range(6):  # nothing, or one buffer off its boundary
        A, Wp, C = off(_dev(a), int(odd == 1)), off(_dev(packed), int(odd == 2)), off(torch.zeros_like(R), int(odd == 3))
        r, pre = off(R, int(odd == 4)), off(torch.zeros_like(R), int(odd == 5))
        for room in sorted({0, need}):
            scratch = torch.empty(room, dtype=torch.uint8, device="cuda") if room else None
            ws = lib.t3_gemm_fwd_act_workspace(A.data_ptr(), Wp.data_ptr(), C.data_ptr(), m, n, k, r.data_ptr(),
                                               pre.data_ptr(), t3.T3_OUT_BF16, room)
            assert ws in (0, m * n)
            C.fill_(7)
            rc = lib.t3_gemm_fwd_act(A.data_ptr(), Wp.data_ptr(), C.data_ptr(), m, n, k, rs.data_ptr(), None, None, 0,
                                     r.data_ptr(), pre.data_ptr(), t3.T3_OUT_BF16, None,
                                     None if scratch is None else scratch.data_ptr(), room,
                                     torch.cuda.current_stream().cuda_stream)
            if ws:
                assert rc == t3.T3_EINVAL and torch.all(C == 7)
            else:
                assert rc == t3.T3_OK and torch.equal(C, want)
        del allocations[:]
        C.fill_(7)
        t3.t3_gemm_fwd_act(A, Wp, K=k, row_scale=rs, residual=r, kind=t3.T3_OUT_BF16, C=C, pre=pre, scratch=scratch)
        assert torch.equal(C, want)
        assert [n for n, dtype in allocations if dtype == torch.int32] == ([m * n] if ws else [])
    assert lib.t3_gemm_fwd_act_workspace(None, None, None, m, n, k, None, None, t3.T3_OUT_F32, 0) == 0


@pytest.mark.gpu
def test_scratch_off_its_boundary_is_not_used():
    m, n, k = 129, 260, 4001
    t3.t3_set_small_product_limit(0)
    g = t3_synth.rng(3)
    a, w = t3_synth.int8_uniform(g, (m, k)), t3_synth.ternary(g, (k, n))
    scratch = torch.full((t3.load().t3_gemm_fwd_act_scratch(m, n, k) + 1,), 9, dtype=torch.uint8, device="cuda")[1:]
    out = t3.t3_gemm_fwd_act(_dev(a), _dev(oracle.pack(w)), kind=t3.T3_OUT_BF16, scratch=scratch)
    assert torch.all(scratch == 9)
    assert torch.equal(out.cpu(), torch.from_numpy((a.astype(np.int64) @ w.astype(np.int64)).astype(np.float32)).bfloat16())
