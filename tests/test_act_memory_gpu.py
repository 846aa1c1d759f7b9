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
