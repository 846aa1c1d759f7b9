"""The norm, recurrence and epilogue operators without a GPU: refusals before
any CUDA call, the binding's checks, and the 64-bit gradients of
tests/operators_ref.py against central differences of its forward forms."""
import ctypes

import numpy as np
import pytest

import operators_ref as ref
import ternary_weight_int8_t3_gb300 as t3

FAKE = ctypes.c_void_p(4096)  # never dereferenced: every case returns first
BF16, F32 = t3.T3_OUT_BF16, t3.T3_OUT_F32
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    return t3.load()


def _norm(lib, x=FAKE, ldx=8, r=None, ldr=0, eps=1e-5, q=FAKE, scale=FAKE, so=None, lds=0, rows=4, cols=8, dt=BF16):
    return lib.t3_rmsnorm_quant(x, ldx, r, ldr, None, eps, q, scale, None, so, lds, rows, cols, dt, None)


def test_norm_refusals(lib):
    bad = [dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(ldx=-1), dict(ldx=BIG),
           dict(r=FAKE, ldr=-1), dict(so=FAKE, lds=7), dict(so=FAKE, lds=-8), dict(eps=0.0), dict(eps=-1.0),
           dict(eps=float("nan")), dict(eps=float("inf")), dict(dt=2), dict(dt=-1), dict(x=None), dict(q=None),
           dict(scale=None), dict(cols=0, scale=None)]
    for kw in bad:
        assert _norm(lib, **kw) == t3.T3_EINVAL, kw
    assert _norm(lib, rows=0, x=None, q=None, scale=None) == t3.T3_OK


def _norm_bwd(lib, dy=FAKE, lddy=8, s=FAKE, lds=8, rstd=FAKE, dsum=None, ldd=0, dx=FAKE, lddx=8, dg=None, rows=4,
              cols=8, dt=BF16, ws=None):
    return lib.t3_rmsnorm_bwd(dy, lddy, s, lds, rstd, None, dsum, ldd, dx, lddx, dg, rows, cols, dt, ws, None)


def test_norm_bwd_refusals(lib):
    bad = [dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(lddy=-1), dict(lds=-1), dict(lddx=7),
           dict(dsum=FAKE, ldd=-1), dict(dt=2), dict(dy=None), dict(s=None), dict(rstd=None), dict(dx=None),
           dict(dg=FAKE)]
    for kw in bad:
        assert _norm_bwd(lib, **kw) == t3.T3_EINVAL, kw
    assert _norm_bwd(lib, cols=0, lddx=0, dy=None, s=None, rstd=None, dx=None) == t3.T3_OK
    assert _norm_bwd(lib, rows=0, dy=None, s=None, rstd=None, dx=None) == t3.T3_OK


def test_colsum_workspace(lib):
    assert lib.t3_colsum_workspace(0, 5) == lib.t3_colsum_workspace(5, 0) == lib.t3_colsum_workspace(-1, 5) == 0
    assert lib.t3_colsum_workspace(3, 5) == 15
    big = lib.t3_colsum_workspace(1 << 20, 8192)
    assert 0 < big <= 2048 * 8192


def _scan(lib, g=FAKE, ldg=8, c=FAKE, ldc=8, h=FAKE, ldh=8, hl=None, b=2, t=3, w=8, dt=BF16):
    return lib.t3_gated_scan_fwd(g, ldg, c, ldc, None, None, h, ldh, hl, b, t, w, dt, None)


def test_scan_refusals(lib):
    bad = [dict(b=-1), dict(t=-1), dict(w=-1), dict(b=BIG), dict(t=BIG), dict(w=BIG), dict(ldg=-1), dict(ldc=-1),
           dict(ldh=7), dict(dt=2), dict(g=None), dict(c=None), dict(h=None)]
    for kw in bad:
        assert _scan(lib, **kw) == t3.T3_EINVAL, kw
    for kw in (dict(b=0), dict(w=0, ldh=0), dict(t=0)):
        assert _scan(lib, g=None, c=None, h=None, **kw) == t3.T3_OK, kw


def _scan_bwd(lib, g=FAKE, c=FAKE, h=FAKE, d=FAKE, dg=FAKE, dc=FAKE, lddg=8, lddc=8, ld=8, dh0=None, b=2, t=3, w=8,
              dt=BF16):
    return lib.t3_gated_scan_bwd(g, ld, c, ld, h, ld, d, ld, None, None, None, dg, lddg, dc, lddc, dh0, b, t, w, dt,
                                 None)


def test_scan_bwd_refusals(lib):
    bad = [dict(b=-1), dict(t=-1), dict(w=-1), dict(b=BIG), dict(t=BIG), dict(w=BIG), dict(ld=-1), dict(lddg=7),
           dict(lddc=7), dict(dt=2), dict(g=None), dict(c=None), dict(h=None), dict(d=None), dict(dg=None),
           dict(dc=None)]
    for kw in bad:
        assert _scan_bwd(lib, **kw) == t3.T3_EINVAL, kw
    for kw in (dict(b=0), dict(w=0), dict(t=0)):
        assert _scan_bwd(lib, g=None, c=None, h=None, d=None, dg=None, dc=None, **kw) == t3.T3_OK, kw


def _act(lib, a=FAKE, wp=FAKE, c=FAKE, m=4, n=8, k=8, act=0, r=None, pre=None, kind=F32, ws=None, room=0):
    return lib.t3_gemm_fwd_act(a, wp, c, m, n, k, None, None, None, act, r, pre, kind, ws, None, room, None)


def test_act_refusals(lib):
    bad = [dict(m=-1), dict(n=-1), dict(k=-1), dict(m=BIG), dict(act=5), dict(act=-1), dict(kind=2), dict(kind=3),
           dict(a=None), dict(wp=None), dict(c=None), dict(r=FAKE), dict(pre=FAKE), dict(room=-1)]
    for kw in bad:
        assert _act(lib, **kw) == t3.T3_EINVAL, kw
    other = ctypes.c_void_p(8192)
    assert _act(lib, r=other, pre=other) == t3.T3_EINVAL
    assert _act(lib, kind=BF16, ws=FAKE) == t3.T3_EINVAL
    assert _act(lib, m=1, k=16777216) == t3.T3_EOVERFLOW
    assert _act(lib, m=0, a=None, wp=None, c=None) == t3.T3_OK
    assert _act(lib, n=0, a=None, wp=None, c=None) == t3.T3_OK


def test_act_scratch(lib):
    f = lib.t3_gemm_fwd_act_scratch
    assert f(32, 729, 243) == f(64, 728, 256) == f(64, 0, 3) == f(64, 3, 0) == f(-1, 3, 3) == 0
    assert f(64, 729, 243) == 64 * 256 + 732 * 64 + 64 * 732 * 4  # A, packed weights, int32 result
    assert f(64, 728, 243) > 0 and f(64, 729, 256) > 0


def _act_bwd(lib, dy=FAKE, z=FAKE, act=1, dz=FAKE, db=None, rows=4, cols=8, dt=BF16, ws=None):
    return lib.t3_act_bwd(dy, z, act, dz, db, rows, cols, dt, ws, None)


def test_act_bwd_refusals(lib):
    bad = [dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(act=5), dict(act=-1), dict(dt=2), dict(dy=None),
           dict(z=None), dict(db=FAKE)]
    for kw in bad:
        assert _act_bwd(lib, **kw) == t3.T3_EINVAL, kw
    assert _act_bwd(lib, cols=0) == t3.T3_OK
    assert _act_bwd(lib, rows=0, dy=None, z=None) == t3.T3_OK
    assert _act_bwd(lib, dz=None) == t3.T3_OK


def test_binding_rejects_cpu_tensors_and_types():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 8))
    for call in (lambda: t3.t3_rmsnorm_quant(x), lambda: t3.t3_rmsnorm_bwd(x, x, x[:, 0]),
                 lambda: t3.t3_gated_scan_fwd(x[None], x[None]),
                 lambda: t3.t3_gated_scan_bwd(x[None], x[None], x[None], x[None]),
                 lambda: t3.t3_act_bwd(x, x, t3.T3_ACT_SILU),
                 lambda: t3.t3_gemm_fwd_act(x.to(torch.int8), torch.zeros((3, 2), dtype=torch.uint8))):
        with pytest.raises(TypeError):
            call()


def test_row_strides_of_the_binding():
    """_rows on CPU tensors (device -1): what counts as evenly spaced rows."""
    torch = pytest.importorskip("torch")

    def rows(t, shape, **kw):
        return t3._rows(t, torch.float32, -1, shape, "t", **kw)
    both = torch.zeros((2, 3, 16))
    assert rows(both[..., 8:], (2, 3, 8)) == (both.data_ptr() + 32, 16)
    assert rows(torch.zeros((4, 8))[::2], (2, 8))[1] == 16
    with pytest.raises(ValueError):  # a gap between sequences
        rows(torch.zeros((3, 3, 8))[::2], (2, 3, 8))
    with pytest.raises(ValueError):  # columns not adjacent
        rows(torch.zeros((8, 4)).t(), (4, 8))
    with pytest.raises(ValueError):  # overlapping output
        rows(torch.zeros((1, 8)).expand(4, 8), (4, 8), out=True)
    assert rows(torch.zeros((1, 8)).expand(4, 8), (4, 8))[1] == 0
    assert rows(torch.zeros((2, 1, 16))[..., :8], (2, 1, 8))[1] == 16
    assert rows(torch.zeros((2, 0, 8)), (2, 0, 8), out=True)[1] >= 8
    with pytest.raises(TypeError):
        rows(both.double(), (2, 3, 16))


# ------------------------------------------- gradients against differences ---

def _differences(fn, x, step=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        out[i] = (fn(a) - fn(b)) / (2 * step)
    return out


def _close(got, want):
    # central differences of an O(1) smooth function: step^2 truncation and
    # 1e-16 / step rounding, both below 1e-8 here
    np.testing.assert_allclose(got, want, rtol=1e-6, atol=1e-7)


def test_norm_gradient_against_differences():
    g = np.random.default_rng(1)
    s, dy, dsum = g.standard_normal((3, 7)), g.standard_normal((3, 7)), g.standard_normal((3, 7))
    gamma = 1 + 0.3 * g.standard_normal(7)
    eps = 0.1

    def loss(s, gamma):
        return (ref.norm(s, gamma, eps)[2] * dy).sum() + (s * dsum).sum()

    rstd = ref.norm(s, gamma, eps)[0]
    dx, dgamma, _, _ = ref.norm_bwd(dy, s, rstd, gamma, dsum)
    _close(dx, _differences(lambda v: loss(v, gamma), s))
    _close(dgamma, _differences(lambda v: loss(s, v), gamma))


def test_scan_gradient_against_differences():
    g = np.random.default_rng(2)
    shape = (2, 5, 3)
    gate, cand, dh = g.standard_normal(shape) + 1, g.standard_normal(shape), g.standard_normal(shape)
    h0, dl = g.standard_normal((2, 3)), g.standard_normal((2, 3))
    resets = np.zeros((2, 5))
    resets[0, 3] = resets[1, 0] = 1

    def loss(gate, cand, h0):
        h = ref.scan(gate, cand, h0, resets)[0]
        return (h * dh).sum() + (h[:, -1] * dl).sum()

    prior = ref.scan(gate, cand, h0, resets)[1]
    (dgate, dcand, dh0), _ = ref.scan_bwd(gate, cand, prior, dh, resets, dl)
    _close(dgate, _differences(lambda v: loss(v, cand, h0), gate))
    _close(dcand, _differences(lambda v: loss(gate, v, h0), cand))
    _close(dh0, _differences(lambda v: loss(gate, cand, v), h0))


@pytest.mark.parametrize("name", ref.ACTS)
def test_act_slope_against_differences(name):
    z = np.array([-9.0, -3.1, -1.2, -0.4, 0.3, 0.9, 2.2, 5.0, 11.0])  # away from the corner at 0
    _close(ref.act(z, name)[1], (ref.act(z + 1e-6, name)[0] - ref.act(z - 1e-6, name)[0]) / 2e-6)
