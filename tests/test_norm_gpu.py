"""GPU tests of t3_rmsnorm_quant and t3_rmsnorm_bwd against the 64-bit forms of
tests/operators_ref.py; the int8 codes bit for bit."""
import numpy as np
import pytest

import operators_ref as ref
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def _np(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _strided(t, ld, offset=0):
    """A copy of t whose rows lie `ld` elements apart, `offset` past an
    aligned base, in a buffer of ones (so a stray write or read shows)."""
    buf = torch.ones(offset + t.shape[0] * ld + 8, dtype=t.dtype, device=t.device)
    v = buf[offset:offset + t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]]
    v.copy_(t)
    return v, buf


def _check_forward(s, gamma, got, dname, finite=None):
    q, scale, rstd, _ = got
    sn = _np(s)
    gn = np.ones(s.shape[1]) if gamma is None else _np(gamma)
    rows = np.ones(len(sn), bool) if finite is None else finite
    want_rstd, want_scale, y = ref.norm(sn[rows], gn, np.float64(np.float32(EPS)))
    # the sum of squares: cols + 1 roundings; the division, sum with eps, root and reciprocal: 4 more
    rel = (s.shape[1] + 8) * ref.U
    np.testing.assert_allclose(_np(rstd)[rows], want_rstd, rtol=rel)
    np.testing.assert_allclose(_np(scale)[rows], want_scale, rtol=rel + 4 * ref.U)
    np.testing.assert_array_equal(q.cpu().numpy()[rows], ref.norm_codes(sn[rows], gn))
    # and as a quantizer: half a step, and the rounding of u and of u * inv (127 ulps at most)
    off = np.abs(q.cpu().numpy()[rows] * want_scale[:, None] - y)
    assert np.all(off <= want_scale[:, None] * (0.5 + 127 * 4 * ref.U))


# widths on every side of the layouts' edges: one warp a row, CTAs of one to four vectors
# a thread, element by element, rows too long for registers
SHAPES = [(1, 1), (3, 8), (5, 27), (2, 243), (27, 729), (1, 8192), (700, 96), (641, 729), (400, 1024),
          (330, 1032), (310, 1280), (3, 2056), (305, 3456), (307, 2050), (2, 16384), (1, 16392), (320, 9000),
          (3, 40000), (2, 33001)]


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dname):
    g = _gen(rows * 31 + cols)
    x = _rand(g, rows, cols, dtype=DT[dname], std=0.7)
    r = _rand(g, rows, cols, dtype=DT[dname], std=2.0)
    gamma = 1 + 0.3 * _rand(g, cols)
    got = t3.t3_rmsnorm_quant(x, gamma, r, EPS)
    s = (x.float() + r.float()).to(DT[dname])
    assert torch.equal(got[3], s)
    _check_forward(s, gamma, got, dname)
    plain = t3.t3_rmsnorm_quant(x, None, None, EPS)
    assert plain[3] is x
    _check_forward(x, None, plain, dname)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,offset", [(310, 128, 8, 0), (310, 128, 3, 0), (310, 128, 8, 1), (5, 2304, 16, 0),
                                                  (5, 1280, 1, 3), (3, 20000, 4, 4)])
def test_forward_strides_and_bases(rows, cols, pad, offset, dname):
    g = _gen(cols + pad)
    x, r = _rand(g, rows, cols, dtype=DT[dname]), _rand(g, rows, cols, dtype=DT[dname])
    xs, _ = _strided(x, cols + pad, offset)
    rs, _ = _strided(r, cols + 2 * pad, offset)
    so, buf = _strided(torch.zeros_like(x), cols + pad, offset)
    gamma = (1 + 0.3 * _rand(g, cols + 1))[1:]  # four bytes off a 16-byte boundary
    got = t3.t3_rmsnorm_quant(xs, gamma, rs, EPS, sum_out=so)
    s = (x.float() + r.float()).to(DT[dname])
    assert torch.equal(so, s)
    so.fill_(1)
    assert torch.all(buf == 1), "written outside the rows"
    _check_forward(s, gamma, (got[0], got[1], got[2], None), dname)
    # a residual shared by all rows (stride 0)
    one = _rand(g, 1, cols, dtype=DT[dname])
    got = t3.t3_rmsnorm_quant(x, gamma, one.expand(rows, cols), EPS)
    _check_forward((x.float() + one.float()).to(DT[dname]), gamma, got, dname)


@pytest.mark.parametrize("cols", [128, 729, 1280, 20001])
def test_residual_stream_in_place(cols):
    g = _gen(cols)
    x, r = _rand(g, 333, cols, dtype=torch.bfloat16), _rand(g, 333, cols, dtype=torch.bfloat16)
    want = t3.t3_rmsnorm_quant(x, None, r, EPS)
    for over in (0, 1):
        a, b = x.clone(), r.clone()
        got = t3.t3_rmsnorm_quant(a, None, b, EPS, sum_out=(a, b)[over])
        assert torch.equal(got[3], want[3]) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [40, 243, 2048, 40008])
def test_rows_of_zeros_and_of_values_that_are_not_finite(cols, dname):
    g = _gen(cols)
    x = _rand(g, 8, cols, dtype=DT[dname])
    x[1] = 0
    x[2, cols // 2] = float("nan")
    x[3, cols - 1] = float("inf")
    x[4, 0] = float("-inf")
    x[5] = 3e38            # squares past the float range
    x[6] = 1e-30
    gamma = 1 + 0.1 * _rand(g, cols)
    q, scale, rstd, _ = got = t3.t3_rmsnorm_quant(x, gamma, None, EPS)
    ok = np.array([True, False, False, False, False, False, True, True])
    _check_forward(x, gamma, got, dname, ok)
    assert torch.all(q[1] == 0) and scale[1] == 0 and torch.isfinite(rstd[1])
    assert torch.isnan(scale[2:6]).all() and torch.all(q[2:6] == 0)
    # an infinite gain shows too
    gamma[1] = float("inf")
    assert torch.isnan(t3.t3_rmsnorm_quant(x, gamma, None, EPS)[1]).all()


def test_empty_shapes():
    z = torch.zeros((0, 16), device="cuda")
    assert t3.t3_rmsnorm_quant(z)[0].shape == (0, 16)
    q, scale, rstd, _ = t3.t3_rmsnorm_quant(torch.zeros((3, 0), device="cuda"), eps=4.0)
    assert q.shape == (3, 0) and torch.all(scale == 0) and torch.all(rstd == 0.5)
    dx, dg = t3.t3_rmsnorm_bwd(z, z, torch.zeros(0, device="cuda"), torch.ones(16, device="cuda"))
    assert dx.shape == (0, 16) and torch.all(dg == 0)


def _check_backward(dy, s, rstd, gamma, dsum, got, dname):
    rows, cols = s.shape
    gn = np.ones(cols) if gamma is None else _np(gamma)
    dn = np.zeros((rows, cols)) if dsum is None else _np(dsum)
    dx, dgamma, mag, gmag = ref.norm_bwd(_np(dy), _np(s), _np(rstd), gn, dn)
    tol = ref.HALF_ULP[dname] * np.abs(dx) + (cols + 16) * ref.U * mag
    assert np.all(np.abs(_np(got[0]) - dx) <= tol), np.max(np.abs(_np(got[0]) - dx) / tol)
    if gamma is not None:
        assert np.all(np.abs(_np(got[1]) - dgamma) <= (rows + 16) * ref.U * gmag)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, dname):
    g = _gen(rows * 17 + cols)
    s = _rand(g, rows, cols, dtype=DT[dname], std=1.7)
    dy, dsum = _rand(g, rows, cols, dtype=DT[dname]), _rand(g, rows, cols, dtype=DT[dname])
    gamma = 1 + 0.3 * _rand(g, cols)
    rstd = (1 / np.sqrt((_np(s) ** 2).mean(1) + EPS)).astype(np.float32)
    rstd = torch.from_numpy(rstd).cuda()
    _check_backward(dy, s, rstd, gamma, dsum, t3.t3_rmsnorm_bwd(dy, s, rstd, gamma, dsum), dname)
    got = t3.t3_rmsnorm_bwd(dy, s, rstd)
    assert got[1] is None
    _check_backward(dy, s, rstd, None, None, got, dname)


@pytest.mark.parametrize("cols,pad", [(128, 8), (128, 1), (1280, 8), (729, 2), (20000, 4)])
def test_backward_strides_and_in_place(cols, pad):
    g = _gen(cols + pad)
    rows = 317
    s, dy, dsum = (_rand(g, rows, cols, dtype=torch.bfloat16) for _ in range(3))
    gamma = 1 + 0.3 * _rand(g, cols)
    rstd = torch.rand(rows, generator=g, device="cuda") + 0.5
    want = t3.t3_rmsnorm_bwd(dy, s, rstd, gamma, dsum)
    a, b, c = (_strided(v, cols + pad)[0] for v in (dy, s, dsum))
    out, buf = _strided(torch.zeros_like(dy), cols + 2 * pad)
    got = t3.t3_rmsnorm_bwd(a, b, rstd, gamma, c, dx=out)
    _check_backward(dy, s, rstd, gamma, dsum, got, "bf16")
    out.fill_(1)
    assert torch.all(buf == 1), "written outside the rows"
    for over in (a, c):
        keep = over.clone()
        got = t3.t3_rmsnorm_bwd(a, b, rstd, gamma, c, dx=over)
        _check_backward(dy, s, rstd, gamma, dsum, got, "bf16")
        over.copy_(keep)
    again = t3.t3_rmsnorm_bwd(dy, s, rstd, gamma, dsum)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1]), "changes from call to call"


# rows that begin on any boundary, all arrays alike: few columns and many, bases off the boundary too, CTAs of
# several rows and of several groups of rows
@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,offset", [(3000, 65, 0), (2600, 67, 3), (5001, 243, 1), (2500, 514, 0), (700, 4099, 5),
                                              (320, 8191, 0), (33, 1003, 7), (4000, 130, 2)])
def test_odd_rows_alike(rows, cols, offset, dname):
    g = _gen(rows + cols)
    v = 8 if dname == "bf16" else 4

    def alike(t):  # the rows one after another, `offset` elements off a boundary
        flat = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
        out = flat[offset:offset + t.numel()].view(t.shape)
        out.copy_(t)
        return out

    x, r, dy, ds = (alike(_rand(g, rows, cols, dtype=DT[dname])) for _ in range(4))
    gamma = 1 + 0.3 * _rand(g, cols)
    q = torch.zeros(rows * cols + 16, dtype=torch.int8, device="cuda")[offset % v:][:rows * cols].view(rows, cols)
    s = (x.float() + r.float()).to(DT[dname])
    got = t3.t3_rmsnorm_quant(x, gamma, r, EPS, q=q, sum_out=r)  # the stream in place
    assert torch.equal(r, s)
    _check_forward(s, gamma, (q, got[1], got[2], None), dname)
    keep = dy.clone()
    back = t3.t3_rmsnorm_bwd(dy, r, got[2], gamma, dsum=ds, dx=dy)  # dx over dy
    _check_backward(keep, s, got[2], gamma, ds, back, dname)


def test_one_row_repeated_as_input():
    """The gradient of a broadcast row (stride 0) counts it once a row."""
    g = _gen(5)
    s = _rand(g, 64, 256)
    rstd = torch.rand(64, generator=g, device="cuda") + 0.5
    dy = _rand(g, 1, 256).expand(64, 256)
    gamma = 1 + 0.3 * _rand(g, 256)
    _check_backward(dy, s, rstd, gamma, None, t3.t3_rmsnorm_bwd(dy, s, rstd, gamma), "f32")


def test_binding_refusals():
    x = torch.zeros((4, 16), device="cuda")
    for bad in (dict(gamma=torch.ones(15, device="cuda")), dict(residual=torch.zeros((4, 15), device="cuda")),
                dict(q=torch.zeros((4, 15), dtype=torch.int8, device="cuda")), dict(row_scale=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            t3.t3_rmsnorm_quant(x, **bad)
    with pytest.raises(TypeError):
        t3.t3_rmsnorm_quant(x, residual=x.bfloat16())
    with pytest.raises(TypeError):
        t3.t3_rmsnorm_quant(x.half())
    with pytest.raises(ValueError):
        t3.t3_rmsnorm_quant(x.t())
    with pytest.raises(t3.T3Error):
        t3.t3_rmsnorm_quant(x, eps=0.0)
    with pytest.raises(ValueError):
        t3.t3_rmsnorm_bwd(x, x, torch.ones(4, device="cuda"), torch.ones(16, device="cuda"),
                          workspace=torch.empty(3, device="cuda"))


def test_another_stream():
    g = _gen(9)
    x = _rand(g, 512, 1280, dtype=torch.bfloat16)
    want = t3.t3_rmsnorm_quant(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(x)
    with torch.cuda.stream(st):
        y.copy_(x)
        got = t3.t3_rmsnorm_quant(y)
    other = t3.t3_rmsnorm_quant(x, stream=st)
    st.synchronize()
    torch.cuda.current_stream().synchronize()
    for a, b, c in zip(want[:3], got[:3], other[:3]):
        assert torch.equal(a, b) and torch.equal(a, c)
