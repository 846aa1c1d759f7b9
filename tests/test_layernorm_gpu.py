"""GPU tests of t3_layernorm_quant and t3_layernorm_bwd against the 64-bit forms of
tests/more_operators_ref.py."""
import numpy as np
import pytest

import more_operators_ref as ref
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


def _rand(g, *shape, dtype=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _strided(t, ld, offset=0):
    """A copy of t whose rows lie `ld` elements apart, `offset` past an
    aligned base, in a buffer of ones (so a stray write or read shows)."""
    buf = torch.ones(offset + t.shape[0] * ld + 8, dtype=t.dtype, device=t.device)
    v = buf[offset:offset + t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]]
    v.copy_(t)
    return v, buf


def _check_forward(s, gamma, beta, got, rows=slice(None)):
    q, scale, mean, rstd = got[:4]
    sn = _np(s)[rows]
    gn = np.ones(s.shape[1]) if gamma is None else _np(gamma)
    bn = np.zeros(s.shape[1]) if beta is None else _np(beta)
    wm, wr, ws, y, (em, er, es, ey) = ref.layer_norm(sn, gn, bn, np.float64(np.float32(EPS)))
    assert np.all(np.abs(_np(mean)[rows] - wm) <= em + ref.U * np.abs(wm))
    assert np.all(np.abs(_np(rstd)[rows] - wr) <= er * wr)
    assert np.all(np.abs(_np(scale)[rows] - ws) <= es)
    # half a step, the values' own error, the scale's (127 of it at most), the product's rounding
    off = np.abs(q.cpu().numpy()[rows] * ws[:, None] - y)
    assert np.all(off <= ws[:, None] * (0.5 + 127 * 6 * ref.U) + ey + 127 * es[:, None])
    assert np.all(np.abs(q.cpu().numpy()[rows]).max(1) == 127 * (ws > 0))


# widths on every side of the layouts' edges: one warp a row, CTAs of one to four vectors
# a thread, element by element, rows too long for registers
SHAPES = [(1, 1), (3, 8), (5, 27), (2, 243), (27, 729), (1, 8192), (700, 96), (641, 729), (400, 1024),
          (330, 1032), (310, 1280), (3, 2056), (305, 3456), (307, 2050), (2, 16384), (1, 16392), (320, 9000),
          (3, 40000), (2, 33001)]


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dname):
    g = _gen(rows * 31 + cols)
    x = _rand(g, rows, cols, dtype=DT[dname], std=0.7, mean=0.5)
    r = _rand(g, rows, cols, dtype=DT[dname], std=2.0, mean=-3.0)
    gamma, beta = 1 + 0.3 * _rand(g, cols), 0.5 * _rand(g, cols) + 0.01
    got = t3.t3_layernorm_quant(x, gamma, beta, r, EPS)
    s = (x.float() + r.float()).to(DT[dname])
    assert torch.equal(got[4], s)
    _check_forward(s, gamma, beta, got)
    if cols > 1:  # a row of one element has no deviation
        plain = t3.t3_layernorm_quant(x, eps=EPS)
        assert plain[4] is x
        _check_forward(x, None, None, plain)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,offset", [(310, 128, 8, 0), (310, 128, 3, 0), (310, 128, 8, 1), (5, 2304, 16, 0),
                                                  (5, 1280, 1, 3), (3, 20000, 4, 4)])
def test_forward_strides_and_bases(rows, cols, pad, offset, dname):
    g = _gen(cols + pad)
    x, r = _rand(g, rows, cols, dtype=DT[dname]), _rand(g, rows, cols, dtype=DT[dname])
    xs, _ = _strided(x, cols + pad, offset)
    rs, _ = _strided(r, cols + 2 * pad, offset)
    so, buf = _strided(torch.zeros_like(x), cols + pad, offset)
    gamma, beta = ((1 + 0.3 * _rand(g, cols + 1))[1:] for _ in range(2))  # four bytes off a 16-byte boundary
    got = t3.t3_layernorm_quant(xs, gamma, beta, rs, EPS, sum_out=so)
    s = (x.float() + r.float()).to(DT[dname])
    assert torch.equal(so, s)
    so.fill_(1)
    assert torch.all(buf == 1), "written outside the rows"
    _check_forward(s, gamma, beta, got)
    one = _rand(g, 1, cols, dtype=DT[dname])  # a residual shared by all rows (stride 0)
    got = t3.t3_layernorm_quant(x, gamma, beta, one.expand(rows, cols), EPS)
    _check_forward((x.float() + one.float()).to(DT[dname]), gamma, beta, got)


@pytest.mark.parametrize("cols", [128, 729, 1280, 20001])
def test_residual_stream_in_place(cols):
    g = _gen(cols)
    x, r = _rand(g, 333, cols, dtype=torch.bfloat16), _rand(g, 333, cols, dtype=torch.bfloat16)
    beta = _rand(g, cols)
    want = t3.t3_layernorm_quant(x, None, beta, r, EPS)
    for over in (0, 1):
        a, b = x.clone(), r.clone()
        got = t3.t3_layernorm_quant(a, None, beta, b, EPS, sum_out=(a, b)[over])
        for i in (0, 1, 2, 3, 4):
            assert torch.equal(got[i], want[i])


@pytest.mark.parametrize("mean", [100.0, -3e4])
@pytest.mark.parametrize("cols", [64, 729, 4096, 8200])
def test_rows_far_from_zero_keep_their_deviation(cols, mean):
    g = _gen(cols)
    x = _rand(g, 40, cols, std=1.0, mean=mean)
    _check_forward(x, None, None, t3.t3_layernorm_quant(x, eps=EPS))


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [40, 243, 2048, 40008])
def test_rows_without_deviation_and_of_values_that_are_not_finite(cols, dname):
    g = _gen(cols)
    x = _rand(g, 8, cols, dtype=DT[dname])
    x[1] = 0
    x[2, cols // 2] = float("nan")
    x[3, cols - 1] = float("inf")
    x[4, 0] = float("-inf")
    x[5, ::2] = 3e38       # squares past the float range
    x[6] = 1e-30 * x[0]
    gamma, beta = 1 + 0.1 * _rand(g, cols), 0.2 * _rand(g, cols)
    q, scale, mean, rstd, _ = got = t3.t3_layernorm_quant(x, gamma, beta, None, EPS)
    _check_forward(x, gamma, beta, got, [0, 1, 6, 7])
    assert torch.isnan(scale[2:6]).all() and torch.all(q[2:6] == 0)
    q, scale, _, rstd, _ = t3.t3_layernorm_quant(x, gamma, None, None, EPS)
    assert torch.all(q[1] == 0) and scale[1] == 0 and torch.isfinite(rstd[1])
    assert torch.isnan(scale[2:6]).all() and torch.all(q[2:6] == 0)
    # values near the bottom of the float range keep their codes
    q, scale, _, _, _ = small = t3.t3_layernorm_quant(x, gamma * 1e-38, None, None, EPS)
    assert torch.equal(q[[0, 7]].abs().amax(1), torch.full((2,), 127, dtype=torch.int8, device="cuda"))
    # an infinite gain or shift shows too
    beta[1] = float("inf")
    assert torch.isnan(t3.t3_layernorm_quant(x, gamma, beta, None, EPS)[1]).all()


def test_empty_shapes():
    z = torch.zeros((0, 16), device="cuda")
    assert t3.t3_layernorm_quant(z)[0].shape == (0, 16)
    q, scale, mean, rstd, _ = t3.t3_layernorm_quant(torch.zeros((3, 0), device="cuda"), eps=4.0)
    assert q.shape == (3, 0) and torch.all(scale == 0) and torch.all(rstd == 0.5) and torch.all(mean == 0)
    none = torch.zeros(0, device="cuda")
    db = torch.ones(16, device="cuda")
    dx, dg, db = t3.t3_layernorm_bwd(z, z, none, none, torch.ones(16, device="cuda"), dbeta=db)
    assert dx.shape == (0, 16) and torch.all(dg == 0) and torch.all(db == 0)


def _check_backward(dy, s, mean, rstd, gamma, dsum, got, dname):
    rows, cols = s.shape
    gn = np.ones(cols) if gamma is None else _np(gamma)
    dn = np.zeros((rows, cols)) if dsum is None else _np(dsum)
    dx, dgamma, dbeta, mag, gmag, bmag = ref.layer_norm_bwd(_np(dy), _np(s), _np(mean), _np(rstd), gn, dn)
    tol = ref.HALF_ULP[dname] * np.abs(dx) + (cols + 16) * ref.U * mag
    assert np.all(np.abs(_np(got[0]) - dx) <= tol), np.max(np.abs(_np(got[0]) - dx) / tol)
    if got[1] is not None:
        assert np.all(np.abs(_np(got[1]) - dgamma) <= (rows + 16) * ref.U * gmag)
    if got[2] is not None:
        assert np.all(np.abs(_np(got[2]) - dbeta) <= (rows + 16) * ref.U * bmag)


def _moments(s):
    sn = _np(s)
    mean = sn.mean(1)
    rstd = 1 / np.sqrt(((sn - mean[:, None]) ** 2).mean(1) + EPS)
    return (torch.from_numpy(v.astype(np.float32)).cuda() for v in (mean, rstd))


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, dname):
    g = _gen(rows * 17 + cols)
    s = _rand(g, rows, cols, dtype=DT[dname], std=1.7, mean=0.6)
    dy, dsum = _rand(g, rows, cols, dtype=DT[dname]), _rand(g, rows, cols, dtype=DT[dname])
    gamma = 1 + 0.3 * _rand(g, cols)
    mean, rstd = _moments(s)
    db = torch.empty(cols, device="cuda")
    got = t3.t3_layernorm_bwd(dy, s, mean, rstd, gamma, dsum, dbeta=db)
    _check_backward(dy, s, mean, rstd, gamma, dsum, got, dname)
    only = t3.t3_layernorm_bwd(dy, s, mean, rstd, gamma, dsum)
    assert only[2] is None and torch.equal(only[1], got[1]) and torch.equal(only[0], got[0])
    got = t3.t3_layernorm_bwd(dy, s, mean, rstd, dbeta=torch.empty(cols, device="cuda"))
    assert got[1] is None
    _check_backward(dy, s, mean, rstd, None, None, got, dname)


@pytest.mark.parametrize("cols,pad", [(128, 8), (128, 1), (1280, 8), (729, 2), (20000, 4)])
def test_backward_strides_and_in_place(cols, pad):
    g = _gen(cols + pad)
    rows = 317
    s, dy, dsum = (_rand(g, rows, cols, dtype=torch.bfloat16) for _ in range(3))
    gamma, beta = 1 + 0.3 * _rand(g, cols), torch.empty(cols, device="cuda")
    mean, rstd = _moments(s)
    want = t3.t3_layernorm_bwd(dy, s, mean, rstd, gamma, dsum, dbeta=torch.empty(cols, device="cuda"))
    a, b, c = (_strided(v, cols + pad)[0] for v in (dy, s, dsum))
    out, buf = _strided(torch.zeros_like(dy), cols + 2 * pad)
    got = t3.t3_layernorm_bwd(a, b, mean, rstd, gamma, c, dx=out, dbeta=beta)
    _check_backward(dy, s, mean, rstd, gamma, dsum, got, "bf16")
    out.fill_(1)
    assert torch.all(buf == 1), "written outside the rows"
    for over in (a, c):
        keep = over.clone()
        got = t3.t3_layernorm_bwd(a, b, mean, rstd, gamma, c, dx=over, dbeta=beta)
        _check_backward(dy, s, mean, rstd, gamma, dsum, got, "bf16")
        over.copy_(keep)
    again = t3.t3_layernorm_bwd(dy, s, mean, rstd, gamma, dsum, dbeta=beta)
    for i in range(3):
        assert torch.equal(again[i], want[i]), "changes from call to call"


# rows that begin on any boundary, all arrays alike
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

    x, r, dy, ds = (alike(_rand(g, rows, cols, dtype=DT[dname], mean=0.3)) for _ in range(4))
    gamma, beta = 1 + 0.3 * _rand(g, cols), _rand(g, cols)
    q = torch.zeros(rows * cols + 16, dtype=torch.int8, device="cuda")[offset % v:][:rows * cols].view(rows, cols)
    s = (x.float() + r.float()).to(DT[dname])
    got = t3.t3_layernorm_quant(x, gamma, beta, r, EPS, q=q, sum_out=r)  # the stream in place
    assert torch.equal(r, s)
    _check_forward(s, gamma, beta, got)
    keep = dy.clone()
    back = t3.t3_layernorm_bwd(dy, r, got[2], got[3], gamma, dsum=ds, dx=dy, dbeta=beta)  # dx over dy
    _check_backward(keep, s, got[2], got[3], gamma, ds, back, dname)


def test_gradient_against_differences():
    """dx, dgamma and dbeta against central differences of the 64-bit form."""
    g = _gen(77)
    rows, cols = 5, 24
    x, dy = _rand(g, rows, cols), _rand(g, rows, cols)
    gamma, beta = 1 + 0.3 * _rand(g, cols), _rand(g, cols)
    _, _, mean, rstd, _ = t3.t3_layernorm_quant(x, gamma, beta, eps=EPS)
    dx, dg, db = t3.t3_layernorm_bwd(dy, x, mean, rstd, gamma, dbeta=torch.empty(cols, device="cuda"))
    xn, gn, bn, d = _np(x), _np(gamma), _np(beta), _np(dy)

    def loss(a, b, c):
        return (ref.layer_norm(a, b, c, EPS)[3] * d).sum()

    step = 1e-6
    for got, at in ((dx, 0), (dg, 1), (db, 2)):
        got = _np(got)
        for i in np.ndindex(got.shape):
            hi, lo = [xn.copy(), gn.copy(), bn.copy()], [xn.copy(), gn.copy(), bn.copy()]
            hi[at][i] += step
            lo[at][i] -= step
            want = (loss(*hi) - loss(*lo)) / (2 * step)
            # float sums of some 24 terms of order one, and the differences' own step^2 and 1e-16 / step
            assert abs(got[i] - want) <= 64 * ref.U * np.abs(d).sum() + 1e-7


def test_binding_refusals():
    x, one = torch.zeros((4, 16), device="cuda"), torch.ones(4, device="cuda")
    for bad in (dict(gamma=torch.ones(15, device="cuda")), dict(beta=torch.ones(15, device="cuda")),
                dict(residual=torch.zeros((4, 15), device="cuda")), dict(mean=torch.zeros(3, device="cuda")),
                dict(q=torch.zeros((4, 15), dtype=torch.int8, device="cuda")), dict(row_scale=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            t3.t3_layernorm_quant(x, **bad)
    for bad in (dict(residual=x.bfloat16()), dict(beta=torch.ones(16, device="cuda").half())):
        with pytest.raises(TypeError):
            t3.t3_layernorm_quant(x, **bad)
    with pytest.raises(TypeError):
        t3.t3_layernorm_quant(x.half())
    with pytest.raises(ValueError):
        t3.t3_layernorm_quant(x.t())
    with pytest.raises(t3.T3Error):
        t3.t3_layernorm_quant(x, eps=0.0)
    grad = torch.ones(16, device="cuda")
    with pytest.raises(ValueError):
        t3.t3_layernorm_bwd(x, x, one, one, grad, workspace=torch.empty(3, device="cuda"))
    with pytest.raises(ValueError):  # enough for one sum, not for two
        t3.t3_layernorm_bwd(x, x, one, one, grad, dbeta=torch.empty(16, device="cuda"),
                            workspace=torch.empty(64, device="cuda"))
    with pytest.raises(t3.T3Error):
        t3.t3_layernorm_bwd(x, x, one, one, grad, dgamma=grad, dbeta=grad)


def test_another_stream():
    g = _gen(9)
    x = _rand(g, 512, 1280, dtype=torch.bfloat16)
    want = t3.t3_layernorm_quant(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(x)
    with torch.cuda.stream(st):
        y.copy_(x)
        got = t3.t3_layernorm_quant(y)
    other = t3.t3_layernorm_quant(x, stream=st)
    st.synchronize()
    torch.cuda.current_stream().synchronize()
    for a, b, c in zip(want[:4], got[:4], other[:4]):
        assert torch.equal(a, b) and torch.equal(a, c)
