"""GPU tests of the product with an activation epilogue (t3_gemm_fwd_act) and
of its gradient (t3_act_bwd).  The product is an exact integer and z a fixed
sequence of float roundings, so `pre` is compared bit for bit in float; the
activation within the bound of tests/operators_ref.py."""
import numpy as np
import pytest

import operators_ref as ref
import oracle
import t3_synth
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
KIND = {"bf16": t3.T3_OUT_BF16, "f32": t3.T3_OUT_F32}


def _np(t):
    return t.detach().double().cpu().numpy()


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _z(x, rs, cs, bias):
    """z in float32, rounding by rounding."""
    z = x.astype(np.float32)
    if rs is not None:
        z = z * rs[:, None]
    if cs is not None:
        z = z * cs
    return z + bias if bias is not None else z


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16()


def _problem(seed, m, n, k):
    g = t3_synth.rng(seed)
    a, w = t3_synth.int8_uniform(g, (m, k)), t3_synth.ternary(g, (k, n))
    rs = (g.random(m) * 0.02 + 0.01).astype(np.float32)
    cs = ((g.random(n) + 0.5) / np.sqrt(max(k, 1))).astype(np.float32)
    bias = (g.standard_normal(n) * 0.5).astype(np.float32)
    res = g.standard_normal((m, n)).astype(np.float32)
    return a, w, rs, cs, bias, res


def _check(out, pre, x, rs, cs, bias, res, act, dname):
    z = _z(x, rs, cs, bias)
    if pre is not None:
        if dname == "f32":
            np.testing.assert_array_equal(pre.cpu().numpy(), z)
        else:
            assert torch.equal(pre.cpu(), _bf16(z))
    y, _, rel = ref.act(z.astype(np.float64), act)
    want = y if res is None else y + res
    tol = (rel + ref.U) * np.abs(y) + (ref.HALF_ULP[dname] + 2 * ref.U) * np.abs(want) + 1e-35
    off = np.abs(_np(out) - want)
    assert np.all(off <= tol), np.max(off / tol)


# each route: the CUDA-core rows of one to eight, the small-M tensor cores, the
# CTA pairs, operands and outputs of any alignment, a split reduction, a small product
SHAPES = [(1, 8192, 1024), (1, 729, 243), (2, 1280, 3456), (5, 640, 640), (8, 300, 512), (16, 8192, 2048),
          (27, 729, 243), (27, 3456, 1280), (32, 256, 512), (33, 192, 128), (256, 192, 1280), (300, 272, 96),
          (300, 273, 96), (129, 1000, 260), (777, 2304, 640), (64, 256, 8192), (1, 16, 16), (3, 1, 5), (200, 8, 16)]


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k, dname):
    a, w, rs, cs, bias, res = _problem(m + n + k, m, n, k)
    x = a.astype(np.int64) @ w.astype(np.int64)
    res = _np(torch.from_numpy(res).to(DT[dname]))
    A, Wp = _dev(a), _dev(oracle.pack(w))
    R = torch.from_numpy(res).to(DT[dname]).cuda()
    act = ref.ACTS[(m + n) % 5]
    for limit in (0, 1 << 29):  # the tensor-core routes, then the default routing
        t3.t3_set_small_product_limit(limit)
        pre = torch.full((m, n), 7.0, dtype=DT[dname], device="cuda")
        out = t3.t3_gemm_fwd_act(A, Wp, K=k, row_scale=_dev(rs), col_scale=_dev(cs), bias=_dev(bias),
                                 act=ref.ACTS.index(act), residual=R, kind=KIND[dname], pre=pre)
        _check(out, pre, x, rs, cs, bias, res, act, dname)
        out = t3.t3_gemm_fwd_act(A, Wp, K=k, kind=KIND[dname])
        _check(out, None, x, None, None, None, None, "none", dname)
    rc, detail = t3.t3_last_device_error()
    assert rc == t3.T3_OK, hex(detail)


# reductions around the 16 codes a lane takes, the 32 and 256 elements a warp and a CTA take, and the
# longest that stay in one CTA; tiles that end inside; operands on every byte boundary
@pytest.mark.parametrize("k", [1, 4, 15, 16, 33, 64, 255, 256, 257, 511, 1535, 1536, 1537])
@pytest.mark.parametrize("m,n", [(9, 17), (31, 200), (33, 15), (70, 48)])
def test_short_reductions_of_few_tiles(m, n, k):
    a, w, rs, cs, bias, res = _problem(m + n + k, m, n, k)
    x = a.astype(np.int64) @ w.astype(np.int64)
    packed = oracle.pack(w)
    R = _dev(res)
    for shift in range(4):
        A = _dev(np.concatenate([np.full(shift, 77, np.int8), a.reshape(-1)]))[shift:].view(m, k)
        Wp = _dev(np.concatenate([np.full(3 - shift, 255, np.uint8), packed.reshape(-1)]))[3 - shift:].view(packed.shape)
        pre = torch.full((m, n), 7.0, device="cuda")
        out = t3.t3_gemm_fwd_act(A, Wp, K=k, row_scale=_dev(rs), col_scale=_dev(cs), bias=_dev(bias),
                                 act=t3.T3_ACT_GELU, residual=R, pre=pre)
        _check(out, pre, x, rs, cs, bias, res, "gelu", "f32")


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 512, 256), (20, 512, 256), (300, 384, 256)])
@pytest.mark.parametrize("act", ref.ACTS)
def test_every_activation_on_every_route(act, m, n, k, dname):
    a, w, rs, cs, bias, _ = _problem(m * 3 + n, m, n, k)
    rs *= 8  # spread z over the activations' whole range
    x = a.astype(np.int64) @ w.astype(np.int64)
    pre = torch.empty((m, n), dtype=DT[dname], device="cuda")
    out = t3.t3_gemm_fwd_act(_dev(a), _dev(oracle.pack(w)), row_scale=_dev(rs), col_scale=_dev(cs), bias=_dev(bias),
                             act=ref.ACTS.index(act), kind=KIND[dname], pre=pre)
    _check(out, pre, x, rs, cs, bias, None, act, dname)


@pytest.mark.parametrize("m", [1, 20, 300])
def test_each_vector_may_be_missing(m):
    a, w, rs, cs, bias, res = _problem(m, m, 384, 256)
    x = a.astype(np.int64) @ w.astype(np.int64)
    for skip in range(4):
        v = [None if i == skip else t for i, t in enumerate((rs, cs, bias, res))]
        d = [None if t is None else _dev(t) for t in v]
        out = t3.t3_gemm_fwd_act(_dev(a), _dev(oracle.pack(w)), row_scale=d[0], col_scale=d[1], bias=d[2], residual=d[3],
                                 act=t3.T3_ACT_SILU)
        _check(out, None, x, *v, "silu", "f32")


@pytest.mark.parametrize("m,n,k", [(1, 512, 256), (20, 512, 256), (300, 384, 256)])
@pytest.mark.parametrize("shift", [1, 2])
def test_unaligned_buffers(m, n, k, shift):
    """Every operand and output `shift` elements past an aligned base; canaries around the outputs."""
    a, w, rs, cs, bias, res = _problem(m + shift, m, n, k)
    x = a.astype(np.int64) @ w.astype(np.int64)

    def off(t):
        buf = torch.full((t.numel() + 64,), 3, dtype=t.dtype, device="cuda")
        v = buf[shift:shift + t.numel()].view(t.shape)
        v.copy_(t)
        return v, buf
    for dname in ("bf16", "f32"):
        r = torch.from_numpy(res).to(DT[dname])
        out, ob = off(torch.zeros((m, n), dtype=DT[dname]))
        pre, pb = off(torch.zeros((m, n), dtype=DT[dname]))
        t3.t3_gemm_fwd_act(off(_dev(a))[0], off(_dev(oracle.pack(w)))[0], row_scale=off(_dev(rs))[0],
                           col_scale=off(_dev(cs))[0], bias=off(_dev(bias))[0], act=t3.T3_ACT_GELU,
                           residual=off(r.cuda())[0], kind=KIND[dname], C=out, pre=pre)
        _check(out, pre, x, rs, cs, bias, _np(r), "gelu", dname)
        for v, b in ((out, ob), (pre, pb)):
            v.fill_(3)
            assert torch.all(b == 3), "written outside the output"


def test_only_one_unaligned_output_or_vector():
    """Aligned operands with one odd buffer at a time: the route may change, the result may not."""
    m, n, k = 300, 384, 256
    a, w, rs, cs, bias, res = _problem(11, m, n, k)
    x = a.astype(np.int64) @ w.astype(np.int64)
    for odd in range(6):
        def make(i, t):
            if i != odd:
                return t
            buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
            v = buf[1:].view(t.shape)
            v.copy_(t)
            return v
        r = torch.from_numpy(res).bfloat16()
        out = make(0, torch.zeros((m, n), dtype=torch.bfloat16, device="cuda"))
        pre = make(1, torch.zeros((m, n), dtype=torch.bfloat16, device="cuda"))
        t3.t3_gemm_fwd_act(_dev(a), _dev(oracle.pack(w)), row_scale=make(2, _dev(rs)), col_scale=make(3, _dev(cs)),
                           bias=make(4, _dev(bias)), residual=make(5, r.cuda()), act=t3.T3_ACT_RELU2,
                           kind=t3.T3_OUT_BF16, C=out, pre=pre)
        _check(out, pre, x, rs, cs, bias, _np(r), "relu2", "bf16")


def test_empty_reduction_and_long_reduction():
    bias, res = np.arange(5, dtype=np.float32), np.ones((3, 5), np.float32)
    out = t3.t3_gemm_fwd_act(torch.zeros((3, 0), dtype=torch.int8, device="cuda"),
                             torch.zeros((5, 0), dtype=torch.uint8, device="cuda"), bias=_dev(bias), residual=_dev(res),
                             act=t3.T3_ACT_RELU2)
    np.testing.assert_array_equal(out.cpu().numpy(), bias[None] ** 2 + res)
    # a reduction longer than one exact accumulation (65536), every term 128
    k = 70_016
    for m in (1, 20, 64):
        a = np.full((m, k), -128, np.int8)
        wp = _dev(oracle.pack(-np.ones((k, 64), np.int8)))
        out = t3.t3_gemm_fwd_act(_dev(a), wp, col_scale=torch.full((64,), 2.0 ** -20, device="cuda"),
                                 bias=torch.ones(64, device="cuda"), kind=t3.T3_OUT_BF16)
        assert torch.equal(out.cpu(), _bf16(np.full((m, 64), np.float32(128 * k) * np.float32(2.0 ** -20) + 1)))


def test_without_workspace():
    """Routes that end in their own epilogue need none; the others say so."""
    lib = t3.load()
    f = lib.t3_gemm_fwd_act
    a = torch.zeros((300, 256), dtype=torch.int8, device="cuda")
    wp = torch.zeros((273, 64), dtype=torch.uint8, device="cuda")
    c = torch.zeros((300, 273), dtype=torch.bfloat16, device="cuda")
    args = [a.data_ptr(), wp.data_ptr(), c.data_ptr(), 300, 273, 256, None, None, None, 0, None, None]
    assert f(*args, t3.T3_OUT_BF16, None, None, 0, None) == t3.T3_EINVAL  # odd output rows
    with pytest.raises(ValueError):
        t3.t3_gemm_fwd_act(a, wp, kind=t3.T3_OUT_F32_ADD)
    with pytest.raises(ValueError):
        t3.t3_gemm_fwd_act(a, wp, bias=torch.zeros(272, device="cuda"))
    with pytest.raises(t3.T3Error):
        t3.t3_gemm_fwd_act(a, wp, act=9)
    with pytest.raises(t3.T3Error):
        t3.t3_gemm_fwd_act(a, wp, C=c, residual=c, kind=t3.T3_OUT_BF16)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(33, 193, 65), (300, 273, 96), (200, 256, 331), (129, 260, 4001), (64, 513, 1280),
                                   (97, 8, 1030), (40, 100, 66_001)])
def test_odd_rows_with_and_without_scratch(m, n, k, dname):
    """Operands laid out aligned in scratch give the bits of those loaded as they lie."""
    a, w, rs, cs, bias, res = _problem(m + n + k, m, n, k)
    R = torch.from_numpy(res).to(DT[dname]).cuda()
    A, Wp = _dev(a), _dev(oracle.pack(w))
    outs = []
    need = t3.load().t3_gemm_fwd_act_scratch(m, n, k)
    assert need > 0
    # none to speak of; too little; what it wants, one byte past it untouched
    for room in (1, need - 1, need):
        buf = torch.full((need + 16,), 0x5A, dtype=torch.uint8, device="cuda")
        pre = torch.full((m, n), 7.0, dtype=DT[dname], device="cuda")
        out = t3.t3_gemm_fwd_act(A, Wp, row_scale=_dev(rs), col_scale=_dev(cs), bias=_dev(bias), act=t3.T3_ACT_SILU,
                                 residual=R, kind=KIND[dname], pre=pre, scratch=buf[:room])
        outs.append((out, pre))
        assert torch.all(buf[room:] == 0x5A)
        if room < need:
            assert torch.all(buf == 0x5A), "used a scratch that is too small"
    x = a.astype(np.int64) @ w.astype(np.int64)
    for out, pre in outs:
        _check(out, pre, x, rs, cs, bias, _np(R), "silu", dname)
        assert torch.equal(out, outs[0][0]) and torch.equal(pre, outs[0][1])


# --------------------------------------------------------------- gradient ---

def _check_bwd(dy, z, act, dz, dbias, dname):
    _, slope, rel = ref.act(_np(z) if z is not None else np.zeros(dy.shape), act)
    want = _np(dy) * slope
    # a slope is a sum of two products: its error is relative to their magnitudes, below 3 in sum here
    near = np.abs(_np(dy)) * rel * (np.abs(slope) + (0 if act in ("none", "relu", "relu2") else 3)) + 4 * ref.U * np.abs(want)
    if dz is not None:
        off = np.abs(_np(dz) - want)
        tol = ref.HALF_ULP[dname] * np.abs(want) + near + 1e-35
        assert np.all(off <= tol), np.max(off / tol)
    if dbias is not None:
        tol = near.sum(0) + (dy.shape[0] + 16) * ref.U * np.abs(want).sum(0) + 1e-35
        assert np.all(np.abs(_np(dbias) - want.sum(0)) <= tol)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8192), (5, 27), (27, 729), (33, 256), (1782, 243), (300, 1288), (700, 264)])
def test_backward(rows, cols, dname):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + cols)
    dy = torch.randn((rows, cols), generator=g, device="cuda").to(DT[dname])
    z = (torch.randn((rows, cols), generator=g, device="cuda") * 3).to(DT[dname])
    z[0, 0] = 0
    for act in ref.ACTS:
        db = torch.full((cols,), 7.0, device="cuda")
        dz, _ = t3.t3_act_bwd(dy, z, ref.ACTS.index(act), dbias=db)
        _check_bwd(dy, z, act, dz, db, dname)
        again = torch.empty_like(db)
        t3.t3_act_bwd(dy, z, ref.ACTS.index(act), dbias=again)
        assert torch.equal(db, again), "changes from call to call"
    assert t3.t3_act_bwd(dy, z, t3.T3_ACT_SILU)[1] is None
    db = torch.empty(cols, device="cuda")
    t3.t3_act_bwd(dy, None, t3.T3_ACT_NONE, dbias=db)
    _check_bwd(dy, None, "none", None, db, dname)
    over = dy.clone()
    t3.t3_act_bwd(over, z, t3.T3_ACT_GELU, dz=over)
    _check_bwd(dy, z, "gelu", over, None, dname)


def test_backward_far_from_zero():
    z = torch.tensor([[-3e38, -1e30, -1e20, -200.0, -90.0, 0.0, 90.0, 200.0, 1e20, 1e30, 3e38, float("nan")]], device="cuda")
    dy = torch.ones_like(z)
    for act in ("relu", "silu", "gelu"):
        got = t3.t3_act_bwd(dy, z, ref.ACTS.index(act))[0].cpu().numpy()[0]
        assert np.all(got[:5] == 0) or np.all(np.abs(got[:5]) < 1e-35), act
        assert np.all(got[6:11] == 1), act
        assert np.isnan(got[11]), act


def test_backward_empty():
    db = torch.ones(6, device="cuda")
    dz, _ = t3.t3_act_bwd(torch.zeros((0, 6), device="cuda"), torch.zeros((0, 6), device="cuda"), t3.T3_ACT_SILU, dbias=db)
    assert dz.shape == (0, 6) and torch.all(db == 0)
