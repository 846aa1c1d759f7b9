"""GPU tests of the gated feed-forward product (t3_gemm_fwd_glu) and of its gradient
(t3_glu_bwd).  The products are exact integers and the pre-activations a fixed sequence of
float roundings, so those are compared bit for bit in float; the activation within the
bound of tests/more_operators_ref.py."""
import numpy as np
import pytest

import more_operators_ref as ref
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


def _problem(seed, m, n, k):
    g = t3_synth.rng(seed)
    a = t3_synth.int8_uniform(g, (m, k))
    w = [t3_synth.ternary(g, (k, n)) for _ in range(2)]
    rs = (g.random(m) * 0.02 + 0.01).astype(np.float32)
    cs = [((g.random(n) + 0.5) / np.sqrt(max(k, 1))).astype(np.float32) for _ in range(2)]
    bias = [(g.standard_normal(n) * 0.5).astype(np.float32) for _ in range(2)]
    return a, w, rs, cs, bias


def _stored(z, dname):
    t = torch.from_numpy(np.ascontiguousarray(z, np.float32))
    return t.bfloat16() if dname == "bf16" else t


def _check(out, pre, x, rs, cs, bias, act, dname):
    z = [ref.glu_z(x[i], rs, cs[i], bias[i]) for i in range(2)]
    for i in range(2):
        if pre[i] is not None:
            assert torch.equal(pre[i].cpu(), _stored(z[i], dname))
    y, _, ey, _ = ref.act(z[0].astype(np.float64), act)
    up = z[1].astype(np.float64)
    want = y * up
    tol = ey * np.abs(up) + (ref.HALF_ULP[dname] + 2 * ref.U) * np.abs(want) + 1e-35
    off = np.abs(_np(out) - want)
    assert np.all(off <= tol), np.max(off / tol)


# each route: the CUDA-core rows of one to eight, the small-M tensor cores, the
# CTA pairs, operands and outputs of any alignment, small products
SHAPES = [(1, 8192, 1024), (1, 729, 243), (2, 1280, 3456), (5, 640, 640), (8, 300, 512), (16, 8192, 2048),
          (27, 729, 243), (27, 3456, 1280), (32, 256, 512), (33, 96, 128), (256, 192, 1280), (300, 272, 96),
          (300, 273, 96), (129, 1000, 260), (777, 2304, 640), (64, 256, 8192), (1, 16, 16), (3, 1, 5), (200, 8, 16),
          (513, 104, 64), (260, 97, 128)]


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k, dname):
    a, w, rs, cs, bias = _problem(m + n + k, m, n, k)
    x = [a.astype(np.int64) @ v.astype(np.int64) for v in w]
    A, W = _dev(a), [_dev(oracle.pack(v)) for v in w]
    act = ref.ACTS[(m + n) % 5]
    kind = KIND[dname]
    for limit in (0, 1 << 29):  # the tensor-core routes, then the default routing
        t3.t3_set_small_product_limit(limit)
        pre = [torch.full((m, n), 7.0, dtype=DT[dname], device="cuda") for _ in range(2)]
        out = t3.t3_gemm_fwd_glu(A, *W, K=k, row_scale=_dev(rs), gate_scale=_dev(cs[0]), up_scale=_dev(cs[1]),
                                 gate_bias=_dev(bias[0]), up_bias=_dev(bias[1]), act=ref.ACTS.index(act), kind=kind,
                                 pre_gate=pre[0], pre_up=pre[1])
        _check(out, pre, x, rs, cs, bias, act, dname)
        one = torch.full((m, n), 7.0, dtype=DT[dname], device="cuda")
        out = t3.t3_gemm_fwd_glu(A, *W, K=k, act=t3.T3_ACT_NONE, kind=kind, pre_up=one)
        _check(out, [None, one], x, None, [None, None], [None, None], "none", dname)
    rc, detail = t3.t3_last_device_error()
    assert rc == t3.T3_OK, hex(detail)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 512, 256), (20, 512, 256), (300, 384, 256)])
@pytest.mark.parametrize("act", ref.ACTS)
def test_every_activation_on_every_route(act, m, n, k, dname):
    a, w, rs, cs, bias = _problem(m * 3 + n, m, n, k)
    rs *= 8  # spread z over the activations' whole range
    x = [a.astype(np.int64) @ v.astype(np.int64) for v in w]
    out = t3.t3_gemm_fwd_glu(_dev(a), _dev(oracle.pack(w[0])), _dev(oracle.pack(w[1])), row_scale=_dev(rs),
                             gate_scale=_dev(cs[0]), up_scale=_dev(cs[1]), gate_bias=_dev(bias[0]),
                             up_bias=_dev(bias[1]), act=ref.ACTS.index(act), kind=KIND[dname])
    _check(out, [None, None], x, rs, cs, bias, act, dname)


# operands, outputs and pre-activations on every boundary; every route gives the same bits
@pytest.mark.parametrize("limit", [0, 1 << 29])
@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (9, 40, 100), (40, 96, 192), (70, 33, 67), (130, 200, 128)])
def test_alignments(m, n, k, limit):
    t3.t3_set_small_product_limit(limit)
    a, w, rs, cs, bias = _problem(m + n + k, m, n, k)
    x = [a.astype(np.int64) @ v.astype(np.int64) for v in w]
    packed = [oracle.pack(v) for v in w]

    def shifted(v, s, fill):
        return _dev(np.concatenate([np.full(s, fill, v.dtype), v.reshape(-1)]))[s:].view(v.shape)

    first = None
    for sa, sg, su, so in ((0, 0, 0, 0), (1, 0, 0, 0), (0, 3, 0, 0), (0, 0, 2, 0), (4, 4, 8, 1), (16, 16, 16, 3), (0, 0, 0, 2)):
        A, G, U = shifted(a, sa, 77), shifted(packed[0], sg, 255), shifted(packed[1], su, 255)
        outs = [torch.zeros(m * n + 8, device="cuda")[so:so + m * n].view(m, n) for _ in range(3)]
        t3.t3_gemm_fwd_glu(A, G, U, K=k, row_scale=_dev(rs), gate_scale=_dev(cs[0]), up_scale=_dev(cs[1]),
                           gate_bias=_dev(bias[0]), up_bias=_dev(bias[1]), act=t3.T3_ACT_SILU, C=outs[0],
                           pre_gate=outs[1], pre_up=outs[2])
        _check(outs[0], outs[1:], x, rs, cs, bias, "silu", "f32")
        first = outs[0].clone() if first is None else first
        assert torch.equal(outs[0], first)


def test_long_reductions():
    """Past one exact chunk of the tensor cores' float sums."""
    m, n, k = 40, 64, 65536 + 192
    a, w, rs, cs, bias = _problem(3, m, n, k)
    x = [a.astype(np.int64) @ v.astype(np.int64) for v in w]
    out = t3.t3_gemm_fwd_glu(_dev(a), _dev(oracle.pack(w[0])), _dev(oracle.pack(w[1])), row_scale=_dev(rs),
                             gate_scale=_dev(cs[0]), up_scale=_dev(cs[1]), act=t3.T3_ACT_SILU)
    _check(out, [None, None], x, rs, cs, [None, None], "silu", "f32")


def test_empty_shapes():
    w = torch.zeros((8, 4), dtype=torch.uint8, device="cuda")
    assert t3.t3_gemm_fwd_glu(torch.zeros((0, 16), dtype=torch.int8, device="cuda"), w, w).shape == (0, 8)
    none = torch.zeros((0, 4), dtype=torch.uint8, device="cuda")
    assert t3.t3_gemm_fwd_glu(torch.zeros((3, 16), dtype=torch.int8, device="cuda"), none, none).shape == (3, 0)
    w = torch.zeros((8, 0), dtype=torch.uint8, device="cuda")
    b = torch.full((8,), 2.0, device="cuda")
    got = t3.t3_gemm_fwd_glu(torch.zeros((3, 0), dtype=torch.int8, device="cuda"), w, w, gate_bias=b, up_bias=b,
                             act=t3.T3_ACT_RELU)
    assert torch.all(got == 4)
    z, s = torch.zeros((0, 8), device="cuda"), torch.ones(8, device="cuda")
    got = t3.t3_glu_bwd(z, z, z, t3.T3_ACT_SILU, dgate_bias=s, dup_bias=torch.ones(8, device="cuda"))
    assert got[0].shape == (0, 8) and torch.all(got[2] == 0) and torch.all(got[3] == 0)


def _check_backward(dy, gate, up, act, got, dname):
    rows = dy.shape[0]
    dg, du, eg, eu = ref.glu_bwd(_np(dy), _np(gate), _np(up), act)
    for t, want, err in ((got[0], dg, eg), (got[1], du, eu)):
        tol = err + ref.HALF_ULP[dname] * np.abs(want) + 1e-35
        assert np.all(np.abs(_np(t) - want) <= tol), np.max(np.abs(_np(t) - want) / tol)
    for t, want, err in ((got[2], dg, eg), (got[3], du, eu)):
        if t is not None:
            assert np.all(np.abs(_np(t) - want.sum(0)) <= err.sum(0) + (rows + 16) * ref.U * np.abs(want).sum(0) + 1e-35)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8192), (3, 5), (27, 729), (333, 96), (700, 1280), (5000, 243), (64, 4096)])
@pytest.mark.parametrize("act", ["none", "relu2", "silu", "gelu"])
def test_backward(act, rows, cols, dname):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + cols)
    dy, gate, up = (torch.randn((rows, cols), generator=g, device="cuda").mul_(s).to(DT[dname]) for s in (1, 4, 2))
    sums = [torch.empty(cols, device="cuda") for _ in range(2)]
    kind = ref.ACTS.index(act)
    got = t3.t3_glu_bwd(dy, gate, up, kind, dgate_bias=sums[0], dup_bias=sums[1])
    _check_backward(dy, gate, up, act, got, dname)
    again = t3.t3_glu_bwd(dy, gate, up, kind, dup_bias=torch.empty(cols, device="cuda"))
    assert again[2] is None and torch.equal(again[3], got[3]), "changes from call to call"
    for over in range(3):  # in place
        args = [dy.clone(), gate.clone(), up.clone()]
        here = t3.t3_glu_bwd(*args, kind, dgate=args[over], dup=args[(over + 1) % 3])
        assert torch.equal(here[0], got[0]) and torch.equal(here[1], got[1])


def test_backward_relu_and_unaligned_rows():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    flat = [torch.randn(50 * 64 + 8, generator=g, device="cuda")[1:1 + 50 * 64].view(50, 64) for _ in range(3)]
    _check_backward(*flat, "relu", t3.t3_glu_bwd(*flat, t3.T3_ACT_RELU), "f32")


def test_gradient_against_differences():
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    for act in ("relu2", "silu", "gelu"):
        dy, gate, up = (torch.randn((4, 16), generator=g, device="cuda") for _ in range(3))
        got = t3.t3_glu_bwd(dy, gate, up, ref.ACTS.index(act))
        d, a, b, h = _np(dy), _np(gate), _np(up), 1e-6
        want = d * (ref.act(a + h, act)[0] - ref.act(a - h, act)[0]) / (2 * h) * b
        assert np.all(np.abs(_np(got[0]) - want) <= 64 * ref.U * (np.abs(want) + np.abs(d * b)) + 1e-8)
        assert np.all(np.abs(_np(got[1]) - d * ref.act(a, act)[0]) <= 64 * ref.U * np.abs(d * a) + 1e-30)


def test_refusals():
    a = torch.zeros((40, 100), dtype=torch.int8, device="cuda")
    w = torch.zeros((9, 25), dtype=torch.uint8, device="cuda")
    for bad in (dict(gate_scale=torch.ones(8, device="cuda")), dict(up_bias=torch.ones(8, device="cuda")),
                dict(row_scale=torch.ones(9, device="cuda")), dict(C=torch.zeros((40, 8), device="cuda")),
                dict(pre_up=torch.zeros((40, 8), device="cuda"))):
        with pytest.raises(ValueError):
            t3.t3_gemm_fwd_glu(a, w, w, **bad)
    with pytest.raises(ValueError):
        t3.t3_gemm_fwd_glu(a, w, w[:8])
    with pytest.raises(ValueError):
        t3.t3_gemm_fwd_glu(a, w, w, kind=t3.T3_OUT_F32_ADD)
    with pytest.raises(TypeError):
        t3.t3_gemm_fwd_glu(a, w, w, pre_gate=torch.zeros((40, 9), device="cuda").bfloat16())
    with pytest.raises(t3.T3Error):
        t3.t3_gemm_fwd_glu(a, w, w, act=9)
    # too little workspace for odd rows on the tensor cores, and one off its boundary
    room = t3.load().t3_gemm_fwd_glu_workspace(a.data_ptr(), w.data_ptr(), w.data_ptr(), 0, 40, 9, 100, None, None,
                                               t3.T3_OUT_F32)
    assert room > 0
    for ws in (torch.empty(room - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(room + 1, dtype=torch.uint8, device="cuda")[1:]):
        with pytest.raises(t3.T3Error):
            t3.t3_gemm_fwd_glu(a, w, w, workspace=ws)
    x = torch.zeros((4, 8), device="cuda")
    with pytest.raises(t3.T3Error):
        t3.t3_glu_bwd(x, x, x, t3.T3_ACT_SILU, dgate=x, dup=x)
    with pytest.raises(TypeError):
        t3.t3_glu_bwd(x, x.bfloat16(), x, t3.T3_ACT_SILU)
