"""The layer norm, the gated feed-forward product and linear attention without a GPU:
refusals before any CUDA call."""
import ctypes

import pytest

import ternary_weight_int8_t3_gb300 as t3

FAKE = ctypes.c_void_p(4096)  # never dereferenced: every case returns first
BF16, F32 = t3.T3_OUT_BF16, t3.T3_OUT_F32
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    return t3.load()


def _norm(lib, x=FAKE, ldx=8, r=None, ldr=0, eps=1e-5, q=FAKE, scale=FAKE, so=None, lds=0, rows=4, cols=8, dt=BF16):
    return lib.t3_layernorm_quant(x, ldx, r, ldr, None, None, eps, q, scale, None, None, so, lds, rows, cols, dt, None)


def test_layer_norm_refusals(lib):
    bad = [dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(ldx=-1), dict(ldx=BIG),
           dict(r=FAKE, ldr=-1), dict(so=FAKE, lds=7), dict(so=FAKE, lds=-8), dict(eps=0.0), dict(eps=-1.0),
           dict(eps=float("nan")), dict(eps=float("inf")), dict(dt=2), dict(dt=-1), dict(x=None), dict(q=None),
           dict(scale=None), dict(cols=0, scale=None)]
    for kw in bad:
        assert _norm(lib, **kw) == t3.T3_EINVAL, kw
    assert _norm(lib, rows=0, x=None, q=None, scale=None) == t3.T3_OK


def _norm_bwd(lib, dy=FAKE, lddy=8, s=FAKE, lds=8, mean=FAKE, rstd=FAKE, dsum=None, ldd=0, dx=FAKE, lddx=8, dg=None,
              db=None, rows=4, cols=8, dt=BF16, ws=None):
    return lib.t3_layernorm_bwd(dy, lddy, s, lds, mean, rstd, None, dsum, ldd, dx, lddx, dg, db, rows, cols, dt, ws, None)


def test_layer_norm_bwd_refusals(lib):
    bad = [dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(lddy=-1), dict(lds=-1), dict(lddx=7),
           dict(dsum=FAKE, ldd=-1), dict(dt=2), dict(dy=None), dict(s=None), dict(mean=None), dict(rstd=None),
           dict(dx=None), dict(dg=FAKE), dict(db=FAKE), dict(dg=FAKE, db=FAKE, ws=FAKE)]
    for kw in bad:
        assert _norm_bwd(lib, **kw) == t3.T3_EINVAL, kw
    assert _norm_bwd(lib, cols=0, lddx=0, dy=None, s=None, mean=None, rstd=None, dx=None) == t3.T3_OK
    assert _norm_bwd(lib, rows=0, dy=None, s=None, mean=None, rstd=None, dx=None) == t3.T3_OK


def _glu(lib, a=FAKE, g=FAKE, u=FAKE, c=FAKE, m=4, n=8, k=8, act=0, pg=None, pu=None, kind=F32, ws=None, room=0):
    return lib.t3_gemm_fwd_glu(a, g, u, c, m, n, k, None, None, None, None, None, act, pg, pu, kind, ws, room, None)


def test_glu_refusals(lib):
    bad = [dict(m=-1), dict(n=-1), dict(k=-1), dict(m=BIG), dict(n=BIG), dict(act=5), dict(act=-1), dict(kind=2),
           dict(kind=3), dict(a=None), dict(g=None), dict(u=None), dict(c=None), dict(pg=FAKE), dict(pu=FAKE),
           dict(room=-1), dict(ws=FAKE, room=1)]
    for kw in bad:
        assert _glu(lib, **kw) == t3.T3_EINVAL, kw
    other = ctypes.c_void_p(8192)
    assert _glu(lib, pg=other, pu=other) == t3.T3_EINVAL
    assert _glu(lib, pg=other, ws=other, room=64) == t3.T3_EINVAL
    assert _glu(lib, m=1, k=16777216) == t3.T3_EOVERFLOW
    assert _glu(lib, m=0, a=None, g=None, u=None, c=None) == t3.T3_OK
    assert _glu(lib, n=0, a=None, g=None, u=None, c=None) == t3.T3_OK
    f = lib.t3_gemm_fwd_glu_workspace
    assert f(FAKE, FAKE, FAKE, FAKE, 0, 8, 8, None, None, F32) == 0
    assert f(FAKE, FAKE, FAKE, FAKE, -1, 8, 8, None, None, F32) == 0
    assert f(FAKE, FAKE, FAKE, FAKE, 8, 8, 8, None, None, 2) == 0


def _glu_bwd(lib, dy=FAKE, gate=FAKE, up=FAKE, act=0, dg=FAKE, du=None, gb=None, ub=None, rows=4, cols=8, dt=BF16, ws=None):
    return lib.t3_glu_bwd(dy, gate, up, act, dg, du, gb, ub, rows, cols, dt, ws, None)


def test_glu_bwd_refusals(lib):
    bad = [dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(act=5), dict(dt=2), dict(dy=None),
           dict(gate=None), dict(up=None), dict(du=FAKE), dict(gb=FAKE), dict(ub=FAKE), dict(gb=FAKE, ub=FAKE, ws=FAKE)]
    for kw in bad:
        assert _glu_bwd(lib, **kw) == t3.T3_EINVAL, kw
    assert _glu_bwd(lib, dg=None) == t3.T3_OK
    assert _glu_bwd(lib, cols=0, dy=None, gate=None, up=None) == t3.T3_OK
    assert _glu_bwd(lib, rows=0, dy=None, gate=None, up=None) == t3.T3_OK


def _lin(lib, q=FAKE, k=FAKE, v=FAKE, o=FAKE, ld=FAKE, ldq=48, ldk=48, ldv=48, ldo=48, b=2, t=3, h=3, dk=16, dv=16, dt=BF16,
         last=None):
    return lib.t3_linear_attn_fwd(q, ldq, k, ldk, v, ldv, ld, None, None, 1.0, o, ldo, last, b, t, h, dk, dv, dt, None, None)


def test_linear_refusals(lib):
    bad = [dict(b=-1), dict(t=-1), dict(h=-1), dict(dk=0), dict(dv=0), dict(dk=129), dict(dv=129), dict(b=BIG), dict(t=BIG),
           dict(h=BIG), dict(b=1 << 20, h=1 << 20), dict(ldq=-1), dict(ldk=BIG), dict(ldv=-1), dict(ldo=47), dict(dt=2),
           dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(ld=None)]
    for kw in bad:
        assert _lin(lib, **kw) == t3.T3_EINVAL, kw
    for kw in (dict(b=0), dict(h=0)):
        assert _lin(lib, q=None, k=None, v=None, o=None, ld=None, **kw) == t3.T3_OK, kw


def _lin_bwd(lib, q=FAKE, k=FAKE, v=FAKE, do=FAKE, ld=FAKE, dq=FAKE, dk_=FAKE, dv_=FAKE, s=48, sq=48, sk=48, sv=48, b=2, t=3,
             h=3, dk=16, dv=16, dt=BF16):
    return lib.t3_linear_attn_bwd(q, s, k, s, v, s, do, s, ld, None, None, 1.0, None, dq, sq, dk_, sk, dv_, sv, None, b, t, h,
                                  dk, dv, dt, None, None)


def test_linear_bwd_refusals(lib):
    bad = [dict(b=-1), dict(t=-1), dict(h=-1), dict(dk=0), dict(dv=129), dict(s=-1), dict(sq=47), dict(sk=47), dict(sv=47),
           dict(dt=2)] + [{n: None} for n in ("q", "k", "v", "do", "ld", "dq", "dk_", "dv_")]
    for kw in bad:
        assert _lin_bwd(lib, **kw) == t3.T3_EINVAL, kw
    assert _lin_bwd(lib, b=0, q=None, k=None, v=None, do=None, ld=None, dq=None, dk_=None, dv_=None) == t3.T3_OK


def test_linear_workspace(lib):
    f = lib.t3_linear_attn_workspace
    assert f(0, 100, 3, 64, 64) == f(2, 32, 3, 64, 64) == f(2, 100, 3, 0, 64) == f(2, 100, 3, 64, 129) == 0
    assert 0 < f(1, 33, 1, 64, 64) <= f(400, 100, 1, 64, 64) <= 610 * 64 * 64
