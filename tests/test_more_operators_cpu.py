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
