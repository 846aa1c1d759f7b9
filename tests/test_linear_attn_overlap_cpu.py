"""Linear attention refuses outputs that are one of its inputs or of each other, before any CUDA call."""
import ctypes
import itertools

import pytest

import ternary_weight_int8_t3_gb300 as t3

AT = {n: ctypes.c_void_p(4096 * (i + 1)) for i, n in enumerate(("q", "k", "v", "ld", "o", "do", "dq", "dk", "dv"))}


@pytest.mark.parametrize("over", ["q", "k", "v"])
def test_an_output_over_an_input(over):
    f = t3.load().t3_linear_attn_fwd
    args = [AT["q"], 48, AT["k"], 48, AT["v"], 48, AT["ld"], None, None, 1.0]
    assert f(*args, AT[over], 48, None, 2, 3, 3, 16, 16, t3.T3_OUT_BF16, None, None) == t3.T3_EINVAL


@pytest.mark.parametrize("at,over", [*itertools.product(("dq", "dk", "dv"), ("q", "k", "v", "do")), ("dq", "dk"), ("dk", "dv"),
                                     ("dv", "dq")])
def test_a_gradient_over_an_input_or_another(at, over):
    p = dict(AT)
    p[at] = p[over]
    args = [p["q"], 48, p["k"], 48, p["v"], 48, p["do"], 48, p["ld"], None, None, 1.0, None, p["dq"], 48, p["dk"], 48, p["dv"], 48]
    assert t3.load().t3_linear_attn_bwd(*args, None, 2, 3, 3, 16, 16, t3.T3_OUT_BF16, None, None) == t3.T3_EINVAL


def test_nothing_to_do_overlaps_nothing():
    x = AT["q"]
    f, b = t3.load().t3_linear_attn_fwd, t3.load().t3_linear_attn_bwd
    assert f(x, 48, x, 48, x, 48, x, None, None, 1.0, x, 48, None, 0, 3, 3, 16, 16, t3.T3_OUT_BF16, None, None) == t3.T3_OK
    assert b(x, 48, x, 48, x, 48, x, 48, x, None, None, 1.0, None, x, 48, x, 48, x, 48, None, 0, 3, 3, 16, 16, t3.T3_OUT_BF16, None,
             None) == t3.T3_OK


BIG = 1 << 31
SIZES = [dict(b=-1), dict(t=-1), dict(h=-1), dict(dk=0), dict(dv=0), dict(dk=129), dict(dv=129), dict(b=BIG), dict(t=BIG), dict(h=BIG),
         dict(b=1 << 20, h=1 << 20), dict(dt=2), dict(dt=-1)]


@pytest.mark.parametrize("bad", SIZES + [dict(sq=-1), dict(sk=BIG), dict(sv=-1), dict(so=47)] + [{n: None} for n in ("q", "k", "v", "ld", "o")])
def test_forward_refusals_of_buffers_apart(bad):
    p = dict(AT, b=2, t=3, h=3, sq=48, sk=48, sv=48, so=48, dt=t3.T3_OUT_BF16)
    size = dict(dk=16, dv=16)
    for n, x in bad.items():
        (size if n in size else p)[n] = x
    assert t3.load().t3_linear_attn_fwd(p["q"], p["sq"], p["k"], p["sk"], p["v"], p["sv"], p["ld"], None, None, 1.0, p["o"], p["so"],
                                        None, p["b"], p["t"], p["h"], size["dk"], size["dv"], p["dt"], None, None) == t3.T3_EINVAL


@pytest.mark.parametrize("bad", SIZES + [dict(s=-1), dict(sq=47), dict(sk=47), dict(sv=47)] +
                         [dict(at=n) for n in ("q", "k", "v", "do", "ld", "dq", "dk", "dv")])
def test_backward_refusals_of_buffers_apart(bad):
    p = dict(b=2, t=3, h=3, dk=16, dv=16, s=48, sq=48, sk=48, sv=48, dt=t3.T3_OUT_BF16)
    p.update(bad)
    a = dict(AT)
    if "at" in bad:
        a[bad["at"]] = None
    assert t3.load().t3_linear_attn_bwd(a["q"], p["s"], a["k"], p["s"], a["v"], p["s"], a["do"], p["s"], a["ld"], None, None, 1.0, None,
                                        a["dq"], p["sq"], a["dk"], p["sk"], a["dv"], p["sv"], None, p["b"], p["t"], p["h"], p["dk"],
                                        p["dv"], p["dt"], None, None) == t3.T3_EINVAL
