"""GPU tests of linear attention with a decay for each head (t3_linear_attn_fwd,
t3_linear_attn_bwd) against the 64-bit recurrence of tests/more_operators_ref.py."""
import numpy as np
import pytest

import more_operators_ref as ref
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _problem(seed, b, t, h, dk, dv, dname, resets=0.0, fused=False):
    g = _gen(seed)
    dt = DT[dname]

    def rand(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    p = {"scale": dk ** -0.5}
    if fused:
        both = torch.full((b, t, h * (2 * dk + dv) + 8), 3.0, dtype=dt, device="cuda")
        p["q"] = both[..., :h * dk].unflatten(-1, (h, dk))
        p["k"] = both[..., h * dk:2 * h * dk].unflatten(-1, (h, dk))
        p["v"] = both[..., 2 * h * dk:h * (2 * dk + dv)].unflatten(-1, (h, dv))
        for n in "qkv":
            p[n].copy_(rand(*p[n].shape))
    else:
        p["q"], p["k"], p["v"] = rand(b, t, h, dk, dtype=dt), rand(b, t, h, dk, dtype=dt), rand(b, t, h, dv, dtype=dt)
    # memories of a few tokens to a few hundred, heads that forget nothing and everything among them
    ld = torch.log1p(-torch.exp2(-(torch.rand(h, generator=g, device="cuda") * 7 + 1)))
    ld[0] = 0.0
    if h > 2:
        ld[1], ld[2] = -float("inf"), -25.0
    p["log_decay"] = ld
    p["state"] = rand(b, h, dk, dv)
    p["resets"] = (torch.rand((b, t), generator=g, device="cuda") < resets).to(torch.uint8) if resets else None
    p["do"], p["dstate_last"] = rand(b, t, h, dv, dtype=dt), rand(b, h, dk, dv)
    return p


def _forward_ref(p, chunks, state=True, resets=True):
    return ref.linear_attend(_np(p["q"]), _np(p["k"]), _np(p["v"]), _np(p["log_decay"]), _np(p["state"]) if state else None,
                             _np(p["resets"]) if resets else None, p["scale"], chunks=chunks)


def _close(got, want, bound, dname, chunks):
    got = _np(got)
    tol = bound + (ref.HALF_ULP[dname] + 2 * ref.U) * (np.abs(want) + bound) + 1e-30
    off = np.abs(got - want)
    assert np.all(off <= tol), np.max(off / tol)
    if chunks and want.size >= 4096:
        # three roundings of at most 2^-8, evenly spread: 2^-8 / sqrt(3) each, 2^-8 together; half again for parts that
        # are larger than their sum
        assert np.sqrt((off ** 2).mean()) <= 1.5 * 2.0 ** -8 * np.sqrt((want ** 2).mean())


def _chunked(p, dname):
    """Whether the call is taken by chunks of 128 tokens on the tensor cores."""
    _, t, _, dk = p["q"].shape
    return dname == "bf16" and t > 16 and dk % 8 == 0 and p["v"].shape[3] % 8 == 0


def _check_forward(p, dname, **kw):
    chunks = _chunked(p, dname)
    o, last, eo, es = _forward_ref(p, chunks)
    got = t3.t3_linear_attn_fwd(p["q"], p["k"], p["v"], p["log_decay"], p["state"], p["resets"], p["scale"], **kw)
    _close(got[0], o, eo, dname, chunks)
    _close(got[1], last, es, "f32", False)
    return got


# token, block and chunk edges; heads of any size; one sequence and many; documents
SHAPES = [(1, 1, 1, 1, 1), (3, 1, 5, 128, 128), (2, 1, 3, 81, 40), (1, 2, 2, 64, 64), (2, 15, 1, 16, 8), (1, 16, 3, 128, 64),
          (1, 17, 3, 128, 64), (2, 31, 2, 24, 128), (1, 32, 3, 64, 64), (1, 33, 4, 100, 50), (1, 127, 2, 128, 128),
          (2, 128, 3, 64, 128), (1, 129, 2, 128, 128), (3, 255, 1, 8, 16), (1, 300, 5, 81, 81), (2, 513, 3, 128, 128),
          (1, 1000, 2, 64, 64), (5, 140, 4, 72, 104)]


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("resets", [0.0, 0.03])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, resets, dname):
    p = _problem(sum(shape), *shape, dname, resets, fused=shape[1] % 2 == 0)
    first = _check_forward(p, dname)
    again = t3.t3_linear_attn_fwd(p["q"], p["k"], p["v"], p["log_decay"], p["state"], p["resets"], p["scale"])
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1]), "changes from call to call"
    rc, detail = t3.t3_last_device_error()
    assert rc == t3.T3_OK, hex(detail)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("resets", [0.0, 0.03])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, resets, dname):
    p = _problem(sum(shape) + 1, *shape, dname, resets, fused=shape[1] % 2 == 1)
    chunks = _chunked(p, dname)
    want = ref.linear_attend_bwd(_np(p["q"]), _np(p["k"]), _np(p["v"]), _np(p["log_decay"]), _np(p["do"]), _np(p["state"]),
                                 _np(p["resets"]), p["scale"], _np(p["dstate_last"]), chunks)
    got = t3.t3_linear_attn_bwd(p["q"], p["k"], p["v"], p["log_decay"], p["do"], p["state"], p["resets"], p["scale"],
                                p["dstate_last"])
    for i, n in enumerate(("q", "k", "v", "state")):
        _close(got[i], *want[n], "f32" if n == "state" else dname, chunks and n != "state")
    # without a state and its gradient
    got = t3.t3_linear_attn_bwd(p["q"], p["k"], p["v"], p["log_decay"], p["do"], scale=p["scale"])
    want = ref.linear_attend_bwd(_np(p["q"]), _np(p["k"]), _np(p["v"]), _np(p["log_decay"]), _np(p["do"]), None, None,
                                 p["scale"], None, chunks)
    for i, n in enumerate(("q", "k", "v", "state")):
        _close(got[i], *want[n], "f32" if n == "state" else dname, chunks and n != "state")
    rc, detail = t3.t3_last_device_error()
    assert rc == t3.T3_OK, hex(detail)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
def test_tokens_one_by_one_and_in_place(dname):
    p = _problem(7, 2, 40, 3, 64, 128, dname, 0.05)
    whole = t3.t3_linear_attn_fwd(p["q"], p["k"], p["v"], p["log_decay"], p["state"], p["resets"], p["scale"])
    o, last, eo, es = _forward_ref(p, True)
    state, parts = p["state"].clone(), []
    for t in range(40):
        parts.append(t3.t3_linear_attn_fwd(*(p[n][:, t:t + 1] for n in "qkv"), p["log_decay"], state,
                                           p["resets"][:, t:t + 1].contiguous(), p["scale"], state_last=state)[0])
    _close(torch.cat(parts, 1), o, eo, dname, False)
    _close(state, last, es, "f32", False)
    state = p["state"].clone()  # a whole prompt in place
    got = t3.t3_linear_attn_fwd(p["q"], p["k"], p["v"], p["log_decay"], state, p["resets"], p["scale"], state_last=state)
    assert torch.equal(got[0], whole[0]) and torch.equal(state, whole[1])


# cut into ranges with and without a workspace, few sequences and more than fill the GPU, in place and not
@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1500, 1, 64, 64), (2, 700, 2, 128, 40), (1, 257, 7, 128, 128), (170, 300, 1, 16, 16),
                                   (9, 400, 23, 32, 64), (320, 200, 1, 8, 8)])
def test_ranges(shape, dname):
    p = _problem(sum(shape), *shape, dname, 0.002)
    got = _check_forward(p, dname)
    b, t, h, dk, dv = shape
    n = t3.load().t3_linear_attn_workspace(b, t, h, dk, dv)
    assert n > 0
    mine = torch.full((n + 8,), float("nan"), device="cuda")
    same = t3.t3_linear_attn_fwd(p["q"], p["k"], p["v"], p["log_decay"], p["state"], p["resets"], p["scale"],
                                 workspace=mine[:n])
    assert torch.equal(same[0], got[0]) and torch.equal(same[1], got[1])
    assert torch.isnan(mine[n:]).all(), "written behind the workspace"
    state = p["state"].clone()
    here = t3.t3_linear_attn_fwd(p["q"], p["k"], p["v"], p["log_decay"], state, p["resets"], p["scale"], state_last=state)
    o, last, eo, es = _forward_ref(p, _chunked(p, dname))
    _close(here[0], o, eo, dname, False)
    _close(state, last, es, "f32", False)
    # the C entry without a workspace: sequences as wholes
    alone, end = torch.empty_like(got[0]), torch.empty_like(got[1])
    rc = t3.load().t3_linear_attn_fwd(
        p["q"].data_ptr(), h * dk, p["k"].data_ptr(), h * dk, p["v"].data_ptr(), h * dv, p["log_decay"].data_ptr(),
        p["state"].data_ptr(), p["resets"].data_ptr(), p["scale"], alone.data_ptr(), h * dv, end.data_ptr(), b, t, h, dk, dv,
        t3.T3_OUT_BF16 if dname == "bf16" else t3.T3_OUT_F32, None, torch.cuda.current_stream().cuda_stream)
    assert rc == t3.T3_OK
    _close(alone, o, eo, dname, False)
    _close(end, last, es, "f32", False)
    back = ref.linear_attend_bwd(_np(p["q"]), _np(p["k"]), _np(p["v"]), _np(p["log_decay"]), _np(p["do"]), _np(p["state"]),
                                 _np(p["resets"]), p["scale"], _np(p["dstate_last"]), _chunked(p, dname))
    d = p["dstate_last"].clone()
    grads = t3.t3_linear_attn_bwd(p["q"], p["k"], p["v"], p["log_decay"], p["do"], p["state"], p["resets"], p["scale"], d,
                                  dstate=d)
    for i, n in enumerate(("q", "k", "v", "state")):
        _close(grads[i], *back[n], "f32" if n == "state" else dname, False)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("offset,pad", [(0, 8), (8, 0), (1, 0), (4, 3)])
def test_strides_and_bases(offset, pad, dname):
    b, t, h, dk, dv = 2, 150, 3, 64, 32
    p = _problem(offset + pad, b, t, h, dk, dv, dname, 0.02)

    def placed(x):
        d = x.shape[3]
        buf = torch.full((offset + b * t * (h * d + pad) + 8,), 5.0, dtype=x.dtype, device="cuda")
        v = buf[offset:offset + b * t * (h * d + pad)].view(b, t, h * d + pad)[..., :h * d].unflatten(-1, (h, d))
        v.copy_(x)
        return v, buf

    for n in ("q", "k", "v", "do"):
        p[n] = placed(p[n])[0]
    o, buf = placed(torch.zeros((b, t, h, dv), dtype=DT[dname], device="cuda"))
    aligned = (offset * DT[dname].itemsize) % 16 == 0 and (pad * DT[dname].itemsize) % 16 == 0
    want, last, eo, es = _forward_ref(p, True)
    got = t3.t3_linear_attn_fwd(p["q"], p["k"], p["v"], p["log_decay"], p["state"], p["resets"], p["scale"], o=o)
    _close(got[0], want, eo, dname, aligned)
    _close(got[1], last, es, "f32", False)
    o.fill_(5)
    assert torch.all(buf == 5), "written outside the rows"
    outs = [placed(torch.zeros_like(p[n])) for n in "qkv"]
    back = ref.linear_attend_bwd(_np(p["q"]), _np(p["k"]), _np(p["v"]), _np(p["log_decay"]), _np(p["do"]), _np(p["state"]),
                                 _np(p["resets"]), p["scale"], None, True)
    got = t3.t3_linear_attn_bwd(p["q"], p["k"], p["v"], p["log_decay"], p["do"], p["state"], p["resets"], p["scale"],
                                dq=outs[0][0], dk=outs[1][0], dv=outs[2][0])
    for i, n in enumerate(("q", "k", "v", "state")):
        _close(got[i], *back[n], "f32" if n == "state" else dname, False)
    for x, buf in outs:
        x.fill_(5)
        assert torch.all(buf == 5), "written outside the rows"


def test_documents_do_not_see_each_other():
    """Documents packed into one row give what each gives alone, and gradients end with them."""
    for dname in DT:
        p = _problem(3, 1, 400, 2, 64, 64, dname)
        r = torch.zeros((1, 400), dtype=torch.bool, device="cuda")
        cuts = [0, 1, 90, 128, 129, 300, 400]
        for c in cuts[:-1]:
            r[0, c] = True
        o, _ = t3.t3_linear_attn_fwd(p["q"], p["k"], p["v"], p["log_decay"], p["state"], r, p["scale"])
        got = t3.t3_linear_attn_bwd(p["q"], p["k"], p["v"], p["log_decay"], p["do"], p["state"], r, p["scale"])
        assert torch.all(got[3] == 0)
        for a, b in zip(cuts, cuts[1:]):
            part = [p[n][:, a:b] for n in ("q", "k", "v", "do")]
            chunks = dname == "bf16"
            w, _, e, _ = ref.linear_attend(*(_np(x) for x in part[:3]), _np(p["log_decay"]), None, None, p["scale"], chunks=chunks)
            _close(o[:, a:b], w, e, dname, False)
            back = ref.linear_attend_bwd(*(_np(x) for x in part[:3]), _np(p["log_decay"]), _np(part[3]), None, None, p["scale"],
                                         None, chunks)
            for i, n in enumerate("qkv"):
                _close(got[i][:, a:b], *back[n], dname, False)


@pytest.mark.parametrize("dname,length,dk,dv", [("bf16", 400, 64, 64), ("bf16", 400, 128, 128), ("bf16", 3000, 128, 64),
                                                ("bf16", 14, 32, 32), ("f32", 400, 40, 33), ("bf16", 200, 27, 27)])
def test_values_that_are_not_finite_stay_in_their_document(dname, length, dk, dv):
    """A document that holds NaN and infinities, and a state in front of the first that does: the others' outputs and
    gradients are, bit for bit, those beside a finite one."""
    p = _problem(dk + length, 2, length, 2, dk, dv, dname)
    at = sorted([0, length // 4, length // 4 + 9, length // 2, length - 3])
    r = torch.zeros((2, length), dtype=torch.bool, device="cuda")
    r[:, at] = True

    def run(q, k, v, do, state):
        o, last = t3.t3_linear_attn_fwd(q, k, v, p["log_decay"], state, r, p["scale"])
        return [o, *t3.t3_linear_attn_bwd(q, k, v, p["log_decay"], do, state, r, p["scale"], p["dstate_last"])[:3]], last
    want, last = run(*(p[n] for n in ("q", "k", "v", "do", "state")))
    nan, inf = float("nan"), float("inf")
    for begin, end in zip(at[:-1], at[1:]):
        bad = {n: p[n].clone() for n in ("q", "k", "v", "do")}
        middle = (begin + end) // 2
        bad["q"][0, middle, 0, 3], bad["k"][0, middle, 0, 1], bad["v"][0, end - 1, 0, 2] = nan, inf, nan
        bad["v"][0, begin, 1], bad["do"][0, middle, 0, 4], bad["do"][0, begin, 1, 0] = -inf, nan, inf
        got, end_state = run(*bad.values(), torch.full_like(p["state"], nan))
        for g, w in zip(got, want):
            assert torch.equal(g[1], w[1])
            assert torch.equal(g[0, :begin], w[0, :begin]) and torch.equal(g[0, end:], w[0, end:])
            assert not torch.isfinite(g[0, begin:end]).all()
        assert torch.equal(end_state, last)


def test_gradient_against_differences():
    """dq, dk, dv and dstate against central differences of the 64-bit recurrence."""
    p = _problem(11, 1, 6, 2, 3, 2, "f32", 0.2)
    args = [_np(p[n]) for n in ("q", "k", "v", "state")]
    do, dl, res, ld = _np(p["do"]), _np(p["dstate_last"]), _np(p["resets"]), _np(p["log_decay"])
    got = t3.t3_linear_attn_bwd(p["q"], p["k"], p["v"], p["log_decay"], p["do"], p["state"], p["resets"], p["scale"],
                                p["dstate_last"])

    def loss(q, k, v, s):
        o, last, _, _ = ref.linear_attend(q, k, v, ld, s, res, p["scale"])
        return (o * do).sum() + (last * dl).sum()

    for at in range(4):
        g = _np(got[at])
        for i in np.ndindex(g.shape):
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[at][i] += 1e-5
            lo[at][i] -= 1e-5
            want = (loss(*hi) - loss(*lo)) / 2e-5
            # some dozens of float terms of order one to ten; the loss is a polynomial whose third derivatives meet 1e-10
            assert abs(g[i] - want) <= 1e-4


def test_empty_shapes():
    ld = torch.zeros(3, device="cuda")
    e = torch.zeros((2, 0, 3, 16), device="cuda")
    s = torch.randn((2, 3, 16, 16), device="cuda")
    o, last = t3.t3_linear_attn_fwd(e, e, e, ld, s)
    assert o.shape == (2, 0, 3, 16) and torch.equal(last, s)
    assert torch.all(t3.t3_linear_attn_fwd(e, e, e, ld)[1] == 0)
    assert torch.equal(t3.t3_linear_attn_bwd(e, e, e, ld, e, dstate_last=s)[3], s)
    e = torch.zeros((0, 5, 3, 16), device="cuda")
    assert t3.t3_linear_attn_fwd(e, e, e, ld)[0].shape == (0, 5, 3, 16)


def test_refusals():
    x, ld = torch.zeros((2, 40, 3, 16), device="cuda"), torch.zeros(3, device="cuda")
    for bad in (dict(state=torch.zeros((2, 3, 16, 15), device="cuda")), dict(resets=torch.zeros((2, 39), dtype=torch.uint8, device="cuda")),
                dict(o=torch.zeros((2, 40, 3, 15), device="cuda")), dict(state_last=torch.zeros((2, 3, 15, 16), device="cuda")),
                dict(workspace=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            t3.t3_linear_attn_fwd(x, x, x, ld, **bad)
    with pytest.raises(ValueError):
        t3.t3_linear_attn_fwd(x, x[:, :, :, :15], x, ld)
    with pytest.raises(ValueError):
        t3.t3_linear_attn_fwd(x, x, x, torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError):
        t3.t3_linear_attn_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), x, x, ld)
    with pytest.raises(TypeError):
        t3.t3_linear_attn_fwd(x, x.bfloat16(), x, ld)
    with pytest.raises(TypeError):
        t3.t3_linear_attn_fwd(x.half(), x.half(), x.half(), ld)
    big = torch.zeros((1, 2, 1, 136), device="cuda")
    with pytest.raises(t3.T3Error):
        t3.t3_linear_attn_fwd(big, big, big, ld[:1])
    with pytest.raises(TypeError):
        t3.t3_linear_attn_bwd(x, x, x, ld, x.bfloat16())
