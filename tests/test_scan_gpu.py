"""GPU tests of the gated recurrence (t3_gated_scan_fwd, t3_gated_scan_bwd)
against the 64-bit forms of tests/operators_ref.py, within the error bounds
that those carry along the sequence."""
import numpy as np
import pytest

import operators_ref as ref
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


def _np(t):
    return t.detach().double().cpu().numpy()


def _make(seed, b, t, d, dname, fused=False, resets=False, mean=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[dname]

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    both = torch.empty((b, t, 2 * d), dtype=dt, device="cuda")
    gate, cand = (both[..., :d], both[..., d:]) if fused else (torch.empty((b, t, d), dtype=dt, device="cuda"),
                                                              torch.empty((b, t, d), dtype=dt, device="cuda"))
    gate.copy_(rand(b, t, d) * 1.7 + mean)
    cand.copy_(rand(b, t, d))
    r = None
    if resets:
        r = (torch.rand((b, t), generator=g, device="cuda") < 0.05).to(torch.uint8) * 7
        r[:, 0] = 0
        if t > 3:
            r[0, 0] = 1
            r[-1, t - 1] = 255
    return gate, cand, rand(b, d), r, rand(b, t, d).to(dt), rand(b, d)


def _resets_np(r, b, t):
    return np.zeros((b, t)) if r is None else _np(r)


def _check_forward(gate, cand, h0, r, got, dname):
    b, t, d = gate.shape
    h, prior, err = ref.scan(_np(gate), _np(cand), np.zeros((b, d)) if h0 is None else _np(h0), _resets_np(r, b, t))
    tol = ref.HALF_ULP[dname] * np.abs(h) + err + 1e-30
    off = np.abs(_np(got[0]) - h)
    assert np.all(off <= tol), np.max(off / tol)
    if t:
        assert np.all(np.abs(_np(got[1]) - h[:, -1]) <= ref.U * np.abs(h[:, -1]) + err[:, -1] + 1e-30)


# lengths around the tokens a thread, a warp, a CTA and a cluster take; odd widths
CASES = [(1, 1, 1), (3, 1, 96), (27, 1, 243), (2, 2, 64), (2, 7, 66), (1, 8, 130), (3, 9, 27), (2, 15, 64), (2, 16, 62),
         (2, 17, 128), (1, 127, 243), (2, 128, 64), (1, 129, 66), (5, 300, 729), (1, 1000, 34), (1, 1024, 64),
         (1, 1025, 63), (1, 5000, 30), (40, 77, 1000), (16, 260, 2050)]


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("b,t,d", CASES)
def test_forward(b, t, d, dname):
    gate, cand, h0, r, _, _ = _make(b + t + d, b, t, d, dname, fused=(t % 2 == 0), resets=True)
    _check_forward(gate, cand, h0, r, t3.t3_gated_scan_fwd(gate, cand, h0, r), dname)
    _check_forward(gate, cand, None, None, t3.t3_gated_scan_fwd(gate, cand), dname)


def _check_backward(gate, cand, h, dh, h0, r, dl, got, dname):
    b, t, d = gate.shape
    first = np.zeros((b, 1, d)) if h0 is None else _np(h0)[:, None]
    rs = _resets_np(r, b, t)
    prior = np.concatenate([first, _np(h)[:, :-1]], 1) * (rs == 0)[..., None]
    want, err = ref.scan_bwd(_np(gate), _np(cand), prior, _np(dh), rs, np.zeros((b, d)) if dl is None else _np(dl))
    for name, g, w, e, ulp in zip(("dgate", "dcand", "dh0"), got, want, err,
                                  (ref.HALF_ULP[dname], ref.HALF_ULP[dname], ref.U)):
        tol = ulp * np.abs(w) + e + 1e-30
        off = np.abs(_np(g) - w)
        assert np.all(off <= tol), (name, np.max(off / tol))


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("b,t,d", CASES)
def test_backward(b, t, d, dname):
    gate, cand, h0, r, dh, dl = _make(3 * b + t + d, b, t, d, dname, fused=(t % 2 == 1), resets=True)
    h = t3.t3_gated_scan_fwd(gate, cand, h0, r)[0]
    _check_backward(gate, cand, h, dh, h0, r, dl, t3.t3_gated_scan_bwd(gate, cand, h, dh, h0, r, dl), dname)
    h = t3.t3_gated_scan_fwd(gate, cand)[0]
    _check_backward(gate, cand, h, dh, None, None, None, t3.t3_gated_scan_bwd(gate, cand, h, dh), dname)


# more tiles than are resident at once: CTAs take parts of several, whose states travel between them
@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("b,t,d", [(13, 210, 2056), (20, 600, 1024), (5, 500, 4104), (41, 129, 520)])
def test_many_tiles(b, t, d, dname):
    gate, cand, h0, r, dh, dl = _make(b * t, b, t, d, dname, fused=True, resets=True)
    state = h0.clone()
    got = t3.t3_gated_scan_fwd(gate, cand, state, r, h_last=state)
    _check_forward(gate, cand, h0, r, got, dname)
    _check_backward(gate, cand, got[0], dh, h0, r, dl, t3.t3_gated_scan_bwd(gate, cand, got[0], dh, h0, r, dl), dname)
    got = t3.t3_gated_scan_fwd(gate, cand)
    _check_forward(gate, cand, None, None, got, dname)
    _check_backward(gate, cand, got[0], dh, None, None, None, t3.t3_gated_scan_bwd(gate, cand, got[0], dh), dname)
    rc, detail = t3.t3_last_device_error()
    assert rc == t3.T3_OK, hex(detail)


def test_backward_against_differences_of_the_kernel():
    """Directional differences of the forward kernel itself.  loss is linear in
    the outputs; a central difference with step 2e-2 truncates at 1e-4 of the
    third derivative's scale, and float rounding of a sum of n terms adds
    sqrt(n) u |loss terms| / step, both below 2e-3 of the gradient's norm here."""
    gate, cand, h0, _, dh, dl = _make(8, 2, 200, 64, "f32")

    def loss(gate, cand, h0):
        h, last = t3.t3_gated_scan_fwd(gate, cand, h0)
        return float((h.double() * dh.double()).sum() + (last.double() * dl.double()).sum())

    h = t3.t3_gated_scan_fwd(gate, cand, h0)[0]
    grads = t3.t3_gated_scan_bwd(gate, cand, h, dh, h0, None, dl)
    for i in range(3):
        args = [gate, cand, h0]
        u = grads[i] / grads[i].double().norm().float()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 2e-2 * u, args[i] - 2e-2 * u
        slope = (loss(*up) - loss(*down)) / 4e-2
        assert abs(slope - float(grads[i].double().norm())) <= 2e-3 * abs(slope), i


@pytest.mark.parametrize("t", [6, 200, 1300])
def test_tokens_one_by_one_advance_the_state_in_place(t):
    gate, cand, h0, r, _, _ = _make(t, 2, t, 70, "f32", resets=True)
    want, last = t3.t3_gated_scan_fwd(gate, cand, h0, r)
    state = h0.clone()
    rows = []
    for i in range(t):
        h, s = t3.t3_gated_scan_fwd(gate[:, i:i + 1], cand[:, i:i + 1], state, r[:, i:i + 1].contiguous(), h_last=state)
        assert s is state
        rows.append(h)
    _, _, err = ref.scan(_np(gate), _np(cand), _np(h0), _np(r))
    off = np.abs(_np(torch.cat(rows, 1)) - _np(want))
    assert np.all(off <= 2 * err + 2 * ref.U * np.abs(_np(want)) + 1e-30)
    whole = h0.clone()
    t3.t3_gated_scan_fwd(gate, cand, whole, r, h_last=whole)
    assert torch.equal(whole, last)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("t", [1, 40, 700])
def test_gates_at_their_limits(t, dname):
    gate, cand, h0, _, dh, dl = _make(t, 3, t, 64, dname)
    gate[0, ::3], gate[0, 1::3] = INF, -INF      # keep all, take all
    gate[1, ::2], gate[1, 1::2] = 3e38, -3e38
    cand[0, ::3] = float("nan")                  # masked tokens may hold anything
    cand[1, ::2] = INF
    gate[2] = INF                                # nothing is ever taken
    cand[2] = float("nan")
    h, last = t3.t3_gated_scan_fwd(gate, cand, h0)
    clean = torch.where(gate > 1e38, torch.zeros_like(cand), cand)
    _check_forward(gate, clean, h0, None, (h, last), dname)
    assert torch.equal(h[2], h0[2].to(DT[dname]).expand(t, -1)) and torch.equal(last[2], h0[2])
    got = t3.t3_gated_scan_bwd(gate, cand, h, dh, h0, None, dl)
    assert torch.all(got[0][gate.abs() > 1e38] == 0) and torch.all(got[1][gate > 1e38] == 0)
    _check_backward(gate, clean, h, dh, h0, None, dl, got, dname)


def test_a_long_memory_is_not_lost_to_rounding():
    """1 - a = 1e-6: the state moves by about half over 700,000 tokens."""
    t = 700_000
    gate = torch.full((1, t, 2), 13.815510, device="cuda")
    cand = torch.ones((1, t, 2), device="cuda")
    last = t3.t3_gated_scan_fwd(gate, cand)[1]
    k = 1 / (1 + np.exp(np.float64(np.float32(13.815510))))
    want = 1 - (1 - k) ** t
    # k itself is within LOGISTIC of the truth, and the state's roundings add
    # at most one ulp a step, both counted in full
    assert abs(float(last[0, 0]) - want) <= want * float(ref.logistic_error(np.float64(13.8))) + 2 * ref.U * 1e6 * 0.5
    assert abs(float(last[0, 0]) - want) <= 2e-3


def test_offsets_past_32_bits():
    """Rows more than 2^32 bytes from the base, reached through the stride."""
    rows, width, ld = 2050, 64, (1 << 20) + 64
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of device memory")
    big = torch.empty((rows - 1) * ld + 2 * width, dtype=torch.bfloat16, device="cuda")
    gate = big.as_strided((1, rows, width), (rows * ld, ld, 1))
    cand = big.as_strided((1, rows, width), (rows * ld, ld, 1), width)
    g2, c2, h0, _, dh, dl = _make(4, 1, rows, width, "bf16")
    gate.copy_(g2)
    cand.copy_(c2)
    want = t3.t3_gated_scan_fwd(g2, c2, h0)
    got = t3.t3_gated_scan_fwd(gate, cand, h0)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    wb = t3.t3_gated_scan_bwd(g2, c2, want[0], dh, h0, None, dl)
    gb = t3.t3_gated_scan_bwd(gate, cand, want[0], dh, h0, None, dl)
    for a, b in zip(wb, gb):
        assert torch.equal(a, b)


@pytest.mark.parametrize("offset", [1, 2, 4])
def test_unaligned_bases_and_outputs_of_wider_tensors(offset):
    b, t, d = 2, 150, 96
    gate, cand, h0, r, dh, dl = _make(offset, b, t, d, "bf16", resets=True)
    wide = torch.ones((b, t, 3 * d + 8), dtype=torch.bfloat16, device="cuda")
    h = wide[..., offset:offset + d]
    want = t3.t3_gated_scan_fwd(gate, cand, h0, r)
    got = t3.t3_gated_scan_fwd(gate, cand, h0, r, h=h)
    assert got[0] is h and torch.equal(h.contiguous(), want[0]) and torch.equal(got[1], want[1])
    dg, dc = wide[..., offset + d:offset + 2 * d], wide[..., offset + 2 * d:offset + 3 * d]
    back = t3.t3_gated_scan_bwd(gate, cand, h, dh, h0, r, dl, dgate=dg, dcand=dc)
    again = t3.t3_gated_scan_bwd(gate, cand, want[0], dh, h0, r, dl)
    for x, y in zip(back, again):
        assert torch.equal(x.contiguous(), y)
    for part in (h, dg, dc):
        part.fill_(1)
    assert torch.all(wide == 1), "written outside the rows"


def test_results_do_not_change_from_call_to_call():
    gate, cand, h0, r, dh, dl = _make(77, 2, 3000, 258, "bf16", resets=True)
    first = t3.t3_gated_scan_fwd(gate, cand, h0, r)
    fb = t3.t3_gated_scan_bwd(gate, cand, first[0], dh, h0, r, dl)
    for _ in range(3):
        again = t3.t3_gated_scan_fwd(gate, cand, h0, r)
        ab = t3.t3_gated_scan_bwd(gate, cand, first[0], dh, h0, r, dl)
        for x, y in zip((*first, *fb), (*again, *ab)):
            assert torch.equal(x, y)


def test_empty_shapes():
    z = torch.zeros((2, 0, 6), device="cuda")
    h0 = torch.arange(12.0, device="cuda").view(2, 6)
    h, last = t3.t3_gated_scan_fwd(z, z, h0)
    assert h.shape == (2, 0, 6) and torch.equal(last, h0)
    assert torch.all(t3.t3_gated_scan_fwd(z, z)[1] == 0)
    assert torch.equal(t3.t3_gated_scan_bwd(z, z, z, z, h0, None, h0)[2], h0)
    assert torch.all(t3.t3_gated_scan_bwd(z, z, z, z)[2] == 0)
    e = torch.zeros((0, 5, 6), device="cuda")
    assert t3.t3_gated_scan_fwd(e, e)[0].shape == (0, 5, 6)


def test_binding_refusals():
    x = torch.zeros((2, 4, 16), device="cuda")
    with pytest.raises(ValueError):
        t3.t3_gated_scan_fwd(x, x[..., :8])
    with pytest.raises(TypeError):
        t3.t3_gated_scan_fwd(x, x.bfloat16())
    with pytest.raises(ValueError):
        t3.t3_gated_scan_fwd(x, x, torch.zeros((2, 15), device="cuda"))
    with pytest.raises(TypeError):
        t3.t3_gated_scan_fwd(x, x, None, torch.zeros((2, 4), device="cuda"))
    with pytest.raises(ValueError):
        t3.t3_gated_scan_fwd(x.transpose(0, 1), x.transpose(0, 1))
    with pytest.raises(ValueError):
        t3.t3_gated_scan_bwd(x, x, x, x, dgate=x[:1].expand(2, 4, 16)[:, :1].expand(2, 4, 16))


def test_another_stream():
    gate, cand, h0, r, dh, dl = _make(6, 2, 500, 128, "bf16", resets=True)
    want = t3.t3_gated_scan_fwd(gate, cand, h0, r)
    wb = t3.t3_gated_scan_bwd(gate, cand, want[0], dh, h0, r, dl)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = t3.t3_gated_scan_fwd(gate, cand, h0, r, stream=st)
    gb = t3.t3_gated_scan_bwd(gate, cand, got[0], dh, h0, r, dl, stream=st)
    st.synchronize()
    for a, b in zip((*want, *wb), (*got, *gb)):
        assert torch.equal(a, b)
