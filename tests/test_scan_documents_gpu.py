"""GPU tests of documents packed into one sequence of the gated recurrence:
masked tokens in front of a reset, values that are not finite on the other side
of one, and the gradient that leaves the sequence.  The wanted values come from the
64-bit forms of tests/operators_ref.py on data whose masked and poisoned
entries are replaced by zeros: a document that is packed behind a reset does not
depend on them, so everything outside them has to agree."""
import numpy as np
import pytest

import operators_ref as ref
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF, NAN = float("inf"), float("nan")


def _np(t):
    return t.detach().double().cpu().numpy()


def _make(seed, b, t, d, dname):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    dt = DT[dname]
    return ((rand(b, t, d) * 1.7 + 1.5).to(dt), rand(b, t, d).to(dt), rand(b, d), rand(b, t, d).to(dt), rand(b, d))


def _resets(rng, b, t, every):
    r = rng.random((b, t)) < 1 / every
    return torch.from_numpy(r.astype(np.uint8)).cuda()


def _within(got, want, err, ulp, where, name):
    tol = ulp * np.abs(want) + err + 1e-30
    off = np.abs(_np(got) - want)
    bad = where & ~(off <= tol)  # NaN counts as off
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist())


# widths whose rows are whole 16-byte pieces, whole words and odd; lengths that end in a
# thread's loop, a lane's run, a warp, a CTA, a cluster and its next rounds; and more tiles than
# are resident at once
SHAPES = [(2, 7, 64), (3, 9, 64), (2, 40, 66), (3, 130, 63), (2, 300, 128), (1, 1300, 62), (1, 5000, 31), (20, 600, 1024)]


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("b,t,d", SHAPES)
def test_masked_tokens_in_front_of_a_reset(b, t, d, dname):
    """Padding at the end of a document: gate +inf and any candidate, 1 to 15
    tokens in front of the next one."""
    gate, cand, h0, dh, dl = _make(b + t + d, b, t, d, dname)
    rng = np.random.default_rng(t)
    r = _resets(rng, b, t, 21)
    mask = np.zeros((b, t), bool)
    for s, at in np.argwhere(_np(r) != 0):
        for back in rng.integers(1, 16, 3):
            if at - back >= 0:
                mask[s, at - back] = True
    m = torch.from_numpy(mask).cuda()
    fill = torch.tensor([NAN, INF, -INF, 3e38], device="cuda").to(DT[dname])
    gate[m] = INF
    dirty = cand.clone()
    dirty[m] = fill[torch.arange(d, device="cuda") % 4].expand(int(mask.sum()), d)
    cand[m] = 0
    h, last = t3.t3_gated_scan_fwd(gate, dirty, h0, r)
    want, prior, err = ref.scan(_np(gate), _np(cand), _np(h0), _np(r))
    everywhere = np.ones((b, t, d), bool)
    _within(h, want, err, ref.HALF_ULP[dname], everywhere, "h")
    _within(last, want[:, -1], err[:, -1], ref.U, everywhere[:, 0], "h_last")
    # what the masked candidates hold changes no bit of either direction
    clean = t3.t3_gated_scan_fwd(gate, cand, h0, r)
    assert torch.equal(h, clean[0]) and torch.equal(last, clean[1])
    got = t3.t3_gated_scan_bwd(gate, dirty, h, dh, h0, r, dl)
    for x, y in zip(got, t3.t3_gated_scan_bwd(gate, cand, h, dh, h0, r, dl)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("t", [6, 9, 40, 300, 1300])
def test_masked_tokens_keep_a_large_state(t, dname):
    """A masked candidate at the other end of the float range, however large the state."""
    gate, cand, h0, _, _ = _make(t, 2, t, 64, dname)
    h0 = torch.full_like(h0, 2e38)
    gate[:], cand[:] = INF, -3e38
    h, last = t3.t3_gated_scan_fwd(gate, cand, h0)
    assert torch.equal(last, h0) and torch.equal(h, h0.to(DT[dname])[:, None].expand_as(h))


def _documents(r):
    """The document's number of each token."""
    return np.cumsum(_np(r) != 0, 1)


def _poison(rng, r):
    """One token in every third document of each sequence, as (sequence, token, document)."""
    docs, out = _documents(r), []
    for s in range(docs.shape[0]):
        for k in np.unique(docs[s]):
            if rng.random() < 0.4:
                out.append((s, int(rng.choice(np.flatnonzero(docs[s] == k))), k))
    return docs, out


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("b,t,d", SHAPES)
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_reset_stops_a_state_that_is_not_finite(value, b, t, d, dname):
    gate, cand, h0, _, _ = _make(b * t + d, b, t, d, dname)
    rng = np.random.default_rng(t + d)
    r = _resets(rng, b, t, 30)
    r[:, 0] = 1  # h0 may be anything, too
    r[-1, t - 1] = 1
    docs, bad = _poison(rng, r)
    dirty, h0d = cand.clone(), h0.clone()
    h0d[:, ::2] = value
    fine = np.ones((b, t, d), bool)
    for s, at, k in bad:
        dirty[s, at, ::3] = value
        end = at + int((docs[s, at:] == k).sum())
        fine[s, at:end, ::3] = False
    h, last = t3.t3_gated_scan_fwd(gate, dirty, h0d, r)
    want, _, err = ref.scan(_np(gate), _np(cand), _np(h0), _np(r))
    _within(h, want, err, ref.HALF_ULP[dname], fine, "h")
    _within(last, want[:, -1], err[:, -1], ref.U, fine[:, -1], "h_last")
    for s, at, k in bad:  # and it shows in its own document
        assert not torch.isfinite(h[s, at, ::3]).any()


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("b,t,d", SHAPES)
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_reset_stops_a_gradient_that_is_not_finite(value, b, t, d, dname):
    gate, cand, h0, dh, dl = _make(b * t + d, b, t, d, dname)
    rng = np.random.default_rng(t + d + 1)
    r = _resets(rng, b, t, 30)
    r[-1, t - 1] = 1
    r[0, 0] = 1
    docs, bad = _poison(rng, r)
    h, _ = t3.t3_gated_scan_fwd(gate, cand, h0, r)
    dirty, dld = dh.clone(), dl.clone()
    fine = np.ones((b, t, d), bool)
    for s, at, k in bad:
        dirty[s, at, ::3] = value
        fine[s, at + 1 - int((docs[s, :at + 1] == k).sum()):at + 1, ::3] = False
    dld[-1, 1::3] = value  # a last document of one token
    fine[-1, t - 1, 1::3] = False
    got = t3.t3_gated_scan_bwd(gate, cand, h, dirty, h0, r, dld)
    rs = _np(r)
    prior = np.concatenate([_np(h0)[:, None], _np(h)[:, :-1]], 1) * (rs == 0)[..., None]
    want, err = ref.scan_bwd(_np(gate), _np(cand), prior, _np(dh), rs, _np(dl))
    for name, x, w, e in zip(("dgate", "dcand"), got, want, err):
        _within(x, w, e, ref.HALF_ULP[dname], fine, name)
    first = fine[:, 0] | (rs[:, :1] != 0)
    _within(got[2], want[2], err[2], ref.U, first, "dh0")
    assert torch.all(got[2][0] == 0)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("t", [1, 5, 9, 40, 300, 1300])
@pytest.mark.parametrize("mean", [-8.0, -12.0, -20.0, 0.0, 9.0])
def test_the_gradient_of_h0_keeps_its_relative_precision(mean, t, dname):
    """dh0 = a_0 G_0 with a_0 far below 1: a_0's own relative error (the
    logistic function's), two roundings, and a_0 times the error of G_0."""
    gate, cand, h0, dh, dl = _make(t, 2, t, 66, dname)
    gate = (gate * 0.1 + mean).to(DT[dname])
    h, _ = t3.t3_gated_scan_fwd(gate, cand, h0)
    got = t3.t3_gated_scan_bwd(gate, cand, h, dh, h0, None, dl)[2]
    g, e = _np(dl), np.zeros((2, 66))
    gt, dn = _np(gate), _np(dh)
    for i in reversed(range(t)):
        e = e + 3 * ref.U * (np.abs(g) + np.abs(dn[:, i]))
        g = g + dn[:, i]
        a, kerr = ref.sigmoid(gt[:, i]), ref.logistic_error(gt[:, i])
        if i == 0:
            e = a * (e + (kerr + 4 * ref.U) * np.abs(g))
        else:
            e = a * e + 3 * (kerr * (1 - a) + ref.U) * np.abs(g)
        g = a * g
    _within(got, g, e, ref.U, np.ones((2, 66), bool), "dh0")


def test_resets_from_a_comparison():
    """resets as torch makes them: bool, the same bytes as uint8."""
    gate, cand, h0, dh, dl = _make(4, 2, 60, 64, "bf16")
    ids = torch.arange(60, device="cuda").expand(2, 60) // 13
    marks = ids != torch.roll(ids, 1, 1)
    r = marks.to(torch.uint8)
    got, want = t3.t3_gated_scan_fwd(gate, cand, h0, marks), t3.t3_gated_scan_fwd(gate, cand, h0, r)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    got = t3.t3_gated_scan_bwd(gate, cand, want[0], dh, h0, marks, dl)
    assert all(torch.equal(x, y) for x, y in zip(got, t3.t3_gated_scan_bwd(gate, cand, want[0], dh, h0, r, dl)))
    with pytest.raises(ValueError):
        t3.t3_gated_scan_fwd(gate, cand, h0, marks[:, :-1])
