"""GPU tests of where values that are not finite go in linear attention without resets: to the tokens
that the recurrence takes them to, and not in front of them, on every kernel."""
import pytest

import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN, INF = float("nan"), float("inf")

# chunks of all head sizes, whole and cut into ranges; blocks of tokens; few tokens
CASES = [("bf16", 1, 300, 64, 64), ("bf16", 1, 300, 128, 128), ("bf16", 2, 200, 128, 64), ("bf16", 1, 200, 40, 104),
         ("bf16", 1, 40, 64, 128), ("bf16", 1, 3000, 64, 64), ("bf16", 1, 200, 27, 27), ("bf16", 1, 14, 64, 64),
         ("f32", 1, 300, 64, 40), ("f32", 1, 1500, 33, 64), ("f32", 1, 5, 16, 16)]


def _problem(dname, batch, length, dk, dv):
    g = torch.Generator(device="cuda")
    g.manual_seed(length + dk + dv)
    heads = 3
    p = {n: torch.randn((batch, length, heads, d), generator=g, device="cuda").to(DT[dname])
         for n, d in (("q", dk), ("k", dk), ("v", dv), ("do", dv))}
    p["state"], p["dlast"] = (torch.randn((batch, heads, dk, dv), generator=g, device="cuda") for _ in range(2))
    # a decay whose power over a chunk is 0 in floats, one that forgets little, one that forgets all
    return p, torch.tensor([-1.0, -0.01, -INF], device="cuda")


def _run(p, ld, marks=None):
    o, last = t3.t3_linear_attn_fwd(p["q"], p["k"], p["v"], ld, p["state"], marks, 0.25)
    dq, dk, dv, ds = t3.t3_linear_attn_bwd(p["q"], p["k"], p["v"], ld, p["do"], p["state"], marks, 0.25, p["dlast"])
    rc, detail = t3.t3_last_device_error()
    assert rc == t3.T3_OK, hex(detail)
    return {"o": o, "last": last, "dq": dq, "dk": dk, "dv": dv, "ds": ds}


def _near(got, want, dname):
    """The same sums by another order and fewer roundings: P and the state rounded to bf16 or not (2^-8 of each term,
    whose magnitudes add up to some ten times the largest result), and the result's own rounding."""
    step = 2.0 ** -8 if dname == "bf16" else 2.0 ** -20
    assert torch.isfinite(got).all()
    if got.numel():
        assert (got.float() - want.float()).abs().max() <= 32 * step * want.float().abs().max()


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("dname,batch,length,dk,dv", CASES)
def test_no_value_reaches_the_tokens_in_front_of_it(dname, batch, length, dk, dv, value):
    p, ld = _problem(dname, batch, length, dk, dv)
    want = _run(p, ld)
    for at in sorted({1, length // 2, length - 1, min(length - 2, 129), max(length - 30, 1)}):
        for name in ("k", "v", "q"):
            bad = dict(p)
            bad[name] = p[name].clone()
            bad[name][0, at, :, 1] = value
            got = _run(bad, ld)
            # in time: o from q, k and v; dq from do, v and k
            for n in ("o", "dq"):
                _near(got[n][0, :at], want[n][0, :at], dname)
                if batch > 1:
                    assert torch.equal(got[n][1], want[n][1])
            if name == "q":
                _near(got["o"][0, at + 1:], want["o"][0, at + 1:], dname)
                # against time: dk and dv from q and do
                for n in ("dk", "dv"):
                    _near(got[n][0, at + 1:], want[n][0, at + 1:], dname)
            elif name == "v":  # one element of v: one column of the outputs
                assert not torch.isfinite(got["o"][0, at, :, 1]).any()
                rest = [c for c in range(dv) if c != 1]
                _near(got["o"][0, :, :, rest], want["o"][0, :, :, rest], dname)
            else:
                assert not torch.isfinite(got["o"][0, at:, 1]).any()
        bad = dict(p)
        bad["do"] = p["do"].clone()
        bad["do"][0, at, :, 1] = value
        got = _run(bad, ld)
        for n in ("dk", "dv"):
            _near(got[n][0, at + 1:], want[n][0, at + 1:], dname)


@pytest.mark.parametrize("dname,batch,length,dk,dv", CASES)
def test_nor_where_documents_meet(dname, batch, length, dk, dv):
    """Next to a reset, and in a sequence with resets elsewhere."""
    p, ld = _problem(dname, batch, length, dk, dv)
    begin = length // 3
    marks = torch.zeros((batch, length), dtype=torch.uint8, device="cuda")
    marks[:, begin] = 1
    want = _run(p, ld, marks)
    for at in sorted({begin, begin + 1, length - 1}):
        for name in ("k", "v", "do"):
            bad = dict(p)
            bad[name] = p[name].clone()
            bad[name][0, at, :, 1] = NAN
            got = _run(bad, ld, marks)
            if name == "do":
                for n in ("dk", "dv"):
                    _near(got[n][0, :begin], want[n][0, :begin], dname)
                    _near(got[n][0, at + 1:], want[n][0, at + 1:], dname)
            else:
                for n in ("o", "dq"):
                    _near(got[n][0, :at], want[n][0, :at], dname)


@pytest.mark.parametrize("dname,batch,length,dk,dv", CASES)
def test_a_state_that_is_not_finite_stays_so(dname, batch, length, dk, dv):
    """Zero times it is NaN: without a reset neither a decay of 0 nor one whose powers run out makes a
    state finite again, and one token, a block, a chunk and a range say the same."""
    p, ld = _problem(dname, batch, length, dk, dv)
    for value in (NAN, INF):
        bad = dict(p)
        bad["state"], bad["dlast"] = torch.full_like(p["state"], value), torch.full_like(p["dlast"], value)
        got = _run(bad, ld)
        for n in ("o", "last", "dq", "dk", "dv", "ds"):
            assert not torch.isfinite(got[n]).any(), n
    bad = dict(p)
    bad["k"] = p["k"].clone()
    bad["k"][0, 0, :, 1] = NAN
    got = _run(bad, ld)
    assert not torch.isfinite(got["last"][0, :, 1]).any()
    assert not torch.isfinite(got["o"][0]).any()


def test_one_token_says_the_same():
    p, ld = _problem("f32", 2, 1, 16, 16)
    for d in (16, 15):  # the single tokens' kernel and the blocks'
        q, k, v = p["q"], p["k"], p["v"][..., :d].contiguous()
        for value in (NAN, INF):
            o, last = t3.t3_linear_attn_fwd(q, k, v, ld, torch.full((2, 3, 16, d), value, device="cuda"))
            assert not torch.isfinite(o).any() and not torch.isfinite(last).any()
