"""GPU tests of linear attention whose states grow (log_decay above 0), on every kernel and in
both directions, against the 64-bit recurrence of tests/more_operators_ref.py."""
import math

import numpy as np
import pytest

import more_operators_ref as ref
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# 3 and 2 as floats round them (a step adds expm1 of them: 2 and 1), a slow growth, and heads that do not grow
GROWTH = [math.log(3.0), math.log(2.0), 0.05, 0.0, -0.3]


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, bound, dname):
    tol = bound + (ref.HALF_ULP[dname] + 2 * ref.U) * (np.abs(want) + bound) + 1e-30
    off = np.abs(_np(got) - want)
    assert np.all(off <= tol), np.max(off / tol)


def _check(batch, length, dk, dv, dname, log_decay, marks):
    heads = len(log_decay)
    g = torch.Generator(device="cuda")
    g.manual_seed(length + dk)

    def rand(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    q, k = (rand(batch, length, heads, dk, dtype=DT[dname]) for _ in range(2))
    v, do = (rand(batch, length, heads, dv, dtype=DT[dname]) for _ in range(2))
    ld = torch.tensor(log_decay, dtype=torch.float32, device="cuda")
    state, dlast = rand(batch, heads, dk, dv), rand(batch, heads, dk, dv)
    resets = None
    if marks:
        resets = torch.zeros((batch, length), dtype=torch.uint8, device="cuda")
        resets[:, length // 3] = 1
    rn = None if resets is None else resets.cpu().numpy()
    chunks = dname == "bf16" and length > 16 and dk % 8 == 0 and dv % 8 == 0
    o, last, eo, es = ref.linear_attend(_np(q), _np(k), _np(v), _np(ld), _np(state), rn, 0.5, chunks=chunks)
    got = t3.t3_linear_attn_fwd(q, k, v, ld, state, resets, 0.5)
    _close(got[0], o, eo, dname)
    _close(got[1], last, es, "f32")
    want = ref.linear_attend_bwd(_np(q), _np(k), _np(v), _np(ld), _np(do), _np(state), rn, 0.5, _np(dlast), chunks)
    got = t3.t3_linear_attn_bwd(q, k, v, ld, do, state, resets, 0.5, dlast)
    for x, n in zip(got, ("q", "k", "v", "state")):
        _close(x, *want[n], "f32" if n == "state" else dname)


@pytest.mark.parametrize("marks", [False, True])
@pytest.mark.parametrize("dname,batch,length,dk,dv", [
    ("bf16", 3, 1, 16, 8), ("f32", 3, 1, 16, 8), ("f32", 3, 1, 16, 7), ("bf16", 2, 2, 64, 64), ("f32", 2, 2, 64, 64),
    ("bf16", 2, 9, 27, 27), ("f32", 2, 9, 27, 27), ("bf16", 2, 16, 32, 40), ("bf16", 2, 20, 27, 40), ("f32", 1, 40, 64, 128),
    ("f32", 2, 60, 128, 32)])
def test_growing_states(dname, batch, length, dk, dv, marks):
    """Token by token, up to 3^60."""
    _check(batch, length, dk, dv, dname, GROWTH, marks)


@pytest.mark.parametrize("dname,length,dk,dv", [("bf16", 700, 64, 64), ("f32", 700, 64, 64), ("bf16", 1500, 40, 33),
                                                ("f32", 1500, 40, 33), ("bf16", 384, 128, 128)])
def test_growing_states_of_long_sequences(dname, length, dk, dv):
    """Whole chunks and ranges (a state in front of each), one sequence: up to e^60."""
    _check(1, length, dk, dv, dname, [60.0 / length, 1.0 / length, 0.0], False)


@pytest.mark.parametrize("marks", [False, True])
@pytest.mark.parametrize("batch,length,dk,dv", [(2, 17, 64, 64), (2, 24, 24, 40), (1, 40, 64, 128), (2, 60, 128, 32), (1, 60, 128, 128)])
def test_growing_states_by_chunks(batch, length, dk, dv, marks):
    """Sequences shorter than a chunk whose growth is a float: what the chunk's other rows would have grown to, 3^127, is none."""
    _check(batch, length, dk, dv, "bf16", GROWTH, marks)


@pytest.mark.parametrize("dname", ["bf16", "f32"])
def test_a_factor_of_any_value_is_a_factor(dname):
    """The floats next to log 3, where a step adds twice the state: the state after two tokens of
    zeros is 9 times what it was, by every float near."""
    near = np.float32(math.log(3.0))
    ld = torch.tensor([near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(2))], device="cuda")
    zeros = torch.zeros((2, 2, 3, 24), dtype=DT[dname], device="cuda")
    state = torch.ones((2, 3, 24, 24), device="cuda")
    _, last = t3.t3_linear_attn_fwd(zeros, zeros, zeros, ld, state)
    assert torch.all((last - 9).abs() <= 1e-4)
