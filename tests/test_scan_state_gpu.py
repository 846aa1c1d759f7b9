"""GPU tests of the recurrence's gradient against that of the float state: the
backward takes h' from the forward's stored rows, whose rounding shows in
h' - c and nowhere else."""
import numpy as np
import pytest

import operators_ref as ref
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("b,t,d", [(3, 1, 64), (2, 9, 66), (2, 300, 128), (1, 1300, 63)])
@pytest.mark.parametrize("mean", [1.5, 6.0])
def test_gradient_of_the_float_state(mean, b, t, d, dname):
    """dgate = G (h' - c) a (1 - a): besides the bound of a float computation on
    the state itself, half a unit of the stored type in h' (the forward's own
    error with it) times |G| a (1 - a).  dcand and dh0 do not depend on h.
    mean 6: states that move by a four-hundredth a token, near their candidates' mean."""
    g = torch.Generator(device="cuda")
    g.manual_seed(b + t + d)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    dt = DT[dname]
    gate, cand = (rand(b, t, d) + mean).to(dt), (0.05 * rand(b, t, d) + 1).to(dt)
    h0, dh, dl = 1 + 0.05 * rand(b, d), rand(b, t, d).to(dt), rand(b, d)
    h, _ = t3.t3_gated_scan_fwd(gate, cand, h0)
    got = t3.t3_gated_scan_bwd(gate, cand, h, dh, h0, None, dl)
    none = np.zeros((b, t))
    _, prior, herr = ref.scan(_np(gate), _np(cand), _np(h0), none)
    want, err = ref.scan_bwd(_np(gate), _np(cand), prior, _np(dh), none, _np(dl))
    a, k = ref.sigmoid(_np(gate)), ref.sigmoid(-_np(gate))
    total = np.abs(want[1]) / k + err[1] / k  # |G| and its error, through dcand = k G
    stored = ref.HALF_ULP[dname] * np.abs(prior) + np.concatenate([np.zeros((b, 1, d)), herr[:, :-1]], 1)
    stored[:, 0] = 0  # h0 is float
    for name, x, w, e, ulp in (("dgate", got[0], want[0], err[0] + a * k * total * stored, ref.HALF_ULP[dname]),
                               ("dcand", got[1], want[1], err[1], ref.HALF_ULP[dname]),
                               ("dh0", got[2], want[2], err[2], ref.U)):
        off, tol = np.abs(_np(x) - w), ulp * np.abs(w) + e + 1e-30
        assert np.all(off <= tol), (name, np.max(off / tol))
