"""GPU tests of the layer norm's moments on rows far from zero: rows of equal elements, and bounds
that a mean or a deviation taken in one pass does not meet."""
import numpy as np
import pytest

import more_operators_ref as ref
import moments_ref
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def _np(t):
    return t.detach().double().cpu().numpy()


def _rows(rows, cols, dtype, lead):
    """Rows `lead` elements past an aligned base: 0 and cols a multiple of 8 for the vector kernels, 1 or odd
    widths for those whose vectors begin inside a row."""
    return torch.zeros(rows * cols + 16, dtype=dtype, device="cuda")[lead:lead + rows * cols].view(rows, cols)


# one warp, several, several vectors a thread, vectors that begin inside a row, element by element
WIDTHS = [(8, 0), (40, 0), (64, 0), (729, 0), (1000, 0), (1000, 1), (1280, 0), (3456, 0), (3457, 1), (8192, 0), (8200, 0),
          (12288, 0), (16392, 0), (40001, 0)]


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("cols,lead", WIDTHS)
def test_rows_of_equal_elements_have_no_deviation(cols, lead, dname):
    values = torch.tensor([-30000.0, 0.1, 3.3, 1e-3, 12345.678, -1.0, 7e4, 1.0 / 3.0], device="cuda").to(DT[dname])
    x = _rows(8, cols, DT[dname], lead)
    x.copy_(values[:, None].expand(8, cols))
    q, scale, mean, rstd, _ = t3.t3_layernorm_quant(x, eps=EPS)
    assert torch.equal(mean, values.float())
    assert torch.all(q == 0) and torch.all(scale == 0)
    assert np.all(np.abs(_np(rstd) * np.sqrt(np.float64(np.float32(EPS))) - 1) <= 8 * ref.U)
    # a shift alone: its codes whatever the row holds
    beta = torch.linspace(-1, 1, cols, device="cuda")
    q, scale, _, _, _ = t3.t3_layernorm_quant(x, beta=beta, eps=EPS)
    assert torch.equal(q, q[:1].expand(8, cols)) and torch.all((scale * 127 - 1).abs() <= 1e-6)


@pytest.mark.parametrize("mean", [100.0, -3e4])
@pytest.mark.parametrize("cols,lead", [(64, 0), (729, 0), (1000, 1), (4096, 0), (8200, 0), (12292, 0), (20000, 0), (33001, 0)])
def test_moments_far_from_zero(cols, lead, mean):
    x = _rows(40, cols, torch.float32, lead)
    x.copy_(torch.from_numpy(moments_ref.rows(40, cols, mean)))
    q, scale, m, rstd, _ = t3.t3_layernorm_quant(x, eps=EPS)
    moments_ref.check(x.cpu().numpy(), EPS, _np(m), _np(rstd), _np(scale), q.cpu().numpy())
