"""GPU tests of t3_rmsnorm_quant on rows so small that 127 / max|u| passes the
float range: the codes still stand for the rows, as at any other size."""
import numpy as np
import pytest

import operators_ref as ref
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [1e-30, 1e-36, 3e-37, 1e-37, 1e-38, 1e-39, 1e-40]


# 16-byte rows, odd rows alike, element by element (a stride that differs from the codes'), beyond the registers
@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("cols,pad", [(40, 0), (2048, 0), (8191, 0), (243, 0), (243, 5), (40008, 0)])
def test_rows_near_the_bottom_of_the_float_range(cols, pad, dname):
    g = torch.Generator(device="cuda")
    g.manual_seed(cols)
    n = len(SIZES)
    x = torch.zeros((n, cols + pad), dtype=DT[dname], device="cuda")[:, :cols]
    x.copy_(torch.randn((n, cols), generator=g, device="cuda").double() * torch.tensor(SIZES, device="cuda").double()[:, None])
    gamma = 1 + 0.3 * torch.rand(cols, generator=g, device="cuda")
    for gain in (None, gamma):
        q, scale, rstd, _ = t3.t3_rmsnorm_quant(x, gain)
        # u = s * gamma as a float product; 2^64 times it and its largest, which changes neither
        # the quotients nor (as the factor is a power of two) their rounding
        s = x.float().cpu().numpy()
        u = s * (np.ones(cols, np.float32) if gain is None else gain.cpu().numpy())
        big = (u.astype(np.float64) * 2.0 ** 64).astype(np.float32)
        inv = np.float32(127) / np.abs(big).max(1)
        np.testing.assert_array_equal(q.cpu().numpy(), np.rint(big * inv[:, None]).astype(np.int8))
        want = np.abs(u.astype(np.float64)).max(1) / 127 / np.sqrt(1e-5)
        # the scale: four float roundings, in units of the last place down to the smallest float
        assert np.all(np.abs(scale.double().cpu().numpy() - want) <= 8 * ref.U * want + 2.0 ** -148 * (1 + 1 / np.sqrt(1e-5)))
