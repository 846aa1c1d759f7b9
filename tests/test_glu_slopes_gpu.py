"""GPU tests of the gated product's gradient for every activation, vectors and single elements, with
gates at exactly 0, where the slopes of relu and its square are 0."""
import pytest

import more_operators_ref as ref
import ternary_weight_int8_t3_gb300 as t3
from test_glu_gpu import DT, _check_backward

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dname", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,lead", [(1, 8, 0), (40, 96, 0), (700, 1280, 0), (3, 5, 0), (333, 243, 0), (50, 64, 1)])
@pytest.mark.parametrize("act", ref.ACTS)
def test_slopes_and_sums(act, rows, cols, lead, dname):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + cols)

    def rand(std):
        flat = torch.randn(rows * cols + 8, generator=g, device="cuda").mul_(std).to(DT[dname])
        return flat[lead:lead + rows * cols].view(rows, cols)

    dy, gate, up = rand(1), rand(4), rand(2)
    gate.view(-1)[::3] = 0.0
    gate.view(-1)[1::6] = -0.0
    sums = [torch.empty(cols, device="cuda") for _ in range(2)]
    got = t3.t3_glu_bwd(dy, gate, up, ref.ACTS.index(act), dgate_bias=sums[0], dup_bias=sums[1])
    _check_backward(dy, gate, up, act, got, dname)
    if act in ("relu", "relu2"):
        assert torch.all(got[0][gate == 0] == 0) and torch.all(got[1][gate == 0] == 0)
