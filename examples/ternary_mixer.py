"""A token mixer whose matrix products are all ternary: norm, gate and candidate
projection, gated recurrence over time, norm, output projection with the
residual in its epilogue.  Runs a prefill, the same tokens one by one, and a few
training steps:

  python examples/ternary_mixer.py

Everything on the GPU's hot path is a call of the library; torch holds the
memory, draws the data and updates the latent weights.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import ternary_weight_int8_t3_gb300 as t3

EPS = 1e-5


class TernaryLinear:
    """Latent float weights [K][N], used as ternary codes and one scale: w =
    scale * clamp(round(latent / scale), -1, 1) with scale = mean |latent|, gradients
    passed straight through."""

    def __init__(self, k, n, gen):
        self.latent = torch.randn((k, n), generator=gen, device="cuda") / k ** 0.5
        self.bias = torch.zeros(n, device="cuda")
        self.pack()

    def pack(self):
        self.scale = self.latent.abs().mean()
        codes = (self.latent / self.scale).round_().clamp_(-1, 1).to(torch.int8)
        self.wp = t3.t3_pack_ternary_device(codes)
        self.col_scale = self.scale.expand(self.latent.shape[1]).contiguous()

    def forward(self, q, row_scale, residual=None):
        return t3.t3_gemm_fwd_act(q, self.wp, K=self.latent.shape[0], row_scale=row_scale, col_scale=self.col_scale,
                                  bias=self.bias, residual=residual, kind=t3.T3_OUT_BF16)

    def backward(self, dy, x):
        """(dx, dlatent, dbias) for dy [M][N] and the product's input x [M][K]
        (its values, bf16): dy is quantized by rows for dx, and both by columns
        for the weights, where the scales have to leave the sum over rows."""
        dbias = torch.empty_like(self.bias)
        t3.t3_act_bwd(dy, None, t3.T3_ACT_NONE, dz=torch.empty_like(dy), dbias=dbias)
        q, s = t3.t3_quantize_rows_bf16(dy)
        dx = t3.t3_gemm_bwd_dx_scaled(q, self.wp, self.latent.shape[0], row_scale=s * self.scale,
                                      kind=t3.T3_OUT_BF16, workspace=torch.empty(x.shape, dtype=torch.int32, device="cuda"))
        (qx, sx), (qy, sy) = (t3.t3_quantize_rows_bf16(v.t().contiguous()) for v in (x, dy))
        dlatent = t3.t3_gemm_bwd_dw_scaled(qx.t().contiguous(), qy.t().contiguous(), row_scale=sx, col_scale=sy)
        return dx, dlatent, dbias


class TernaryMixer:
    def __init__(self, width, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.width = width
        self.gamma_in = torch.ones(width, device="cuda")
        self.gamma_out = torch.ones(width, device="cuda")
        self.inp = TernaryLinear(width, 2 * width, gen)   # gate logits | candidates
        self.inp.bias[:width] = 2.0                       # start with a memory of some ten tokens
        self.out = TernaryLinear(width, width, gen)

    def forward(self, x, state=None, saved=None):
        """(y, state): x bf16 [batch][length][width], state float [batch][width],
        advanced in place when given."""
        b, t, d = x.shape
        rows = x.view(b * t, d)
        q, s, rstd, _ = t3.t3_rmsnorm_quant(rows, self.gamma_in, eps=EPS)
        both = self.inp.forward(q, s).view(b, t, 2 * d)
        gate, cand = both[..., :d], both[..., d:]
        h, state = t3.t3_gated_scan_fwd(gate, cand, state, h_last=state)
        q2, s2, rstd2, _ = t3.t3_rmsnorm_quant(h.view(b * t, d), self.gamma_out, eps=EPS)
        y = self.out.forward(q2, s2, residual=rows)
        if saved is not None:
            saved.update(rows=rows, q=q, s=s, rstd=rstd, gate=gate, cand=cand, h=h, q2=q2, s2=s2, rstd2=rstd2)
        return y.view(b, t, d), state

    def backward(self, dy, saved):
        """Gradients of everything that forward(..., saved=saved) used: (dx,
        [(parameter, gradient)])."""
        b, t, d = dy.shape
        dy = dy.reshape(b * t, d)
        values = lambda q, s: (q * s[:, None]).to(torch.bfloat16)  # noqa: E731
        dn2, dw_out, db_out = self.out.backward(dy, values(saved["q2"], saved["s2"]))
        dh, dgamma_out = t3.t3_rmsnorm_bwd(dn2, saved["h"].view(b * t, d), saved["rstd2"], self.gamma_out)
        dboth = torch.empty((b, t, 2 * d), dtype=torch.bfloat16, device="cuda")
        t3.t3_gated_scan_bwd(saved["gate"], saved["cand"], saved["h"], dh.view(b, t, d),
                             dgate=dboth[..., :d], dcand=dboth[..., d:])
        dn1, dw_in, db_in = self.inp.backward(dboth.view(b * t, 2 * d), values(saved["q"], saved["s"]))
        dx, dgamma_in = t3.t3_rmsnorm_bwd(dn1, saved["rows"], saved["rstd"], self.gamma_in, dsum=dy)
        grads = [(self.out.latent, dw_out), (self.out.bias, db_out), (self.gamma_out, dgamma_out),
                 (self.inp.latent, dw_in), (self.inp.bias, db_in), (self.gamma_in, dgamma_in)]
        return dx.view(b, t, d), grads

    def train_step(self, x, target, rate):
        """One step of gradient descent on the mean squared error; the loss."""
        saved = {}
        y, _ = self.forward(x, saved=saved)
        diff = y.float() - target.float()
        _, grads = self.backward((diff * (2 / diff.shape[-1])).to(torch.bfloat16), saved)
        for parameter, grad in grads:
            parameter -= rate / (diff.shape[0] * diff.shape[1]) * grad
        self.inp.pack()
        self.out.pack()
        return float(diff.square().mean())


def main(width=512, batch=2, length=300, steps=20):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    mixer = TernaryMixer(width)
    x = torch.randn((batch, length, width), generator=gen, device="cuda").to(torch.bfloat16)
    y, state = mixer.forward(x, torch.zeros((batch, width), device="cuda"))
    token_state = torch.zeros((batch, width), device="cuda")
    tokens = [mixer.forward(x[:, t:t + 1].contiguous(), token_state)[0] for t in range(length)]
    off = (torch.cat(tokens, 1).float() - y.float()).abs().max() / y.float().square().mean().sqrt()
    print(f"prefill of {batch} x {length} tokens against one by one: largest difference {float(off):.4f} of the output's rms")
    target = torch.roll(x, 3, 1)  # what came three tokens ago
    losses = [mixer.train_step(x, target, 0.5) for _ in range(steps)]
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    status, detail = t3.t3_last_device_error()
    assert status == t3.T3_OK, hex(detail)
    return float(off), losses, (state - token_state).abs().max()


if __name__ == "__main__":
    main()
