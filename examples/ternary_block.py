"""A block of a language model whose matrix products are all ternary: layer norm,
query, key and value projections, linear attention with a decay for each head,
layer norm, output projection, and a gated feed-forward layer with its own
norm and the residual stream around both.  Runs a prefill, the same tokens one
by one from the state, and a few training steps:

  python examples/ternary_block.py

Everything on the GPU's hot path is a call of the library; torch holds the
memory, draws the data and updates the latent weights.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import torch
from ternary_mixer import EPS, TernaryLinear

import ternary_weight_int8_t3_gb300 as t3


class Norm:
    """Layer norm whose rows leave as int8 codes, one scale each."""

    def __init__(self, width):
        self.gamma = torch.ones(width, device="cuda")
        self.beta = torch.zeros(width, device="cuda")

    def forward(self, x, residual=None):
        """((codes, scales), what backward takes)."""
        q, s, mean, rstd, total = t3.t3_layernorm_quant(x, self.gamma, self.beta, residual, EPS)
        return (q, s), (total, mean, rstd)

    def backward(self, dy, saved, dsum=None):
        """(dx, [(parameter, gradient)])"""
        dbeta = torch.empty_like(self.beta)
        dx, dgamma, _ = t3.t3_layernorm_bwd(dy, *saved, self.gamma, dsum, dbeta=dbeta)
        return dx, [(self.gamma, dgamma), (self.beta, dbeta)]


class TernaryBlock:
    def __init__(self, width, heads, hidden, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.width, self.heads, self.dim = width, heads, width // heads
        self.scale = self.dim ** -0.5
        # memories of some four tokens to some five hundred
        self.log_decay = torch.log1p(-torch.exp2(-torch.linspace(2, 9, heads, device="cuda")))
        self.norm_in, self.norm_out, self.norm_ff = Norm(width), Norm(width), Norm(width)
        self.inp, self.out = TernaryLinear(width, 3 * width, gen), TernaryLinear(width, width, gen)
        self.gate, self.up = TernaryLinear(width, hidden, gen), TernaryLinear(width, hidden, gen)
        self.down = TernaryLinear(hidden, width, gen)

    def empty_state(self, batch):
        return torch.zeros((batch, self.heads, self.dim, self.dim), device="cuda")

    def _qkv(self, both, b, t):
        return (both[:, i * self.width:(i + 1) * self.width].view(b, t, self.heads, self.dim) for i in range(3))

    def forward(self, x, state=None, saved=None):
        """(y, state): x bf16 [batch][length][width], state float [batch][heads][dim][dim], advanced in place
        when given."""
        b, t, d = x.shape
        rows = x.view(b * t, d)
        n1, norm1 = self.norm_in.forward(rows)
        qkv = self.inp.forward(*n1)
        q, k, v = self._qkv(qkv, b, t)
        o, state = t3.t3_linear_attn_fwd(q, k, v, self.log_decay, state, None, self.scale, state_last=state)
        n2, norm2 = self.norm_out.forward(o.view(b * t, d))
        a = self.out.forward(*n2)
        n3, norm3 = self.norm_ff.forward(a, residual=rows)
        g, u = self.gate, self.up
        pre = [torch.empty((b * t, g.bias.numel()), dtype=x.dtype, device=x.device) for _ in range(2)] if saved is not None else [None] * 2
        h = t3.t3_gemm_fwd_glu(n3[0], g.wp, u.wp, d, n3[1], g.col_scale, u.col_scale, g.bias, u.bias, t3.T3_ACT_SILU,
                               t3.T3_OUT_BF16, pre_gate=pre[0], pre_up=pre[1])
        y = self.down.forward(*t3.t3_quantize_rows_bf16(h), residual=norm3[0])
        if saved is not None:
            saved.update(n1=n1, norm1=norm1, qkv=qkv, o=o, n2=n2, norm2=norm2, a=a, n3=n3, norm3=norm3, pre=pre, h=h)
        return y.view(b, t, d), state

    def backward(self, dy, saved):
        """Gradients of everything that forward(..., saved=saved) used, from zero states: (dx,
        [(parameter, gradient)]); what lies between is left in `saved`."""
        b, t, d = dy.shape
        dy = dy.reshape(b * t, d)
        grads = []

        def through(linear, grad, x):
            dx, dlatent, dbias = linear.backward(grad, x)
            grads.extend([(linear.latent, dlatent), (linear.bias, dbias)])
            return dx
        values = lambda n: (n[0] * n[1][:, None]).to(torch.bfloat16)  # noqa: E731
        dh = through(self.down, dy, saved["h"])
        dgate, dup, _, _ = t3.t3_glu_bwd(dh, *saved["pre"], t3.T3_ACT_SILU)
        x3 = values(saved["n3"])
        dn3 = through(self.gate, dgate, x3) + through(self.up, dup, x3)
        da, norm = self.norm_ff.backward(dn3, saved["norm3"], dsum=dy)
        grads += norm
        dn2 = through(self.out, da, values(saved["n2"]))
        do, norm = self.norm_out.backward(dn2, saved["norm2"])
        grads += norm
        dqkv = torch.empty_like(saved["qkv"])
        dq, dk, dv = self._qkv(dqkv, b, t)
        t3.t3_linear_attn_bwd(*self._qkv(saved["qkv"], b, t), self.log_decay, do.view(b, t, self.heads, self.dim),
                              scale=self.scale, dq=dq, dk=dk, dv=dv)
        dn1 = through(self.inp, dqkv, values(saved["n1"]))
        dx, norm = self.norm_in.backward(dn1, saved["norm1"], dsum=da)
        grads += norm
        saved.update(dh=dh, dgate=dgate, dup=dup, dn3=dn3, da=da, dn2=dn2, do=do, dqkv=dqkv, dn1=dn1)
        return dx.view(b, t, d), grads

    def train_step(self, x, target, rate):
        """One step of gradient descent on the mean squared error; the loss."""
        saved = {}
        y, _ = self.forward(x, saved=saved)
        diff = y.float() - target.float()
        _, grads = self.backward((diff * (2 / diff.shape[-1])).to(torch.bfloat16), saved)
        for parameter, grad in grads:
            parameter -= rate / (diff.shape[0] * diff.shape[1]) * grad
        for linear in (self.inp, self.out, self.gate, self.up, self.down):
            linear.pack()
        return float(diff.square().mean())


def main(width=512, heads=8, hidden=1280, batch=2, length=300, steps=10):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    block = TernaryBlock(width, heads, hidden)
    x = torch.randn((batch, length, width), generator=gen, device="cuda").to(torch.bfloat16)
    y, state = block.forward(x, block.empty_state(batch))
    token_state = block.empty_state(batch)
    tokens = torch.cat([block.forward(x[:, t:t + 1].contiguous(), token_state)[0] for t in range(length)], 1)
    off = (tokens.float() - y.float()).square().mean().sqrt() / y.float().square().mean().sqrt()
    print(f"prefill of {batch} x {length} tokens against one by one: {float(off):.4f} of the output's rms apart")
    target = torch.roll(x, 3, 1)  # what came three tokens ago
    losses = [block.train_step(x, target, 0.5) for _ in range(steps)]
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    status, detail = t3.t3_last_device_error()
    assert status == t3.T3_OK, hex(detail)
    return y, tokens, losses


if __name__ == "__main__":
    main()
