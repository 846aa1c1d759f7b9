"""Layer norm, linear attention and the gated feed-forward product together, as a
language model's block uses them: the example's forward, single tokens and gradient, each step
against its 64-bit form on what the step before left; and the calls in a row, allocating nothing, in a
captured graph and from two host threads on two streams."""
import importlib.util
import os
import threading

import numpy as np
import pytest

import more_operators_ref as ref
import oracle
import t3_synth
import ternary_weight_int8_t3_gb300 as t3

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("ternary_block", os.path.join(ROOT, "examples", "ternary_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(got, want, bound):
    """Within a bound before the rounding to bf16, and that rounding."""
    off, tol = np.abs(_np(got) - want), bound + (ref.HALF_ULP["bf16"] + 2 * ref.U) * (np.abs(want) + bound) + 1e-30
    assert np.all(off <= tol), np.max(off / tol)


def _check_norm(norm, codes, saved, eps):
    total, mean, rstd = saved
    wm, wr, ws, y, (em, er, es, ey) = ref.layer_norm(_np(total), _np(norm.gamma), _np(norm.beta), np.float64(np.float32(eps)))
    assert np.all(np.abs(_np(mean) - wm) <= em + ref.U * np.abs(wm)) and np.all(np.abs(_np(rstd) - wr) <= er * wr)
    q, s = _np(codes[0]), _np(codes[1])
    assert np.all(np.abs(s - ws) <= es)
    assert np.all(np.abs(q * ws[:, None] - y) <= ws[:, None] * (0.5 + 127 * 6 * ref.U) + ey + 127 * es[:, None])


def _check_norm_bwd(norm, dy, saved, dsum, got):
    """The roundings of a row's sums: n + 16 float terms and some factors of them; the columns' likewise."""
    total, mean, rstd = (_np(t) for t in saved)
    dsum = 0.0 if dsum is None else _np(dsum)
    dx, dg, db, mag, mg, mb = ref.layer_norm_bwd(_np(dy), total, mean, rstd, _np(norm.gamma), dsum)
    rows, n = total.shape
    _near(got[0], dx, (n + 32) * ref.U * mag)
    assert np.all(np.abs(_np(got[1]) - dg) <= (rows + 32) * ref.U * mg + 1e-30)
    assert np.all(np.abs(_np(got[2]) - db) <= (rows + 32) * ref.U * mb + 1e-30)


def _attend(block, qkv, b, t, state=None, chunks=False):
    q, k, v = (_np(x) for x in block._qkv(qkv, b, t))
    return ref.linear_attend(q, k, v, _np(block.log_decay), state, None, float(np.float32(block.scale)), chunks=chunks)


# (batch, length, width, heads, hidden): chunks on the tensor cores with heads of 64, one
# of them cut; odd heads, token by token
SIZES = [(2, 300, 512, 8, 1280), (3, 40, 243, 9, 729)]


@pytest.mark.parametrize("b,t,width,heads,hidden", SIZES)
def test_a_block_step_by_step(example, b, t, width, heads, hidden):
    block = example.TernaryBlock(width, heads, hidden, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    for n in (block.norm_in, block.norm_out, block.norm_ff):
        n.gamma += 0.2 * torch.randn(width, generator=g, device="cuda")
        n.beta += 0.2 * torch.randn(width, generator=g, device="cuda")
    chunks = block.dim % 8 == 0
    x = torch.randn((b, t, width), generator=g, device="cuda").to(BF)
    dy = torch.randn((b, t, width), generator=g, device="cuda").to(BF)
    saved = {}
    y, state = block.forward(x, saved=saved)
    _check_norm(block.norm_in, saved["n1"], saved["norm1"], example.EPS)
    o, last, eo, es = _attend(block, saved["qkv"], b, t, chunks=chunks)
    _near(saved["o"], o, eo)
    assert np.all(np.abs(_np(state) - last) <= es)
    _check_norm(block.norm_out, saved["n2"], saved["norm2"], example.EPS)
    assert torch.equal(saved["norm3"][0], (saved["a"].float() + x.view(b * t, width).float()).to(BF))
    _check_norm(block.norm_ff, saved["n3"], saved["norm3"], example.EPS)
    codes, scales = saved["n3"]
    z = []
    for linear, pre in ((block.gate, saved["pre"][0]), (block.up, saved["pre"][1])):
        ternary = (linear.latent / linear.scale).round().clamp(-1, 1).cpu().numpy().astype(np.int64)
        exact = codes.cpu().numpy().astype(np.int64) @ ternary
        z.append(ref.glu_z(exact, scales.cpu().numpy(), linear.col_scale.cpu().numpy(), linear.bias.cpu().numpy()))
        assert torch.equal(pre.cpu(), torch.from_numpy(z[-1]).to(BF))
    gated, _, eg, _ = ref.act(z[0].astype(np.float64), "silu")
    _near(saved["h"], gated * z[1], eg * np.abs(z[1]) + 2 * ref.U * np.abs(gated * z[1]))

    dx, grads = block.backward(dy, saved)
    grad_of = {id(p): v for p, v in grads}
    of = lambda n: (grad_of[id(n.gamma)], grad_of[id(n.beta)])  # noqa: E731
    dgate, dup, eg, eu = ref.glu_bwd(_np(saved["dh"]), _np(saved["pre"][0]), _np(saved["pre"][1]), "silu")
    _near(saved["dgate"], dgate, eg)
    _near(saved["dup"], dup, eu)
    _check_norm_bwd(block.norm_ff, saved["dn3"], saved["norm3"], dy.view(b * t, width), (saved["da"], *of(block.norm_ff)))
    _check_norm_bwd(block.norm_out, saved["dn2"], saved["norm2"], None, (saved["do"], *of(block.norm_out)))
    q, k, v = (_np(a) for a in block._qkv(saved["qkv"], b, t))
    want = ref.linear_attend_bwd(q, k, v, _np(block.log_decay), _np(saved["do"]).reshape(v.shape), None, None,
                                 float(np.float32(block.scale)), None, chunks)
    for name, got in zip("qkv", block._qkv(saved["dqkv"], b, t)):
        _near(got, *want[name])
    _check_norm_bwd(block.norm_in, saved["dn1"], saved["norm1"], saved["da"], (dx.view(b * t, width), *of(block.norm_in)))


@pytest.mark.parametrize("b,t,width,heads,hidden", SIZES)
def test_tokens_from_a_prefills_state(example, b, t, width, heads, hidden):
    """A prefill's state, advanced in place by single tokens, is the recurrence's over all of them: each from the
    queries, keys and values that its call made."""
    block = example.TernaryBlock(width, heads, hidden, seed=7)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    x = torch.randn((b, t + 3, width), generator=g, device="cuda").to(BF)
    state, seen, outs = block.empty_state(b), [], []
    for part in (x[:, :t], x[:, t:t + 1], x[:, t + 1:t + 2], x[:, t + 2:]):
        saved = {}
        y, last = block.forward(part.contiguous(), state, saved)
        assert last is state and torch.isfinite(y).all()
        seen.append(saved["qkv"].view(b, part.shape[1], 3 * width))
        outs.append(saved["o"].view(b, part.shape[1], heads, block.dim))
    qkv = torch.cat(seen, 1).reshape(b * (t + 3), 3 * width)
    o, last, eo, es = _attend(block, qkv, b, t + 3, chunks=block.dim % 8 == 0)
    _near(torch.cat(outs, 1), o, eo)
    assert np.all(np.abs(_np(state) - last) <= es)


def test_the_example_runs(example):
    y, tokens, losses = example.main(width=256, heads=4, hidden=640, length=50, steps=3)
    assert y.shape == tokens.shape and torch.isfinite(y).all() and torch.isfinite(tokens).all()
    assert len(losses) == 3 and all(np.isfinite(losses))


# ------------------------------------------------------- the calls in a row ---

def _calls(seed, b, length, heads, dim, hidden):
    """Buffers of a block's forward and gradient, and the calls in order; every output and workspace is here already."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows, d = b * length, heads * dim

    def rand(*shape, dtype=BF):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    def room(*shape, dtype=BF):
        return torch.zeros(shape, dtype=dtype, device="cuda")
    rng = t3_synth.rng(seed)
    wqkv, wg, wu = (torch.from_numpy(oracle.pack(t3_synth.ternary(rng, (d, n)))).cuda() for n in (3 * d, hidden, hidden))
    x, res, gamma, beta, dy = rand(rows, d), rand(rows, d), 1 + 0.1 * rand(d, dtype=F32), 0.1 * rand(d, dtype=F32), rand(rows, hidden)
    codes, s, total = room(rows, d, dtype=torch.int8), room(rows, dtype=F32), room(rows, d)
    mean, rstd, mean2, rstd2 = (room(rows, dtype=F32) for _ in range(4))
    both, cs = room(rows, 3 * d), torch.full((3 * d,), 0.02, device="cuda")
    view = [both[:, i * d:(i + 1) * d].view(b, length, heads, dim) for i in range(3)]
    ld = torch.log1p(-torch.exp2(-torch.linspace(1, 8, heads, device="cuda")))
    h0, last, dh0 = rand(b, heads, dim, dim, dtype=F32), room(b, heads, dim, dim, dtype=F32), room(b, heads, dim, dim, dtype=F32)
    resets = (torch.rand((b, length), generator=g, device="cuda") < 0.02).to(torch.uint8)
    o, codes2, s2 = room(b, length, heads, dim), room(rows, d, dtype=torch.int8), room(rows, dtype=F32)
    out, pg, pu, dg, du = (room(rows, hidden) for _ in range(5))
    dgb, dub, cg = room(hidden, dtype=F32), room(hidden, dtype=F32), torch.full((hidden,), 0.02, device="cuda")
    do, dboth, dx, dgamma, dbeta = rand(b, length, heads, dim), room(rows, 3 * d), room(rows, d), room(d, dtype=F32), room(d, dtype=F32)
    dview = [dboth[:, i * d:(i + 1) * d].view(b, length, heads, dim) for i in range(3)]
    lib = t3.load()
    attn = room(max(1, lib.t3_linear_attn_workspace(b, length, heads, dim, dim)), dtype=F32)
    glu = room(1 << 26, dtype=torch.uint8)
    sums = room(lib.t3_colsum_workspace(rows, max(2 * hidden, 2 * d)), dtype=F32)
    ws = room(rows, 3 * d, dtype=torch.int32)
    scratch = room(max(lib.t3_gemm_fwd_act_scratch(rows, 3 * d, d), 16), dtype=torch.uint8)

    def run(stream=None):
        t3.t3_layernorm_quant(x, gamma, beta, res, q=codes, row_scale=s, mean=mean, rstd=rstd, sum_out=total, stream=stream)
        t3.t3_gemm_fwd_act(codes, wqkv, K=d, row_scale=s, col_scale=cs, kind=t3.T3_OUT_BF16, C=both, workspace=ws,
                           scratch=scratch, stream=stream)
        t3.t3_linear_attn_fwd(*view, ld, h0, resets, dim ** -0.5, o=o, state_last=last, workspace=attn, stream=stream)
        t3.t3_layernorm_quant(o.view(rows, d), gamma, beta, q=codes2, row_scale=s2, mean=mean2, rstd=rstd2, stream=stream)
        t3.t3_gemm_fwd_glu(codes2, wg, wu, d, s2, cg, cg, act=t3.T3_ACT_GELU, kind=t3.T3_OUT_BF16, C=out, pre_gate=pg,
                           pre_up=pu, workspace=glu, stream=stream)
        t3.t3_glu_bwd(dy, pg, pu, t3.T3_ACT_GELU, dgate=dg, dup=du, dgate_bias=dgb, dup_bias=dub, workspace=sums, stream=stream)
        t3.t3_linear_attn_bwd(*view, ld, do, h0, resets, dim ** -0.5, h0, dq=dview[0], dk=dview[1], dv=dview[2], dstate=dh0,
                              workspace=attn, stream=stream)
        t3.t3_layernorm_bwd(dboth[:, :d], total, mean, rstd, gamma, x, dx=dx, dgamma=dgamma, dbeta=dbeta, workspace=sums,
                            stream=stream)
    outs = [codes, s, total, mean, rstd, both, last, o, codes2, s2, mean2, rstd2, out, pg, pu, dg, du, dgb, dub, dh0, dboth,
            dx, dgamma, dbeta]
    return run, outs


# single tokens; a few rows of odd heads; heads of 64 in several chunks; few long sequences, cut into ranges
CALLS = [(4, 1, 8, 64, 1024), (2, 12, 9, 27, 729), (3, 200, 5, 64, 1000), (1, 2048, 5, 128, 1280)]


@pytest.mark.parametrize("b,length,heads,dim,hidden", CALLS)
def test_calls_allocate_nothing_and_replay(b, length, heads, dim, hidden):
    run, outs = _calls(length, b, length, heads, dim, hidden)
    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    torch.cuda.synchronize()
    before, free = torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]
    run()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    assert torch.cuda.mem_get_info()[0] == free
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        run()
    for _ in range(3):
        for t in outs:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(outs, want):
            assert torch.equal(t, w)
    assert t3.t3_last_device_error()[0] == t3.T3_OK


def test_two_threads_on_two_streams():
    blocks = [_calls(17, 1, 2048, 5, 128, 1280), _calls(18, 2, 12, 9, 27, 729)]
    want = []
    for run, outs in blocks:
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.fill_(3)
    torch.cuda.synchronize()
    errors = []

    def work(run):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                run(stream)
            stream.synchronize()
        except Exception as e:  # reported by the assertion below
            errors.append(e)
    threads = [threading.Thread(target=work, args=(run,)) for run, _ in blocks]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for (_, outs), ws in zip(blocks, want):
        for t, w in zip(outs, ws):
            assert torch.equal(t, w)
    assert t3.t3_last_device_error()[0] == t3.T3_OK
