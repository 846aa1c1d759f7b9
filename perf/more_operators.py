"""Workloads of three more operators around the ternary products: the layer norm
with its 8-bit output and both gradients, the gated feed-forward product (two
ternary projections, activation and product in one) with its gradient, and
linear attention with a decay for each head (whole sequences, single tokens,
gradient).  Each is one call of a ternary layer's forward or training step, in a
plain torch form (32 bits, rounded once at the end) and through this library's
entry points.

Shapes are those of the library's own workloads (the 16384 x 3456 x 1280
layer, N = K = 8192 for few rows, the widths 243 and 729 at 27 and 1782 rows)
and general sizes between one row and 16384.
"""
import math

import torch

own = False

EPS = 1e-5
ACTS = ("none", "relu", "relu2", "silu", "gelu")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
CHUNK = 64  # tokens of a piece of the plain linear attention


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one new token of a serving loop: latency, a few 16 KB rows
        {"name": "layer_norm_decode", "op": "norm", "train": False, "rows": 1, "cols": 8192,
         "dtype": "bf16", "residual": True, "beta": True},
        # a prefill's residual stream in front of the 1280-wide projections
        {"name": "layer_norm_prefill", "op": "norm", "train": False, "rows": 16384, "cols": 1280,
         "dtype": "bf16", "residual": True, "beta": True},
        # a training step's norm in front of the widest projection, both directions
        {"name": "layer_norm_train", "op": "norm", "train": True, "rows": 16384, "cols": 3456,
         "dtype": "bf16", "residual": True, "beta": True},
        # the odd width of the small model, float activations, no residual
        {"name": "layer_norm_train_odd", "op": "norm", "train": True, "rows": 1782, "cols": 729,
         "dtype": "f32", "residual": False, "beta": True},
        # one new token through the widest block: bound by both packed matrices
        {"name": "glu_decode", "op": "glu", "train": False, "m": 1, "n": 8192, "k": 8192,
         "dtype": "bf16", "act": "silu", "bias": False},
        # a prefill through the large block
        {"name": "glu_prefill", "op": "glu", "train": False, "m": 16384, "n": 3456, "k": 1280,
         "dtype": "bf16", "act": "silu", "bias": False},
        # a training step's forward, which saves both pre-activations, and the gradient
        {"name": "glu_train", "op": "glu", "train": True, "m": 4096, "n": 3456, "k": 1280,
         "dtype": "bf16", "act": "gelu", "bias": True},
        # the small model's ragged block at 27 rows, float output
        {"name": "glu_odd", "op": "glu", "train": False, "m": 27, "n": 729, "k": 243,
         "dtype": "f32", "act": "silu", "bias": True},
        # single tokens of 27 sequences advance their states
        {"name": "linear_step", "op": "linear", "train": False, "batch": 27, "length": 1, "heads": 64,
         "dk": 128, "dv": 128, "dtype": "bf16", "resets": False, "fused": True},
        # one long document's prefill: few heads, so time has to be split
        {"name": "linear_long", "op": "linear", "train": False, "batch": 1, "length": 16384,
         "heads": 10, "dk": 128, "dv": 128, "dtype": "bf16", "resets": False, "fused": True},
        # a training step over eight sequences, both directions
        {"name": "linear_train", "op": "linear", "train": True, "batch": 8, "length": 2048,
         "heads": 27, "dk": 128, "dv": 128, "dtype": "bf16", "resets": False, "fused": False},
        # documents packed into odd-sized rows and heads, float activations
        {"name": "linear_train_packed", "op": "linear", "train": True, "batch": 3, "length": 1782,
         "heads": 9, "dk": 81, "dv": 81, "dtype": "f32", "resets": True, "fused": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """A width: half of them multiples of 128, the others any number."""
    w = _log_int(rng, lo, hi)
    return max(128, w // 128 * 128) if rng.random() < 0.5 else w


def _head(rng):
    """A head's size: the usual ones, or any."""
    return rng.choice((64, 128)) if rng.random() < 0.6 else rng.randint(16, 128)


def draw(rng):
    op = rng.choice(("norm", "glu", "linear"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    train = rng.random() < 0.5
    limit = 28_000_000 if dtype == "f32" else 56_000_000  # elements, as in the largest listed ones
    if op == "norm":
        cols = _width(rng, 96, 8192)
        return {"op": op, "train": train, "rows": _log_int(rng, 1, min(16384, limit // cols)),
                "cols": cols, "dtype": dtype, "residual": rng.random() < 0.7, "beta": rng.random() < 0.7}
    if op == "glu":
        n, k = _width(rng, 96, 8192), _width(rng, 96, 8192)
        m = _log_int(rng, 1, max(1, min(16384, limit // n, 72_000_000_000 // (n * k))))
        return {"op": op, "train": train, "m": m, "n": n, "k": k, "dtype": dtype,
                "act": rng.choice(ACTS), "bias": rng.random() < 0.5}
    dk = _head(rng)
    dv = dk if rng.random() < 0.7 else _head(rng)
    if rng.random() < 0.25:
        heads = rng.randint(1, 64)
        return {"op": op, "train": False, "batch": _log_int(rng, 1, 27 * 64 // heads), "length": 1,
                "heads": heads, "dk": dk, "dv": dv, "dtype": dtype, "resets": False,
                "fused": rng.random() < 0.5}
    if dtype == "f32":
        limit = 5_000_000
    heads = _log_int(rng, 1, 32)
    tokens = max(16, min(16384, limit // (heads * max(dk, dv))))
    batch = _log_int(rng, 1, 16)
    return {"op": op, "train": train, "batch": batch,
            "length": _log_int(rng, 16, max(16, tokens // batch)), "heads": heads, "dk": dk, "dv": dv,
            "dtype": dtype, "resets": rng.random() < 0.4, "fused": rng.random() < 0.5}


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        n = r * c
        b = n * e + (2 * n * e if case["residual"] else 0) + n + 2 * n + 12 * r + (8 if case["beta"] else 4) * c
        f = 10 * n
        if case["train"]:
            b += 2 * n * e + (n * e if case["residual"] else 0) + 8 * c
            f += 14 * n
        return {"bytes": b, "flops": f}
    if case["op"] == "glu":
        m, n, k = case["m"], case["n"], case["k"]
        b = m * k + 2 * n * ((k + 3) // 4) + m * n * e + 4 * m + 8 * n + (8 * n if case["bias"] else 0)
        f = 4 * m * n * k + 10 * m * n
        if case["train"]:
            b += 7 * m * n * e + (8 * n if case["bias"] else 0)
            f += 10 * m * n
        return {"bytes": b, "flops": f}
    s = case["batch"] * case["heads"]
    dk, dv = case["dk"], case["dv"]
    n = s * case["length"]
    b = n * (2 * dk + 2 * dv) * e + 8 * s * dk * dv + (case["batch"] * case["length"] if case["resets"] else 0)
    f = 4 * n * dk * dv
    if case["train"]:
        b += n * (2 * dk + 2 * dv) * e + 8 * s * dk * dv
        f += 12 * n * dk * dv
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------------- inputs ---

def _pack(w):
    """Two-bit codes of w [k][n], four per byte along k: 0, 1 for +1, 2 for -1."""
    k, n = w.shape
    codes = torch.zeros((n, (k + 3) // 4 * 4), dtype=torch.uint8, device="cuda")
    codes[:, :k] = torch.where(w == -1, 2, w).to(torch.uint8).t()
    codes = codes.view(n, -1, 4)
    return (codes[..., 0] | codes[..., 1] << 2 | codes[..., 2] << 4 | codes[..., 3] << 6).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, mean=0.0, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    def empty(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda")

    f32 = torch.float32
    s = {"case": case}
    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        s["x"] = normal(r, c, mean=0.2, std=0.7)
        s["residual"] = normal(r, c, std=1.5) if case["residual"] else None
        s["gamma"] = normal(c, mean=1.0, std=0.2, dtype=f32)
        s["beta"] = normal(c, std=0.2, dtype=f32) if case["beta"] else None
        s["q"] = empty(r, c, dtype=torch.int8)
        s["values"] = empty(r, c, dtype=torch.bfloat16)
        s["row_scale"], s["mean"], s["rstd"] = empty(r, dtype=f32), empty(r, dtype=f32), empty(r, dtype=f32)
        s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
        if case["train"]:
            s["dy"] = normal(r, c)
            s["dsum"] = normal(r, c) if case["residual"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dgamma"] = empty(c, dtype=f32)
            s["dbeta"] = empty(c, dtype=f32) if case["beta"] else None
    elif case["op"] == "glu":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
        for side in ("gate", "up"):
            w = torch.randint(-1, 2, (k, n), generator=g, device="cuda", dtype=torch.int8)
            s[side + "_packed"] = _pack(w)
            s[side + "_w"] = w.to(f32)
            s[side + "_scale"] = (torch.rand(n, generator=g, device="cuda") + 0.5) / math.sqrt(k)
            s[side + "_bias"] = normal(n, std=0.3, dtype=f32) if case["bias"] else None
        s["row_scale"] = torch.rand(m, generator=g, device="cuda") * 0.02 + 0.01
        s["out"] = empty(m, n)
        s["pre_gate"] = s["pre_up"] = None
        if case["train"]:
            s["pre_gate"], s["pre_up"] = empty(m, n), empty(m, n)
            # a pipeline's step: one micro-batch forward, and the gradient of an earlier
            # one from the pre-activations that it left
            s["saved_gate"], s["saved_up"] = normal(m, n), normal(m, n)
            s["dy"] = normal(m, n)
            s["dgate"], s["dup"] = empty(m, n), empty(m, n)
            s["dgate_bias"] = empty(n, dtype=f32) if case["bias"] else None
            s["dup_bias"] = empty(n, dtype=f32) if case["bias"] else None
    else:
        b, t, h, dk, dv = (case[i] for i in ("batch", "length", "heads", "dk", "dv"))
        if case["fused"]:  # query, key and value side by side, as one projection writes them
            whole = empty(b, t, h * (2 * dk + dv))
            s["q"] = whole[..., :h * dk].unflatten(-1, (h, dk))
            s["k"] = whole[..., h * dk:2 * h * dk].unflatten(-1, (h, dk))
            s["v"] = whole[..., 2 * h * dk:].unflatten(-1, (h, dv))
        else:
            s["q"], s["k"], s["v"] = empty(b, t, h, dk), empty(b, t, h, dk), empty(b, t, h, dv)
        for name in ("q", "k", "v"):
            s[name].copy_(normal(*s[name].shape))
        s["scale"] = 1 / math.sqrt(dk)
        # memories of some four to five hundred tokens, each head its own
        spread = torch.rand(h, generator=g, device="cuda") * 7 + 2
        s["log_decay"] = torch.log1p(-torch.exp2(-spread))
        s["state"] = normal(b, h, dk, dv, dtype=f32)
        s["resets"] = None
        if case["resets"]:  # a document starts about every 300 tokens
            s["resets"] = (torch.rand((b, t), generator=g, device="cuda") < 1 / 300).to(torch.uint8)
        s["o"] = empty(b, t, h, dv)
        s["state_last"] = empty(b, h, dk, dv, dtype=f32)
        if case["train"]:
            s["do"] = normal(b, t, h, dv)
            s["dstate_last"] = normal(b, h, dk, dv, dtype=f32)
            s["dq"], s["dk"], s["dv"] = empty(b, t, h, dk), empty(b, t, h, dk), empty(b, t, h, dv)
            s["dstate"] = empty(b, h, dk, dv, dtype=f32)
    return s


# ------------------------------------------------------------ plain forms ---

def _plain_norm(s):
    case = s["case"]
    dt = s["x"].dtype
    total = s["x"].float()
    if case["residual"]:
        total = (total + s["residual"].float()).to(dt).float()
    mean = total.mean(1)
    centred = total - mean[:, None]
    rstd = torch.rsqrt(centred.square().mean(1) + EPS)
    hat = centred * rstd[:, None]
    y = hat * s["gamma"]
    if case["beta"]:
        y = y + s["beta"]
    amax = y.abs().amax(1)
    q = torch.round(y * (127.0 / amax)[:, None]).clamp(-127, 127)
    row_scale = amax / 127.0
    out = {"values": (q * row_scale[:, None]).to(torch.bfloat16), "row_scale": row_scale, "mean": mean,
           "rstd": rstd}
    if case["residual"]:
        out["sum"] = total.to(dt)
    if case["train"]:
        dy = s["dy"].float()
        dn = dy * s["gamma"]
        dx = (dn - dn.mean(1, keepdim=True) - hat * (dn * hat).mean(1, keepdim=True)) * rstd[:, None]
        if case["residual"]:
            dx = dx + s["dsum"].float()
        out["dx"] = dx.to(dt)
        out["dgamma"] = (dy * hat).sum(0)
        if case["beta"]:
            out["dbeta"] = dy.sum(0)
    return out


def _plain_act(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).float()
    if act == "relu2":
        p = z.clamp(min=0)
        return p * p, 2 * p
    if act == "silu":
        g = torch.sigmoid(z)
        return z * g, g * (1 + z * (1 - g))
    c = math.sqrt(2 / math.pi)  # gelu, its tanh form
    th = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + th), 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)


def _plain_glu(s):
    case = s["case"]
    dt = s["out"].dtype
    a = s["a"].float()
    z = {}
    for side in ("gate", "up"):
        z[side] = (a @ s[side + "_w"]) * s["row_scale"][:, None] * s[side + "_scale"]
        if case["bias"]:
            z[side] = z[side] + s[side + "_bias"]
    out = {"out": (_plain_act(z["gate"], case["act"])[0] * z["up"]).to(dt)}
    if case["train"]:
        out["pre_gate"], out["pre_up"] = z["gate"].to(dt), z["up"].to(dt)
        dy = s["dy"].float()
        value, slope = _plain_act(s["saved_gate"].float(), case["act"])
        dgate = dy * s["saved_up"].float() * slope
        dup = dy * value
        out["dgate"], out["dup"] = dgate.to(dt), dup.to(dt)
        if case["bias"]:
            out["dgate_bias"], out["dup_bias"] = dgate.sum(0), dup.sum(0)
    return out


def _prefix(a, b):
    """h_i = a_i h_(i-1) + b_i along dim 1 from zero: each pass doubles the span
    that an element sums up."""
    n = 1
    while n < a.shape[1]:
        b = torch.cat((b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]), 1)
        a = torch.cat((a[:, :n], a[:, n:] * a[:, :-n]), 1)
        n *= 2
    return b


def _plain_attend(q, k, v, log_decay, state, cuts, first):
    """o_t = sum over j <= t of decay^(t - j) (q_t . k_j) v_j plus decay^(t + first)
    q_t . state, within the stretches that begin where `cuts` is set; and the state
    behind the last token.  Pieces of CHUNK tokens, each with the state in front of
    it, which a prefix over the pieces gives."""
    batch, length, heads, _ = q.shape
    size = min(CHUNK, length)
    pieces = (length + size - 1) // size
    pad = pieces * size - length

    def split(x):  # [batch][pieces][heads][size][d], zeros behind the last token
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, pad))
        return x.unflatten(1, (pieces, size)).transpose(2, 3)

    q, k, v = split(q), split(k), split(v)
    # how often the state has decayed at each token, and in front of each piece
    count = torch.arange(pieces * size, device=q.device).clamp(max=length - 1).view(pieces, size)
    before = torch.cat((count.new_full((1,), -first), count[:-1, -1]))[:, None]
    rate = log_decay[:, None]
    ago = count[:, None, :, None] - count[:, None, None, :]
    decay = torch.exp(ago.clamp(min=0) * rate[..., None])
    decay = decay * torch.ones((size, size), device=q.device).tril()  # [pieces][heads][size][size]
    into = torch.exp((count - before)[:, None] * rate)
    outof = torch.exp((count[:, -1:] - count)[:, None] * rate)
    through = torch.exp((count[:, -1:] - before)[:, None] * rate)[..., None]
    if cuts is not None:
        part = torch.nn.functional.pad(cuts.int(), (0, pad)).unflatten(1, (pieces, size)).cumsum(2)[:, :, None]
        decay = decay * (part[..., :, None] == part[..., None, :])
        into = into * (part == 0)
        outof = outof * (part == part[..., -1:])
        through = through * (part[..., -1:, None] == 0)
    through = through.expand(batch, pieces, heads, 1, 1)
    end = (k * outof[..., None]).transpose(3, 4) @ v
    end[:, 0] += through[:, 0] * state
    end = _prefix(through, end)
    begin = torch.cat((state[:, None], end[:, :-1]), 1)
    o = ((q @ k.transpose(3, 4)) * decay) @ v + (q @ begin) * into[..., None]
    return o.transpose(2, 3).flatten(1, 2)[:, :length], end[:, -1]


def _plain_linear(s):
    case = s["case"]
    dt = s["o"].dtype
    q, k, v, ld, scale, resets = s["q"], s["k"], s["v"], s["log_decay"], s["scale"], s["resets"]
    o, last = _plain_attend(q, k, v, ld, s["state"], resets, 1)
    out = {"o": (o * scale).to(dt), "state_last": last}
    if case["train"]:
        do = s["do"]
        out["dq"] = (_plain_attend(do, v, k, ld, s["state"].transpose(2, 3), resets, 1)[0] * scale).to(dt)
        # backward in time: what cut in front of a token cuts behind it
        cuts = None
        if resets is not None:
            cuts = torch.cat((torch.zeros_like(resets[:, :1]), resets[:, 1:].flip(1)), 1)
        qs = (q.float() * scale).flip(1)
        kr, vr, dor = k.flip(1), v.flip(1), do.flip(1)
        dv, dstate = _plain_attend(kr, qs, dor, ld, s["dstate_last"], cuts, 0)
        dk, _ = _plain_attend(vr, dor, qs, ld, s["dstate_last"].transpose(2, 3), cuts, 0)
        dstate = dstate * torch.exp(ld)[:, None, None]
        if resets is not None:
            dstate = dstate * (resets[:, 0] == 0)[:, None, None, None]
        out["dk"], out["dv"], out["dstate"] = dk.flip(1).to(dt), dv.flip(1).to(dt), dstate
    return out


# ------------------------------------------------------------ the library ---

def _own_norm(s):
    import ternary_weight_int8_t3_gb300 as t3
    case = s["case"]
    t3.t3_layernorm_quant(s["x"], s["gamma"], s["beta"], s["residual"], EPS, q=s["q"], row_scale=s["row_scale"],
                          mean=s["mean"], rstd=s["rstd"], sum_out=s["sum"])
    # the 8-bit rows, as the values they stand for
    torch.mul(s["q"], s["row_scale"][:, None], out=s["values"])
    out = {"values": s["values"], "row_scale": s["row_scale"], "mean": s["mean"], "rstd": s["rstd"]}
    if case["residual"]:
        out["sum"] = s["sum"]
    if case["train"]:
        total = s["sum"] if case["residual"] else s["x"]
        t3.t3_layernorm_bwd(s["dy"], total, s["mean"], s["rstd"], s["gamma"], dsum=s["dsum"], dx=s["dx"],
                            dgamma=s["dgamma"], dbeta=s["dbeta"])
        out["dx"], out["dgamma"] = s["dx"], s["dgamma"]
        if case["beta"]:
            out["dbeta"] = s["dbeta"]
    return out


def _own_glu(s):
    import ternary_weight_int8_t3_gb300 as t3
    case = s["case"]
    act = getattr(t3, "T3_ACT_" + case["act"].upper())
    kind = t3.T3_OUT_BF16 if case["dtype"] == "bf16" else t3.T3_OUT_F32
    t3.t3_gemm_fwd_glu(s["a"], s["gate_packed"], s["up_packed"], row_scale=s["row_scale"],
                       gate_scale=s["gate_scale"], up_scale=s["up_scale"], gate_bias=s["gate_bias"],
                       up_bias=s["up_bias"], act=act, kind=kind, C=s["out"], pre_gate=s["pre_gate"],
                       pre_up=s["pre_up"])
    out = {"out": s["out"]}
    if case["train"]:
        t3.t3_glu_bwd(s["dy"], s["saved_gate"], s["saved_up"], act, dgate=s["dgate"], dup=s["dup"],
                      dgate_bias=s["dgate_bias"], dup_bias=s["dup_bias"])
        for name in ("pre_gate", "pre_up", "dgate", "dup"):
            out[name] = s[name]
        if case["bias"]:
            out["dgate_bias"], out["dup_bias"] = s["dgate_bias"], s["dup_bias"]
    return out


def _own_linear(s):
    import ternary_weight_int8_t3_gb300 as t3
    t3.t3_linear_attn_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["resets"], s["scale"], o=s["o"],
                          state_last=s["state_last"])
    out = {"o": s["o"], "state_last": s["state_last"]}
    if s["case"]["train"]:
        t3.t3_linear_attn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], s["state"], s["resets"], s["scale"],
                              dstate_last=s["dstate_last"], dq=s["dq"], dk=s["dk"], dv=s["dv"],
                              dstate=s["dstate"])
        for name in ("dq", "dk", "dv", "dstate"):
            out[name] = s[name]
    return out


def run(state):
    plain = {"norm": _plain_norm, "glu": _plain_glu, "linear": _plain_linear}
    calls = {"norm": _own_norm, "glu": _own_glu, "linear": _own_linear}
    return (calls if own else plain)[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits ---

def _exact_norm(s):
    case = s["case"]
    dt = s["x"].dtype
    x = s["x"].double()
    if case["residual"]:
        x = x.add(s["residual"].double()).to(dt).double()  # the sum is kept in the stream's type
    gamma = s["gamma"].double()
    mu = x.sum(1, keepdim=True) / case["cols"]
    dev = ((x - mu).pow(2).sum(1, keepdim=True) / case["cols"] + EPS).sqrt()
    z = (x - mu) / dev
    y = z * gamma
    if case["beta"]:
        y += s["beta"].double()
    step = y.abs().max(1, keepdim=True).values / 127
    out = {"values": torch.round(y / step) * step, "row_scale": step[:, 0], "mean": mu[:, 0], "rstd": 1 / dev[:, 0]}
    if case["residual"]:
        out["sum"] = x
    if case["train"]:
        dy = s["dy"].double()
        dz = dy * gamma
        # through the row's mean and deviation
        ddev = -(dz * z).sum(1, keepdim=True) / dev
        dx = dz / dev + ddev * z / case["cols"]
        dx -= (dz / dev).sum(1, keepdim=True) / case["cols"]
        if case["residual"]:
            dx += s["dsum"].double()
        out["dx"] = dx
        out["dgamma"] = (dy * z).sum(0)
        if case["beta"]:
            out["dbeta"] = dy.sum(0)
    return out


def _exact_act(z, act):
    """act(z) and its derivative."""
    zero = torch.zeros_like(z)
    if act == "none":
        return z, zero + 1
    if act == "relu":
        return torch.maximum(z, zero), torch.where(z > 0, 1.0, zero)
    if act == "relu2":
        return torch.maximum(z, zero) ** 2, 2 * torch.maximum(z, zero)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return z * sg, sg + z * sg * (1 - sg)
    # 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
    k = 2 * math.sqrt(2 / math.pi)
    sg = 1 / (1 + torch.exp(-k * (z + 0.044715 * z ** 3)))
    return z * sg, sg + z * sg * (1 - sg) * k * (1 + 0.134145 * z ** 2)


def _exact_glu(s):
    case = s["case"]

    def project(side):
        z = torch.matmul(s["a"].double(), s[side + "_w"].double())
        z = z * s["row_scale"].double()[:, None] * s[side + "_scale"].double()[None, :]
        return z + s[side + "_bias"].double() if case["bias"] else z

    zg, zu = project("gate"), project("up")
    out = {"out": _exact_act(zg, case["act"])[0] * zu}
    if case["train"]:
        out["pre_gate"], out["pre_up"] = zg, zu
        value, slope = _exact_act(s["saved_gate"].double(), case["act"])
        dy = s["dy"].double()
        out["dup"] = dy * value
        out["dgate"] = dy * s["saved_up"].double() * slope
        if case["bias"]:
            out["dgate_bias"], out["dup_bias"] = out["dgate"].sum(0), out["dup"].sum(0)
    return out


def _exact_linear(s):
    """Token by token, from the recurrence and its gradient."""
    case = s["case"]
    length, scale = case["length"], s["scale"]
    gamma = torch.exp(s["log_decay"].double())[None, :, None, None]
    live = None if s["resets"] is None else (s["resets"] == 0).double()

    def outer(x, y):
        return x.double()[..., :, None] * y.double()[..., None, :]

    def alive(t):
        return gamma if live is None else gamma * live[:, t, None, None, None]

    def times(x, m):  # row vectors x [b][h][i] by matrices m [b][h][i][j]
        return (x.double()[..., None, :] @ m)[..., 0, :]

    shape = s["o"].shape
    o = torch.empty(shape, dtype=torch.float64, device="cuda")
    if case["train"]:
        dq = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    state = s["state"].double()
    for t in range(length):
        state = state * alive(t) + outer(s["k"][:, t], s["v"][:, t])
        o[:, t] = scale * times(s["q"][:, t], state)
        if case["train"]:
            dq[:, t] = scale * times(s["do"][:, t], state.transpose(2, 3))
    out = {"o": o, "state_last": state}
    if case["train"]:
        dk, dv = torch.empty_like(dq), torch.empty_like(o)
        back = s["dstate_last"].double()
        for t in reversed(range(length)):
            back = back + scale * outer(s["q"][:, t], s["do"][:, t])
            dk[:, t] = times(s["v"][:, t], back.transpose(2, 3))
            dv[:, t] = times(s["k"][:, t], back)
            back = back * alive(t)
        out["dq"], out["dk"], out["dv"], out["dstate"] = dq, dk, dv, back
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "glu": _exact_glu, "linear": _exact_linear}[case["op"]](s)
