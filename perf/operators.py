"""Workloads of the operators around the ternary products: the residual add
with the root-mean-square norm and its 8-bit output, the gated linear
recurrence over a sequence, and the ternary product with bias, activation and
residual in its epilogue.  Each is one call of a ternary layer's forward or
training step, in a plain torch form (32 bits, rounded once at the end) and
through this library's entry points.

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


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one new token of a serving loop: latency, a few 16 KB rows
        {"name": "norm_decode", "op": "norm", "train": False, "rows": 1, "cols": 8192, "dtype": "bf16",
         "residual": True},
        # a prefill's residual stream in front of the 1280-wide projections
        {"name": "norm_prefill", "op": "norm", "train": False, "rows": 16384, "cols": 1280,
         "dtype": "bf16", "residual": True},
        # a training step's norm in front of the widest projection, both directions
        {"name": "norm_train", "op": "norm", "train": True, "rows": 16384, "cols": 3456,
         "dtype": "bf16", "residual": True},
        # the odd width of the small model, float activations, no residual
        {"name": "norm_train_odd", "op": "norm", "train": True, "rows": 1782, "cols": 729,
         "dtype": "f32", "residual": False},
        # single tokens of 27 sequences advance their states
        {"name": "scan_step", "op": "scan", "train": False, "batch": 27, "length": 1, "width": 8192,
         "dtype": "bf16", "resets": False, "fused": True},
        # one long document's prefill: few channels, so time has to be split
        {"name": "scan_long", "op": "scan", "train": False, "batch": 1, "length": 16384,
         "width": 1280, "dtype": "bf16", "resets": False, "fused": True},
        # a training step over eight sequences, both directions
        {"name": "scan_train", "op": "scan", "train": True, "batch": 8, "length": 2048,
         "width": 3456, "dtype": "bf16", "resets": False, "fused": True},
        # documents packed into odd-sized rows, float activations
        {"name": "scan_train_packed", "op": "scan", "train": True, "batch": 3, "length": 1782,
         "width": 729, "dtype": "f32", "resets": True, "fused": False},
        # one new token through the widest layer: bound by its packed weights
        {"name": "product_decode", "op": "product", "train": False, "m": 1, "n": 8192, "k": 8192,
         "dtype": "bf16", "act": "silu", "bias": True, "residual": True},
        # a prefill through the large layer
        {"name": "product_prefill", "op": "product", "train": False, "m": 16384, "n": 3456,
         "k": 1280, "dtype": "bf16", "act": "gelu", "bias": True, "residual": True},
        # a training step's forward with the saved pre-activation, and the epilogue's gradient
        {"name": "product_train", "op": "product", "train": True, "m": 4096, "n": 3456, "k": 1280,
         "dtype": "bf16", "act": "relu2", "bias": True, "residual": False},
        # the small model's ragged layer at 27 rows, float output
        {"name": "product_odd", "op": "product", "train": False, "m": 27, "n": 729, "k": 243,
         "dtype": "f32", "act": "silu", "bias": True, "residual": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """A width: half of them multiples of 128, the others any number."""
    w = _log_int(rng, lo, hi)
    return max(128, w // 128 * 128) if rng.random() < 0.5 else w


def draw(rng):
    op = rng.choice(("norm", "scan", "product"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    train = rng.random() < 0.5
    limit = 28_000_000 if dtype == "f32" else 56_000_000  # elements, as in the largest listed ones
    if op == "norm":
        cols = _width(rng, 96, 8192)
        return {"op": op, "train": train, "rows": _log_int(rng, 1, min(16384, limit // cols)),
                "cols": cols, "dtype": dtype, "residual": rng.random() < 0.7}
    if op == "scan":
        width = _width(rng, 96, 8192)
        tokens = min(16384, limit // width)
        if rng.random() < 0.25:
            return {"op": op, "train": False, "batch": _log_int(rng, 1, 64), "length": 1,
                    "width": width, "dtype": dtype, "resets": False, "fused": rng.random() < 0.5}
        batch = _log_int(rng, 1, 16)
        return {"op": op, "train": train, "batch": batch,
                "length": _log_int(rng, 16, max(16, tokens // batch)), "width": width,
                "dtype": dtype, "resets": rng.random() < 0.4, "fused": rng.random() < 0.5}
    n, k = _width(rng, 96, 8192), _width(rng, 96, 8192)
    m = _log_int(rng, 1, max(1, min(16384, limit // n, 72_000_000_000 // (n * k))))
    return {"op": op, "train": train, "m": m, "n": n, "k": k, "dtype": dtype,
            "act": rng.choice(ACTS), "bias": rng.random() < 0.7, "residual": rng.random() < 0.5}


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        n = r * c
        b = n * e + (2 * n * e if case["residual"] else 0) + n + 2 * n + 8 * r + 4 * c
        f = 8 * n
        if case["train"]:
            b += 2 * n * e + (n * e if case["residual"] else 0) + 4 * c
            f += 12 * n
        return {"bytes": b, "flops": f}
    if case["op"] == "scan":
        s = case["batch"] * case["width"]
        n = s * case["length"]
        b = 3 * n * e + 8 * s + (case["batch"] * case["length"] if case["resets"] else 0)
        f = 8 * n
        if case["train"]:
            b += 3 * n * e + 8 * s
            f += 14 * n
        return {"bytes": b, "flops": f}
    m, n, k = case["m"], case["n"], case["k"]
    b = m * k + n * ((k + 3) // 4) + m * n * e + 4 * m + 4 * n
    b += (4 * n if case["bias"] else 0) + (m * n * e if case["residual"] else 0)
    f = 2 * m * n * k + 8 * m * n
    if case["train"]:
        b += 3 * m * n * e + (4 * n if case["bias"] else 0)
        f += 8 * m * n
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------------- inputs ---

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, mean=0.0, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        s["x"] = normal(r, c, std=0.7)
        s["residual"] = normal(r, c, std=1.5) if case["residual"] else None
        s["gamma"] = normal(c, mean=1.0, std=0.2, dtype=torch.float32)
        s["q"] = torch.empty((r, c), dtype=torch.int8, device="cuda")
        s["values"] = torch.empty((r, c), dtype=torch.bfloat16, device="cuda")
        s["row_scale"] = torch.empty(r, device="cuda")
        s["rstd"] = torch.empty(r, device="cuda")
        s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
        if case["train"]:
            s["dy"] = normal(r, c)
            s["dsum"] = normal(r, c) if case["residual"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dgamma"] = torch.empty(c, device="cuda")
    elif case["op"] == "scan":
        b, t, d = case["batch"], case["length"], case["width"]
        if case["fused"]:  # gate and candidate side by side, as one projection writes them
            both = torch.empty((b, t, 2 * d), dtype=dt, device="cuda")
            s["gate"], s["cand"] = both[..., :d], both[..., d:]
        else:
            s["gate"] = torch.empty((b, t, d), dtype=dt, device="cuda")
            s["cand"] = torch.empty((b, t, d), dtype=dt, device="cuda")
        s["gate"].copy_(normal(b, t, d, mean=1.5, std=1.7))
        s["cand"].copy_(normal(b, t, d))
        s["h0"] = normal(b, d, dtype=torch.float32)
        s["resets"] = None
        if case["resets"]:  # a document starts about every 300 tokens
            s["resets"] = (torch.rand((b, t), generator=g, device="cuda") < 1 / 300).to(torch.uint8)
        s["h"] = torch.empty((b, t, d), dtype=dt, device="cuda")
        s["h_last"] = torch.empty((b, d), device="cuda")
        if case["train"]:
            s["dh"] = normal(b, t, d)
            s["dh_last"] = normal(b, d, dtype=torch.float32)
            if case["fused"]:
                both = torch.empty((b, t, 2 * d), dtype=dt, device="cuda")
                s["dgate"], s["dcand"] = both[..., :d], both[..., d:]
            else:
                s["dgate"], s["dcand"] = torch.empty_like(s["gate"]), torch.empty_like(s["cand"])
            s["dh0"] = torch.empty((b, d), device="cuda")
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
        w = torch.randint(-1, 2, (k, n), generator=g, device="cuda", dtype=torch.int8)
        # two-bit codes, four per byte along k: 0, 1 for +1, 2 for -1
        codes = torch.zeros((n, (k + 3) // 4 * 4), dtype=torch.uint8, device="cuda")
        codes[:, :k] = torch.where(w == -1, 2, w).to(torch.uint8).t()
        codes = codes.view(n, -1, 4)
        s["packed"] = (codes[..., 0] | codes[..., 1] << 2 | codes[..., 2] << 4 | codes[..., 3] << 6).contiguous()
        s["w"] = w.to(torch.float32)
        s["row_scale"] = torch.rand(m, generator=g, device="cuda") * 0.02 + 0.01
        s["col_scale"] = (torch.rand(n, generator=g, device="cuda") + 0.5) / math.sqrt(k)
        s["bias"] = normal(n, std=0.3, dtype=torch.float32) if case["bias"] else None
        s["residual"] = normal(m, n) if case["residual"] else None
        s["out"] = torch.empty((m, n), dtype=dt, device="cuda")
        s["workspace"] = torch.empty((m, n), dtype=torch.int32, device="cuda")
        s["pre"] = None
        if case["train"]:
            s["pre"] = torch.empty((m, n), dtype=dt, device="cuda")
            s["dy"] = normal(m, n)
            s["dz"] = torch.empty((m, n), dtype=dt, device="cuda")
            s["dbias"] = torch.empty(n, device="cuda") if case["bias"] else None
    return s


# ------------------------------------------------------------ plain forms ---

def _plain_norm(s):
    case = s["case"]
    dt = s["x"].dtype
    total = s["x"].float()
    if case["residual"]:
        total = (total + s["residual"].float()).to(dt).float()
    rstd = torch.rsqrt(total.square().mean(1) + EPS)
    y = total * rstd[:, None] * s["gamma"]
    amax = y.abs().amax(1)
    q = torch.round(y * (127.0 / amax)[:, None]).clamp(-127, 127)
    row_scale = amax / 127.0
    out = {"values": (q * row_scale[:, None]).to(torch.bfloat16), "row_scale": row_scale, "rstd": rstd}
    if case["residual"]:
        out["sum"] = total.to(dt)
    if case["train"]:
        dy = s["dy"].float()
        dn = dy * s["gamma"]
        hat = total * rstd[:, None]
        dx = (dn - hat * (dn * hat).mean(1, keepdim=True)) * rstd[:, None]
        if case["residual"]:
            dx = dx + s["dsum"].float()
        out["dx"] = dx.to(dt)
        out["dgamma"] = (dy * hat).sum(0)
    return out


def _prefix(a, b):
    """h_t = a_t h_(t-1) + b_t along dim 1 from zero: each pass doubles the span
    of steps that an element sums up, so ceil(log2 length) passes do."""
    n = 1
    while n < a.shape[1]:
        b = torch.cat((b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]), 1)
        a = torch.cat((a[:, :n], a[:, n:] * a[:, :-n]), 1)
        n *= 2
    return b


def _plain_scan(s):
    case = s["case"]
    dt = s["h"].dtype
    gate, cand = s["gate"].float(), s["cand"].float()
    keep, take = torch.sigmoid(gate), torch.sigmoid(-gate)
    carry = keep if s["resets"] is None else keep * (s["resets"] == 0)[..., None]
    b = take * cand
    b[:, 0] += carry[:, 0] * s["h0"]
    h = _prefix(carry, b)
    out = {"h": h.to(dt), "h_last": h[:, -1].clone()}
    if case["train"]:
        dh = s["dh"].float().clone()
        dh[:, -1] += s["dh_last"]
        # total gradient of h_t: dh_t + carry_(t+1) times that of h_(t+1)
        after = torch.cat((carry[:, 1:], torch.zeros_like(carry[:, :1])), 1)
        total = _prefix(after.flip(1), dh.flip(1)).flip(1)
        before = torch.cat((s["h0"][:, None], h[:, :-1]), 1)
        if s["resets"] is not None:
            before = before * (s["resets"] == 0)[..., None]
        out["dgate"] = (total * (before - cand) * keep * take).to(dt)
        out["dcand"] = (total * take).to(dt)
        out["dh0"] = total[:, 0] * carry[:, 0]
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


def _plain_product(s):
    case = s["case"]
    dt = s["out"].dtype
    z = (s["a"].float() @ s["w"]) * s["row_scale"][:, None] * s["col_scale"]
    if case["bias"]:
        z = z + s["bias"]
    y, _ = _plain_act(z, case["act"])
    if case["residual"]:
        y = y + s["residual"].float()
    out = {"out": y.to(dt)}
    if case["train"]:
        # the gradient is taken at the saved pre-activation, in the type it is kept in
        out["pre"] = z.to(dt)
        dz = s["dy"].float() * _plain_act(out["pre"].float(), case["act"])[1]
        out["dz"] = dz.to(dt)
        if case["bias"]:
            out["dbias"] = dz.sum(0)
    return out


# ------------------------------------------------------------ the library ---

def _own_norm(s):
    import ternary_weight_int8_t3_gb300 as t3
    case = s["case"]
    t3.t3_rmsnorm_quant(s["x"], s["gamma"], s["residual"], EPS, q=s["q"], row_scale=s["row_scale"],
                        rstd=s["rstd"], sum_out=s["sum"])
    # the 8-bit rows, as the values they stand for
    torch.mul(s["q"], s["row_scale"][:, None], out=s["values"])
    out = {"values": s["values"], "row_scale": s["row_scale"], "rstd": s["rstd"]}
    if case["residual"]:
        out["sum"] = s["sum"]
    if case["train"]:
        total = s["sum"] if case["residual"] else s["x"]
        t3.t3_rmsnorm_bwd(s["dy"], total, s["rstd"], s["gamma"], dsum=s["dsum"], dx=s["dx"],
                          dgamma=s["dgamma"])
        out["dx"], out["dgamma"] = s["dx"], s["dgamma"]
    return out


def _own_scan(s):
    import ternary_weight_int8_t3_gb300 as t3
    t3.t3_gated_scan_fwd(s["gate"], s["cand"], s["h0"], s["resets"], h=s["h"], h_last=s["h_last"])
    out = {"h": s["h"], "h_last": s["h_last"]}
    if s["case"]["train"]:
        t3.t3_gated_scan_bwd(s["gate"], s["cand"], s["h"], s["dh"], s["h0"], s["resets"],
                             dh_last=s["dh_last"], dgate=s["dgate"], dcand=s["dcand"], dh0=s["dh0"])
        out["dgate"], out["dcand"], out["dh0"] = s["dgate"], s["dcand"], s["dh0"]
    return out


def _own_product(s):
    import ternary_weight_int8_t3_gb300 as t3
    case = s["case"]
    act = getattr(t3, "T3_ACT_" + case["act"].upper())
    kind = t3.T3_OUT_BF16 if case["dtype"] == "bf16" else t3.T3_OUT_F32
    t3.t3_gemm_fwd_act(s["a"], s["packed"], row_scale=s["row_scale"], col_scale=s["col_scale"],
                       bias=s["bias"], act=act, residual=s["residual"], kind=kind, C=s["out"],
                       pre=s["pre"], workspace=s["workspace"])
    out = {"out": s["out"]}
    if case["train"]:
        t3.t3_act_bwd(s["dy"], s["pre"], act, dz=s["dz"], dbias=s["dbias"])
        out["pre"], out["dz"] = s["pre"], s["dz"]
        if case["bias"]:
            out["dbias"] = s["dbias"]
    return out


def run(state):
    plain = {"norm": _plain_norm, "scan": _plain_scan, "product": _plain_product}
    calls = {"norm": _own_norm, "scan": _own_scan, "product": _own_product}
    return (calls if own else plain)[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits ---

def _exact_norm(s):
    case = s["case"]
    dt = s["x"].dtype
    x = s["x"].double()
    if case["residual"]:
        x = x.add(s["residual"].double()).to(dt).double()  # the sum is kept in the stream's type
    gamma = s["gamma"].double()
    rms = (x.pow(2).sum(1, keepdim=True) / case["cols"] + EPS).sqrt()
    y = x / rms * gamma
    step = y.abs().max(1, keepdim=True).values / 127
    out = {"values": torch.round(y / step) * step, "row_scale": step[:, 0], "rstd": 1 / rms[:, 0]}
    if case["residual"]:
        out["sum"] = x
    if case["train"]:
        dy = s["dy"].double()
        inner = (dy * gamma * x).sum(1, keepdim=True)
        dx = dy * gamma / rms - x * inner / (case["cols"] * rms.pow(3))
        if case["residual"]:
            dx += s["dsum"].double()
        out["dx"] = dx
        out["dgamma"] = (dy * x / rms).sum(0)
    return out


def _exact_scan(s):
    case = s["case"]
    gate, cand = s["gate"].double(), s["cand"].double()
    a = 1 / (1 + torch.exp(-gate))
    na = 1 / (1 + torch.exp(gate))
    live = torch.ones(gate.shape[:2], dtype=torch.float64, device=gate.device)
    if s["resets"] is not None:
        live = 1.0 - s["resets"].double()
    h = torch.empty_like(gate)
    prior = torch.empty_like(gate)
    state = s["h0"].double()
    for t in range(case["length"]):
        prior[:, t] = state * live[:, t, None]
        state = a[:, t] * prior[:, t] + na[:, t] * cand[:, t]
        h[:, t] = state
    out = {"h": h, "h_last": state}
    if case["train"]:
        dh = s["dh"].double()
        dgate, dcand = torch.empty_like(gate), torch.empty_like(gate)
        back = s["dh_last"].double()
        for t in reversed(range(case["length"])):
            back = back + dh[:, t]
            dcand[:, t] = back * na[:, t]
            dgate[:, t] = back * (prior[:, t] - cand[:, t]) * a[:, t] * na[:, t]
            back = back * a[:, t] * live[:, t, None]
        out["dgate"], out["dcand"], out["dh0"] = dgate, dcand, back
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


def _exact_product(s):
    case = s["case"]
    z = torch.matmul(s["a"].double(), s["w"].double())
    z = z * s["row_scale"].double()[:, None] * s["col_scale"].double()[None, :]
    if case["bias"]:
        z += s["bias"].double()
    y = _exact_act(z, case["act"])[0]
    if case["residual"]:
        y = y + s["residual"].double()
    out = {"out": y}
    if case["train"]:
        dz = s["dy"].double() * _exact_act(z.to(DTYPES[case["dtype"]]).double(), case["act"])[1]
        out["pre"], out["dz"] = z, dz
        if case["bias"]:
            out["dbias"] = dz.sum(0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "scan": _exact_scan, "product": _exact_product}[case["op"]](s)
