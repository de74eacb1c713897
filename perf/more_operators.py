"""The operators of a state-space block around the token mixers, as a program calls them: their cases, inputs,
plain forms and 64-bit values.

  ssm    the selective state space scan over packed sequences, h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t and
         y_t = (C_t h_t + skip x_t) silu(z_t), forward, training and one token per sequence against a state pool;
  rn     the root-mean-square norm of whole rows with the residual's addition, in the input's type or in 8 bits with
         scales, forward and training.

`own` selects the package's kernels; otherwise `run` computes the plain forms below in 32 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
# lengths from one token to 16384, some empty, as one batch of a mixed service or data set
SKEWED = "16384,17,0,1033,5000,1,211,8191,64,65,3,2999,640,0,12001,129,450,77,2048,31"


def listed():
    return [
        # one decoding step of a small serving batch: latency counts
        {"name": "scan, one token for 8 sequences", "op": "ssm_decode", "N": 8, "D": 2048, "S": 16, "G": 1, "x": "bf16",
         "z": True, "softplus": True, "pool": "f32", "P": 16},
        # one decoding step of a large serving batch: the states' bytes count
        {"name": "scan, one token for 512 sequences", "op": "ssm_decode", "N": 512, "D": 8192, "S": 16, "G": 1,
         "x": "bf16", "z": True, "softplus": True, "pool": "f32", "P": 1024},
        # a prompt batch of three sequences
        {"name": "scan forward, three sequences", "op": "ssm_fwd", "lens": "1000,1500,1596", "D": 2048, "S": 16, "G": 1,
         "x": "bf16", "z": True, "softplus": True},
        # the dense batch, 8 x 8192 tokens of 4096 channels
        {"name": "scan forward, dense batch", "op": "ssm_fwd", "lens": "8x8192", "D": 4096, "S": 16, "G": 1,
         "x": "bf16", "z": True, "softplus": True},
        # one long prompt with few channels: the time axis has to be split
        {"name": "scan forward, one long sequence", "op": "ssm_fwd", "lens": "131072", "D": 1000, "S": 16, "G": 1,
         "x": "bf16", "z": False, "softplus": True},
        # a small training batch with grouped B and C, an odd state size and step sizes given as they are
        {"name": "scan training, groups, ragged", "op": "ssm_train", "lens": "100,0,1,700,333", "D": 600, "S": 23, "G": 3,
         "x": "bf16", "z": False, "softplus": False},
        # a skewed training batch in 32 bits
        {"name": "scan training, skewed batch in fp32", "op": "ssm_train", "lens": SKEWED, "D": 1024, "S": 16, "G": 1,
         "x": "f32", "z": True, "softplus": True},
        # the dense training batch
        {"name": "scan training, dense batch", "op": "ssm_train", "lens": "8x8192", "D": 2048, "S": 16, "G": 1,
         "x": "bf16", "z": True, "softplus": True},
        # the norm of a decoding step before an 8-bit projection
        {"name": "norm of 64 tokens, 8 bits", "op": "rn_fwd", "T": 64, "V": 4096, "x": "bf16", "w": "f32", "r": "bf16",
         "q": "row"},
        # the norm of the dense batch before an 8-bit projection, scales as block-scaled products take them
        {"name": "norm of the dense batch, 8 bits", "op": "rn_fwd", "T": 65536, "V": 4096, "x": "bf16", "w": "bf16",
         "r": "bf16", "q": "mx"},
        # the norm in training, the residual stream held in 32 bits
        {"name": "norm training, dense batch", "op": "rn_train", "T": 65536, "V": 4096, "x": "bf16", "w": "f32",
         "r": "f32", "q": "none"},
        # rows of an odd width, the residual in the activations' type
        {"name": "norm training, odd rows", "op": "rn_train", "T": 4099, "V": 1001, "x": "bf16", "w": "bf16", "r": "bf16",
         "q": "none"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lens(rng, most):
    """Sequence lengths summing to at most `most`, now and then with empty ones and single tokens."""
    n = _log_int(rng, 1, 48)
    total = _log_int(rng, 1, most)
    kind = rng.choice(["even", "ragged", "one"])
    if kind == "one":
        return str(total)
    if kind == "even":
        return "%dx%d" % (n, max(1, total // n))
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    return ",".join(str(v) for v in lens)


def draw(rng):
    op = rng.choice(["ssm_decode", "ssm_fwd", "ssm_fwd", "ssm_train", "ssm_train", "rn_fwd", "rn_fwd", "rn_train"])
    c = {"op": op, "x": rng.choice(["bf16", "bf16", "f32"])}
    if op.startswith("rn"):
        c["V"] = rng.choice([_log_int(rng, 1, 16384), 128 * _log_int(rng, 1, 128)])
        c["q"] = rng.choice(["none", "row", "block", "mx"]) if op == "rn_fwd" else "none"
        c["T"] = _log_int(rng, 1, max(1, min(65536, (1 << 27) // c["V"])))
        c["w"] = rng.choice(["bf16", "f32"])
        c["r"] = rng.choice(["none", "f32"] if c["x"] == "f32" else ["none", "bf16", "f32"])
        return c
    c["S"] = rng.choice([16, 16, _log_int(rng, 1, 64)])
    c["G"] = rng.choice([1, 1, _log_int(rng, 1, 8)])
    c["z"] = rng.random() < 0.7
    c["softplus"] = rng.random() < 0.7
    width = rng.choice([_log_int(rng, 1, 8192), 64 * _log_int(rng, 1, 128)])
    c["D"] = c["G"] * max(1, width // c["G"])
    if op == "ssm_decode":
        c["N"] = _log_int(rng, 1, max(1, min(1024, (1 << 26) // (c["D"] * c["S"]))))
        c["P"] = c["N"] + _log_int(rng, 1, 256)
        c["pool"] = rng.choice(["bf16", "f32", "f32"])
    else:
        c["lens"] = _draw_lens(rng, min(131072, (1 << (31 if op == "ssm_fwd" else 30)) // (c["D"] * c["S"])))
    return c


def _lens(text):
    if "x" in text:
        n, L = text.split("x")
        return [int(L)] * int(n)
    return [int(v) for v in text.split(",")]


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 29)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (scale * torch.randn(shape, generator=gen, device=DEV)).to(dtype)

    op, xt = c["op"], DTYPES[c["x"]]
    s = {"case": c}
    if op.startswith("rn"):
        T, V = c["T"], c["V"]
        s["x"] = randn(T, V, dtype=xt)
        s["w"] = (1.0 + randn(V, scale=0.1)).to(DTYPES[c["w"]])
        s["r"] = None if c["r"] == "none" else randn(T, V, dtype=DTYPES[c["r"]], scale=2.0)
        if op == "rn_train":
            s["dy"] = randn(T, V, dtype=xt)
            s["dr"] = None if s["r"] is None else randn(T, V, dtype=s["r"].dtype)
        return s
    D, S, G = c["D"], c["S"], c["G"]
    if op == "ssm_decode":
        rows = c["N"]
        s["pool"] = randn(c["P"], D, S, dtype=DTYPES[c["pool"]], scale=0.5)
        s["idx"] = torch.randperm(c["P"], generator=gen, device=DEV)[:rows].to(torch.int32)
    else:
        lens = _lens(c["lens"])
        rows, cu = sum(lens), [0]
        for L in lens:
            cu.append(cu[-1] + L)
        s["lens"], s["most"] = lens, max(lens)
        s["have"] = torch.tensor([i for i, L in enumerate(lens) if L], dtype=torch.int64, device=DEV)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["s0"] = randn(len(lens), D, S, scale=0.5)
    s["x"] = randn(rows, D, dtype=xt)
    s["b"] = randn(rows, G, S, dtype=xt)
    s["c"] = randn(rows, G, S, dtype=xt)
    # rates -1, -2, ... as they are initialised, moved by training; steps between 1/1000 and 1/10 at their biases
    s["a"] = -torch.arange(1, S + 1, device=DEV) * torch.exp(randn(D, S, scale=0.3))
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(D, generator=gen, device=DEV))
    if c["softplus"]:
        s["dt"] = randn(rows, D, dtype=xt)
        s["bias"] = step + torch.log(-torch.expm1(-step))
    else:
        s["dt"] = (step * torch.exp(randn(rows, D, scale=0.5))).to(xt)
        s["bias"] = None
    s["skip"] = 1.0 + randn(D, scale=0.1)
    s["z"] = randn(rows, D, dtype=xt) if c["z"] else None
    if op == "ssm_train":
        s["dy"] = randn(rows, D, dtype=xt)
        s["dfin"] = randn(len(lens), D, S)
    return s


# ---------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------
def _run_own(s):
    import gated_delta_rule_29_gb300 as la
    c = s["case"]
    op = c["op"]
    if op == "rn_fwd":
        quantize = None if c["q"] == "none" else c["q"]
        y, r, scales = la.rn_fwd(s["x"], s["w"], s["r"], quantize=quantize, eps=EPS)
        if quantize is None:
            return y, (None if s["r"] is None else r)
        values = _dequantised(y, scales, quantize)
        return values, (None if quantize == "mx" else scales), (None if s["r"] is None else r)
    if op == "rn_train":
        y, r, _ = la.rn_fwd(s["x"], s["w"], s["r"], eps=EPS)
        dx, dw, dr = la.rn_bwd(r, s["w"], s["dy"], d_residual=s["dr"], eps=EPS)
        return y, (None if s["r"] is None else r), dx, dw, (None if s["r"] is None else dr)
    kw = {"skip": s["skip"], "z": s["z"], "dt_bias": s["bias"], "dt_softplus": c["softplus"]}
    if op == "ssm_decode":
        y = la.ssm_decode(s["x"], s["dt"], s["a"], s["b"], s["c"], s["pool"], state_indices=s["idx"], **kw)
        return y, s["pool"]
    ops = (s["x"], s["dt"], s["a"], s["b"], s["c"], s["cu"])
    if op == "ssm_fwd":
        y, fin, _ = la.ssm_fwd(*ops, initial_state=s["s0"], **kw)
        return y, fin
    y, fin, states = la.ssm_fwd(*ops, initial_state=s["s0"], output_checkpoints=True, **kw)
    grads = la.ssm_bwd(*ops, s["dy"], initial_state=s["s0"], d_final_state=s["dfin"], checkpoints=states, **kw)
    return (y, fin) + tuple(grads)


WIDTH = {"block": 128, "mx": 32}  # channels that share a scale; "row": all of them


def _dequantised(q, scales, kind):
    """What 8-bit values [T, V] stand for, in 16 bits; exact where the scales are powers of two."""
    T, V = q.shape
    width = WIDTH.get(kind, V)
    v, scales = q.to(torch.bfloat16), scales.to(torch.bfloat16 if kind == "mx" else torch.float32)
    if V % width:
        scales = scales.repeat_interleave(width, 1)[:, :V]
        return (v * scales).to(torch.bfloat16)
    return (v.view(T, -1, width) * scales[:, :, None]).to(torch.bfloat16).view(T, V)


# ---------------------------------------------------------------------------------------------
# plain forms, 32 bits
# ---------------------------------------------------------------------------------------------
def _scan(a, b, most):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; a is 0 where a sequence starts."""
    s = 1
    while s < most:
        b = torch.cat([b[:s], b[s:] + a[s:] * b[:-s]])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _silu(z):
    """silu(z) and its derivative."""
    sg = 1.0 / (1.0 + torch.exp(-z))
    return z * sg, sg * (1.0 + z * (1.0 - sg))


def _steps(s):
    """The step sizes and their derivative by what they are given as."""
    raw = s["dt"].float()
    if s["bias"] is not None:
        raw = raw + s["bias"]
    if not s["case"]["softplus"]:
        return raw, None
    return torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())), 1.0 / (1.0 + torch.exp(-raw))


def _wide(v, D):
    """Each group's vector beside its channels: [rows, G, S] as [rows, D, S]."""
    return v.float().repeat_interleave(D // v.shape[1], 1)


def _by_group(v, G):
    """[rows, D, S] summed over each group's channels."""
    return v.view(v.shape[0], G, -1, v.shape[2]).sum(2)


def _ssm_plain(s):
    c = s["case"]
    D, G, xt = c["D"], c["G"], s["x"].dtype
    x, (dt, slope) = s["x"].float(), _steps(s)
    a = torch.exp(dt[:, :, None] * s["a"])
    u = dt * x
    gate, dgate = (None, None) if s["z"] is None else _silu(s["z"].float())
    if c["op"] == "ssm_decode":
        idx = s["idx"].long()
        h = a * s["pool"][idx].float() + u[:, :, None] * _wide(s["b"], D)
        s["pool"][idx] = h.to(s["pool"].dtype)
        p = (h * _wide(s["c"], D)).sum(2) + s["skip"] * x
        return (p if gate is None else p * gate).to(xt), s["pool"]
    have = s["have"]
    first, last = s["cu"][:-1][have].long(), s["cu"][1:][have].long() - 1
    b = u[:, :, None] * _wide(s["b"], D)
    b.index_add_(0, first, a[first] * s["s0"][have])
    h = _scan(a.index_fill(0, first, 0.0), b, s["most"])
    del b
    fin = s["s0"].clone()
    fin[have] = h[last]
    p = (h * _wide(s["c"], D)).sum(2) + s["skip"] * x
    out = ((p if gate is None else p * gate).to(xt), fin)
    if c["op"] == "ssm_fwd":
        return out
    dy = s["dy"].float()
    dp, dz = (dy, None) if gate is None else (dy * gate, (dy * p * dgate).to(xt))
    dc = _by_group(dp[:, :, None] * h, G).to(xt)
    e = dp[:, :, None] * _wide(s["c"], D)
    e.index_add_(0, last, s["dfin"][have])
    e = _scan(torch.roll(a, -1, 0).index_fill_(0, last, 0.0).flip(0), e.flip(0), s["most"]).flip(0)
    prev = torch.roll(h, 1, 0)
    del h
    prev[first] = s["s0"][have]
    db = _by_group(e * u[:, :, None], G).to(xt)
    du = (e * _wide(s["b"], D)).sum(2)
    e *= a
    ds0 = s["dfin"].clone()
    ds0[have] = e[first]
    e *= prev
    da = (e * dt[:, :, None]).sum(0)
    ddt = du * x + (e * s["a"]).sum(2)
    if slope is not None:
        ddt = ddt * slope
    dx = du * dt + dp * s["skip"]
    dbias = None if s["bias"] is None else ddt.sum(0)
    return out + (dx.to(xt), ddt.to(xt), da, db, dc, (dp * x).sum(0), dz, dbias, ds0)


def _quantise(y, kind):
    """8-bit values and what they are scaled with."""
    T, V = y.shape
    width = WIDTH.get(kind, V)
    blocks = -(-V // width)
    wide = torch.zeros(T, blocks * width, device=DEV)
    wide[:, :V] = y
    wide = wide.view(T, blocks, width)
    scale = torch.clamp(wide.abs().amax(2), min=2.0 ** -100) / 448.0
    if kind == "mx":
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    q = torch.clamp(wide / scale[:, :, None], -448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(T, -1)[:, :V], scale


def _rn_plain(s):
    c = s["case"]
    x, w = s["x"], s["w"].float()
    r = x if s["r"] is None else (x.float() + s["r"].float()).to(s["r"].dtype)
    t = r.float()
    inv = 1.0 / torch.sqrt((t * t).mean(1, keepdim=True) + EPS)
    n = t * inv
    y = n * w
    kept = None if s["r"] is None else r
    if c["q"] != "none":
        q, scale = _quantise(y, c["q"])
        return _dequantised(q, scale, c["q"]), (None if c["q"] == "mx" else scale), kept
    y = y.to(x.dtype)
    if c["op"] == "rn_fwd":
        return y, kept
    dy = s["dy"].float()
    dw = (dy * n).sum(0).to(s["w"].dtype)
    dn = dy * w
    d = inv * (dn - n * (dn * n).mean(1, keepdim=True))
    if s["dr"] is not None:
        d = d + s["dr"].float()
    return y, kept, d.to(x.dtype), dw, (None if s["r"] is None else d.to(s["r"].dtype))


def run(state):
    if own:
        return _run_own(state)
    return _rn_plain(state) if state["case"]["op"].startswith("rn") else _ssm_plain(state)


# ---------------------------------------------------------------------------------------------
# the least work
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    op, sx = c["op"], SIZE[c["x"]]
    if op.startswith("rn"):
        n, w = c["T"] * c["V"], c["V"] * SIZE[c["w"]]
        rr = 0 if c["r"] == "none" else SIZE[c["r"]]
        if op == "rn_fwd":
            out = sx if c["q"] == "none" else 1
            scales = {"none": 0, "row": 4, "block": 4 * -(-c["V"] // 128), "mx": -(-c["V"] // 32)}[c["q"]]
            return {"bytes": n * (sx + 2 * rr + out) + w + c["T"] * scales, "flops": 6 * n}
        # the sum that the forward leaves is read again by no one who keeps it; without a residual the input is
        back = sx + rr + rr + (sx if rr != sx else 0) if rr else 2 * sx
        return {"bytes": n * (2 * sx + 2 * rr + back) + 2 * w, "flops": 18 * n}
    D, S, G = c["D"], c["S"], c["G"]
    par = D * S * 4 + D * 8
    if op == "ssm_decode":
        N = c["N"]
        return {"bytes": N * (D * (3 + c["z"]) * sx + 2 * G * S * sx + 2 * D * S * SIZE[c["pool"]] + 4) + par,
                "flops": 8 * N * D * S}
    lens = _lens(c["lens"])
    T, N = sum(lens), len(lens)
    rows = T * D * sx
    if op == "ssm_fwd":
        return {"bytes": rows * (3 + c["z"]) + 2 * T * G * S * sx + 8 * N * D * S + par, "flops": 8 * T * D * S}
    return {"bytes": rows * (6 + 2 * c["z"]) + 4 * T * G * S * sx + 16 * N * D * S + 2 * par, "flops": 26 * T * D * S}


# ---------------------------------------------------------------------------------------------
# 64-bit values, from the definitions
# ---------------------------------------------------------------------------------------------
def _exact_silu(z):
    return z * torch.sigmoid(z), torch.sigmoid(z) * (1.0 + z * torch.sigmoid(-z))


def _exact_step(s, dt):
    raw = dt.double() if s["bias"] is None else dt.double() + s["bias"].double()
    if not s["case"]["softplus"]:
        return raw, torch.ones_like(raw)
    return torch.logaddexp(raw, torch.zeros_like(raw)), torch.sigmoid(raw)


def _exact_ssm(c, s):
    """Token by token, all the sequences that have one at a time, the longest first."""
    D, G, S = c["D"], c["G"], c["S"]
    train = c["op"] == "ssm_train"
    order = sorted(range(len(s["lens"])), key=lambda i: -s["lens"][i])
    places = torch.tensor(order, device=DEV)
    starts = s["cu"][:-1].long()[places]
    lens = [s["lens"][i] for i in order]
    A, skip = s["a"].double(), s["skip"].double()
    T = s["x"].shape[0]
    p = torch.empty(T, D, dtype=torch.float64, device=DEV)
    st = s["s0"].double()[places]
    kept = torch.empty(T, D, S, dtype=torch.float64, device=DEV) if train else None

    def rows_at(t):
        m = sum(L > t for L in lens)
        return m, starts[:m] + t

    def spread(v):  # [m, G, S] beside the channels
        return v.double() if G == 1 else v.double().repeat_interleave(D // G, 1)

    def by_group(v):
        return v.view(v.shape[0], G, D // G, S).sum(2)

    x, (dt, slope) = s["x"].double(), _exact_step(s, s["dt"])
    u = dt * x
    for t in range(lens[0] if lens else 0):
        m, rows = rows_at(t)
        if train:
            kept[rows] = st[:m]
        st[:m] *= torch.exp(dt[rows][:, :, None] * A)
        st[:m].addcmul_(u[rows][:, :, None], spread(s["b"][rows]))
        p[rows] = (st[:m] * spread(s["c"][rows])).sum(2)
    p += skip * x
    fin = torch.empty_like(st)
    fin[places] = st
    f, df = (1.0, None) if s["z"] is None else _exact_silu(s["z"].double())
    y = p * f
    if not train:
        return y, fin
    dy = s["dy"].double()
    dp, dz = dy * f, None if df is None else dy * p * df
    e = s["dfin"].double()[places]
    dx, ddt = torch.empty_like(p), torch.empty_like(p)
    db, dc = (torch.empty(T, G, S, dtype=torch.float64, device=DEV) for _ in range(2))
    da = torch.zeros_like(A)
    for t in range(lens[0] - 1 if lens else -1, -1, -1):
        m, rows = rows_at(t)
        step, bw, g, old = dt[rows], spread(s["b"][rows]), dp[rows][:, :, None], kept[rows]
        a = torch.exp(step[:, :, None] * A)
        e[:m] += g * spread(s["c"][rows])
        dc[rows] = by_group(g * (a * old + u[rows][:, :, None] * bw))
        db[rows] = by_group(e[:m] * u[rows][:, :, None])
        du = (e[:m] * bw).sum(2)
        e[:m] *= a
        w = e[:m] * old
        da += (w * step[:, :, None]).sum(0)
        dx[rows] = du * step
        ddt[rows] = du * x[rows] + (w * A).sum(2)
    dx += dp * skip
    ddt *= slope
    ds0 = torch.empty_like(e)
    ds0[places] = e
    dbias = None if s["bias"] is None else ddt.sum(0)
    return y, fin, dx, ddt, da, db, dc, (dp * x).sum(0), dz, dbias, ds0


def _exact_decode(c, s):
    """Sequence by sequence."""
    D, G, S = c["D"], c["G"], c["S"]
    pool, out = s["pool"].double(), []
    f = None if s["z"] is None else _exact_silu(s["z"].double())[0]
    dt, _ = _exact_step(s, s["dt"])
    for i, k in enumerate(s["idx"].tolist()):
        x, h = s["x"][i].double(), pool[k].view(G, D // G, S)
        h = torch.exp(dt[i][:, None] * s["a"].double()).view_as(h) * h \
            + torch.einsum("gd,gs->gds", (dt[i] * x).view(G, -1), s["b"][i].double())
        pool[k] = h.view(D, S)
        p = torch.einsum("gds,gs->gd", h, s["c"][i].double()).reshape(D) + s["skip"].double() * x
        out.append(p if f is None else p * f[i])
    return torch.stack(out), pool


def _e4m3(v):
    """Rounded to e4m3: 3 bits after the first down to 2^-6, steps of 2^-9 below; ties to even."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** -20))), min=-6.0) - 3.0)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def _exact_rn(c, s):
    """Some rows at a time, so that the largest batch needs little memory."""
    w = s["w"].double()
    rows = max(1, (1 << 25) // c["V"])
    parts, dw = [], torch.zeros_like(w)
    for t in range(0, c["T"], rows):
        at = slice(t, t + rows)
        r = s["x"][at].double()
        if s["r"] is not None:
            r = r + s["r"][at].double()  # rounded once, to what the stream is held in
        held = r.to(s["x"].dtype if s["r"] is None else s["r"].dtype).double()
        inv = (held.square().mean(1, keepdim=True) + EPS).rsqrt()
        n = held * inv
        y, scale, dn = n * w, None, None
        if c["q"] != "none":
            V = c["V"]
            width = WIDTH.get(c["q"], V)
            most = torch.nn.functional.pad(y.abs(), (0, -V % width)).view(y.shape[0], -1, width).amax(2)
            scale = torch.clamp(most, min=2.0 ** -100) / 448.0
            if c["q"] == "mx":
                scale = torch.exp2(torch.ceil(torch.log2(scale)))
            each = scale.repeat_interleave(width, 1)[:, :V]
            y = _e4m3(y / each) * each
        if c["op"] == "rn_train":
            dy = s["dy"][at].double()
            dw += (dy * n).sum(0)
            dn = dy * w
            dn = inv * (dn - n * (dn * n).mean(1, keepdim=True))
            if s["dr"] is not None:
                dn = dn + s["dr"][at].double()
            dn = dn.float() if c["x"] == "bf16" and c["r"] != "f32" else dn
        parts.append((y.float() if c["x"] == "bf16" or c["q"] != "none" else y, scale,
                      None if s["r"] is None else r.to(torch.float64 if c["r"] == "f32" else torch.float32), dn))
    y, scale, r, d = (None if parts[0][j] is None else torch.cat([v[j] for v in parts]) for j in range(4))
    kept = None if s["r"] is None else r
    if c["q"] != "none":
        return y, (None if c["q"] == "mx" else scale), kept
    if c["op"] == "rn_fwd":
        return y, kept
    return y, kept, d, dw, (None if s["r"] is None else d)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rn"):
        return _exact_rn(case, s)
    return _exact_decode(case, s) if case["op"] == "ssm_decode" else _exact_ssm(case, s)
