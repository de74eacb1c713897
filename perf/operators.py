"""The token-mixer operators around the gated delta rule, as a program calls them: their cases, inputs,
plain forms and 64-bit values.

Three operators share the packed token layout (tokens of all sequences concatenated, cu_seqlens):

  glr    the gated linear recurrence h_t = a_t h_{t-1} + m_t x_t per channel, forward, training and
         one token per sequence against a state pool;
  gn     the per-token group norm over each head's channels with an activation or a gate, forward and
         training;
  sconv  the short causal convolution along each sequence with an activation, forward, training and one
         token per sequence against a state pool.

`own` selects the package's kernels; otherwise `run` computes the plain forms below in 32 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a small serving batch: latency counts
        {"name": "recurrence, one token for 8 sequences", "op": "glr_decode", "N": 8, "D": 2048, "x": "bf16",
         "g": "f32", "gate": "log", "complement": False, "P": 16},
        # the three-sequence batch of the framework's page example; gate logits as a projection leaves them
        {"name": "recurrence forward, three sequences", "op": "glr_fwd", "lens": "1000,1500,1596", "D": 2048,
         "x": "bf16", "g": "bf16", "gate": "logsigmoid", "complement": True},
        # the dense training batch, 8 x 8192 tokens, 32 heads of 128 channels
        {"name": "recurrence forward, dense batch", "op": "glr_fwd", "lens": "8x8192", "D": 4096, "x": "bf16",
         "g": "f32", "gate": "log", "complement": False},
        # one long prompt with few channels: only the time axis can be split
        {"name": "recurrence forward, one long sequence", "op": "glr_fwd", "lens": "131072", "D": 1000,
         "x": "bf16", "g": "bf16", "gate": "bound", "complement": False},
        # a small training batch in 32 bits
        {"name": "recurrence training, three sequences in fp32", "op": "glr_train", "lens": "1000,1500,1596",
         "D": 2048, "x": "f32", "g": "f32", "gate": "log", "complement": True},
        # the dense training batch through forward and backward
        {"name": "recurrence training, dense batch", "op": "glr_train", "lens": "8x8192", "D": 4096, "x": "bf16",
         "g": "bf16", "gate": "logsigmoid", "complement": True},
        # the output norm of a decoding step, gated
        {"name": "norm of 64 tokens, gated", "op": "gn_fwd", "T": 64, "H": 32, "V": 128, "x": "bf16", "w": "f32",
         "per_head": False, "bias": False, "center": False, "act": "silu", "gate": True},
        # the output norm of the dense batch, gated, through forward and backward
        {"name": "norm training, dense batch, gated", "op": "gn_train", "T": 65536, "H": 32, "V": 128, "x": "bf16",
         "w": "f32", "per_head": False, "bias": False, "center": False, "act": "silu", "gate": True},
        # centred groups of an odd width with weights of their own and an activation on the result
        {"name": "norm training, odd groups", "op": "gn_train", "T": 4099, "H": 10, "V": 100, "x": "bf16",
         "w": "bf16", "per_head": True, "bias": True, "center": True, "act": "silu", "gate": False},
        # the convolution of q, k and v in one decoding step of a large serving batch
        {"name": "convolution, one token for 512 sequences", "op": "sconv_decode", "N": 512, "D": 8192, "W": 4,
         "x": "bf16", "w": "bf16", "bias": False, "act": "silu", "P": 1024},
        # the convolution before the dense training batch
        {"name": "convolution forward, dense batch", "op": "sconv_fwd", "lens": "8x8192", "D": 4096, "W": 4,
         "x": "bf16", "w": "bf16", "bias": False, "act": "silu"},
        # a skewed batch through forward and backward
        {"name": "convolution training, skewed batch", "op": "sconv_train", "lens": SKEWED, "D": 2048, "W": 4,
         "x": "bf16", "w": "f32", "bias": True, "act": "silu"},
    ]


# lengths from one token to 16384, some empty, as one batch of a mixed service or data set
SKEWED = "16384,17,0,1033,5000,1,211,8191,64,65,3,2999,640,0,12001,129,450,77,2048,31"


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
    op = rng.choice(["glr_decode", "glr_fwd", "glr_fwd", "glr_train", "glr_train", "gn_fwd", "gn_train", "gn_train",
                     "sconv_decode", "sconv_fwd", "sconv_train"])
    c = {"op": op, "x": rng.choice(["bf16", "bf16", "f32"])}
    if op.startswith("gn"):
        c["H"] = _log_int(rng, 1, 64)
        c["V"] = rng.choice([64, 96, 128, 256, rng.randint(4, 512)])
        c["T"] = _log_int(rng, 1, max(1, min(65536, (1 << 26) // (c["H"] * c["V"]))))
        c["w"] = rng.choice(["bf16", "f32"])
        c["per_head"] = rng.random() < 0.5
        c["bias"] = rng.random() < 0.5
        c["center"] = rng.random() < 0.5
        c["gate"] = rng.random() < 0.5
        c["act"] = rng.choice(["silu", "sigmoid", "none"]) if not c["gate"] else rng.choice(["silu", "sigmoid"])
        return c
    c["D"] = rng.choice([_log_int(rng, 1, 8192), 64 * _log_int(rng, 1, 128)])
    if op.endswith("decode"):
        c["N"] = _log_int(rng, 1, 1024)
        c["P"] = c["N"] + _log_int(rng, 1, 256)
    else:
        c["lens"] = _draw_lens(rng, min(131072, (1 << 26) // c["D"]))
    if op.startswith("glr"):
        c["g"] = rng.choice(["bf16", "f32"])
        c["gate"] = rng.choice(["log", "bound", "logsigmoid"])
        c["complement"] = rng.random() < 0.5
    else:
        c["W"] = rng.choice([2, 3, 4, 4])
        c["w"] = rng.choice(["bf16", "f32"])
        c["bias"] = rng.random() < 0.5
        c["act"] = rng.choice(["silu", "silu", "none"])
    return c


def _lens(text):
    if "x" in text:
        n, L = text.split("x")
        return [int(L)] * int(n)
    return [int(v) for v in text.split(",")]


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
GATE_BOUND = -0.5


def _gate_input(shape, kind, dtype, gen):
    """g as the layer before produces it: natural-log decays -softplus(N(0,1)) with every other channel decaying a
    hundred times slower, or logits (around 3 for the log sigmoid: forget gates mostly open)."""
    r = torch.randn(shape, generator=gen, device=DEV)
    if kind == "log":
        r = -torch.log1p(torch.exp(r))
        r[..., 1::2] *= 0.01
    elif kind == "logsigmoid":
        r = r + 3.0
    return r.to(dtype)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 17)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (scale * torch.randn(shape, generator=gen, device=DEV)).to(dtype)

    op, xt = c["op"], DTYPES[c["x"]]
    s = {"case": c}
    if op.startswith("gn"):
        T, H, V, wt = c["T"], c["H"], c["V"], DTYPES[c["w"]]
        s["x"] = randn(T, H, V, dtype=xt) + 0.25
        wshape = (H, V) if c["per_head"] else (V,)
        s["w"] = (1.0 + randn(*wshape, scale=0.1)).to(wt)
        s["b"] = randn(*wshape, dtype=wt, scale=0.1) if c["bias"] else None
        s["z"] = randn(T, H, V, dtype=xt) if c["gate"] else None
        if op == "gn_train":
            s["dy"] = randn(T, H, V, dtype=xt)
        return s
    D = c["D"]
    if op.endswith("decode"):
        N, P = c["N"], c["P"]
        s["x"] = randn(N, D, dtype=xt)
        s["idx"] = torch.randperm(P, generator=gen, device=DEV)[:N].to(torch.int32)
    else:
        lens = _lens(c["lens"])
        N, T = len(lens), sum(lens)
        cu = [0]
        for L in lens:
            cu.append(cu[-1] + L)
        s["lens"], s["most"] = lens, max(lens)
        s["have"] = torch.tensor([i for i, L in enumerate(lens) if L], dtype=torch.int64, device=DEV)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["x"] = randn(T, D, dtype=xt)
    if op.startswith("glr"):
        s["g"] = _gate_input(tuple(s["x"].shape), c["gate"], DTYPES[c["g"]], gen)
        if op == "glr_decode":
            s["pool"] = randn(P, D, scale=0.5)
        else:
            s["s0"] = randn(N, D, scale=0.5)
            if op == "glr_train":
                s["dh"] = randn(T, D, dtype=xt)
                s["dfin"] = randn(N, D)
    else:
        W, wt = c["W"], DTYPES[c["w"]]
        s["w"] = randn(D, W, dtype=wt, scale=0.5)
        s["b"] = randn(D, dtype=wt, scale=0.5) if c["bias"] else None
        if op == "sconv_decode":
            s["pool"] = randn(P, W - 1, D, dtype=xt)
        else:
            s["s0"] = randn(N, W - 1, D, dtype=xt)
            if op == "sconv_train":
                s["dy"] = randn(T, D, dtype=xt)
    return s


# ---------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------
def _gate_args(c):
    return {"gate_logsigmoid": c["gate"] == "logsigmoid",
            "gate_lower_bound": GATE_BOUND if c["gate"] == "bound" else None,
            "complement_input": c["complement"]}


def _run_own(s):
    import gated_delta_rule_29_gb300 as la
    c = s["case"]
    op = c["op"]
    if op == "glr_decode":
        h = la.glr_decode(s["x"], s["g"], s["pool"], state_indices=s["idx"], **_gate_args(c))
        return h, s["pool"]
    if op == "glr_fwd":
        h, fin, _ = la.glr_fwd(s["x"], s["g"], s["cu"], initial_state=s["s0"], **_gate_args(c))
        return h, fin
    if op == "glr_train":
        h, fin, states = la.glr_fwd(s["x"], s["g"], s["cu"], initial_state=s["s0"], output_checkpoints=True,
                                    **_gate_args(c))
        dx, dg, ds0 = la.glr_bwd(s["x"], s["g"], s["cu"], s["dh"], initial_state=s["s0"], d_final_state=s["dfin"],
                                 checkpoints=states, **_gate_args(c))
        return h, fin, dx, dg, ds0
    if op == "gn_fwd":
        return la.gn_fwd(s["x"], s["w"], s["b"], z=s["z"], center=c["center"], activation=c["act"])
    if op == "gn_train":
        y = la.gn_fwd(s["x"], s["w"], s["b"], z=s["z"], center=c["center"], activation=c["act"])
        dx, dw, db, dz = la.gn_bwd(s["x"], s["w"], s["dy"], s["b"], z=s["z"], center=c["center"], activation=c["act"])
        return y, dx, dw, db, dz
    if op == "sconv_decode":
        y = la.sconv_decode(s["x"], s["w"], s["pool"], s["b"], state_indices=s["idx"], activation=c["act"])
        return y, s["pool"]
    y, fin = la.sconv_fwd(s["x"], s["w"], s["cu"], s["b"], initial_state=s["s0"], activation=c["act"])
    if op == "sconv_fwd":
        return y, fin
    dx, dw, db, ds0 = la.sconv_bwd(s["x"], s["w"], s["cu"], s["dy"], s["b"], initial_state=s["s0"],
                                   activation=c["act"])
    return y, fin, dx, dw, db, ds0


# ---------------------------------------------------------------------------------------------
# plain forms, 32 bits
# ---------------------------------------------------------------------------------------------
def _decay(c, g):
    """(a, m, dlog a / dg): the decay, the input's factor and the gate's derivative."""
    g = g.float()
    if c["gate"] == "log":
        a, slope = torch.exp(g), None
        rest = -torch.expm1(g)
    elif c["gate"] == "bound":
        sg = 1.0 / (1.0 + torch.exp(-g))
        lg = GATE_BOUND * sg
        a, rest, slope = torch.exp(lg), -torch.expm1(lg), lg * (1.0 - sg)
    else:
        a = 1.0 / (1.0 + torch.exp(-g))
        rest = 1.0 / (1.0 + torch.exp(g))
        slope = rest
    return a, (rest if c["complement"] else None), slope


def _scan(a, b, most):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; a is 0 where a sequence starts."""
    s = 1
    while s < most:
        b = torch.cat([b[:s], b[s:] + a[s:] * b[:-s]])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _places(s):
    """The numbers of the sequences that have tokens, and their first and last ones."""
    have = s["have"]
    return have, s["cu"][:-1][have].long(), s["cu"][1:][have].long() - 1


def _glr_plain(s):
    c = s["case"]
    x, (a, m, slope) = s["x"].float(), _decay(c, s["g"])
    have, first, last = _places(s)
    s0 = s["s0"]
    b = x if m is None else m * x
    b = b.index_add(0, first, a[first] * s0[have])
    h = _scan(a.index_fill(0, first, 0.0), b, s["most"])
    fin = s0.clone()
    fin[have] = h[last]
    out = (h.to(s["x"].dtype), fin)
    if c["op"] == "glr_fwd":
        return out
    prev = torch.roll(h, 1, 0)
    prev[first] = s0[have]
    e = s["dh"].float().index_add(0, last, s["dfin"][have])
    an = torch.roll(a, -1, 0).index_fill(0, last, 0.0)
    e = _scan(an.flip(0), e.flip(0), s["most"]).flip(0)
    dx = e if m is None else m * e
    dl = e * a * (prev if m is None else prev - x)
    dg = dl if slope is None else dl * slope
    ds0 = s["dfin"].clone()
    ds0[have] = (a * e)[first]
    return out + (dx.to(s["x"].dtype), dg.to(s["g"].dtype), ds0)


def _act(kind, p):
    """act(p) and its derivative."""
    if kind == "none":
        return p, torch.ones_like(p)
    sg = 1.0 / (1.0 + torch.exp(-p))
    if kind == "sigmoid":
        return sg, sg * (1.0 - sg)
    return p * sg, sg * (1.0 + p * (1.0 - sg))


def _gn_plain(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"].float()
    mu = x.mean(-1, keepdim=True) if c["center"] else 0.0
    d = x - mu
    r = 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5)
    n = d * r
    p = n * w if s["b"] is None else n * w + s["b"].float()
    if s["z"] is None:
        y, dact = _act(c["act"], p)
    else:
        az, dz = _act(c["act"], s["z"].float())
        y = p * az
    y = y.to(s["x"].dtype)
    if c["op"] == "gn_fwd":
        return y
    dy = s["dy"].float()
    if s["z"] is None:
        dp, dz = dy * dact, None
    else:
        dp, dz = dy * az, (dy * p * dz).to(s["x"].dtype)
    over = (0,) if c["per_head"] else (0, 1)
    dw = (dp * n).sum(over).to(s["w"].dtype)
    db = dp.sum(over).to(s["w"].dtype) if s["b"] is not None else None
    dn = dp * w
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if c["center"]:
        dx = dx - dn.mean(-1, keepdim=True)
    return y, (r * dx).to(s["x"].dtype), dw, db, dz


def _conv_rows(s, W):
    """The rows of [x; states] that hold token t's inputs x_{t-W+1}, ..., x_t ([W, T]), and those of the states
    that follow each sequence ([N, W - 1])."""
    lens, T = s["lens"], s["x"].shape[0]
    cu = s["cu"].long()
    L = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), L, output_size=T)
    t = torch.arange(T, device=DEV)
    off = torch.arange(W - 1, -1, -1, device=DEV)[:, None]
    pos = t - cu[seq] - off
    rows = torch.where(pos >= 0, t - off, T + seq * (W - 1) + (W - 1) + pos)
    k = torch.arange(W - 1, device=DEV)
    pf = L[:, None] - (W - 1) + k
    n = torch.arange(len(lens), device=DEV)[:, None]
    frows = torch.where(pf >= 0, cu[:-1, None] + pf, T + n * (W - 1) + (W - 1) + pf)
    return rows, frows


def _sconv_plain(s):
    c = s["case"]
    W, D, T = c["W"], c["D"], s["x"].shape[0]
    w = s["w"].float()
    rows, frows = _conv_rows(s, W)
    src = torch.cat([s["x"], s["s0"].reshape(-1, D)])
    tap = lambda j: src[rows[j]].float()  # noqa: E731
    p = s["b"].float().expand(T, D) if s["b"] is not None else torch.zeros(T, D, device=DEV)
    p = p + torch.stack([tap(j) * w[:, j] for j in range(W)]).sum(0)
    y, dact = _act(c["act"], p)
    out = (y.to(s["x"].dtype), src[frows])
    if c["op"] == "sconv_fwd":
        return out
    dp = s["dy"].float() * dact
    dsrc = torch.zeros(src.shape, device=DEV)
    dw = torch.stack([_tap_back(dsrc, rows[j], dp, w[:, j], tap(j)) for j in range(W)], 1)
    db = dp.sum(0).to(s["w"].dtype) if s["b"] is not None else None
    xt = s["x"].dtype
    return out + (dsrc[:T].to(xt), dw.to(s["w"].dtype), db, dsrc[T:].reshape(s["s0"].shape).to(xt))


def _tap_back(dsrc, rows, dp, wj, xj):
    """One tap's part of the inputs' gradient, added into dsrc, and its weight's gradient."""
    dsrc[rows] += dp * wj  # the rows of one tap are all different
    return (dp * xj).sum(0)


def _decode_plain(s):
    c = s["case"]
    idx, x = s["idx"].long(), s["x"].float()
    if c["op"] == "glr_decode":
        a, m, _ = _decay(c, s["g"])
        h = a * s["pool"][idx] + (x if m is None else m * x)
        s["pool"][idx] = h
        return h.to(s["x"].dtype), s["pool"]
    seen = torch.cat([s["pool"][idx], s["x"][:, None]], 1)
    p = (seen.float() * s["w"].float().t()).sum(1)
    if s["b"] is not None:
        p = p + s["b"].float()
    s["pool"][idx] = seen[:, 1:]
    return _act(c["act"], p)[0].to(s["x"].dtype), s["pool"]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op.endswith("decode"):
        return _decode_plain(state)
    if op.startswith("glr"):
        return _glr_plain(state)
    if op.startswith("gn"):
        return _gn_plain(state)
    return _sconv_plain(state)


# ---------------------------------------------------------------------------------------------
# the least work
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    op, sx = c["op"], SIZE[c["x"]]
    if op.startswith("gn"):
        n = c["T"] * c["H"] * c["V"]
        rows = 2 + c["gate"] if op == "gn_fwd" else 4 + 2 * c["gate"]
        par = (c["H"] if c["per_head"] else 1) * c["V"] * (1 + c["bias"]) * SIZE[c["w"]] * (1 if op == "gn_fwd" else 2)
        return {"bytes": n * sx * rows + par, "flops": n * (12 if op == "gn_fwd" else 36)}
    D = c["D"]
    if op == "glr_decode":
        n = c["N"] * D
        return {"bytes": n * (2 * sx + SIZE[c["g"]] + 8) + 4 * c["N"], "flops": 6 * n}
    if op == "sconv_decode":
        n, W = c["N"] * D, c["W"]
        return {"bytes": n * sx * (2 + 2 * (W - 1)) + D * (W + c["bias"]) * SIZE[c["w"]] + 4 * c["N"],
                "flops": n * (2 * W + 5)}
    lens = _lens(c["lens"])
    n, N = sum(lens) * D, len(lens)
    if op == "glr_fwd":
        return {"bytes": n * (2 * sx + SIZE[c["g"]]) + 8 * N * D, "flops": 6 * n}
    if op == "glr_train":
        return {"bytes": n * (4 * sx + 2 * SIZE[c["g"]]) + 16 * N * D, "flops": 20 * n}
    W = c["W"]
    par = D * (W + c["bias"]) * SIZE[c["w"]]
    st = N * (W - 1) * D * sx
    if op == "sconv_fwd":
        return {"bytes": 2 * n * sx + 2 * st + par, "flops": n * (2 * W + 5)}
    return {"bytes": 4 * n * sx + 3 * st + 2 * par, "flops": n * (8 * W + 16)}


# ---------------------------------------------------------------------------------------------
# 64-bit values, from the definitions token by token
# ---------------------------------------------------------------------------------------------
def _exact_gate(c, g):
    g = g.double()
    if c["gate"] == "log":
        lg, slope = g, torch.ones_like(g)
    elif c["gate"] == "bound":
        lg = GATE_BOUND * torch.sigmoid(g)
        slope = GATE_BOUND * torch.sigmoid(g) * torch.sigmoid(-g)
    else:
        lg, slope = torch.nn.functional.logsigmoid(g), torch.sigmoid(-g)
    return torch.exp(lg), (-torch.expm1(lg) if c["complement"] else torch.ones_like(lg)), slope


def _exact_glr(c, s):
    a, m, slope = _exact_gate(c, s["g"])
    x = s["x"].double()
    h, prev = torch.empty_like(x), torch.empty_like(x)
    fin = s["s0"].double().clone()
    u = m * x
    start = 0
    for i, L in enumerate(s["lens"]):
        st = fin[i].clone()
        for t in range(start, start + L):
            prev[t] = st
            st = torch.addcmul(u[t], a[t], st, out=h[t])
        fin[i] = st
        start += L
    if c["op"] == "glr_fwd":
        return h, fin
    e = s["dh"].double()
    ds0 = s["dfin"].double().clone()
    end = sum(s["lens"])
    for i in range(len(s["lens"]) - 1, -1, -1):
        st = ds0[i].clone()
        for t in range(end - 1, end - 1 - s["lens"][i], -1):
            e[t] += st
            st = a[t] * e[t]
        ds0[i] = st
        end -= s["lens"][i]
    dl = e * a * (prev - x) if c["complement"] else e * a * prev
    return h, fin, e * m, dl * slope, ds0


def _exact_act(kind, p):
    if kind == "none":
        return p, torch.ones_like(p)
    sg = torch.sigmoid(p)
    return (sg, sg * torch.sigmoid(-p)) if kind == "sigmoid" else (p * sg, sg + p * sg * torch.sigmoid(-p))


def _exact_gn(c, s):
    """Head by head, so that the largest batch needs little memory."""
    parts = []
    H, w_all, b_all = c["H"], s["w"].double(), None if s["b"] is None else s["b"].double()
    for k in range(H):
        x = s["x"][:, k].double()
        w = w_all[k] if c["per_head"] else w_all
        b = 0.0 if b_all is None else b_all[k] if c["per_head"] else b_all
        if c["center"]:
            x = x - x.mean(1, keepdim=True)
        r = (x.square().mean(1, keepdim=True) + 1e-5).rsqrt()
        n = x * r
        p = n * w + b
        if s["z"] is None:
            y, q = _exact_act(c["act"], p)
        else:
            f, df = _exact_act(c["act"], s["z"][:, k].double())
            y = p * f
        if c["op"] == "gn_fwd":
            parts.append((y,))
            continue
        dy = s["dy"][:, k].double()
        dp, dz = (dy * q, None) if s["z"] is None else (dy * f, dy * p * df)
        dn = dp * w
        dx = dn - n * (dn * n).mean(1, keepdim=True)
        if c["center"]:
            dx = dx - dn.mean(1, keepdim=True)
        parts.append((y, dx * r, (dp * n).sum(0), dp.sum(0), dz))
    y = torch.stack([v[0] for v in parts], 1)
    if c["op"] == "gn_fwd":
        return y
    dx = torch.stack([v[1] for v in parts], 1)
    dw, db = (torch.stack([v[j] for v in parts]) for j in (2, 3))
    if not c["per_head"]:
        dw, db = dw.sum(0), db.sum(0)
    dz = None if s["z"] is None else torch.stack([v[4] for v in parts], 1)
    return y, dx, dw, (db if s["b"] is not None else None), dz


def _exact_sconv(c, s):
    """Sequence by sequence on the state followed by the tokens."""
    W, T, D = c["W"], s["x"].shape[0], c["D"]
    train = c["op"] == "sconv_train"
    w = s["w"].double()
    y, fin = torch.empty(T, D, dtype=torch.float64, device=DEV), s["s0"].double().clone()
    dx, ds0 = torch.empty_like(y), torch.zeros_like(fin)
    dw, db = torch.zeros_like(w), torch.zeros(D, dtype=torch.float64, device=DEV)
    t = 0
    for i, L in enumerate(s["lens"]):
        line = torch.cat([s["s0"][i].double(), s["x"][t:t + L].double()])
        p = torch.zeros(L, D, dtype=torch.float64, device=DEV)
        if s["b"] is not None:
            p += s["b"].double()
        for j in range(W):
            p += w[:, j] * line[j:j + L]
        y[t:t + L], q = _exact_act(c["act"], p)
        fin[i] = line[L:]
        if train:
            dp = s["dy"][t:t + L].double() * q
            dline = torch.zeros_like(line)
            for j in range(W):
                dline[j:j + L] += w[:, j] * dp
                dw[:, j] += (dp * line[j:j + L]).sum(0)
            db += dp.sum(0)
            ds0[i], dx[t:t + L] = dline[:W - 1], dline[W - 1:]
        t += L
    return (y, fin, dx, dw, (db if s["b"] is not None else None), ds0) if train else (y, fin)


def _exact_decode(c, s):
    slots = s["idx"].tolist()
    pool = s["pool"].double()
    out = []
    if c["op"] == "glr_decode":
        a, m, _ = _exact_gate(c, s["g"])
        for i, k in enumerate(slots):
            pool[k] = a[i] * pool[k] + m[i] * s["x"][i].double()
            out.append(pool[k].clone())
        return torch.stack(out), pool
    w = s["w"].double()
    for i, k in enumerate(slots):
        line = torch.cat([pool[k], s["x"][i].double()[None]])
        p = (line.t() * w).sum(1)
        if s["b"] is not None:
            p = p + s["b"].double()
        out.append(_exact_act(c["act"], p)[0])
        pool[k] = line[1:]
    return torch.stack(out), pool


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].endswith("decode"):
        return _exact_decode(case, s)
    if case["op"].startswith("glr"):
        return _exact_glr(case, s)
    if case["op"].startswith("gn"):
        return _exact_gn(case, s)
    return _exact_sconv(case, s)
