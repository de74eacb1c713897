"""The selective scan and the residual norm together, as a model uses them, and at their edges: the example's stacks, a
block against 64 bits with all its gradients, captured and replayed calls, calls on two streams, guard regions."""
import os
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_29_gb300 as la
import test_gpu_ssm as S

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import token_mixer  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
dev, cu_of = S.dev, S.cu_of


def models(kind):
    torch.manual_seed(1)
    if kind == "selective":
        return token_mixer.SelectiveMixer(256, 320, 16)
    return token_mixer.Stack([token_mixer.TokenMixer(256, 4, 64, "delta"), token_mixer.SelectiveMixer(256, 512, 8),
                              token_mixer.TokenMixer(256, 4, 64, "diagonal")], 256)


@pytest.mark.parametrize("kind", ["selective", "stack"])
def test_example_trains(kind):
    """A few steps run, every parameter gets a finite gradient that is not all zeros, and moves."""
    lengths = [300, 17, 129, 64]
    h = torch.randn(sum(lengths), 256, generator=torch.Generator().manual_seed(2)).to(BF).to(dev())
    model = models(kind)
    before = [p.detach().clone() for p in model.parameters()]
    losses = token_mixer.train(model, h, 0.5 * torch.roll(h, 1, 0).float(), cu_of(lengths), steps=3)
    assert np.isfinite(losses).all()
    for name, p in model.named_parameters():
        if p.grad is None:  # the gate's parameters of the mixers that have none
            assert name.endswith(("a_log", "dt_bias")), name
            continue
        assert bool(torch.isfinite(p.grad).all()) and bool(p.grad.any()), name
    assert all(bool((a != p).any()) for a, p in zip(before, model.parameters()) if p.grad is not None)


@pytest.mark.parametrize("kind,stages", [("selective", 7), ("stack", 25)])
def test_example_decodes(kind, stages):
    """A prefill and single tokens give the whole sequence's outputs: every stage between rounds to bf16 on either side, half
    a step of 2^-8 each, and every projection adds up some hundred of them (at most sixfold in a sum of random signs)."""
    lengths = [60, 17, 129, 64]
    h = torch.randn(sum(lengths), 256, generator=torch.Generator().manual_seed(3)).to(BF).to(dev())
    assert token_mixer.decode_error(models(kind), h, lengths, 5) <= 6 * stages * 2.0 ** -9


def plain_scan(x, dt, a, b, c, lens, skip, z, bias):
    """Token by token, for autograd in 64 bits."""
    step, out, t = torch.nn.functional.softplus(dt + bias), [], 0
    for L in lens:
        h = torch.zeros_like(a)
        for t in range(t, t + L):
            h = torch.exp(step[t][:, None] * a) * h + (step[t] * x[t])[:, None] * b[t]
            out.append((h * c[t]).sum(1) + skip * x[t])
        t = t + 1 if L else t
    return torch.stack(out) * torch.nn.functional.silu(z)


def plain_norm(h, w, stream):
    s = h + stream
    return s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-5) * w, s


def test_a_block_and_its_gradients_against_64_bits():
    """Norm, projections, scan, projection, norm, in 32 bits on the GPU: results and the gradients of every input and
    parameter against autograd through the plain forms in 64 bits.  Each operator's own bound is some hundred units of
    2^-24 of its terms' absolute values, a projection's is its 48 terms; ten of them on the way give less than 10^4
    units, 6e-4 of the largest value; held to 2e-4."""
    lens, D, N = [11, 1, 20], 48, 4
    T = sum(lens)
    gen = torch.Generator().manual_seed(4)

    def randn(*shape, scale=1.0):
        return scale * torch.randn(*shape, generator=gen)

    leaves = dict(h=randn(T, D), stream=randn(T, D), w0=1 + randn(D, scale=0.1), w1=1 + randn(D, scale=0.1),
                  pin=randn(D, 3 * D, scale=D ** -0.5), pbc=randn(D, 2 * N, scale=D ** -0.5), pout=randn(D, D, scale=D ** -0.5),
                  a_log=randn(D, N, scale=0.3), skip=randn(D), bias=randn(D) - 2)
    cot, cot_s = randn(T, D), randn(T, D)

    def block(v, norm, scan):
        y, s = norm(v["h"], v["w0"], v["stream"])
        x, dt, z = (y @ v["pin"]).split(D, 1)
        b, c = (y @ v["pbc"]).split(N, 1)
        o = scan(x, dt, -torch.exp(v["a_log"]), b, c, v["skip"], z, v["bias"]) @ v["pout"]
        return norm(o, v["w1"], s)

    def run(cast, norm, scan):
        v = {k: cast(t).requires_grad_() for k, t in leaves.items()}
        y, s = block(v, norm, scan)
        ((y * cast(cot)).sum() + (s * cast(cot_s)).sum()).backward()
        return {"y": y.detach(), "s": s.detach(), **{k: t.grad for k, t in v.items()}}

    cu = cu_of(lens)
    got = run(lambda t: t.clone().to(dev()), la.residual_norm,
              lambda x, dt, a, b, c, skip, z, bias: la.selective_scan(x, dt, a, b, c, cu, skip=skip, z=z, dt_bias=bias, dt_softplus=True)[0])
    ref = run(lambda t: t.double().clone(), plain_norm, lambda x, dt, a, b, c, skip, z, bias: plain_scan(x, dt, a, b, c, lens, skip, z, bias))
    for k, r in ref.items():
        assert float((got[k].cpu().double() - r).abs().max()) <= 2e-4 * float(r.abs().max()), k


def test_autograd_forms():
    """What the wrappers return is what the calls return: unused outputs, expanded cotangents, inputs that need no
    gradient, without the saved states, states in bf16."""
    lens = [30, 45]
    t = S.draw(lens, 64, 16, G=2, seed=5)
    cu = cu_of(lens)
    names = ("x", "dt", "a", "b", "c", "skip", "z", "bias", "s0")
    for save in (True, False):
        v = {k: t[k].clone().requires_grad_() for k in names}
        y, fin = la.selective_scan(v["x"], v["dt"], v["a"], v["b"], v["c"], cu, skip=v["skip"], z=v["z"], dt_bias=v["bias"],
                                   dt_softplus=True, initial_state=v["s0"], save_checkpoints=save, time_block=64)
        (y.float() * t["dy"].float()).sum().backward(retain_graph=True)
        want = la.ssm_bwd(t["x"], t["dt"], t["a"], t["b"], t["c"], cu, t["dy"], skip=t["skip"], z=t["z"], dt_bias=t["bias"],
                          dt_softplus=True, initial_state=t["s0"])
        order = ("x", "dt", "a", "b", "c", "skip", "z", "bias", "s0")
        assert all(torch.equal(v[k].grad, g) for k, g in zip(order, want))
        for p in v.values():
            p.grad = None
        fin.sum().backward()  # an expanded cotangent, y unused
        want = la.ssm_bwd(t["x"], t["dt"], t["a"], t["b"], t["c"], cu, torch.zeros_like(t["x"]), skip=t["skip"], z=t["z"], dt_bias=t["bias"],
                          dt_softplus=True, initial_state=t["s0"], d_final_state=torch.ones_like(fin))
        assert all(torch.equal(v[k].grad, g) for k, g in zip(order, want))
    s0 = t["s0"].to(BF).requires_grad_()
    y, _ = la.selective_scan(t["x"], t["dt"], t["a"], t["b"], t["c"], cu, initial_state=s0)
    y.sum().backward()
    assert s0.grad.dtype == BF and bool(s0.grad.any())

    x, w, r = torch.randn(9, 128, device=dev()).to(BF), torch.ones(128, device=dev()), torch.randn(9, 128, device=dev())
    for res in (None, r, r.to(BF)):
        xv, wv, rv = x.clone().requires_grad_(), w.clone().requires_grad_(), None if res is None else res.clone().requires_grad_()
        out = la.residual_norm(xv, wv, rv)
        y, s = (out, None) if res is None else out
        loss = y.float().sum() if s is None else y.float().sum() + 2 * s.float().sum()
        loss.backward()
        stream = x if res is None else (x.float() + res.float()).to(res.dtype)
        dx, dw, ds = la.rn_bwd(stream, w, torch.ones_like(x), d_residual=None if res is None else torch.full_like(stream, 2.0))
        assert torch.equal(xv.grad, dx) and torch.equal(wv.grad, dw) and (rv is None or torch.equal(rv.grad, ds))
    xv, rv = x.clone().requires_grad_(), r.clone().requires_grad_()
    _, s = la.residual_norm(xv, w, rv)
    s.sum().backward()  # y unused
    assert torch.equal(rv.grad, torch.ones_like(r)) and torch.equal(xv.grad, torch.ones_like(x))


def test_results_over_operands():
    """Single tokens over x, dt or z (both kernels: the second takes large batches), norms over x or the residual."""
    for N, D, states in ((9, 70, 16), (70, 8192, 16), (4100, 64, 64)):
        t = S.draw([1] * N, D, states, seed=N, xt=BF)
        vec = [t[k] for k in "abc"]
        opts = dict(skip=t["skip"], dt_bias=t["bias"], dt_softplus=True)
        want = la.ssm_decode(t["x"], t["dt"], *vec, t["s0"].clone(), z=t["z"], **opts)
        for name in ("x", "dt", "z"):
            v = {k: t[k].clone() for k in ("x", "dt", "z")}
            la.ssm_decode(v["x"], v["dt"], *vec, t["s0"].clone(), z=v["z"], y=v[name], **opts)
            assert torch.equal(v[name], want), (N, name)
    for T, V in ((1300, 4096), (700, 37), (300, 12288)):
        x, r = (torch.randn(T, V, device=dev()).to(BF) for _ in range(2))
        w = torch.randn(V, device=dev())
        y, s, _ = la.rn_fwd(x, w, r)
        xv, rv = x.clone(), r.clone()
        la.rn_fwd(xv, w, rv, y=xv, residual_out=rv)
        assert torch.equal(xv, y) and torch.equal(rv, s)
        rv = r.clone()
        s2 = la.rn_fwd(x, w, rv, y=rv)[1]
        assert torch.equal(rv, y) and torch.equal(s2, s)
        xv = s.clone()
        la.rn_fwd(xv, w, y=xv)
        assert torch.equal(xv, y)
        with pytest.raises(la.binding.LinAttnError):
            la.rn_fwd(x, w, r, y=rv, residual_out=rv)


def test_steps_of_zero_keep_the_state():
    """Bit by bit, whatever the number of tokens and of states."""
    for lens, states in (([1, 2, 3, 17, 33], 16), ([5, 64], 40), ([130], 3)):
        t = S.draw(lens, 40, states, seed=1, softplus=False, z=False)
        t["dt"].zero_()
        y, fin, *grads = S.call(t, cu_of(lens), time_block=64)
        assert torch.equal(fin, t["s0"])
        assert not grads[2].any() and not grads[3].any()  # no decay and no input: rates and inputs' vectors do not matter


def graph_of(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def test_captured_training_calls_replay_with_new_inputs():
    """Two graphs with one workspace between them, replayed in turn."""
    lens = [200, 3, 150]
    cu = cu_of(lens)
    sets = [S.draw(lens, 70, 16, seed=s) for s in (1, 2)]
    buf = {k: v.clone() for k, v in sets[0].items()}
    need = max(la.binding.load().la_ssm_bwd_workspace_bytes(353, 3, 70, 16, 1, 1), la.binding.load().la_ssm_fwd_workspace_bytes(353, 3, 70, 16, 1, 64))
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    opts = dict(skip=buf["skip"], z=buf["z"], dt_bias=buf["bias"], dt_softplus=True)
    ops = [buf[k] for k in "x dt a b c".split()]
    out = {}

    def forward():
        out["f"] = la.ssm_fwd(*ops, cu, initial_state=buf["s0"], output_checkpoints=True, time_block=64, workspace=ws, **opts)

    def backward():
        out["b"] = la.ssm_bwd(*ops, cu, buf["dy"], initial_state=buf["s0"], d_final_state=buf["dfin"], checkpoints=out["f"][2], workspace=ws, **opts)

    gf = graph_of(forward)
    gb = graph_of(backward)
    for t in (sets[1], sets[0], sets[1]):
        for k, v in t.items():
            buf[k].copy_(v)
        gf.replay()
        gb.replay()
        want = S.call(t, cu, time_block=64)
        assert all(torch.equal(a, b) for a, b in zip(out["f"][:2] + out["b"], want))


def test_captured_decoding_steps():
    N, D, steps = 5, 64, 4
    lens = [steps] * N
    t = S.draw(lens, D, 16, seed=6)
    at = torch.arange(N, device=dev()) * steps
    pool = t["s0"].clone()
    buf = {k: t[k][at].clone() for k in ("x", "dt", "z", "b", "c")}
    w, stream = torch.ones(D, device=dev()), torch.zeros(N, D, device=dev())
    out = {}

    def step():
        y = la.ssm_decode(buf["x"], buf["dt"], t["a"], buf["b"], buf["c"], pool, skip=t["skip"], z=buf["z"], dt_bias=t["bias"], dt_softplus=True)
        out["y"], out["q"] = y, la.rn_fwd(y, w, stream, quantize="block")

    g = graph_of(step)
    pool.copy_(t["s0"])
    check = t["s0"].clone()
    for k in range(steps):
        for n, v in buf.items():
            v.copy_(t[n][at + k])
        g.replay()
        y = la.ssm_decode(buf["x"], buf["dt"], t["a"], buf["b"], buf["c"], check, skip=t["skip"], z=buf["z"], dt_bias=t["bias"], dt_softplus=True)
        q = la.rn_fwd(y, w, stream, quantize="block")
        assert torch.equal(out["y"], y) and torch.equal(pool, check)
        assert torch.equal(out["q"][0].view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(out["q"][2], q[2])


def test_two_streams_at_once():
    lens = [3000, 1500]
    cu = cu_of(lens)
    sets = [S.draw(lens, 256, 16, seed=s) for s in (3, 4)]
    x = [torch.randn(4096, 1024, device=dev()).to(BF) for _ in sets]
    w = torch.randn(1024, device=dev())

    def both(t, x, **kw):
        opts = dict(skip=t["skip"], z=t["z"], dt_bias=t["bias"], dt_softplus=True, initial_state=t["s0"])
        ops = [t[k] for k in "x dt a b c".split()] + [cu]
        y, fin, ck = la.ssm_fwd(*ops, output_checkpoints=True, **opts, **kw)
        n, s, _ = la.rn_fwd(x, w, x, **kw)
        return (y, fin, n) + la.ssm_bwd(*ops, t["dy"], d_final_state=t["dfin"], checkpoints=ck, **opts, **kw) + la.rn_bwd(s, w, x, **kw)

    want = [both(t, v) for t, v in zip(sets, x)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = [both(t, v, stream=s) for t, v, s in zip(sets, x, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_only_the_results_are_written():
    """Rows behind the last sequence, neighbouring columns and the ends of every buffer are left as they were."""
    lens, D, N = [20, 0, 33], 40, 16
    T = sum(lens)
    t = S.draw(lens, D, N, seed=8)
    cu = cu_of(lens)
    opts = dict(skip=t["skip"], z=t["z"], dt_bias=t["bias"], dt_softplus=True, initial_state=t["s0"])
    ops = [t[k] for k in "x dt a b c".split()]

    def rows(extra=7):
        buf = torch.full((T + 3, D + extra), 7.0, dtype=BF, device=dev())
        return buf, buf[1:T + 1, 3:D + 3]

    def flat(n, dtype=F32):
        buf = torch.full((n + 512,), 7.0, dtype=dtype, device=dev())
        return buf, buf[256:256 + n]

    y, fin, ck = la.ssm_fwd(*ops, cu, output_checkpoints=True, **opts)
    by, vy = rows()
    bf, vf = flat(3 * D * N)
    bc, vc = flat(la.ssm_checkpoint_rows(T, 3) * D * N)
    la.ssm_fwd(*ops, cu, y=vy, final_state=vf.view(3, D, N), checkpoints=vc.view(-1, D, N), time_block=64, **opts)
    assert torch.equal(vy, y) and torch.equal(vf.view(3, D, N), fin)
    outs = [rows() for _ in range(3)]
    need = la.binding.load().la_ssm_bwd_workspace_bytes(T, 3, D, N, 1, 1)
    ws = torch.full((need + 512,), 9, dtype=torch.uint8, device=dev())
    la.ssm_bwd(*ops, cu, t["dy"], checkpoints=vc.view(-1, D, N), dx=outs[0][1], ddt=outs[1][1], dz=outs[2][1], workspace=ws[256:256 + need], **opts)
    want = la.ssm_bwd(*ops, cu, t["dy"], checkpoints=ck, **opts)
    for (buf, v), g in zip([(by, vy)] + outs, (y, want[0], want[1], want[6])):
        assert torch.equal(v, g)
        v.fill_(7.0)
        assert bool((buf == 7).all())
    for buf, v in ((bf, vf), (bc, vc)):
        assert bool((buf[:256] == 7).all()) and bool((buf[256 + v.numel():] == 7).all())
    assert bool((ws[:256] == 9).all()) and bool((ws[256 + need:] == 9).all())


@pytest.mark.parametrize("N", [33, 1025])
def test_many_sequences(N):
    """More sequences than one round of the block search holds, some empty, some long, against each sequence alone."""
    rng = np.random.default_rng(N)
    lens = [int(v) for v in rng.integers(0, 5, N)]
    lens[N // 2], lens[N - 1] = 500, 130
    t = S.draw(lens, 48, 16, seed=N)
    cu = cu_of(lens)
    whole = S.call(t, cu, time_block=64)
    starts = np.concatenate([[0], np.cumsum(lens)])
    for i in [0, 1, 31, 32, N // 2 - 1, N // 2, N // 2 + 1, N - 2, N - 1] + [int(v) for v in rng.integers(0, N, 6)]:
        a, b = starts[i], starts[i + 1]
        one = {k: v[a:b] if k in ("x", "dt", "b", "c", "z", "dy") else v[i:i + 1] if k in ("s0", "dfin") else v for k, v in t.items()}
        alone = S.call(one, cu_of([lens[i]]), time_block=64)
        for k in (0, 2, 3, 5, 6, 8):
            assert torch.equal(alone[k], whole[k][a:b]), (i, k)
        assert torch.equal(alone[1][0], whole[1][i]) and torch.equal(alone[10][0], whole[10][i])


@pytest.mark.parametrize("S_,pool_dtype,xt", [(16, F32, BF), (16, F32, F32), (32, F32, BF), (4, F32, BF), (8, F32, BF), (64, F32, BF), (16, BF, BF)])
def test_large_decoding_batches(S_, pool_dtype, xt):
    """Batches on the other side of the choice of kernel: some of their sequences as small batches, bad slots left alone."""
    N, D = 1030, 8192 * 16 // S_ // 16 * 2
    N = max(N, (1 << 23) // (D * S_) + 3)
    gen = torch.Generator(device=dev()).manual_seed(S_)

    def randn(*shape, dtype=xt):
        return torch.randn(*shape, generator=gen, device=dev()).to(dtype)

    x, dt, z = (randn(N, D) for _ in range(3))
    b, c = (randn(N, 1, S_) for _ in range(2))
    a, skip, bias = -torch.exp(randn(D, S_, dtype=F32)), randn(D, dtype=F32), randn(D, dtype=F32) - 3
    pool = randn(N + 5, D, S_, dtype=pool_dtype)
    before = pool.clone()
    idx = torch.randperm(N + 5, generator=torch.Generator().manual_seed(1))[:N].to(torch.int32).to(dev())
    idx[7], idx[N - 1] = -1, N + 5
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    y0 = torch.full((N, D), 7.0, dtype=xt, device=dev())
    opts = dict(skip=skip, z=z, dt_bias=bias, dt_softplus=True)
    y = la.ssm_decode(x, dt, a, b, c, pool, state_indices=idx, y=y0, status=status, **opts)
    assert la.read_status(status) == la.binding.LA_ERR_BAD_STATE_INDEX
    assert bool((y[[7, N - 1]] == 7).all())
    some = torch.tensor([0, 1, 2, 3, 5, 6, 8, 9, N // 2, N - 3, N - 2], device=dev())
    few = before.clone()
    opts["z"] = z[some]
    y1 = la.ssm_decode(x[some], dt[some], a, b[some], c[some], few, state_indices=idx[some].contiguous(), **opts)
    # the two sum the states in other orders
    tol = 2.0 ** -7 if xt == BF else 1e-5
    assert float((y[some].float() - y1.float()).abs().max()) <= tol * float(y1.float().abs().max())
    rows = idx[some].long()
    assert float((pool[rows].float() - few[rows].float()).abs().max()) <= 1e-6 * float(few.abs().max())
    used = torch.zeros(N + 5, dtype=torch.bool, device=dev())
    ok = (idx >= 0) & (idx < N + 5)
    used[idx[ok].long()] = True
    assert torch.equal(pool[~used], before[~used])
