"""The per-head group norm with an activation or gate on the GPU against its 64-bit form.

Bounds (fixed before the first run): an output is rounded once to its type; before that a row's sums of V terms,
r and the activation may be off by 2 V + 64 units of 2^-24 of their scales, and the sums over R rows by R more."""
import pytest
import torch

import gated_delta_rule_29_gb300 as la
import mixer_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def draw(T, H, V, xt, wt, per_head, bias, gate, seed, mean=0.25):
    gen = torch.Generator().manual_seed(seed)
    shape = (H, V) if per_head else (V,)
    t = dict(x=(torch.randn(T, H, V, generator=gen) + mean).to(xt), w=(1 + 0.1 * torch.randn(shape, generator=gen)).to(wt),
             b=(0.1 * torch.randn(shape, generator=gen)).to(wt) if bias else None,
             z=torch.randn(T, H, V, generator=gen).to(xt) if gate else None,
             dy=torch.randn(T, H, V, generator=gen).to(xt))
    return {k: None if v is None else v.to(dev()) for k, v in t.items()}


def check(t, center, act, views=None, eps=1e-5):
    v = dict(t, **(views or {}))
    kw = dict(center=center, activation=act, eps=eps)
    y = la.gn_fwd(v["x"], t["w"], t["b"], z=v["z"], **kw)
    dx, dw, db, dz = la.gn_bwd(v["x"], t["w"], v["dy"], t["b"], z=v["z"], **kw)
    args = [R.f64(t[k]) for k in ("x", "w", "b", "z", "dy")]
    ref = R.gn(*args, **kw)
    sc = R.gn_scales(*args, **kw)
    T, H, V = t["x"].shape
    row = 2 * V + 64
    many = row + T * (1 if t["w"].dim() == 2 else H)
    xt, wt = t["x"].dtype, t["w"].dtype
    R.within("y", y, ref[0], xt, row, sc[0])
    R.within("dx", dx, ref[1], xt, 2 * row, sc[1])
    R.within("dw", dw, ref[2], wt, many, sc[2])
    R.within("db", db, ref[3], wt, many, sc[3])
    R.within("dz", dz, ref[4], xt, row, sc[4])
    return y, dx, dw, db, dz


@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 33, 64, 96, 100, 128, 250, 256, 257, 512, 1000, 1024, 1025, 2048, 4099, 8192])
@pytest.mark.parametrize("xt", [BF, F32])
def test_widths(V, xt):
    check(draw(5, 3, V, xt, F32, False, True, True, seed=V), False, "silu")


@pytest.mark.parametrize("V", [4, 60, 128, 1040])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("act,gate", [("none", False), ("silu", False), ("sigmoid", False), ("silu", True),
                                      ("sigmoid", True), ("none", True)])
def test_forms(V, per_head, center, act, gate):
    check(draw(9, 4, V, BF, BF, per_head, act != "none", gate, seed=V), center, act)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 64), (257, 1), (63, 5), (1030, 16), (2, 300)])
@pytest.mark.parametrize("per_head", [False, True])
def test_tokens_and_heads(T, H, per_head):
    check(draw(T, H, 32, BF, F32, per_head, True, True, seed=T), True, "silu")


def test_many_rows():
    check(draw(4100, 8, 64, F32, F32, False, False, True, seed=2), False, "silu")
    check(draw(4100, 8, 64, F32, F32, True, True, False, seed=3), True, "silu")


def test_no_tokens():
    t = draw(0, 3, 64, BF, F32, False, True, True, seed=1)
    y = la.gn_fwd(t["x"], t["w"], t["b"], z=t["z"])
    dx, dw, db, dz = la.gn_bwd(t["x"], t["w"], t["dy"], t["b"], z=t["z"])
    assert y.numel() == dx.numel() == dz.numel() == 0
    assert torch.equal(dw, torch.zeros_like(t["w"])) and torch.equal(db, torch.zeros_like(t["b"]))


def test_constant_rows_and_large_means():
    """A constant row has variance 0: n = 0 and r = eps^-1/2.  A mean a hundred times the deviation leaves the
    deviations their bits (they are taken after the mean)."""
    t = draw(6, 2, 64, F32, F32, False, True, False, seed=8)
    t["x"][0] = 3.0
    t["x"][1] = 0.0
    check(t, True, "silu")
    check(draw(6, 2, 64, F32, F32, False, True, False, seed=8, mean=100.0), True, "silu")


def test_nan_and_infinity_stay_in_their_row():
    t = draw(8, 4, 128, BF, F32, False, False, True, seed=5)
    clean = la.gn_fwd(t["x"], t["w"], z=t["z"], center=True)
    t["x"][3, 1, 7] = float("nan")
    t["x"][5, 2, 0] = float("inf")
    got = la.gn_fwd(t["x"], t["w"], z=t["z"], center=True)
    keep = torch.ones(8, 4, dtype=torch.bool, device=dev())
    keep[3, 1] = keep[5, 2] = False
    assert torch.equal(got[keep], clean[keep])
    assert bool(torch.isnan(got[3, 1].float()).all()) and bool(torch.isnan(got[5, 2].float()).any())


@pytest.mark.parametrize("V", [128, 100])
def test_views(V):
    """x and z as column slices of one projection, at an odd offset and at an aligned one; a broadcast gradient; results
    written into a slice leave the rest alone."""
    t = draw(50, 4, V, BF, F32, True, True, True, seed=6)
    packed = check(t, True, "silu")
    for shift in (1, 8):
        wide = torch.full((50, shift + 8 * V), float("nan"), dtype=BF, device=dev())
        x = wide[:, shift:shift + 4 * V].view(50, 4, V)
        z = wide[:, shift + 4 * V:].view(50, 4, V)
        x.copy_(t["x"])
        z.copy_(t["z"])
        got = check(t, True, "silu", views=dict(x=x, z=z))
        assert all(torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=1e-5) for a, b in zip(got, packed))
        out = torch.full((50, 4, V + 2 * shift), 7.0, dtype=BF, device=dev())
        y = la.gn_fwd(x, t["w"], t["b"], z=z, y=out[:, :, shift:shift + V])
        assert torch.equal(y, got[0]) and bool((out[:, :, :shift] == 7).all()) and bool((out[:, :, shift + V:] == 7).all())
    t["dy"] = t["dy"][:1].expand(50, 4, V).contiguous()
    check(t, True, "silu", views=dict(dy=t["dy"][:1].expand(50, 4, V)))


def test_rows_do_not_depend_on_the_batch():
    t = draw(300, 4, 128, BF, F32, False, False, True, seed=12)
    y = la.gn_fwd(t["x"], t["w"], z=t["z"])
    dx = la.gn_bwd(t["x"], t["w"], t["dy"], z=t["z"])[0]
    for a, b in ((0, 1), (17, 60), (299, 300)):
        assert torch.equal(la.gn_fwd(t["x"][a:b], t["w"], z=t["z"][a:b]), y[a:b])
        assert torch.equal(la.gn_bwd(t["x"][a:b], t["w"], t["dy"][a:b], z=t["z"][a:b])[0], dx[a:b])


def test_autograd_and_repeatability():
    t = draw(700, 4, 128, BF, BF, False, True, True, seed=14)
    x, w, b, z = (t[k].clone().requires_grad_() for k in ("x", "w", "b", "z"))
    y = la.group_norm(x, w, b, z=z, center=False)
    got = torch.autograd.grad(y, (x, w, b, z), t["dy"])
    want = la.gn_bwd(t["x"], t["w"], t["dy"], t["b"], z=t["z"], center=False)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    dx, = torch.autograd.grad(la.group_norm(x, w).sum(), (x,))
    assert torch.equal(dx, la.gn_bwd(t["x"], t["w"], torch.ones_like(t["x"]))[0])


def test_graph_and_stream():
    t = draw(70, 4, 128, BF, F32, True, True, True, seed=15)
    u = draw(70, 4, 128, BF, F32, True, True, True, seed=16)

    def both(v, **kw):
        return (la.gn_fwd(v["x"], v["w"], v["b"], z=v["z"], **kw),) + la.gn_bwd(v["x"], v["w"], v["dy"], v["b"], z=v["z"], **kw)

    want, want_u = both(t), both(u)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(t, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(t)
    for k in t:
        t[k].copy_(u[k])
    for _ in range(2):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want_u))


def test_wrapper_refusals():
    t = draw(4, 2, 8, BF, F32, False, True, True, seed=1)
    x, w, b, z = t["x"], t["w"], t["b"], t["z"]
    with pytest.raises(TypeError):
        la.gn_fwd(x.half(), w)
    with pytest.raises(TypeError):
        la.gn_fwd(x, w, b.to(BF))
    with pytest.raises(TypeError):
        la.gn_fwd(x, w, z=z.float())
    with pytest.raises(ValueError):
        la.gn_fwd(x, w[:4])
    with pytest.raises(ValueError):
        la.gn_fwd(x[0], w)
    with pytest.raises(ValueError):
        la.gn_fwd(x.transpose(1, 2), w)
    with pytest.raises(ValueError):
        la.gn_fwd(x, w, activation="relu")
    with pytest.raises(la.binding.LinAttnError):
        la.gn_fwd(x, w, eps=0.0)
    with pytest.raises(ValueError):
        la.gn_bwd(x, w, t["dy"][:2])
    with pytest.raises(la.binding.LinAttnError):
        la.gn_fwd(torch.zeros(1, 1, 8193, device=dev()), torch.zeros(8193, device=dev()))
