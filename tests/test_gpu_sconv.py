"""The short causal convolution on the GPU against its 64-bit form.

Bounds (fixed before the first run): an output is rounded once to its type; before that a token's W + 1 terms and the
activation may be off by 32 units of 2^-24 of their scale, and the sums over T tokens by T units more."""
import numpy as np
import pytest
import torch

import gated_delta_rule_29_gb300 as la
import mixer_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def cu_of(lens, dtype=torch.int32):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=dtype, device=dev())


def draw(lens, D, W, xt, wt, bias, seed):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    t = dict(x=torch.randn(T, D, generator=gen).to(xt), w=(0.5 * torch.randn(D, W, generator=gen)).to(wt),
             b=(0.5 * torch.randn(D, generator=gen)).to(wt) if bias else None,
             s0=torch.randn(N, W - 1, D, generator=gen).to(xt), dy=torch.randn(T, D, generator=gen).to(xt),
             dfin=torch.randn(N, W - 1, D, generator=gen).to(xt))
    return {k: None if v is None else v.to(dev()) for k, v in t.items()}


def check(t, lens, act="silu", cu=None, views=None, state=True):
    v = dict(t, **(views or {}))
    cu = cu_of(lens) if cu is None else cu
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    s0, dfin = (t["s0"], t["dfin"]) if state else (None, None)
    y, fin = la.sconv_fwd(v["x"], t["w"], cu, t["b"], activation=act, initial_state=s0, status=status)
    dx, dw, db, ds0 = la.sconv_bwd(v["x"], t["w"], cu, v["dy"], t["b"], activation=act, initial_state=s0,
                                   d_final_state=dfin, status=status)
    assert la.read_status(status) == 0
    args = [R.f64(t["x"]), R.f64(t["w"]), R.f64(t["b"]), lens, R.f64(s0), R.f64(t["dy"]), R.f64(dfin)]
    ref, sc = R.sconv(*args, activation=act), R.sconv(*args, activation=act, absolute=True)
    xt, wt, T = t["x"].dtype, t["w"].dtype, sum(lens)
    R.within("y", y, ref[0], xt, 32, sc[0])
    assert np.array_equal(R.f64(fin), ref[1])  # copies of inputs
    R.within("dx", dx, ref[2], xt, 32, sc[2])
    R.within("dw", dw, ref[3], wt, 32 + T, sc[3])
    R.within("db", db, ref[4], wt, 32 + T, sc[4])
    R.within("d_initial_state", ds0, ref[5], xt, 32, sc[5])
    return y, fin, dx, dw, db, ds0


LENGTHS = {"one token": [1], "empty": [0, 0], "mixed": [1, 0, 2, 3, 127, 128, 129, 0, 64, 300, 4],
           "long": [1500], "many short": [3] * 70}


@pytest.mark.parametrize("lens", LENGTHS.values(), ids=LENGTHS.keys())
@pytest.mark.parametrize("D", [1, 8, 63, 64, 264])
def test_lengths_and_widths(lens, D):
    check(draw(lens, D, 4, BF, F32, True, seed=D), lens)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("xt,wt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("act,bias", [("silu", True), ("none", False), ("sigmoid", True)])
def test_forms(W, xt, wt, act, bias):
    lens = [130, 1, 0, 2, 260]
    check(draw(lens, 72, W, xt, wt, bias, seed=W), lens, act)
    check(draw(lens, 72, W, xt, wt, bias, seed=W), lens, act, state=False)


def test_int64_boundaries():
    lens = [700, 0, 33]
    check(draw(lens, 64, 4, BF, BF, False, seed=1), lens, cu=cu_of(lens, torch.int64))


@pytest.mark.parametrize("D", [64, 66])
def test_views(D):
    """x as a column slice of a projection at odd and aligned offsets, a broadcast gradient, a strided result."""
    lens = [150, 3, 200]
    t = draw(lens, D, 4, BF, F32, True, seed=2)
    packed = check(t, lens)
    T = sum(lens)
    for shift in (1, 8):
        wide = torch.full((T, D + 16 + shift), float("nan"), dtype=BF, device=dev())
        x = wide[:, shift:shift + D]
        x.copy_(t["x"])
        got = check(t, lens, views=dict(x=x))
        assert all(torch.equal(a, b) for a, b in zip(got, packed))
        out = torch.full((T, D + 16 + shift), 7.0, dtype=BF, device=dev())
        y, _ = la.sconv_fwd(x, t["w"], cu_of(lens), t["b"], initial_state=t["s0"], y=out[:, shift:shift + D])
        assert torch.equal(y, packed[0]) and bool((out[:, :shift] == 7).all()) and bool((out[:, shift + D:] == 7).all())
    t["dy"] = t["dy"][:1].expand(T, D).contiguous()
    check(t, lens, views=dict(dy=t["dy"][:1].expand(T, D)))


def test_rows_do_not_depend_on_the_batch():
    lens = [1, 500, 0, 131, 77]
    t = draw(lens, 64, 4, BF, F32, False, seed=3)
    y, fin, dx, _, _, ds0 = check(t, lens)
    for i, L in enumerate(lens):
        a = sum(lens[:i])
        y1, fin1 = la.sconv_fwd(t["x"][a:a + L], t["w"], cu_of([L]), initial_state=t["s0"][i:i + 1])
        dx1, _, _, ds1 = la.sconv_bwd(t["x"][a:a + L], t["w"], cu_of([L]), t["dy"][a:a + L],
                                      initial_state=t["s0"][i:i + 1], d_final_state=t["dfin"][i:i + 1])
        assert torch.equal(y1, y[a:a + L]) and torch.equal(fin1, fin[i:i + 1])
        assert torch.equal(dx1, dx[a:a + L]) and torch.equal(ds1, ds0[i:i + 1])


def test_nan_reaches_only_its_taps():
    lens = [100, 200]
    t = draw(lens, 64, 4, BF, F32, False, seed=4)
    clean, _ = la.sconv_fwd(t["x"], t["w"], cu_of(lens))
    t["x"][98, 7] = float("nan")
    t["x"][150, 9] = float("nan")
    got, _ = la.sconv_fwd(t["x"], t["w"], cu_of(lens))
    same = torch.ones_like(got, dtype=torch.bool)
    same[98:100, 7] = False  # not into the next sequence
    same[150:154, 9] = False
    assert torch.equal(got[same], clean[same]) and bool(torch.isnan(got[~same].float()).all())
    # backwards: dx_t reads dp_t .. dp_{t+3}, and dp is NaN where y is
    dx = la.sconv_bwd(t["x"], t["w"], cu_of(lens), t["dy"])[0].float()
    same[95:98, 7] = same[147:150, 9] = False
    assert bool(torch.isfinite(dx[same]).all()) and bool(torch.isnan(dx[~same]).all())


@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("D", [64, 67])
def test_state_pool_prefill_and_decode(W, D):
    """A prefill into pool slots followed by single tokens equals one run over the whole sequences."""
    lens, P, steps = [130, 0, 1, 2, 515], 9, 5
    full = [L + steps for L in lens]
    t = draw(full, D, W, BF, BF, True, seed=5)
    idx = torch.tensor([4, 0, 8, 2, 1], dtype=torch.int32, device=dev())
    pool = torch.randn(P, W - 1, D, generator=torch.Generator().manual_seed(2)).to(BF).to(dev())
    before = pool.clone()
    pool[idx.long()] = t["s0"]
    want, fin = la.sconv_fwd(t["x"], t["w"], cu_of(full), t["b"], initial_state=t["s0"])
    starts = np.concatenate([[0], np.cumsum(full)])
    rows = torch.cat([torch.arange(s, s + L) for s, L in zip(starts, lens)]).to(dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    y, none = la.sconv_fwd(t["x"][rows], t["w"], cu_of(lens), t["b"], initial_state=pool, state_indices=idx, status=status)
    assert none is None and torch.equal(y, want[rows])
    for k in range(steps):
        at = torch.tensor([s + L + k for s, L in zip(starts, lens)], device=dev())
        assert torch.equal(la.sconv_decode(t["x"][at], t["w"], pool, t["b"], state_indices=idx, status=status), want[at])
    assert la.read_status(status) == 0
    assert torch.equal(pool[idx.long()], fin)
    others = [i for i in range(P) if i not in idx.tolist()]
    assert torch.equal(pool[others], before[others])


@pytest.mark.parametrize("xt", [BF, F32])
def test_decode_without_indices(xt):
    t = draw([1] * 37, 130, 3, xt, F32, False, seed=6)
    pool = t["s0"].clone()
    y = la.sconv_decode(t["x"], t["w"], pool, activation="none")
    args = (R.f64(t["x"]), R.f64(t["w"]), None, [1] * 37, R.f64(t["s0"]))
    ref, sc = R.sconv(*args, activation="none"), R.sconv(*args, absolute=True)
    R.within("y", y, ref[0], xt, 32, sc[0])
    assert np.array_equal(R.f64(pool), ref[1])


def test_device_side_errors():
    t = draw([100, 200], 64, 4, BF, F32, False, seed=1)
    for cu in ([0, 250, 200], [1, 100, 300], [0, 100, 299], [0, 100, 301], [0, -5, 300], [0, 100000, 300]):
        status = torch.zeros(1, dtype=torch.int32, device=dev())
        c = torch.tensor(cu, dtype=torch.int32, device=dev())
        la.sconv_fwd(t["x"], t["w"], c, status=status)
        assert la.read_status(status) == la.binding.LA_ERR_BAD_SEQLENS, cu
        status.zero_()
        la.sconv_bwd(t["x"], t["w"], c, t["dy"], status=status)
        assert la.read_status(status) == la.binding.LA_ERR_BAD_SEQLENS, cu
    for bad in (-1, 4, 2 ** 31 - 1):
        pool = torch.ones(4, 3, 64, dtype=BF, device=dev())
        idx = torch.tensor([1, bad], dtype=torch.int32, device=dev())
        status = torch.zeros(1, dtype=torch.int32, device=dev())
        la.sconv_decode(t["x"][:2], t["w"], pool, state_indices=idx, status=status)
        assert la.read_status(status) == la.binding.LA_ERR_BAD_STATE_INDEX
        status.zero_()
        la.sconv_fwd(t["x"], t["w"], cu_of([100, 200]), initial_state=pool, state_indices=idx, status=status)
        assert la.read_status(status) == la.binding.LA_ERR_BAD_STATE_INDEX
        assert bool((pool[[0, 2, 3]] == 1).all())


def test_autograd_and_repeatability():
    lens = [700, 0, 9]
    t = draw(lens, 64, 4, F32, F32, True, seed=7)
    x, w, b, s0 = (t[k].clone().requires_grad_() for k in ("x", "w", "b", "s0"))
    y, fin = la.short_conv(x, w, cu_of(lens), b, initial_state=s0)
    got = torch.autograd.grad((y * t["dy"]).sum() + (fin * t["dfin"]).sum(), (x, w, b, s0))
    want = la.sconv_bwd(t["x"], t["w"], cu_of(lens), t["dy"], t["b"], initial_state=t["s0"], d_final_state=t["dfin"])
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    dx, = torch.autograd.grad(la.short_conv(x, w, cu_of(lens))[0].sum(), (x,))
    assert torch.equal(dx, la.sconv_bwd(t["x"], t["w"], cu_of(lens), torch.ones_like(t["x"]))[0])


def test_graph_and_stream():
    lens = [300, 41]
    t, u = draw(lens, 64, 4, BF, F32, True, seed=8), draw(lens, 64, 4, BF, F32, True, seed=9)
    cu = cu_of(lens)

    def both(v, **kw):
        return la.sconv_fwd(v["x"], v["w"], cu, v["b"], initial_state=v["s0"], **kw) + \
            la.sconv_bwd(v["x"], v["w"], cu, v["dy"], v["b"], initial_state=v["s0"], **kw)

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
    t = draw([4], 8, 4, BF, F32, True, seed=1)
    cu, x, w = cu_of([4]), t["x"], t["w"]
    with pytest.raises(TypeError):
        la.sconv_fwd(x.half(), w, cu)
    with pytest.raises(TypeError):
        la.sconv_fwd(x, w.half(), cu)
    with pytest.raises(ValueError):
        la.sconv_fwd(x, w[:4], cu)
    with pytest.raises(la.binding.LinAttnError):
        la.sconv_fwd(x, torch.zeros(8, 5, device=dev()), cu)
    with pytest.raises(TypeError):
        la.sconv_fwd(x, w, cu, initial_state=t["s0"].float())
    with pytest.raises(ValueError):
        la.sconv_fwd(x, w, cu, activation="tanh")
    with pytest.raises(ValueError):
        la.sconv_fwd(x, w, cu, state_indices=torch.zeros(1, dtype=torch.int32, device=dev()))
    with pytest.raises(ValueError):
        la.sconv_decode(x, w, torch.zeros(4, 2, 8, dtype=BF, device=dev()))
    with pytest.raises(TypeError):
        la.sconv_bwd(x, w, cu, t["dy"].float())
