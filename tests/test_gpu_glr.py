"""The gated linear recurrence on the GPU against its 64-bit form.

Bounds (fixed before the first run): an output is rounded once to its type; before that every step of the
recurrence is off by at most 16 units of 2^-24 of the running error scale (expf and expm1f by 2 units of their
last place, the gate's few operations, the products and sums, the joining of blocks)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_29_gb300 as la
import mixer_reference as R

pytestmark = pytest.mark.gpu

UNITS = 16
BF, F32 = torch.bfloat16, torch.float32
GATES = {"log": {}, "logsigmoid": {"gate_logsigmoid": True}, "bound": {"gate_lower_bound": -0.5}}
REF = {"log": {}, "logsigmoid": {"logsigmoid": True}, "bound": {"lower_bound": -0.5}}


def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def cu_of(lens, dtype=torch.int32):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=dtype, device=dev())


def draw(lens, D, xt, gt, gate, seed):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    g = torch.randn(T, D, generator=gen)
    if gate == "log":
        g = -torch.nn.functional.softplus(g)
        g[:, 1::2] *= 0.01
    elif gate == "logsigmoid":
        g = g + 3
    t = dict(x=torch.randn(T, D, generator=gen).to(xt), g=g.to(gt), s0=torch.randn(N, D, generator=gen),
             dh=torch.randn(T, D, generator=gen).to(xt), dfin=torch.randn(N, D, generator=gen))
    return {k: v.to(dev()) for k, v in t.items()}


def check(t, lens, gate, complement, cu=None, checkpoints=True, x=None, g=None, dh=None):
    """Forward and backward of one batch; x, g, dh replace the packed operands by views of the same values."""
    kw = dict(GATES[gate], complement_input=complement)
    ref_kw = dict(REF[gate], complement=complement)
    x, g, dh = (t[k] if v is None else v for k, v in (("x", x), ("g", g), ("dh", dh)))
    cu = cu_of(lens) if cu is None else cu
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    h, fin, ck = la.glr_fwd(x, g, cu, initial_state=t["s0"], output_checkpoints=checkpoints, status=status, **kw)
    dx, dg, ds0 = la.glr_bwd(x, g, cu, dh, initial_state=t["s0"], d_final_state=t["dfin"], checkpoints=ck,
                             status=status, **kw)
    assert la.read_status(status) == 0
    xs, gs, s0, dhs, dfin = (R.f64(t[k]) for k in ("x", "g", "s0", "dh", "dfin"))
    rh, rfin = R.glr_fwd(xs, gs, lens, s0, **ref_kw)
    rdx, rdg, rds0 = R.glr_bwd(xs, gs, lens, dhs, s0, dfin, **ref_kw)
    sh, sfin, sdx, sdg, sds0 = R.glr_scales(xs, gs, lens, s0, dhs, dfin, **ref_kw)
    R.within("h", h, rh, x.dtype, UNITS, sh)
    R.within("final_state", fin, rfin, F32, UNITS, sfin)
    R.within("dx", dx, rdx, x.dtype, UNITS, sdx)
    R.within("dg", dg, rdg, g.dtype, UNITS, sdg)
    R.within("d_initial_state", ds0, rds0, F32, UNITS, sds0)
    return h, fin, dx, dg, ds0


LENGTHS = {"one token": [1], "empty": [0, 0], "mixed": [1, 0, 127, 128, 129, 0, 64, 300, 2],
           "long": [2500], "many short": [3] * 70}


@pytest.mark.parametrize("lens", LENGTHS.values(), ids=LENGTHS.keys())
@pytest.mark.parametrize("D", [1, 2, 63, 64, 130])
def test_lengths_and_widths(lens, D):
    check(draw(lens, D, BF, F32, "log", seed=D + len(lens)), lens, "log", False)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("xt,gt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_types_and_gates(xt, gt, gate, complement):
    lens = [200, 5, 0, 391]
    check(draw(lens, 96, xt, gt, gate, seed=7), lens, gate, complement)


@pytest.mark.parametrize("xt,gt", [(BF, BF), (BF, F32), (F32, F32)])
def test_many_blocks(xt, gt):
    """Two sequences of more blocks than any group of them, slow decays: states travel through all."""
    lens = [6300, 5111]
    check(draw(lens, 72, xt, gt, "log", seed=11), lens, "log", True)


def test_no_initial_state_no_checkpoints_int64():
    lens = [700, 0, 33]
    t = draw(lens, 64, BF, F32, "log", seed=3)
    cu = cu_of(lens, torch.int64)
    h, fin, ck = la.glr_fwd(t["x"], t["g"], cu)
    assert ck is None
    dx, dg, ds0 = la.glr_bwd(t["x"], t["g"], cu, t["dh"])
    xs, gs, dhs = (R.f64(t[k]) for k in ("x", "g", "dh"))
    rh, rfin = R.glr_fwd(xs, gs, lens)
    rdx, rdg, rds0 = R.glr_bwd(xs, gs, lens, dhs)
    sh, sfin, sdx, sdg, sds0 = R.glr_scales(xs, gs, lens, None, dhs)
    R.within("h", h, rh, BF, UNITS, sh)
    R.within("final_state", fin, rfin, F32, UNITS, sfin)
    R.within("dx", dx, rdx, BF, UNITS, sdx)
    R.within("dg", dg, rdg, F32, UNITS, sdg)
    R.within("d_initial_state", ds0, rds0, F32, UNITS, sds0)
    # the kept and the recomputed states are the same bits
    _, _, ck = la.glr_fwd(t["x"], t["g"], cu, output_checkpoints=True)
    again = la.glr_bwd(t["x"], t["g"], cu, t["dh"], checkpoints=ck)
    assert all(torch.equal(a, b) for a, b in zip((dx, dg, ds0), again))


def test_strided_and_unaligned_views():
    """Column slices of one projection, a base that is only element-aligned, odd strides, a broadcast cotangent."""
    lens = [150, 260]
    t = draw(lens, 66, BF, BF, "logsigmoid", seed=5)
    T, D = t["x"].shape
    wide = torch.full((T, 2 * D + 3), float("nan"), dtype=BF, device=dev())
    wide[:, 1:1 + D] = t["x"]
    wide[:, 2 + D:2 + 2 * D] = t["g"]
    t["dh"] = t["dh"][:1].expand(T, D).contiguous()
    got = check(t, lens, "logsigmoid", True, x=wide[:, 1:1 + D], g=wide[:, 2 + D:2 + 2 * D], dh=t["dh"][:1].expand(T, D))
    packed = check(t, lens, "logsigmoid", True)
    assert all(torch.equal(a, b) for a, b in zip(got, packed))
    out = torch.full((T, D + 5), 7.0, dtype=BF, device=dev())
    la.glr_fwd(t["x"], t["g"], cu_of(lens), initial_state=t["s0"], h=out[:, 3:3 + D], gate_logsigmoid=True,
               complement_input=True)
    assert torch.equal(out[:, 3:3 + D], packed[0]) and bool((out[:, :3] == 7).all()) and bool((out[:, 3 + D:] == 7).all())


def test_batch_invariance():
    """A sequence's results are the same bits alone and inside a batch."""
    lens = [1, 500, 0, 131, 4000, 77]
    t = draw(lens, 64, BF, F32, "log", seed=9)
    kw = dict(complement_input=True)
    h, fin, ck = la.glr_fwd(t["x"], t["g"], cu_of(lens), initial_state=t["s0"], output_checkpoints=True, **kw)
    dx, dg, ds0 = la.glr_bwd(t["x"], t["g"], cu_of(lens), t["dh"], initial_state=t["s0"], checkpoints=ck,
                             d_final_state=t["dfin"], **kw)
    for i, L in enumerate(lens):
        a = sum(lens[:i])
        x, g, dh = (t[k][a:a + L] for k in ("x", "g", "dh"))
        h1, fin1, _ = la.glr_fwd(x, g, cu_of([L]), initial_state=t["s0"][i:i + 1], **kw)
        dx1, dg1, ds1 = la.glr_bwd(x, g, cu_of([L]), dh, initial_state=t["s0"][i:i + 1],
                                   d_final_state=t["dfin"][i:i + 1], **kw)
        for whole, alone in ((h[a:a + L], h1), (fin[i:i + 1], fin1), (dx[a:a + L], dx1), (dg[a:a + L], dg1),
                             (ds0[i:i + 1], ds1)):
            assert torch.equal(whole, alone)


def test_nan_stays_in_its_sequence_and_channel_and_minus_infinity_resets():
    lens = [140, 300, 20]
    t = draw(lens, 64, BF, F32, "log", seed=13)
    clean = la.glr_fwd(t["x"], t["g"], cu_of(lens), initial_state=t["s0"])[0]
    t["x"][141 + 9, 5] = float("nan")
    got = la.glr_fwd(t["x"], t["g"], cu_of(lens), initial_state=t["s0"])[0]
    same = torch.ones_like(got, dtype=torch.bool)
    same[141 + 9:440, 5] = False
    assert torch.equal(got[same], clean[same]) and bool(torch.isnan(got[141 + 9:440, 5].float()).all())
    # a = 0: the state before has no part in what follows, in either direction
    t = draw(lens, 64, BF, F32, "log", seed=13)
    t["g"][200] = float("-inf")
    check(t, lens, "log", False)


@pytest.mark.parametrize("pool_dtype", [F32, BF])
def test_state_pool_prefill_and_decode(pool_dtype):
    """A prefill into pool slots followed by single tokens equals one run over the whole sequences."""
    lens, D, P, steps = [130, 0, 1, 515], 70, 9, 3
    t = draw([L + steps for L in lens], D, BF, F32, "bound", seed=21)
    kw = dict(GATES["bound"], complement_input=True)
    idx = torch.tensor([4, 0, 8, 2], dtype=torch.int32, device=dev())
    pool = torch.randn(P, D, generator=torch.Generator().manual_seed(2)).to(pool_dtype).to(dev())
    before = pool.clone()
    starts = np.concatenate([[0], np.cumsum([L + steps for L in lens])])
    rows = torch.cat([torch.arange(s, s + L) for s, L in zip(starts, lens)]).to(dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    h, fin, _ = la.glr_fwd(t["x"][rows], t["g"][rows], cu_of(lens), initial_state=pool, state_indices=idx, status=status, **kw)
    assert fin is None
    state = R.f64(before[idx.long()])
    rk = dict(REF["bound"], complement=True)
    xs, gs = R.f64(t["x"]), R.f64(t["g"])
    rr = rows.cpu().numpy()
    rh, rfin = R.glr_fwd(xs[rr], gs[rr], lens, state, **rk)
    sh, sfin = R.glr_scales(xs[rr], gs[rr], lens, state, **rk)
    R.within("h", h, rh, BF, UNITS, sh)
    R.within("pool", pool[idx.long()], rfin, pool_dtype, UNITS, sfin)
    for k in range(steps):
        at = torch.tensor([s + L + k for s, L in zip(starts, lens)], device=dev())
        state = R.f64(pool[idx.long()])
        y = la.glr_decode(t["x"][at], t["g"][at], pool, state_indices=idx, status=status, **kw)
        ones = [1] * len(lens)
        aa = at.cpu().numpy()
        rh, rfin = R.glr_fwd(xs[aa], gs[aa], ones, state, **rk)
        sh, sfin = R.glr_scales(xs[aa], gs[aa], ones, state, **rk)
        R.within("decode", y, rh, BF, UNITS, sh)
        R.within("pool", pool[idx.long()], rfin, pool_dtype, UNITS, sfin)
    assert la.read_status(status) == 0
    others = [i for i in range(P) if i not in idx.tolist()]
    assert torch.equal(pool[others], before[others])


@pytest.mark.parametrize("N,D", [(1, 1), (3, 33), (130, 64)])
@pytest.mark.parametrize("gt", [BF, F32])
def test_decode_without_indices(N, D, gt):
    t = draw([1] * N, D, F32, gt, "logsigmoid", seed=N)
    pool = t["s0"].clone()
    y = la.glr_decode(t["x"], t["g"], pool, gate_logsigmoid=True)
    args = (R.f64(t["x"]), R.f64(t["g"]), [1] * N, R.f64(t["s0"]))
    rh, rfin = R.glr_fwd(*args, logsigmoid=True)
    sh, sfin = R.glr_scales(*args, logsigmoid=True)
    R.within("h", y, rh, F32, UNITS, sh)
    R.within("pool", pool, rfin, F32, UNITS, sfin)


def test_device_side_errors():
    """Invalid cu_seqlens and slots outside the pool set the status word; every access stays inside the operands and
    the other sequences' slots keep their values."""
    t = draw([100, 200], 64, BF, F32, "log", seed=1)
    for cu in ([0, 250, 200], [1, 100, 300], [0, 100, 299], [0, 100, 301], [0, -5, 300], [0, 100000, 300]):
        status = torch.zeros(1, dtype=torch.int32, device=dev())
        c = torch.tensor(cu, dtype=torch.int32, device=dev())
        la.glr_fwd(t["x"], t["g"], c, status=status)
        assert la.read_status(status) == la.binding.LA_ERR_BAD_SEQLENS, cu
        status.zero_()
        la.glr_bwd(t["x"], t["g"], c, t["dh"], status=status)
        assert la.read_status(status) == la.binding.LA_ERR_BAD_SEQLENS, cu
    for bad in (-1, 4, 2 ** 31 - 1):
        pool = torch.ones(4, 64, device=dev())
        idx = torch.tensor([1, bad], dtype=torch.int32, device=dev())
        status = torch.zeros(1, dtype=torch.int32, device=dev())
        la.glr_decode(t["x"][:2], t["g"][:2], pool, state_indices=idx, status=status)
        assert la.read_status(status) == la.binding.LA_ERR_BAD_STATE_INDEX
        assert torch.equal(pool[[0, 2, 3]], torch.ones(3, 64, device=dev()))
        status.zero_()
        la.glr_fwd(t["x"], t["g"], cu_of([100, 200]), initial_state=pool, state_indices=idx, status=status)
        assert la.read_status(status) == la.binding.LA_ERR_BAD_STATE_INDEX
        assert torch.equal(pool[[0, 2, 3]], torch.ones(3, 64, device=dev()))


def test_wrapper_refusals():
    t = draw([4], 8, BF, F32, "log", seed=1)
    cu, x, g = cu_of([4]), t["x"], t["g"]
    with pytest.raises(TypeError):
        la.glr_fwd(x.half(), g, cu)
    with pytest.raises(ValueError):
        la.glr_fwd(x, g[:3], cu)
    with pytest.raises(ValueError):
        la.glr_fwd(x[:, ::2], g[:, ::2], cu)
    with pytest.raises(TypeError):
        la.glr_fwd(x, g, cu.float())
    with pytest.raises(ValueError):
        la.glr_fwd(x, g, cu, gate_logsigmoid=True, gate_lower_bound=-1.0)
    with pytest.raises(la.binding.LinAttnError):
        la.glr_fwd(x, g, cu, gate_lower_bound=1.0)
    with pytest.raises(ValueError):
        la.glr_fwd(x, g, cu, initial_state=torch.zeros(2, 8, device=dev()))
    with pytest.raises(ValueError):
        la.glr_fwd(x, g, cu, state_indices=torch.zeros(1, dtype=torch.int32, device=dev()))
    with pytest.raises(TypeError):
        la.glr_bwd(x, g, cu, t["dh"].float())
    with pytest.raises(ValueError):
        la.glr_bwd(x, g, cu, t["dh"], checkpoints=torch.zeros(3, 8, device=dev()))
    with pytest.raises(ValueError):
        la.glr_decode(x, g, torch.zeros(4, 9, device=dev()))


@pytest.mark.parametrize("save", [True, False])
def test_autograd(save):
    lens = [150, 0, 7]
    t = draw(lens, 40, F32, F32, "logsigmoid", seed=4)
    x, g, s0 = (t[k].clone().requires_grad_() for k in ("x", "g", "s0"))
    h, fin = la.gated_linear_recurrence(x, g, cu_of(lens), initial_state=s0, gate_logsigmoid=True,
                                        save_checkpoints=save)
    got = torch.autograd.grad((h * t["dh"]).sum() + (fin * t["dfin"]).sum(), (x, g, s0))
    want = la.glr_bwd(t["x"], t["g"], cu_of(lens), t["dh"], initial_state=t["s0"], d_final_state=t["dfin"],
                      gate_logsigmoid=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # an expanded cotangent, and an output that nothing uses
    h, fin = la.gated_linear_recurrence(x, g, cu_of(lens), gate_logsigmoid=True)
    dx, = torch.autograd.grad(h.sum(), (x,))
    assert torch.equal(dx, la.glr_bwd(t["x"], t["g"], cu_of(lens), torch.ones_like(t["x"]), gate_logsigmoid=True)[0])
    h, fin = la.gated_linear_recurrence(x, g, cu_of(lens), gate_logsigmoid=True)
    dx, = torch.autograd.grad(fin.sum(), (x,))
    assert torch.equal(dx, la.glr_bwd(t["x"], t["g"], cu_of(lens), torch.zeros_like(t["x"]), gate_logsigmoid=True,
                                      d_final_state=torch.ones_like(t["dfin"]))[0])


def test_other_stream_and_graph():
    """On a stream of its own, and captured into a graph that is replayed on new inputs."""
    lens = [900, 41]
    t = draw(lens, 64, BF, F32, "log", seed=17)
    u = draw(lens, 64, BF, F32, "log", seed=18)
    cu = cu_of(lens)

    def both(v, **kw):
        h, fin, ck = la.glr_fwd(v["x"], v["g"], cu, initial_state=v["s0"], output_checkpoints=True, **kw)
        return (h, fin) + la.glr_bwd(v["x"], v["g"], cu, v["dh"], initial_state=v["s0"], checkpoints=ck, **kw)

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
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    for k in t:
        t[k].copy_(u[k])
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want_u))
