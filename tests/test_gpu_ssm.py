"""The selective scan on the GPU against its 64-bit form.

Bounds (fixed before the first run): an output is rounded once to its type; before that it is off by at most twice the
first-order bound of ssm_scales (block_reference.py), the two being for what products of errors and the joining of time
blocks add."""
import numpy as np
import pytest
import torch

import block_reference as R
import gated_delta_rule_29_gb300 as la
from gated_delta_rule_29_gb300 import binding as B

pytestmark = pytest.mark.gpu

UNITS = 2
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dx", "ddt", "da", "db", "dc", "d_skip", "dz", "d_dt_bias", "d_initial_state")


def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def cu_of(lens, dtype=torch.int32):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=dtype, device=dev())


def draw(lens, D, S, G=1, xt=BF, seed=1, z=True, skip=True, softplus=True, slow=False):
    """Operands as a model has them: rates from -1 to -S, steps around 1/30 (or 1/1000, slow) by softplus of a bias."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)

    def randn(*shape):
        return torch.randn(*shape, generator=gen)

    step = (1e-3 if slow else 0.03) * torch.exp(randn(D))
    t = dict(x=randn(T, D).to(xt), b=randn(T, G, S).to(xt), c=randn(T, G, S).to(xt),
             a=-torch.arange(1, S + 1) * torch.exp(0.3 * randn(D, S)), s0=randn(N, D, S), dy=randn(T, D).to(xt), dfin=randn(N, D, S))
    if softplus:
        t["dt"], t["bias"] = randn(T, D).to(xt), step + torch.log(-torch.expm1(-step))
    else:
        t["dt"] = (step * torch.exp(0.5 * randn(T, D))).to(xt)
    if skip:
        t["skip"] = 1 + 0.1 * randn(D)
    if z:
        t["z"] = randn(T, D).to(xt)
    return {k: v.to(dev()) for k, v in t.items()}


def call(t, cu, checkpoints=True, backward=True, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    ops = [t[k] for k in ("x", "dt", "a", "b", "c")] + [cu]
    opts = dict(skip=t.get("skip"), z=t.get("z"), dt_bias=t.get("bias"), dt_softplus="bias" in t, status=status)
    y, fin, ck = la.ssm_fwd(*ops, initial_state=t.get("s0"), output_checkpoints=checkpoints, **opts, **kw)
    out = (y, fin)
    if backward:
        out += la.ssm_bwd(*ops, t["dy"], initial_state=t.get("s0"), d_final_state=t.get("dfin"), checkpoints=ck, **opts)
    assert la.read_status(status) == 0
    return out


def reference(t, lens, backward=True, scales=False):
    v = {k: R.f64(t.get(k)) for k in ("x", "dt", "a", "b", "c", "skip", "z", "bias", "s0", "dy", "dfin")}
    for k in ("b", "c"):
        v[k] = v[k][:, None] if v[k].ndim == 2 else v[k]
    if not backward:
        v["dy"] = v["dfin"] = None
    return (R.ssm_scales if scales else R.ssm)(v.pop("x"), v.pop("dt"), v.pop("a"), v.pop("b"), v.pop("c"), lens,
                                               use_softplus="bias" in t, **v)


def compare(got, t, lens, backward=True):
    ref, scale = reference(t, lens, backward), reference(t, lens, backward, scales=True)
    xt = t["x"].dtype
    types = (xt, F32, xt, xt, F32, xt, xt, F32, xt, F32, F32)
    for name, g, r, s, ty in zip(("y", "final_state") + NAMES, got, ref, scale, types):
        if r is not None and g is not None and g.shape != r.shape:
            g = g.reshape(r.shape)
        R.within(name, g, r, ty, UNITS, s)


LENGTHS = {"one token": [1], "empty": [0, 0], "mixed": [1, 0, 31, 32, 33, 0, 64, 300, 2], "long": [1500], "many short": [3] * 70}


@pytest.mark.parametrize("lens", LENGTHS.values(), ids=LENGTHS.keys())
@pytest.mark.parametrize("D", [1, 2, 33, 130])
def test_lengths_and_widths(lens, D):
    t = draw(lens, D, 16, seed=D + len(lens))
    compare(call(t, cu_of(lens)), t, lens)


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("S", [1, 3, 4, 5, 8, 9, 16, 23, 32, 33, 64])
def test_state_sizes(S, xt):
    lens = [70, 0, 45]
    t = draw(lens, 40, S, G=2, xt=xt, seed=S)
    compare(call(t, cu_of(lens)), t, lens)


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("opts", [dict(z=False), dict(skip=False), dict(softplus=False), dict(z=False, skip=False, softplus=False)],
                         ids=lambda o: "-".join("no_" + k for k in o))
@pytest.mark.parametrize("G", [1, 3])
def test_options_and_types(opts, xt, G):
    lens = [100, 5, 0, 91]
    t = draw(lens, 96, 16, G=G, xt=xt, seed=7, **opts)
    compare(call(t, cu_of(lens)), t, lens)


@pytest.mark.parametrize("time_block", [0, 64, 256])
def test_split_along_time(time_block):
    """Slow states that travel through many blocks."""
    lens = [1300, 0, 64, 65, 700]
    t = draw(lens, 36, 16, seed=11, slow=True)
    compare(call(t, cu_of(lens), time_block=time_block), t, lens)


def test_no_states_no_checkpoints_int64():
    lens = [300, 0, 33]
    t = draw(lens, 64, 16, seed=3)
    del t["s0"], t["dfin"]
    cu = cu_of(lens, torch.int64)
    got = call(t, cu, checkpoints=False, time_block=64)
    compare(got, t, lens)
    # the kept and the recomputed states are the same bits where the blocks are the same
    again = call(t, cu, checkpoints=False)
    kept = call(t, cu, checkpoints=True)
    assert all(torch.equal(a, b) for a, b in zip(again, kept))


def test_batch_invariance_and_repeats():
    """With a given block a sequence's results are the same bits alone and in a batch; the gradients always."""
    lens = [500, 33, 0, 1100]
    t = draw(lens, 70, 16, seed=5)
    whole = call(t, cu_of(lens), time_block=256)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(whole, call(t, cu_of(lens), time_block=256)))
    at = 0
    for i, L in enumerate(lens):
        one = {k: v[at:at + L].contiguous() if k in ("x", "dt", "b", "c", "z", "dy") else v[i:i + 1] if k in ("s0", "dfin") else v
               for k, v in t.items()}
        alone = call(one, cu_of([L]), time_block=256)
        for k in (0, 2, 3, 5, 6, 8):  # y, dx, ddt, db, dc, dz
            assert torch.equal(alone[k], whole[k][at:at + L]), k
        assert torch.equal(alone[1][0], whole[1][i]) and torch.equal(alone[10][0], whole[10][i])
        at += L


def test_strided_and_unaligned_views():
    """Column slices of one projection, a base that is only element-aligned, broadcast vectors and cotangents."""
    lens = [60, 45]
    t = draw(lens, 66, 16, seed=9)
    want = call(t, cu_of(lens))
    T, D = t["x"].shape
    v = dict(t)
    wide = torch.full((T, 4 * D + 37), float("nan"), dtype=BF, device=dev())
    for i, k in enumerate(("x", "dt", "z", "dy")):
        wide[:, 1 + i * D:1 + (i + 1) * D] = t[k]
        v[k] = wide[:, 1 + i * D:1 + (i + 1) * D]
    wide[:, 4 * D + 3:4 * D + 19] = t["b"][:, 0]
    v["b"] = wide[:, 4 * D + 3:4 * D + 19]
    got = call(v, cu_of(lens))
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(got, want))
    # one vector for every token and group
    t["b"], t["c"] = (t[k][:1].expand(T, 2, 16) for k in ("b", "c"))
    t["dy"] = t["dy"][:1].expand(T, D)
    compare(call(t, cu_of(lens)), t, lens)


def test_results_into_views_and_in_place():
    lens = [40, 90]
    t = draw(lens, 64, 16, seed=4)
    y, fin = call(t, cu_of(lens), backward=False)
    T, D = t["x"].shape
    buf = torch.full((T + 2, 2 * D), 7.0, dtype=BF, device=dev())
    got, fin2, _ = la.ssm_fwd(*[t[k] for k in "x dt a b c".split()], cu_of(lens), skip=t["skip"], z=t["z"], dt_bias=t["bias"],
                              dt_softplus=True, initial_state=t["s0"], y=buf[1:-1, 5:5 + D])
    assert torch.equal(got, y) and torch.equal(fin, fin2) and int((buf != 7).sum()) <= T * D
    for k in ("x", "dt", "z"):
        w = {n: v.clone() for n, v in t.items()}
        got, _, _ = la.ssm_fwd(*[w[n] for n in "x dt a b c".split()], cu_of(lens), skip=w["skip"], z=w["z"], dt_bias=w["bias"],
                               dt_softplus=True, initial_state=w["s0"], y=w[k], time_block=64)
        ref, _, _ = la.ssm_fwd(*[t[n] for n in "x dt a b c".split()], cu_of(lens), skip=t["skip"], z=t["z"], dt_bias=t["bias"],
                               dt_softplus=True, initial_state=t["s0"], time_block=64)
        assert got is w[k] and torch.equal(got, ref)


@pytest.mark.parametrize("pool_dtype", [F32, BF])
@pytest.mark.parametrize("time_block", [0, 64])
def test_state_pool(pool_dtype, time_block):
    lens = [100, 0, 37, 200]
    t = draw(lens, 48, 16, seed=6)
    idx = torch.tensor([5, 0, 3, 2], dtype=torch.int32, device=dev())
    pool = torch.randn(7, 48, 16, device=dev()).to(pool_dtype)
    before = pool.clone()
    t["s0"] = pool[idx.long()].clone()
    y, fin = call(t, cu_of(lens), backward=False, time_block=time_block)
    got, none, _ = la.ssm_fwd(*[t[k] for k in "x dt a b c".split()], cu_of(lens), skip=t["skip"], z=t["z"], dt_bias=t["bias"],
                              dt_softplus=True, initial_state=pool, state_indices=idx, time_block=time_block)
    assert none is None and torch.equal(got, y) and torch.equal(pool[idx.long()], fin.to(pool_dtype))
    rest = [1, 4, 6]
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("xt,pool_dtype", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("D,S,G", [(1, 1, 1), (40, 16, 2), (130, 23, 1), (33, 64, 3), (256, 4, 1)])
def test_decode(xt, pool_dtype, D, S, G):
    lens = [1] * 5
    t = draw(lens, D, S, G=G, xt=xt, seed=D)
    pool = torch.randn(9, D, S, device=dev()).to(pool_dtype)
    before = pool.clone()
    idx = torch.tensor([4, 8, 0, 3, 7], dtype=torch.int32, device=dev())
    t["s0"] = pool[idx.long()].float()
    y = la.ssm_decode(*[t[k] for k in "x dt a b c".split()], pool, state_indices=idx, skip=t["skip"], z=t["z"], dt_bias=t["bias"],
                      dt_softplus=True)
    ref, scale = reference(t, lens, False), reference(t, lens, False, scales=True)
    R.within("y", y, ref[0], xt, UNITS, scale[0])
    R.within("state", pool[idx.long()], ref[1], pool_dtype, UNITS, scale[1])
    assert torch.equal(pool[[1, 2, 5, 6]], before[[1, 2, 5, 6]])
    # without indices slot i, and no gate
    del t["z"]
    t["s0"] = before[:5].float().clone()
    y = la.ssm_decode(*[t[k] for k in "x dt a b c".split()], before, skip=t["skip"], dt_bias=t["bias"], dt_softplus=True)
    ref, scale = reference(t, lens, False), reference(t, lens, False, scales=True)
    R.within("y", y, ref[0], xt, UNITS, scale[0])
    R.within("state", before[:5], ref[1], pool_dtype, UNITS, scale[1])


@pytest.mark.parametrize("softplus", [False, True])
def test_a_bf16_pool_rounds_what_the_formula_gives(softplus):
    """The states that a token leaves in a bf16 pool are the formula's in 32 bits, operation by operation, rounded once: all
    of them, where the exponential and logarithm are the ones of elementary operations."""
    N, D, S = 37, 520, 16
    t = draw([1] * N, D, S, seed=11, xt=F32)
    pool = t["s0"].to(BF)
    raw = t["dt"] + t["bias"]
    step = raw if not softplus else torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    b = t["b"].reshape(N, 1, S)
    want = (torch.exp(step[:, :, None] * t["a"]) * pool.float() + (step * t["x"])[:, :, None] * b).to(BF)
    la.ssm_decode(t["x"], t["dt"], t["a"], t["b"], t["c"], pool, dt_bias=t["bias"], dt_softplus=softplus)
    assert torch.equal(pool, want)


def test_prefill_then_tokens_give_the_whole():
    lens = [50, 7, 90]
    t = draw(lens, 64, 16, xt=F32, seed=8)
    whole, fin = call(t, cu_of(lens), backward=False)
    N, k = len(lens), 5
    ends = cu_of(lens)[1:].long()
    first = torch.cat([torch.arange(int(e) - L, int(e) - k, device=dev()) for e, L in zip(ends, lens)])
    pool, idx = torch.zeros(N, 64, 16, device=dev()), torch.tensor([2, 0, 1], dtype=torch.int32, device=dev())
    pool[idx.long()] = t["s0"]
    opts = dict(skip=t["skip"], dt_bias=t["bias"], dt_softplus=True)
    la.ssm_fwd(*[t[n][first] if n != "a" else t[n] for n in "x dt a b c".split()], cu_of([L - k for L in lens]), z=t["z"][first],
               initial_state=pool, state_indices=idx, **opts)
    for i in range(k):
        at = ends - k + i
        y = la.ssm_decode(*[t[n][at] if n != "a" else t[n] for n in "x dt a b c".split()], pool, state_indices=idx, z=t["z"][at], **opts)
        # each is within 8 units per step of the running scale of the 64-bit value, and all values are of order 10
        assert float((y - whole[at]).abs().max()) <= 1e-4 * float(whole.abs().max())
    assert float((pool[idx.long()] - fin).abs().max()) <= 1e-4 * float(fin.abs().max())


def test_closed_and_extreme_steps():
    """Steps of 0, raw steps far from 0 either way, decays that underflow, gates that close."""
    lens = [64]
    t = draw(lens, 32, 16, xt=F32, seed=12)
    t["dt"][::7] = -200.0
    t["dt"][3::7] = 60.0
    t["z"][::5] = -200.0
    t["z"][2::5] = 300.0
    t["bias"][:4] = 0.0
    compare(call(t, cu_of(lens)), t, lens)
    t = draw(lens, 32, 16, xt=F32, seed=13, softplus=False)
    t["dt"][::3] = 0.0
    compare(call(t, cu_of(lens)), t, lens)


def test_not_a_number_stays_where_it_is():
    """A NaN in a channel's row reaches that channel from that token on and, of the shared vectors' gradients, that token's
    and those before; other channels, sequences and earlier tokens keep their bits."""
    lens = [40, 40]
    t = draw(lens, 64, 16, seed=2)
    good = call(t, cu_of(lens))
    t["x"][50, 9] = float("nan")
    bad = call(t, cu_of(lens))
    keep = torch.ones_like(good[0], dtype=torch.bool)
    keep[50:, 9] = False
    assert torch.equal(good[0][keep], bad[0][keep]) and bool(torch.isnan(bad[0][50:, 9]).all())
    assert torch.equal(good[5][:40], bad[5][:40])


def test_bad_boundaries_and_indices_set_the_status():
    lens = [40, 30]
    t = draw(lens, 32, 16, seed=3)
    opts = dict(skip=t["skip"], z=t["z"], dt_bias=t["bias"], dt_softplus=True)
    ops = [t[k] for k in "x dt a b c".split()]
    for cu in ([0, 50, 40], [0, 80, 70], [1, 40, 70], [0, 40, 60], [0, -5, 70]):
        for block in (0, 64):
            status = torch.zeros(1, dtype=torch.int32, device=dev())
            la.ssm_fwd(*ops, torch.tensor(cu, dtype=torch.int32, device=dev()), status=status, time_block=block, **opts)
            assert la.read_status(status) == B.LA_ERR_BAD_SEQLENS
        status = torch.zeros(1, dtype=torch.int32, device=dev())
        la.ssm_bwd(*ops, torch.tensor(cu, dtype=torch.int32, device=dev()), t["dy"], status=status, **opts)
        assert la.read_status(status) == B.LA_ERR_BAD_SEQLENS
    pool = torch.randn(4, 32, 16, device=dev())
    before = pool.clone()
    idx = torch.tensor([4, 1], dtype=torch.int32, device=dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    la.ssm_fwd(*ops, cu_of(lens), initial_state=pool, state_indices=idx, status=status, **opts)
    assert la.read_status(status) == B.LA_ERR_BAD_STATE_INDEX and torch.equal(pool[[0, 2, 3]], before[[0, 2, 3]])
    status.zero_()
    before = pool.clone()
    two = [v[:2] if v is not t["a"] else v for v in ops]
    la.ssm_decode(*two, pool, state_indices=torch.tensor([-1, 2], dtype=torch.int32, device=dev()), status=status, skip=t["skip"])
    assert la.read_status(status) == B.LA_ERR_BAD_STATE_INDEX and torch.equal(pool[[0, 1, 3]], before[[0, 1, 3]])


def test_nothing_to_do():
    t = draw([0, 0], 32, 16, seed=3)
    got = call(t, cu_of([0, 0]))
    assert got[0].shape == (0, 32) and torch.equal(got[1], t["s0"]) and torch.equal(got[10], t["dfin"])
    assert not got[4].any() and not got[7].any() and not got[9].any()
    empty = {k: v[:0] if k in ("s0", "dfin") else v for k, v in t.items()}
    got = call(empty, cu_of([]))
    assert got[1].shape == (0, 32, 16) and not got[4].any()
    y = la.ssm_decode(*[t[k] for k in "x dt a b c".split()], torch.zeros(2, 32, 16, device=dev()))
    assert y.shape == (0, 32)


def test_wrapper_refusals():
    t = draw([8], 32, 16, G=2, seed=3)
    ops, cu = [t[k] for k in "x dt a b c".split()], cu_of([8])

    def swap(i, v):
        return ops[:i] + [v] + ops[i + 1:]

    for args, error in ((swap(1, t["dt"].float()), TypeError), (swap(1, t["dt"][:, :31]), ValueError), (swap(2, t["a"].to(BF)), TypeError),
                        (swap(2, t["a"].t()), ValueError), (swap(3, t["b"].float()), TypeError), (swap(3, t["b"][:, :1]), ValueError),
                        (swap(3, t["b"][:4]), ValueError), (swap(0, t["x"].half()), TypeError)):
        with pytest.raises(error):
            la.ssm_fwd(*args, cu)
        with pytest.raises(error):
            la.ssm_bwd(*args, cu, t["dy"])
    three = [v[:, None, 0].expand(8, 3, 16) if v.dim() == 3 else v for v in ops]
    with pytest.raises(ValueError, match="multiple"):
        la.ssm_fwd(*three, cu)
    with pytest.raises(ValueError, match="time_block"):
        la.ssm_fwd(*ops, cu, time_block=100)
    with pytest.raises(B.LinAttnError):  # S above 64
        la.ssm_fwd(t["x"], t["dt"], torch.zeros(32, 65, device=dev()), *[torch.zeros(8, 65, dtype=BF, device=dev())] * 2, cu)
    with pytest.raises(ValueError):
        la.ssm_fwd(*ops, cu, z=t["z"][:4])
    with pytest.raises(ValueError):
        la.ssm_fwd(*ops, cu, state_indices=torch.zeros(1, dtype=torch.int32, device=dev()))
    with pytest.raises(B.LinAttnError):  # the next rows
        buf = torch.zeros(9, 32, dtype=BF, device=dev())
        la.ssm_fwd(*swap(0, buf[:8]), cu, y=buf[1:])


def test_rows_beyond_32_bits():
    """Operands whose last rows start more than 2^31 elements in."""
    T, D, S = 40, 64, 16
    t = draw([T], D, S, seed=21)
    want = call(t, cu_of([T]))
    stride = (1 << 31) // 32 + 8
    big = torch.empty(T * stride, dtype=BF, device=dev())
    v = dict(t)
    for i, k in enumerate(("x", "dt", "z", "dy")):
        v[k] = big.as_strided((T, D), (stride, 1), i * D)
        v[k].copy_(t[k])
    for i, k in enumerate(("b", "c")):
        v[k] = big.as_strided((T, 1, S), (stride, S, 1), 4 * D + i * S)
        v[k].copy_(t[k])
    got = call(v, cu_of([T]))
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(got, want))
    y = big.as_strided((T, D), (stride, 1), 5 * D)
    la.ssm_fwd(*[v[k] for k in "x dt a b c".split()], cu_of([T]), skip=t["skip"], z=v["z"], dt_bias=t["bias"], dt_softplus=True,
               initial_state=t["s0"], y=y)
    assert torch.equal(y, want[0])
