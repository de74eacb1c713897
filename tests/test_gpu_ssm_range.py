"""The selective scan at the ends of its range: sums over many tokens, states that grow."""
import numpy as np
import pytest
import torch

import block_reference as R
import gated_delta_rule_29_gb300 as la
from test_gpu_ssm import F32, UNITS, compare, cu_of, dev, draw
import test_gpu_ssm as S

pytestmark = pytest.mark.gpu


def test_sums_over_many_tokens():
    """Steady states under constant tokens, so that every token adds the same to dA, d_skip and d_dt_bias and a running sum is
    off by the same rounding again and again.  A sum goes over 64 tokens of a block, a part's blocks (52 here), the parts (5)
    and some threads: 128 additions at most in the way of a token, half a unit of 2^-23 each.  The terms themselves: the
    steady state and gradient are off by (8 + 6 roundings) / (1 - a), 28 units each for a = 1/2."""
    T, D = 16384, 8192
    gen = torch.Generator().manual_seed(1)

    def draw_one(lo, hi):
        return (lo + (hi - lo) * torch.rand(D, generator=gen)).to(dev())

    dt, x, dy, skip = draw_one(0.5, 1.0), draw_one(1.0, 2.0), draw_one(1.0, 2.0), draw_one(0.5, 1.0)
    bias = torch.zeros(D, device=dev())
    a = -np.log(2.0).astype(np.float32) / dt
    one = torch.ones(1, 1, 1, device=dev())
    A, d = a.double(), dt.double()
    f = torch.exp(d * A)
    h, e = d * x.double() / (1 - f), dy.double() / (1 - f)  # the steady state; the gradient of a state, with what comes back
    g = f * e
    t = dict(x=x.expand(T, D), dt=dt.expand(T, D), b=one.expand(T, 1, 1), c=one.expand(T, 1, 1), dy=dy.expand(T, D))
    cu = cu_of([T])
    s0, dfin = h.float()[None, :, None].contiguous(), g.float()[None, :, None].contiguous()
    da, d_skip, d_bias = (la.ssm_bwd(t["x"], t["dt"], a[:, None].contiguous(), t["b"], t["c"], cu, t["dy"], skip=skip, dt_bias=bias,
                                     initial_state=s0, d_final_state=dfin)[k] for k in (2, 5, 7))
    w = g * h
    for name, got, term, own in (("d_skip", d_skip, dy.double() * x.double(), 2), ("da", da[:, 0], w * d, 64),
                                 ("d_dt_bias", d_bias, e * x.double() + w * A, 2 * 64 * (w * A).abs() / (e * x.double() + w * A).abs() + 64)):
        off = (got.double() / (T * term) - 1).abs() * 2.0 ** 24
        assert bool((off <= 128 + own).all()), (name, float(off.max()))


@pytest.mark.parametrize("time_block", [64, 256])
def test_growing_states(time_block):
    """Rates above 0: a block's factor leaves the range, but the states it stands beside are 0 until the last tokens."""
    T, D, N = 600, 5, 4
    t = draw([T], D, N, xt=F32, seed=1, softplus=False, z=False)
    del t["s0"], t["dfin"]
    t["a"] = torch.full((D, N), 0.5, device=dev())
    t["a"][:, 1] = 2.0
    t["a"][:, 2] = -1.0
    t["dt"] = torch.ones_like(t["dt"])
    t["x"][:-10] = 0  # states are 0 up to here
    t["dy"][10:] = 0  # gradients are 0 from here on
    compare(S.call(t, cu_of([T]), time_block=time_block), t, [T])


def test_tiny_states_that_grow():
    """States of 1e-30 that grow by e^73 and e^90 in one block, the second being beyond the 32-bit range as a factor."""
    T, D, N = 3 * 256, 3, 2
    t = draw([T], D, N, xt=F32, seed=1, softplus=False, z=False)
    t["a"] = torch.full((D, N), 0.30, device=dev())
    t["a"][:, 1] = 0.37
    t["dt"] = torch.zeros_like(t["dt"])
    t["dt"][100:500] = 1.0
    t["x"].zero_()
    t["s0"] *= 1e-30
    t["dy"].zero_()
    t["dfin"] *= 1e-30
    got = S.call(t, cu_of([T]), backward=False, time_block=256)
    ref, scale = S.reference(t, [T], False), S.reference(t, [T], False, scales=True)
    assert np.isfinite(ref[1]).all()
    R.within("final_state", got[1], ref[1], F32, UNITS, scale[1])
