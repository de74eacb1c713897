"""Steps of the selective scan with a bias and softplus one without the other, which test_gpu_ssm.py has only together: forward,
backward and single tokens against the 64-bit form, within the bounds of test_gpu_ssm.py."""
import pytest
import torch

import block_reference as R
import gated_delta_rule_29_gb300 as la
import test_gpu_ssm as S
from test_gpu_ssm import BF, F32, UNITS, cu_of, dev, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softplus,bias", [(True, False), (False, True)])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("time_block", [0, 64])
def test_bias_and_softplus_are_independent(softplus, bias, xt, time_block):
    lens = [200, 0, 33, 1]
    D, N = 70, 16
    t = draw(lens, D, N, xt=xt, seed=4, softplus=False)
    t["dt"] = (torch.randn(sum(lens), D, generator=torch.Generator().manual_seed(1)) - 3).to(xt).to(dev()) if softplus else t["dt"]
    extra = torch.linspace(0.01, 0.1, D, device=dev()) if bias else None
    cu = cu_of(lens)
    opts = dict(skip=t["skip"], z=t["z"], dt_bias=extra, dt_softplus=softplus, initial_state=t["s0"])
    ops = [t[k] for k in ("x", "dt", "a", "b", "c")]
    y, fin, ck = la.ssm_fwd(*ops, cu, output_checkpoints=True, time_block=time_block, **opts)
    got = (y, fin) + la.ssm_bwd(*ops, cu, t["dy"], d_final_state=t["dfin"], checkpoints=ck, **opts)
    v = [R.f64(t[k]) for k in ("x", "dt", "a", "b", "c")]
    kw = dict(skip=R.f64(t["skip"]), z=R.f64(t["z"]), bias=R.f64(extra), use_softplus=softplus, s0=R.f64(t["s0"]), dy=R.f64(t["dy"]),
              dfin=R.f64(t["dfin"]))
    types = (xt, F32, xt, xt, F32, xt, xt, F32, xt, F32, F32)
    for name, g, r, s, ty in zip(("y", "final_state") + S.NAMES, got, R.ssm(*v, lens, **kw), R.ssm_scales(*v, lens, **kw), types):
        R.within(name, g, r, ty, UNITS, s)
    # the same for single tokens
    pool = t["s0"][[0, 2, 3]].clone()
    at = torch.tensor([0, 200, 233], device=dev())
    y1 = la.ssm_decode(*[o if o is t["a"] else o[at] for o in ops], pool, skip=t["skip"], z=t["z"][at], dt_bias=extra, dt_softplus=softplus)
    first = [o if i == 2 else o[[0, 200, 233]] for i, o in enumerate(v)]
    kw.update(z=kw["z"][[0, 200, 233]], s0=kw["s0"][[0, 2, 3]], dy=None, dfin=None)
    ref, scale = R.ssm(*first, [1] * 3, **kw), R.ssm_scales(*first, [1] * 3, **kw)
    R.within("y", y1, ref[0], xt, UNITS, scale[0])
    R.within("state", pool, ref[1], F32, UNITS, scale[1])
