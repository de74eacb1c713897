"""Invalid sequence boundaries with more sequences than the scan takes side by side: the status word says so, no access
leaves the operands, and no block waits for one that is not there (a wait that ends by its limit takes a second)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_29_gb300 as la

pytestmark = pytest.mark.gpu


def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def batches():
    early = 300 * np.arange(41)
    early[21] = early[20] - 512
    yield "one sequence begins early", early, 12000
    rng = np.random.default_rng(8)
    for N, T in ((33, 9000), (120, 30000), (1100, 40000)):
        cu = rng.integers(0, T + 1, N + 1)
        cu[0], cu[-1] = 0, T
        yield f"{N} in no order", cu, T
        cu = rng.integers(-300, T + 300, N + 1)
        yield f"{N} inside and outside", cu, T


@pytest.mark.parametrize("name,cu,T", list(batches()), ids=lambda v: v if isinstance(v, str) else "")
@pytest.mark.parametrize("D", [64, 66])
def test_many_sequences_with_invalid_boundaries(name, cu, T, D):
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, D, generator=gen).to(torch.bfloat16).to(dev())
    g = -torch.rand(T, D, generator=gen).to(dev())
    w = torch.randn(D, 4, generator=gen).to(dev())
    N = len(cu) - 1
    good = torch.tensor(np.linspace(0, T, N + 1).astype(np.int32), device=dev())
    bad = torch.tensor(cu.astype(np.int32), device=dev())
    s0 = torch.randn(N, D, generator=gen).to(dev())
    status = torch.zeros(1, dtype=torch.int32, device=dev())

    def calls(c):
        yield lambda: la.glr_fwd(x, g, c, initial_state=s0, output_checkpoints=True, status=status)
        yield lambda: la.glr_bwd(x, g, c, x, initial_state=s0, d_final_state=s0, status=status)
        yield lambda: la.sconv_fwd(x, w, c, status=status)
        yield lambda: la.sconv_bwd(x, w, c, x, status=status)

    want = [call() for call in calls(good)]
    torch.cuda.synchronize()
    assert la.read_status(status) == 0
    for call in calls(bad):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        call()
        end.record()
        end.synchronize()
        assert la.read_status(status) == la.binding.LA_ERR_BAD_SEQLENS
        assert begin.elapsed_time(end) < 500.0
        status.zero_()
    for outs, call in zip(want, calls(good)):
        assert all(torch.equal(a, b) for a, b in zip(outs, call()) if a is not None and a.shape[0] != T // 128 + N)
    assert la.read_status(status) == 0
