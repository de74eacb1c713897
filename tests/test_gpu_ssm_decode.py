"""Single tokens of the selective scan: many of them against the scan and the 64-bit decay, small batches against large
ones (two kernels), and the large batches' kernel over what it takes, against the 64-bit form."""
import numpy as np
import pytest
import torch

import block_reference as R
import gated_delta_rule_29_gb300 as la
import test_gpu_ssm as S
from test_gpu_ssm import BF, F32, UNITS, dev

pytestmark = pytest.mark.gpu


def batch(N, D, states, G=1, xt=BF, seed=1, z=True, skip=True, softplus=True):
    """Operands of N tokens, drawn on the GPU."""
    gen = torch.Generator(device=dev()).manual_seed(seed)

    def randn(*shape, dtype=F32):
        return torch.randn(*shape, generator=gen, device=dev()).to(dtype)

    t = dict(x=randn(N, D, dtype=xt), b=randn(N, G, states, dtype=xt), c=randn(N, G, states, dtype=xt),
             a=-torch.arange(1, states + 1, device=dev()) * torch.exp(0.3 * randn(D, states)), s0=randn(N, D, states))
    step = 0.03 * torch.exp(randn(D))
    if softplus:
        t["dt"], t["bias"] = randn(N, D, dtype=xt), step + torch.log(-torch.expm1(-step))
    else:
        t["dt"] = (step * torch.exp(0.5 * randn(N, D))).to(xt)
    if z:
        t["z"] = randn(N, D, dtype=xt)
    if skip:
        t["skip"] = 1 + 0.1 * randn(D)
    return t


def options(t):
    return dict(skip=t.get("skip"), z=t.get("z"), dt_bias=t.get("bias"), dt_softplus="bias" in t)


def rows_of(t, at):
    """The tokens `at` alone, their states with them."""
    return {k: v if k in ("a", "skip", "bias") else v[at].contiguous() for k, v in t.items()}


def operands(t):
    return [t[k] for k in ("x", "dt", "a", "b", "c")]


LARGE = 1 << 23  # states from which on a batch takes the other kernel


# N tokens, D channels; 1 + LARGE / (D S) tokens at least
@pytest.mark.parametrize("N,D,states", [(3, 70, 16), (5, 33, 3), (2, 40, 64), (65, 8192, 16), (1040, 2000, 4), (130, 2048, 32)])
def test_tokens_give_the_scans_states(N, D, states):
    """Token by token an fp32 pool holds the very bits that the scan leaves, whose sequences are whole here."""
    L = 24
    t = batch(N * L, D, states, seed=N)
    s0 = t.pop("s0")[:N].clone()
    cu = torch.arange(0, N * L + 1, L, dtype=torch.int32, device=dev())
    _, fin, _ = la.ssm_fwd(*operands(t), cu, initial_state=s0, **options(t))
    pool = s0.clone()
    for k in range(L):
        one = rows_of(t, cu[:-1].long() + k)
        la.ssm_decode(*operands(one), pool, **options(one))
    assert torch.equal(pool, fin)


@pytest.mark.parametrize("lo,hi,steps", [(2.5e-4, 2e-3, 2000), (0.01, 0.05, 1000)], ids=["slow", "medium"])
@pytest.mark.parametrize("how", ["small", "large", "scan"])
def test_decays_over_many_tokens(lo, hi, steps, how):
    """Decays near 1 without inputs, by both kernels for single tokens and by the scan: the mean of their errors stays within
    0.15 units of 2^-24 a token, where ex2 as it is has up to 0.35 (single ones are off by up to 2, at random)."""
    N, D, states = (66, 8192, 16) if how == "large" else (2, 64, 16)
    gen = torch.Generator(device=dev()).manual_seed(5)
    a = -(0.5 + torch.rand(D, states, generator=gen, device=dev()))
    start = 1 + torch.rand(N, D, states, generator=gen, device=dev())
    x, v = torch.zeros(N, D, device=dev()), torch.zeros(N, 1, states, device=dev())
    total = torch.zeros(N, D, dtype=torch.float64, device=dev())
    pool, all_steps = start.clone(), []
    for _ in range(steps):
        dt = lo / 0.5 + (hi / 1.5 - lo / 0.5) * torch.rand(N, D, generator=gen, device=dev())
        total += dt.double()
        if how == "scan":
            all_steps.append(dt)
        else:
            la.ssm_decode(x, dt, a, v, v, pool)
    if how == "scan":
        dt = torch.stack(all_steps, 1).view(N * steps, D)
        zeros = torch.zeros(N * steps, 1, states, device=dev())
        cu = torch.arange(0, N * steps + 1, steps, dtype=torch.int32, device=dev())
        pool = la.ssm_fwd(torch.zeros_like(dt), dt, a, zeros, zeros, cu, initial_state=start, time_block=1 << 12)[1]
    off = (pool.double() / (start.double() * torch.exp(total[:, :, None] * a.double())) - 1) * 2.0 ** 24
    assert abs(float(off.mean())) <= 0.15 * steps, float(off.mean()) / steps
    assert float(off.abs().max()) <= 2 * steps


SHAPES = [(8192, 16, 1), (8192, 4, 1), (4096, 8, 1), (2048, 32, 2), (1024, 64, 1), (2048, 12, 2), (1512, 24, 3), (1000, 48, 1), (1064, 64, 1)]


@pytest.mark.parametrize("opts", [{}, dict(z=False, softplus=False), dict(skip=False)], ids=["all", "plain_steps", "no_skip"])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("D,states,G", SHAPES)
def test_a_sequence_does_not_depend_on_the_batch(D, states, G, xt, opts):
    """The same bits in y and in an fp32 pool, alone, among a few and in a batch of the other kernel."""
    N = LARGE // (D * states) + 5
    t = batch(N, D, states, G, xt, seed=states, **opts)
    pool = t["s0"].clone()
    y = la.ssm_decode(*operands(t), pool, **options(t))
    for at in ([0], [N - 1], [0, 1, 2, 5, N // 2, N - 3, N - 2]):
        few = rows_of(t, at)
        y1 = la.ssm_decode(*operands(few), few["s0"], **options(few))
        assert torch.equal(y1, y[at]) and torch.equal(few["s0"], pool[at])


@pytest.mark.parametrize("opts", [{}, dict(z=False), dict(softplus=False), dict(skip=False), dict(z=False, skip=False, softplus=False)],
                         ids=["all", "no_z", "plain_steps", "no_skip", "none"])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("D,states,G", SHAPES)
def test_large_batches_against_64_bits(D, states, G, xt, opts):
    """Groups, states that leave lanes idle, channels that do not fill the last CTA."""
    N = LARGE // (D * states) + 6
    t = batch(N, D, states, G, xt, seed=D + states, **opts)
    pool = torch.randn(N + 3, D, states, device=dev())
    idx = torch.randperm(N + 3, generator=torch.Generator().manual_seed(2))[:N].to(torch.int32).to(dev())
    pool[idx.long()] = t["s0"]
    before = pool.clone()
    y = la.ssm_decode(*operands(t), pool, state_indices=idx, **options(t))
    at = sorted({0, 1, 2, 3, 4, N // 2, N - 2, N - 1})
    some = rows_of(t, at)
    ref, scale = S.reference(some, [1] * len(at), False), S.reference(some, [1] * len(at), False, scales=True)
    R.within("y", y[at], ref[0], xt, UNITS, scale[0])
    R.within("state", pool[idx[at].long()], ref[1], F32, UNITS, scale[1])
    unused = torch.from_numpy(np.setdiff1d(np.arange(N + 3), idx.cpu().numpy())).to(dev())
    assert torch.equal(pool[unused], before[unused])
