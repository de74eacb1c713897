"""The mixer operators together and at their edges: the example's training and decoding, offsets beyond 32 bits, many
sequences, two streams at once."""
import os
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_29_gb300 as la

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import token_mixer  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev())


@pytest.mark.parametrize("kind", ["delta", "diagonal"])
def test_example_trains_and_decodes(kind):
    """Training lowers the loss; a prefill and single tokens give the whole sequence's outputs.  Bound of the second:
    every stage between (projection, convolution, recurrence, norm, projection) rounds to bf16, half a step of 2^-8
    each, on either side, and the last projection adds up 256 of them (at most sixfold in a sum of random signs)."""
    torch.manual_seed(1)
    lengths = [300, 17, 129, 64]
    h = torch.randn(sum(lengths), 256, device=dev()).to(BF)
    mixer = token_mixer.TokenMixer(256, 4, 64, kind)
    losses = token_mixer.train(mixer, h, 0.5 * torch.roll(h, 1, 0).float(), cu_of(lengths), steps=20)
    assert np.isfinite(losses).all() and losses[-1] < 0.9 * losses[0], losses
    assert all(torch.isfinite(p.grad.float()).all() for p in mixer.parameters() if p.grad is not None)
    assert token_mixer.decode_error(mixer, h, lengths, 5) <= 6 * 10 * 2.0 ** -9


def test_rows_beyond_32_bits():
    """Two rows 2^31 elements apart (and results as far apart) against the same rows packed."""
    far = 2 ** 31
    buf = torch.zeros(far + 4096, dtype=BF, device=dev())
    out = torch.zeros(far + 4096, dtype=BF, device=dev())
    gen = torch.Generator().manual_seed(1)
    for D in (64, 65):
        x = torch.randn(2, D, generator=gen).to(BF).to(dev())
        g = -torch.rand(2, D, generator=gen).to(dev())
        w = torch.randn(D, 4, generator=gen).to(dev())
        v, o = buf.as_strided((2, D), (far, 1)), out.as_strided((2, D), (far, 1))
        v.copy_(x)
        cu = cu_of([2])
        assert torch.equal(la.glr_fwd(v, g, cu, h=o)[0], la.glr_fwd(x, g, cu)[0])
        assert all(torch.equal(a, b) for a, b in zip(la.glr_bwd(v, g, cu, v, dx=o), la.glr_bwd(x, g, cu, x)))
        assert torch.equal(la.sconv_fwd(v, w, cu, y=o)[0], la.sconv_fwd(x, w, cu)[0])
        assert all(torch.equal(a, b) for a, b in zip(la.sconv_bwd(v, w, cu, v, dx=o)[:2], la.sconv_bwd(x, w, cu, x)[:2]))
        pool, pool2 = torch.ones(2, D, device=dev()), torch.ones(2, D, device=dev())
        assert torch.equal(la.glr_decode(v, g, pool, h=o), la.glr_decode(x, g, pool2)) and torch.equal(pool, pool2)
        n = torch.ones(D, device=dev())
        v3, o3 = buf.as_strided((2, 1, D), (far, D, 1)), out.as_strided((2, 1, D), (far, D, 1))
        x3 = x.view(2, 1, D)
        assert torch.equal(la.gn_fwd(v3, n, y=o3), la.gn_fwd(x3, n))
        assert all(torch.equal(a, b) for a, b in zip(la.gn_bwd(v3, n, v3, dx=o3)[:2], la.gn_bwd(x3, n, x3)[:2]))


@pytest.mark.parametrize("N", [33, 1025, 3000])
def test_many_sequences(N):
    """More sequences than one round of the block search holds, some empty, some of several blocks, against each
    sequence alone."""
    rng = np.random.default_rng(N)
    lens = [int(v) for v in rng.integers(0, 5, N)]
    lens[N // 2], lens[N - 1] = 700, 130
    D, gen = 48, torch.Generator().manual_seed(N)
    T = sum(lens)
    x, dy = (torch.randn(T, D, generator=gen).to(BF).to(dev()) for _ in range(2))
    g = -torch.rand(T, D, generator=gen).to(dev())
    s0, w = torch.randn(N, D, generator=gen).to(dev()), torch.randn(D, 3, generator=gen).to(dev())
    c0 = torch.randn(N, 2, D, generator=gen).to(BF).to(dev())
    cu = cu_of(lens)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    h, fin, ck = la.glr_fwd(x, g, cu, initial_state=s0, output_checkpoints=True, status=status)
    dx, dg, ds0 = la.glr_bwd(x, g, cu, dy, initial_state=s0, checkpoints=ck, status=status)
    y, cfin = la.sconv_fwd(x, w, cu, initial_state=c0, status=status)
    cdx, _, _, cds0 = la.sconv_bwd(x, w, cu, dy, initial_state=c0, status=status)
    assert la.read_status(status) == 0
    starts = np.concatenate([[0], np.cumsum(lens)])
    for i in [0, 1, 31, 32, N // 2 - 1, N // 2, N // 2 + 1, N - 2, N - 1] + [int(v) for v in rng.integers(0, N, 12)]:
        a, b, one = starts[i], starts[i + 1], cu_of([lens[i]])
        h1, fin1, _ = la.glr_fwd(x[a:b], g[a:b], one, initial_state=s0[i:i + 1])
        dx1, dg1, ds1 = la.glr_bwd(x[a:b], g[a:b], one, dy[a:b], initial_state=s0[i:i + 1])
        y1, cfin1 = la.sconv_fwd(x[a:b], w, one, initial_state=c0[i:i + 1])
        cdx1, _, _, cds1 = la.sconv_bwd(x[a:b], w, one, dy[a:b], initial_state=c0[i:i + 1])
        for whole, alone in ((h[a:b], h1), (fin[i:i + 1], fin1), (dx[a:b], dx1), (dg[a:b], dg1), (ds0[i:i + 1], ds1),
                             (y[a:b], y1), (cfin[i:i + 1], cfin1), (cdx[a:b], cdx1), (cds0[i:i + 1], cds1)):
            assert torch.equal(whole, alone), i


def test_two_streams_at_once():
    """Calls on two streams, overlapping, each with its own workspace: the results of one after the other."""
    gen = torch.Generator().manual_seed(3)
    D, lens = 512, [9000, 3000]
    T, cu = sum(lens), cu_of(lens)
    sets = [[torch.randn(T, D, generator=gen).to(BF).to(dev()), -torch.rand(T, D, generator=gen).to(dev()),
             torch.randn(T, D, generator=gen).to(BF).to(dev())] for _ in range(2)]

    def both(x, g, dh, **kw):
        h, fin, ck = la.glr_fwd(x, g, cu, output_checkpoints=True, **kw)
        return (h, fin) + la.glr_bwd(x, g, cu, dh, checkpoints=ck, **kw)

    want = [both(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [both(*s, stream=t) for s, t in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_repeated_calls_give_the_same_bits():
    gen = torch.Generator().manual_seed(4)
    D, lens = 320, [5000, 1, 2500]
    T, cu = sum(lens), cu_of(lens)
    x, dh = (torch.randn(T, D, generator=gen).to(BF).to(dev()) for _ in range(2))
    g = (-0.05 * torch.rand(T, D, generator=gen)).to(dev())
    want = None
    for _ in range(20):
        h, fin, ck = la.glr_fwd(x, g, cu, output_checkpoints=True)
        got = (h, fin) + la.glr_bwd(x, g, cu, dh, checkpoints=ck)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("N", [2, 7, 31, 32])
@pytest.mark.parametrize("D", [64, 200])
def test_sequences_side_by_side(N, D):
    """Up to 32 sequences are taken block by block in turn, single ones block after block: the same bits, for sequences of
    no, one and many blocks, forwards and backwards, and through pool slots."""
    rng = np.random.default_rng(N + D)
    lens = [int(v) for v in rng.integers(0, 1500, N)]
    lens[0], lens[-1] = 4000, 128
    if N > 5:
        lens[2], lens[3], lens[4] = 0, 1, 129
    T, gen = sum(lens), torch.Generator().manual_seed(N)
    x, dh = (torch.randn(T, D, generator=gen).to(BF).to(dev()) for _ in range(2))
    g = (-0.1 * torch.rand(T, D, generator=gen)).to(dev())
    s0, dfin = (torch.randn(N, D, generator=gen).to(dev()) for _ in range(2))
    cu = cu_of(lens)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    h, fin, ck = la.glr_fwd(x, g, cu, initial_state=s0, output_checkpoints=True, status=status)
    dx, dg, ds0 = la.glr_bwd(x, g, cu, dh, initial_state=s0, d_final_state=dfin, checkpoints=ck, status=status)
    pool = torch.zeros(N + 2, D, device=dev())
    slots = torch.randperm(N + 2, generator=gen)[:N].to(torch.int32).to(dev())
    pool[slots.long()] = s0
    hp, _, _ = la.glr_fwd(x, g, cu, initial_state=pool, state_indices=slots, status=status)
    assert la.read_status(status) == 0
    assert torch.equal(hp, h) and torch.equal(pool[slots.long()], fin)
    starts = np.concatenate([[0], np.cumsum(lens)])
    for i in range(N):
        a, b, one = starts[i], starts[i + 1], cu_of([lens[i]])
        h1, fin1, ck1 = la.glr_fwd(x[a:b], g[a:b], one, initial_state=s0[i:i + 1], output_checkpoints=True)
        dx1, dg1, ds1 = la.glr_bwd(x[a:b], g[a:b], one, dh[a:b], initial_state=s0[i:i + 1],
                                   d_final_state=dfin[i:i + 1], checkpoints=ck1)
        for whole, alone in ((h[a:b], h1), (fin[i:i + 1], fin1), (dx[a:b], dx1), (dg[a:b], dg1), (ds0[i:i + 1], ds1)):
            assert torch.equal(whole, alone), i
