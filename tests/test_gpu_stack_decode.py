"""Decoding with the example's stack, by the root mean square over each sequence: tight enough that a state handed over
wrongly shows."""
import pytest
import torch

from test_gpu_block import BF, dev, models

pytestmark = pytest.mark.gpu

LENGTHS, STEPS = [60, 17, 129, 64], 5
# The two ways round some 25 stages to bf16, by at most 2^-8 of a value and 2^-8 / sqrt(3) in the root mean square, at random on
# either side.  A stage passes on the relative errors of what it is given as they are: projections and the norms' sums by a row's
# length, products one factor's beside the other's (each is a stage), and the stream, in 32 bits, takes only its share of them.
BOUND = (2 * 25 / 3) ** 0.5 * 2.0 ** -8


def handed_over(model, h, spoil=None):
    """Each sequence's relative errors (root mean squares) against the whole: its single tokens' outputs, and what every pool
    holds at the end; spoil(pools, slots) between the prefill and the tokens."""
    N = len(LENGTHS)
    starts = torch.tensor([0] + LENGTHS, device=h.device).cumsum(0)
    cu = starts.to(torch.int32)
    slots = torch.tensor([5, 0, 3, 2], dtype=torch.int32, device=h.device)
    ends, pools = model.pools(N + 3), model.pools(N + 3)
    whole = model.prefill(h, cu, ends, slots).float()
    first = torch.cat([torch.arange(starts[i], starts[i + 1] - STEPS, device=h.device) for i in range(N)])
    model.prefill(h[first], cu - STEPS * torch.arange(N + 1, device=h.device, dtype=torch.int32), pools, slots)
    if spoil:
        spoil(pools, slots)

    def error(got, want):
        off, size = ((v.float().flatten(1)).square().sum(1) for v in (got.float() - want.float(), want))
        return (off / size).sqrt()

    at = [starts[1:] - STEPS + k for k in range(STEPS)]
    tokens = torch.stack([model.step(h[rows], pools, slots) for rows in at], 1)
    out = {"outputs": error(tokens, torch.stack([whole[rows] for rows in at], 1))}
    for i, (got, want) in enumerate(zip(pools, ends)):
        for key in got:
            out[i, key] = error(got[key][slots.long()], want[key][slots.long()])
    return out


def test_the_stack_hands_its_states_over():
    h = torch.randn(sum(LENGTHS), 256, generator=torch.Generator().manual_seed(3)).to(BF).to(dev())
    model = models("stack")
    good = handed_over(model, h)
    assert all(bool((v <= BOUND).all()) for v in good.values()), good
    for layer in range(3):
        for key in model.pools(1)[layer]:
            def spoil(pools, slots):
                pools[layer][key][slots[2].long()] = 0
            bad = handed_over(model, h, spoil)
            assert max(float(v[2]) for v in bad.values()) > BOUND, (layer, key, bad)
            assert all(torch.equal(bad[k][[0, 1, 3]], good[k][[0, 1, 3]]) for k in good)
