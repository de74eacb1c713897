"""What the differentiable scan asks of its forward (CPU: the forward is a stand-in)."""
import pytest
import torch

import gated_delta_rule_29_gb300 as la
from gated_delta_rule_29_gb300 import block


@pytest.fixture
def asked(monkeypatch):
    calls = []

    def stand_in(x, *args, initial_state=None, output_checkpoints=False, **kw):
        calls.append(output_checkpoints)
        return torch.zeros_like(x), torch.zeros(1, 8, 2), torch.zeros(1) if output_checkpoints else None

    monkeypatch.setattr(block, "ssm_fwd", stand_in)
    return calls


def test_states_are_kept_only_for_a_backward_pass(asked):
    x, a, v, cu = torch.zeros(4, 8), torch.zeros(8, 2, requires_grad=True), torch.zeros(4, 2), torch.tensor([0, 4])
    la.selective_scan(x, x, a, v, v, cu)
    la.selective_scan(x, x, a, v, v, cu, save_checkpoints=False)
    with torch.no_grad():
        la.selective_scan(x, x, a, v, v, cu)
    with torch.inference_mode():
        la.selective_scan(x, x, a, v, v, cu)
    la.selective_scan(x, x, a.detach(), v, v, cu)
    for name in ("skip", "z", "dt_bias", "initial_state"):
        la.selective_scan(x, x, a.detach(), v, v, cu, **{name: torch.zeros(8, requires_grad=True)})
    assert asked == [True, False, False, False, False, True, True, True, True]
