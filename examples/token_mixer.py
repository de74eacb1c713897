"""A token mixer from the library's operators: short convolution, recurrence, gated group norm.

    h -> projection -> short_conv -> gdn_attention | gated_linear_recurrence -> group_norm (gate z) -> projection

over packed variable-length sequences for training, and with state pools for serving (a prefill that leaves every
sequence's state in its slot, then one token a step).  Run as a program it trains a small mixer for a few steps and
then decodes with it, checking that single tokens give what the whole sequence gives.

    python examples/token_mixer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_29_gb300 as la  # noqa: E402


class TokenMixer(torch.nn.Module):
    """kind "delta": the gated delta rule, a [head_dim, head_dim] state a head; kind "diagonal": the gated linear
    recurrence, a state of one value a channel."""

    def __init__(self, dim: int, heads: int, head_dim: int, kind: str = "delta", taps: int = 4, device="cuda"):
        super().__init__()
        self.heads, self.head_dim, self.kind, self.taps = heads, head_dim, kind, taps
        inner = heads * head_dim
        self.width = 3 * inner if kind == "delta" else inner
        kw = dict(bias=False, device=device, dtype=torch.bfloat16)
        self.proj_in = torch.nn.Linear(dim, self.width, **kw)
        self.proj_gate = torch.nn.Linear(dim, 2 * heads if kind == "delta" else inner, **kw)
        self.proj_z = torch.nn.Linear(dim, inner, **kw)
        self.proj_out = torch.nn.Linear(inner, dim, **kw)
        self.conv = torch.nn.Parameter(torch.randn(self.width, taps, device=device) * taps ** -0.5)
        self.norm = torch.nn.Parameter(torch.ones(head_dim, device=device))
        self.a_log = torch.nn.Parameter(torch.zeros(heads, device=device))
        self.dt_bias = torch.nn.Parameter(torch.full((heads,), -2.0, device=device))

    def _split(self, x):
        T = x.shape[0]
        return (v.reshape(T, self.heads, self.head_dim) for v in x.view(T, 3, -1).unbind(1))

    def _gates(self, h):
        gate = self.proj_gate(h)
        if self.kind != "delta":
            return gate, None
        return gate[:, :self.heads].float(), gate[:, self.heads:].float()

    def _norm(self, o, h):
        shape = (h.shape[0], self.heads, self.head_dim)
        y = la.group_norm(o.view(shape), self.norm, z=self.proj_z(h).view(shape), center=False)
        return self.proj_out(y.view(h.shape[0], -1))

    def forward(self, h, cu_seqlens):
        """h [T, dim] over packed sequences."""
        x, _ = la.short_conv(self.proj_in(h), self.conv, cu_seqlens)
        gate, beta = self._gates(h)
        if self.kind == "delta":
            o, _ = la.gdn_attention(*self._split(x), gate, beta, cu_seqlens, a_log=self.a_log, dt_bias=self.dt_bias,
                                    beta_sigmoid=True)
        else:
            o, _ = la.gated_linear_recurrence(x, gate, cu_seqlens, gate_logsigmoid=True, complement_input=True)
        return self._norm(o, h)

    def pools(self, slots: int) -> dict:
        """State pools for `slots` sequences, all starting from nothing."""
        dev = self.conv.device
        state = (self.heads, self.head_dim, self.head_dim) if self.kind == "delta" else (self.heads * self.head_dim,)
        return {"conv": torch.zeros(slots, self.taps - 1, self.width, dtype=torch.bfloat16, device=dev),
                "state": torch.zeros(slots, *state, device=dev)}

    @torch.no_grad()
    def prefill(self, h, cu_seqlens, pools, slots):
        """Whole sequences (or their next parts), whose states go on from and back to pools[slots]."""
        x, _ = la.sconv_fwd(self.proj_in(h), self.conv, cu_seqlens, initial_state=pools["conv"], state_indices=slots)
        gate, beta = self._gates(h)
        if self.kind == "delta":
            o, _, _ = la.gdn_fwd(*self._split(x), gate, beta, cu_seqlens, initial_state=pools["state"],
                                 state_indices=slots, a_log=self.a_log, dt_bias=self.dt_bias, beta_sigmoid=True)
        else:
            o, _, _ = la.glr_fwd(x, gate, cu_seqlens, initial_state=pools["state"], state_indices=slots,
                                 gate_logsigmoid=True, complement_input=True)
        return self._norm(o, h)

    @torch.no_grad()
    def step(self, h, pools, slots):
        """One token of each sequence, h [N, dim]."""
        x = la.sconv_decode(self.proj_in(h), self.conv, pools["conv"], state_indices=slots)
        gate, beta = self._gates(h)
        if self.kind == "delta":
            o = la.gdn_decode(*self._split(x), gate, beta, pools["state"], state_indices=slots, a_log=self.a_log,
                              dt_bias=self.dt_bias, beta_sigmoid=True)
        else:
            o = la.glr_decode(x, gate, pools["state"], state_indices=slots, gate_logsigmoid=True,
                              complement_input=True)
        return self._norm(o, h)


def train(mixer, h, target, cu_seqlens, steps: int = 20, lr: float = 3e-3):
    """Least squares towards `target`; returns the loss before every step."""
    opt = torch.optim.Adam(mixer.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        loss = (mixer(h, cu_seqlens).float() - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def decode_error(mixer, h, lengths, steps: int):
    """Largest difference of a prefill and `steps` single tokens from the whole sequences, over the largest value."""
    dev, N = h.device, len(lengths)
    starts = torch.tensor([0] + lengths, device=dev).cumsum(0)
    cu = starts.to(torch.int32)
    with torch.no_grad():
        whole = mixer(h, cu)
    pools, slots = mixer.pools(N + 3), torch.randperm(N + 3, device=dev)[:N].to(torch.int32)
    first = torch.cat([torch.arange(starts[i], starts[i + 1] - steps, device=dev) for i in range(N)])
    got = torch.empty_like(whole)
    got[first] = mixer.prefill(h[first], cu - steps * torch.arange(N + 1, device=dev, dtype=torch.int32), pools, slots)
    for k in range(steps):
        at = starts[1:] - steps + k
        got[at] = mixer.step(h[at], pools, slots)
    return float((got.float() - whole.float()).abs().max() / whole.float().abs().max())


def main():
    torch.manual_seed(0)
    lengths = [300, 17, 129, 64]
    cu = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    h = torch.randn(sum(lengths), 256, device="cuda").to(torch.bfloat16)
    for kind in ("delta", "diagonal"):
        mixer = TokenMixer(256, 4, 64, kind)
        target = 0.5 * torch.roll(h, 1, 0).float()
        losses = train(mixer, h, target, cu)
        print(f"{kind}: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps, "
              f"decoding differs from the whole by {decode_error(mixer, h, lengths, 5):.1e} of the largest value")


if __name__ == "__main__":
    main()
