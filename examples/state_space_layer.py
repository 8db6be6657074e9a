"""A state-space layer on the library's operators: residual norm, input
projection, short convolution, selective scan, output projection. Trains it on
packed sequences, runs prompts with their states carried out, and continues
them token by token.

    python examples/state_space_layer.py

The projections are plain torch products; everything between them is one call
of the library each.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_18_gb300 as gdn  # noqa: E402
from gated_delta_rule_18_gb300 import autograd as gdr  # noqa: E402


class StateSpaceLayer(torch.nn.Module):
    """norm(x + residual) -> (x, z) -> conv -> (dt, B, C) -> scan * silu(z) -> out."""

    def __init__(self, d_model, expand=2, d_state=16, taps=4, device="cuda", seed=0):
        super().__init__()
        g = torch.Generator(device="cpu").manual_seed(seed)
        d, rank = expand * d_model, max(8, d_model // 16)

        def param(*shape, std, dtype=torch.bfloat16):
            return torch.nn.Parameter((torch.randn(shape, generator=g) * std).to(device, dtype))

        f32 = torch.float32
        self.rank, self.d_state = rank, d_state
        self.norm = torch.nn.Parameter(torch.ones(d_model, device=device))
        self.w_in = param(d_model, 2 * d, std=d_model**-0.5)
        self.taps, self.conv_bias = param(d, taps, std=taps**-0.5, dtype=f32), param(d, std=0.02, dtype=f32)
        self.w_x = param(d, rank + 2 * d_state, std=d**-0.5)
        self.w_dt = param(rank, d, std=rank**-0.5)
        step = torch.exp(torch.empty(d).uniform_(math.log(1e-3), math.log(1e-1), generator=g))
        self.dt_bias = torch.nn.Parameter((step + torch.log(-torch.expm1(-step))).to(device))
        self.a_log = torch.nn.Parameter(torch.log(torch.arange(1.0, d_state + 1)).repeat(d, 1).to(device))
        self.skip = torch.nn.Parameter(torch.ones(d, device=device))
        self.w_out = param(d, d_model, std=d**-0.5)

    def _split(self, p):
        r, n = self.rank, self.d_state
        return p[..., :r] @ self.w_dt, p[..., r : r + n], p[..., r + n :]

    def forward(self, x, residual, cu_seqlens=None):
        """Training: (B, T, d_model) -> (y, residual stream)."""
        y, residual = gdr.rms_norm(x, self.norm, residual)
        x, z = (y @ self.w_in).chunk(2, dim=-1)
        x, _ = gdr.causal_conv(x, self.taps, self.conv_bias, cu_seqlens=cu_seqlens)
        dt, bm, cm = self._split(x @ self.w_x)
        y, _ = gdr.selective_scan(x, dt, -torch.exp(self.a_log), bm, cm, self.skip, z, self.dt_bias, cu_seqlens=cu_seqlens)
        return y @ self.w_out, residual

    @torch.no_grad()
    def prompt(self, x, residual, cu_seqlens=None):
        """(y, residual, state): the state is (windows, scan states) of every sequence."""
        n = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        d, taps = self.taps.shape
        window = torch.empty(n, taps - 1, d, dtype=x.dtype, device=x.device)
        h = torch.empty(n, d, self.d_state, device=x.device)
        r = gdn.gdn_rmsnorm_fwd(x, self.norm, residual=residual)
        x, z = (r["out"] @ self.w_in).chunk(2, dim=-1)
        x = gdn.gdn_conv_fwd(x, self.taps, bias=self.conv_bias, cu_seqlens=cu_seqlens, final_state=window)
        dt, bm, cm = self._split(x @ self.w_x)
        y = gdn.gdn_ssm_fwd(x, dt, -torch.exp(self.a_log), bm, cm, D=self.skip, z=z, dt_bias=self.dt_bias,
                            cu_seqlens=cu_seqlens, h_final=h)
        return y @ self.w_out, r["residual"], (window, h)

    @torch.no_grad()
    def step(self, x, residual, state, slots=None, eight_bit=False):
        """One token of n requests, the states updated in place. eight_bit: the
        norm leaves e4m3 values and a scale for 128 channels, as an 8-bit
        input projection takes them; here they are multiplied out before it."""
        window, h = state
        if eight_bit:
            r = gdn.gdn_rmsnorm_fwd(x, self.norm, residual=residual, out_dtype=torch.float8_e4m3fn, group=128)
            y = (r["out"].float() * r["scale"].repeat_interleave(128, -1)[:, : x.shape[1]]).to(x.dtype)
        else:
            r = gdn.gdn_rmsnorm_fwd(x, self.norm, residual=residual)
            y = r["out"]
        x, z = (y @ self.w_in).chunk(2, dim=-1)
        x = gdn.gdn_conv_step(x, window, self.taps, bias=self.conv_bias, slots=slots)
        dt, bm, cm = self._split(x @ self.w_x)
        y = gdn.gdn_ssm_step(x, dt, -torch.exp(self.a_log), bm, cm, h, D=self.skip, z=z, dt_bias=self.dt_bias, slots=slots)
        return y @ self.w_out, r["residual"]


def train(layer, steps=20, lengths=(50, 1, 77, 128), seed=1):
    """Losses of a few steps towards each sequence's input delayed by one token."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, total = layer.norm.numel(), sum(lengths)
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    x = torch.randn(1, total, d, generator=g, device="cuda", dtype=torch.bfloat16)
    want = torch.cat([torch.nn.functional.pad(s, (0, 0, 1, 0))[:, :-1] for s in x.split(list(lengths), 1)], 1)
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        y, _ = layer(x, torch.zeros_like(x), cu)
        loss = (y.float() - want.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


def continue_prompt(layer, prompt=61, tokens=5, requests=3, eight_bit=False, seed=2):
    """The largest difference between continuing token by token and one long
    prompt, relative to the largest output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = layer.norm.numel()
    x = torch.randn(requests, prompt + tokens, d, generator=g, device="cuda", dtype=torch.bfloat16)
    res = torch.randn(requests, prompt + tokens, d, generator=g, device="cuda")
    whole, _, _ = layer.prompt(x, res)
    _, _, (window, h) = layer.prompt(x[:, :prompt].contiguous(), res[:, :prompt].contiguous())
    # a pool of states, as a server keeps it: request i in row 2 i
    pool = (window.new_zeros(2 * requests, *window.shape[1:]), h.new_zeros(2 * requests, *h.shape[1:]))
    slots = torch.arange(0, 2 * requests, 2, dtype=torch.int32, device="cuda")
    pool[0][::2], pool[1][::2] = window, h
    worst = 0.0
    for t in range(prompt, prompt + tokens):
        y, _ = layer.step(x[:, t], res[:, t], pool, slots, eight_bit)
        worst = max(worst, ((y - whole[:, t]).float().abs().max() / whole.float().abs().max()).item())
    return worst


def main():
    torch.cuda.set_device(0)
    layer = StateSpaceLayer(256)
    losses = train(layer)
    print(f"training on packed sequences: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    print(f"token by token against one prompt: {continue_prompt(layer):.2e} of the largest output, "
          f"with the 8-bit norm {continue_prompt(layer, eight_bit=True):.2e}")


if __name__ == "__main__":
    main()
