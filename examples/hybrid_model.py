"""A small recurrent language model made of the library's operators: trained for a few steps, then run as a server
would, a packed batch of prompts first and token by token after it.

Each block is  x, h <- rms_norm(mixer output + h);  h's mixer is either the gated delta rule or the selective scan,
both behind a short causal convolution.  Run from the repository's root:

    python examples/hybrid_model.py
"""

from __future__ import annotations

import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_38_gb300 as gdr  # noqa: E402

BF = torch.bfloat16


class Conv(nn.Module):
    """Short causal convolution through SiLU; ``state`` holds a row's last three inputs between calls."""

    def __init__(self, width):
        super().__init__()
        self.weight = nn.Parameter(torch.randn(width, 4, dtype=BF, device="cuda") * 0.5)

    def forward(self, x, cu, state):
        if state is None:
            y, _ = gdr.short_conv(x, self.weight, activation="silu", cu_seqlens=cu)
            return y
        if x.shape[1] == 1 and "conv" in state:
            return gdr.short_conv_step(x, state["conv"], self.weight, activation="silu")
        y, state["conv"] = gdr.short_conv_fwd(x, self.weight, activation="silu", initial_state=state.get("conv"),
                                              output_final_state=True, cu_seqlens=cu)
        return y


def linear(i, o):
    return nn.Linear(i, o, bias=False, dtype=BF, device="cuda")


class DeltaMixer(nn.Module):
    """Gated delta rule with 128-wide heads."""

    def __init__(self, width, heads=2):
        super().__init__()
        self.heads, self.inner = heads, heads * 128
        self.qkv, self.gates, self.out = linear(width, 3 * self.inner), linear(width, 2 * heads), linear(self.inner, width)
        self.conv = Conv(3 * self.inner)

    def forward(self, x, cu, state):
        B, T, _ = x.shape
        q, k, v = self.conv(self.qkv(x), cu, state).view(B, T, 3, self.heads, 128).unbind(2)
        g, beta = self.gates(x).view(B, T, 2, self.heads).unbind(2)
        act = dict(use_qk_l2norm_in_kernel=True, use_gate_in_kernel=True, use_beta_sigmoid_in_kernel=True)
        if state is None:
            o, _ = gdr.chunk_gated_delta_rule(q, k, v, g + 2, beta, cu_seqlens=cu, **act)
        elif T == 1 and "delta" in state:
            o, _ = gdr.recurrent_gated_delta_rule(*(t.contiguous() for t in (q, k, v, g + 2, beta)),
                                                  initial_state=state["delta"], inplace=True, **act)
        else:
            o, state["delta"] = gdr.chunk_gated_delta_rule(q, k, v, g + 2, beta, initial_state=state.get("delta"), cu_seqlens=cu,
                                                           output_final_state=True, **act)
        return self.out(o.reshape(B, T, self.inner))


class ScanMixer(nn.Module):
    """Selective state space scan, 16 states a channel; x, z, the step and B, C are slices of two projections."""

    def __init__(self, width, states=16):
        super().__init__()
        self.inner, self.states = 2 * width, states
        self.xz, self.dbc, self.out = linear(width, 2 * self.inner), linear(self.inner, self.inner + 2 * states), linear(self.inner, width)
        self.conv = Conv(self.inner)
        step = torch.exp(torch.empty(self.inner).uniform_(-6.9, -2.3))  # between 1e-3 and 1e-1
        self.dt_bias = nn.Parameter((step + torch.log(-torch.expm1(-step))).cuda())
        self.log_a = nn.Parameter(torch.log(torch.arange(1, states + 1, dtype=torch.float32)).repeat(self.inner, 1).cuda())
        self.skip = nn.Parameter(torch.ones(self.inner, device="cuda"))

    def forward(self, x, cu, state):
        u, z = self.xz(x).split(self.inner, -1)
        u = self.conv(u, cu, state)
        dt, b, c = self.dbc(u).split((self.inner, self.states, self.states), -1)
        args = (u, dt, -torch.exp(self.log_a), b.unsqueeze(2), c.unsqueeze(2))
        opt = dict(D=self.skip, z=z, dt_bias=self.dt_bias, dt_softplus=True)
        if state is None:
            y, _ = gdr.selective_scan(*args, cu_seqlens=cu, **opt)
        elif x.shape[1] == 1 and "scan" in state:
            y = gdr.selective_scan_step(*args, state["scan"], **opt)
        else:
            y, state["scan"], _ = gdr.selective_scan_fwd(*args, initial_state=state.get("scan"), cu_seqlens=cu, **opt)
        return self.out(y)


class Model(nn.Module):
    def __init__(self, vocab=64, width=128):
        super().__init__()
        self.embed = nn.Embedding(vocab, width, dtype=BF, device="cuda")
        self.mixers = nn.ModuleList([ScanMixer(width), DeltaMixer(width), ScanMixer(width)])
        self.norms = nn.ParameterList([nn.Parameter(torch.ones(width, device="cuda")) for _ in range(len(self.mixers) + 1)])
        self.head = linear(width, vocab)

    def forward(self, tokens, cu=None, states=None):
        """Logits; ``states`` (a list of one dict a block) is filled by a prompt and advanced by single tokens or by more
        of the prompts."""
        h = self.embed(tokens).float()  # the residual stream is fp32
        y = torch.zeros_like(h, dtype=BF)
        for i, mixer in enumerate(self.mixers):
            x, h = gdr.rms_norm(y, self.norms[i], h)
            y = mixer(x, cu, None if states is None else states[i])
        x, _ = gdr.rms_norm(y, self.norms[-1], h)
        return self.head(x)


def batch(B, T, vocab, gen):
    """Walks through a fixed permutation of the tokens from random starts: each token tells the next."""
    after = torch.randperm(vocab, generator=torch.Generator().manual_seed(7))
    seq = [torch.randint(vocab, (B,), generator=gen)]
    for _ in range(T - 1):
        seq.append(after[seq[-1]])
    return torch.stack(seq, 1).cuda()


def train(steps=60, seed=0):
    torch.manual_seed(seed)
    gen = torch.Generator().manual_seed(seed)
    model = Model()
    opt = torch.optim.AdamW(model.parameters(), lr=5e-3)
    losses = []
    for _ in range(steps):
        t = batch(16, 129, 64, gen)
        logits = model(t[:, :-1])
        loss = nn.functional.cross_entropy(logits.flatten(0, 1).float(), t[:, 1:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return model, losses


@torch.no_grad()
def serve(model, lens=(40, 3, 64, 17), new=12, seed=1):
    """Prompts of different lengths as one packed batch, then ``new`` tokens of every row, one by one.  Returns the
    tokens and their logits from the states, and the logits of the same tokens from whole sequences."""
    gen = torch.Generator().manual_seed(seed)
    prompts = [batch(1, n, 64, gen)[0] for n in lens]
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    states = [{} for _ in model.mixers]
    logits = model(torch.cat(prompts)[None], cu, states)[0, cu[1:].long() - 1]
    rows, steps = [list(p) for p in prompts], [logits]
    for _ in range(new - 1):
        nxt = steps[-1].argmax(-1)
        for r, t in zip(rows, nxt):
            r.append(t)
        steps.append(model(nxt[:, None], None, states)[:, 0])
    whole = [model(torch.stack(r)[None])[0, n - 1:] for r, n in zip(rows, lens)]
    return rows, torch.stack(steps, 1), torch.stack(whole)


if __name__ == "__main__":
    model, losses = train()
    print("loss %.3f -> %.3f over %d steps" % (losses[0], losses[-1], len(losses)))
    rows, stepped, whole = serve(model)
    off = float((stepped - whole).float().norm() / whole.float().norm())
    print("logits token by token against whole sequences: relative difference %.1e" % off)
    print("continuation of row 0:", [int(t) for t in rows[0][32:]])
