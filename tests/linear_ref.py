"""Plain fp64 forms of linear attention, the gated norm and the block norm for the tests, straight from their definitions;
gradients come from torch's autograd on them."""

from __future__ import annotations

import torch

from layer_ref import U, ranges

# Linear attention's 16-bit results carry three roundings: a product's left side (P, or the state's copy) of each term, and
# the result's own.  One is off by at most U of the value, evenly spread within that, which is U / sqrt(3) in the mean
# square; three independent ones give U, and a quarter more is for the spread of small samples.  The states are sums of keys
# held as two or three 16-bit numbers, each term off by at most U^2, and of fp32 operations (2e-6 together).
def attn_bound(t, dt) -> float:
    if t.dtype == torch.float32:
        return U[dt] ** 2 + 2e-6
    return 1.25 * U[t.dtype]


def check(got, want, bound, name):
    assert got.shape == want.shape, (name, tuple(got.shape), tuple(want.shape))
    a, b = got.detach().double().cpu(), want.detach().double().cpu()
    assert torch.isfinite(a).all(), name + ": non-finite values"
    err = float((a - b).norm() / b.norm().clamp(min=1e-30)) if b.numel() else 0.0
    assert err <= bound, "%s: relative L2 error %.3e > %.3e" % (name, err, bound)


def attn(q, k, v, decay, scale, state, lens, piece=512):
    """(o, final states): every sequence in pieces of tokens, each by the sums over its pairs, from the state before it."""
    B, T, Hk, K = q.shape
    H = v.shape[2]
    q, k = (t.repeat_interleave(H // Hk, 2) for t in (q, k))
    outs, fins = [[] for _ in range(B)], []
    for n, (b, t0, t1) in enumerate(ranges(B, T, lens)):
        S = torch.zeros(H, K, v.shape[3], dtype=q.dtype) if state is None else state[n]
        for p0 in range(t0, t1, piece):
            p1 = min(t1, p0 + piece)
            qq, kk, vv = (t[b, p0:p1].transpose(0, 1) for t in (q, k, v))
            i = torch.arange(p1 - p0, dtype=q.dtype)
            d = i[:, None] - i
            g = torch.where(d >= 0, torch.exp(decay[:, None, None] * d.clamp(min=0)), 0.0)
            o = ((qq @ kk.transpose(1, 2)) * g) @ vv + torch.exp(decay[:, None] * (i + 1))[..., None] * (qq @ S)
            outs[b].append(scale * o.transpose(0, 1))
            left = torch.exp(decay[:, None] * (p1 - p0 - 1 - i))[..., None]
            S = torch.exp(decay * (p1 - p0))[:, None, None] * S + (kk * left).transpose(1, 2) @ vv
        fins.append(S)
    o = torch.stack([torch.cat(r) if r else v[b] for b, r in enumerate(outs)])
    return o, torch.stack(fins)


def act(name, g):
    return torch.sigmoid(g) if name == "sigmoid" else g * torch.sigmoid(g) if name == "silu" else g


def rms(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def gated(x, g, w, name, eps=1e-6):
    return rms(x, eps) * w * act(name, g)


def block_sum(x, res, pw, g, name, s, eps=1e-6):
    b = x if pw is None else rms(x, eps) * pw
    return res + s * (b if g is None else b * act(name, g))
