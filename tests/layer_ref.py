"""Plain fp64 forms of the layer operators, token by token, for the tests.  Gradients come from torch's autograd on
these forms and from central differences of them."""

from __future__ import annotations

import torch

# Unit roundoff of the 16-bit types: a result rounded once is off by at most this, relative to itself.
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def bound(t) -> float:
    """Relative L2 bound of one output: a 16-bit one is rounded once (the fp32 arithmetic before it adds less than a
    hundredth of that in bf16 and a twentieth in fp16); an fp32 one holds sums and recurrences of fp32 operations and
    2^-22 exponentials, whose errors of about 5e-7 a step gather over the some forty steps that a state remembers."""
    if t.dtype == torch.float32:
        return 2e-5
    return 1.05 * U[t.dtype]


def check(got, want, name):
    assert got.shape == want.shape, (name, tuple(got.shape), tuple(want.shape))
    a, b = got.detach().double().cpu(), want.detach().double().cpu()
    assert torch.isfinite(a).all(), name + ": non-finite values"
    err = float((a - b).norm() / b.norm().clamp(min=1e-30)) if b.numel() else 0.0
    assert err <= bound(got), "%s: relative L2 error %.3e > %.3e" % (name, err, bound(got))


def ranges(B, T, lens):
    if lens is None:
        return [(b, 0, T) for b in range(B)]
    out, at = [], 0
    for n in lens:
        out.append((0, at, at + n))
        at += n
    return out


def norm(x, w, res, eps=1e-6):
    h = x if res is None else x + res
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w, h


def conv(x, w, bias, silu, state, lens):
    """(y, final state): state [N, W-1, D] or None."""
    B, T, D = x.shape
    W = w.shape[1]
    ys, fins = [[] for _ in range(B)], []
    for n, (b, t0, t1) in enumerate(ranges(B, T, lens)):
        past = torch.zeros(W - 1, D, dtype=x.dtype) if state is None else state[n]
        ext = torch.cat([past, x[b, t0:t1]])
        for t in range(t1 - t0):
            pre = (ext[t:t + W] * w.T).sum(0)
            if bias is not None:
                pre = pre + bias
            ys[b].append(pre * torch.sigmoid(pre) if silu else pre)
        fins.append(ext[t1 - t0:])
    y = torch.stack([torch.stack(r) if r else x[b] for b, r in enumerate(ys)])
    return y, torch.stack(fins)


def scan(x, dt, A, B, C, D, z, bias, softplus, state, lens):
    """(y, final state): state [N_seqs, D, N] or None."""
    nb, T, width = x.shape
    N, G = A.shape[1], B.shape[2]
    raw = dt if bias is None else dt + bias
    delta = torch.nn.functional.softplus(raw, threshold=1e9) if softplus else raw
    Bw, Cw = (m.repeat_interleave(width // G, 2) for m in (B, C))
    ys, fins = [[] for _ in range(nb)], []
    for n, (b, t0, t1) in enumerate(ranges(nb, T, lens)):
        h = torch.zeros(width, N, dtype=x.dtype) if state is None else state[n]
        for t in range(t0, t1):
            h = torch.exp(delta[b, t, :, None] * A) * h + (delta[b, t] * x[b, t])[:, None] * Bw[b, t]
            ys[b].append((h * Cw[b, t]).sum(-1))
        fins.append(h)
    y = torch.stack([torch.stack(r) if r else x[b] * 0 for b, r in enumerate(ys)])
    if D is not None:
        y = y + D * x
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return y, torch.stack(fins)


def f64(t, grad=True):
    """The tensor's values in fp64 on the CPU, as a leaf."""
    return None if t is None else t.detach().double().cpu().requires_grad_(grad)


def directional(f, args, seed=0, h=1e-5):
    """For every fp64 leaf of args: (a random direction, the central difference of the scalar f along it)."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, a in enumerate(args):
        if a is None:
            out.append(None)
            continue
        d = torch.randn(a.shape, generator=g, dtype=torch.float64)
        with torch.no_grad():
            up, down = list(args), list(args)
            up[i], down[i] = a + h * d, a - h * d
            out.append((d, float((f(*up) - f(*down)) / (2 * h))))
    return out
