"""The layer operators at the sizes they are for: several rounds of rows a block (norm), walks longer than the ring of
copies (convolution), several groups of rows a block (scan step), memories of thousands of tokens (scan), and tensors
of more than 2^31 elements.  References in fp64 on the GPU, whole tensors at once."""

import pytest
import torch

import gated_delta_rule_38_gb300 as gdr
import layer_ref as ref
from test_gpu_layer_ops import BF, DT, F32, FH, cu_of

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=F32, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * scale

    return randn


def check(got, want, name, more=0.0):
    """layer_ref.check on the GPU; `more` is added to the bound."""
    assert got.shape == want.shape, (name, tuple(got.shape), tuple(want.shape))
    a, b = got.detach().double(), want.detach()
    assert torch.isfinite(a).all(), name + ": non-finite values"
    err = float((a - b).norm() / b.norm().clamp(min=1e-30))
    assert err <= ref.bound(got) + more, "%s: relative L2 error %.3e > %.3e" % (name, err, ref.bound(got) + more)


def f64(t):
    return None if t is None else t.detach().double().requires_grad_()


# ---------------------------------------------------------------- RMS norm: several rounds of rows a block

ROWS = [(3000, 4096), (25000, 256), (700, 16384), (1501, 4099), (10007, 250), (3001, 1031), (701, 9001), (613, 16377)]


@DT
@pytest.mark.parametrize("res", [None, "same", "fp32"])
@pytest.mark.parametrize("R,D", ROWS)
def test_norm_rounds(R, D, res, dt):
    randn = gen(R + D)
    x, dy, w = randn(R, D, dtype=dt), randn(R, D, dtype=dt), 1 + 0.1 * randn(D)
    rt = {None: None, "same": dt, "fp32": F32}[res]
    r = None if rt is None else randn(R, D, dtype=rt, scale=2.0)
    y, h, _ = gdr.rms_norm_fwd(x, w, residual=r)
    want, hw = ref.norm(x.double(), w.double(), None if r is None else r.double())
    check(y, want, "y")
    dres = None
    if r is not None:
        check(h, hw, "residual_out")
        dres = randn(R, D, dtype=rt)
    at = x if h is None else h
    dx, dr, dw = gdr.rms_norm_bwd(at, w, dy, dresidual=dres)
    h64, w64 = f64(at), f64(w)
    (ref.norm(h64, w64, None)[0] * dy.double()).sum().backward()
    grad = h64.grad if dres is None else h64.grad + dres.double()
    check(dx, grad, "dx")
    check(dw, w64.grad, "dweight")
    if dr is not None:
        check(dr, grad, "dresidual")


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("R,D", ROWS)
def test_norm_e4m3_rounds(R, D, group):
    randn = gen(R - D)
    x, r, w = randn(R, D, dtype=BF), randn(R, D), 1 + 0.1 * randn(D)
    q, h, scale = gdr.rms_norm_fwd(x, w, residual=r, quant="e4m3", scale_group=group)
    y, hw = ref.norm(x.double(), w.double(), r.double())
    check(h, hw, "residual_out")
    parts = y.split(group or D, -1)
    sw = torch.stack([p.abs().amax(-1) for p in parts], -1) / 448
    check(scale, sw, "scale")
    v = torch.cat([p / sw[..., i:i + 1] for i, p in enumerate(parts)], -1)
    # half a step of e4m3 (2^-4 of the value, 2^-10 below the smallest normal), and the scale's own error
    assert ((q.float().double() - v).abs() <= v.abs() * (2.0 ** -4 + 4e-5) + 2.0 ** -10).all()


# ---------------------------------------------------------------- convolution: walks longer than the ring

def conv(x, w, b, state, lens):
    """(y, final states) through SiLU, every sequence at once."""
    W = w.shape[1]
    ys, fins = [], []
    for n, (row, t0, t1) in enumerate(ref.ranges(x.shape[0], x.shape[1], lens)):
        ext = torch.cat([state[n], x[row, t0:t1]])
        pre = b + sum(ext[i:i + t1 - t0] * w[:, i] for i in range(W))
        ys.append(pre * torch.sigmoid(pre))
        fins.append(ext[t1 - t0:])
    return torch.cat(ys).view(x.shape), torch.stack(fins)


@DT
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,D,lens", [(1, 1024, 12288, None), (1, 1024, 12287, None), (3, 1000, 4099, None),
                                        (1, 1024, 12288, (300, 0, 5, 1, 400, 318)), (1, 1024, 12287, (1, 511, 2, 510, 0))])
def test_conv_long_walks(B, T, D, lens, W, dt):
    randn = gen(T + D + W)
    n = B if lens is None else len(lens)
    x, dy, w, b = randn(B, T, D, dtype=dt), randn(B, T, D, dtype=dt), randn(D, W, scale=W ** -0.5), randn(D, scale=0.3)
    s0, ds, cu = randn(n, W - 1, D, dtype=dt), randn(n, W - 1, D, dtype=dt), cu_of(lens)
    y, fin = gdr.short_conv_fwd(x, w, b, "silu", s0, True, cu)
    grads = gdr.short_conv_bwd(x, w, dy, b, "silu", s0, ds, cu)
    leaves = [f64(t) for t in (x, w, b, s0)]
    yw, fw = conv(*leaves, lens)
    check(y, yw, "y")
    check(fin, fw, "final_state")
    ((yw * dy.double()).sum() + (fw * ds.double()).sum()).backward()
    for got, leaf, name in zip(grads, leaves, ("dx", "dweight", "dbias", "dinitial_state")):
        check(got, leaf.grad, name)


# ---------------------------------------------------------------- scan step: several groups of rows a block

def scan(x, dt, A, B, C, D, z, bias, h):
    """(y, final states) of dense rows, with softplus; h [B,D,N]."""
    delta = torch.nn.functional.softplus(dt + bias, threshold=1e9)
    G = B.shape[2]
    B, C = (m.repeat_interleave(x.shape[2] // G, 2) for m in (B, C))
    ys = []
    for t in range(x.shape[1]):
        h = torch.exp(delta[:, t, :, None] * A) * h + (delta[:, t] * x[:, t])[..., None] * B[:, t]
        ys.append((h * C[:, t]).sum(-1))
    return (torch.stack(ys, 1) + D * x) * z * torch.sigmoid(z), h


def scan_inputs(B, T, D, N, G, dt, seed, step=-2.3, rate=None):
    randn = gen(seed)
    A = -(0.2 + randn(D, N).abs()) if rate is None else torch.full((D, N), -rate, device="cuda")
    return [randn(B, T, D, dtype=dt), (0.3 * randn(B, T, D) + step).to(dt), A, randn(B, T, G, N, dtype=dt),
            randn(B, T, G, N, dtype=dt)], [randn(D), randn(B, T, D, dtype=dt), randn(D, scale=0.1)], randn(B, D, N), randn


@DT
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("B,D,N,G", [(512, 4096, 16, 1), (130, 4100, 16, 2), (250, 4096, 5, 1), (62, 2048, 64, 1), (250, 8193, 3, 3),
                                     (61, 4096, 24, 4)])
def test_scan_step_groups(B, D, N, G, T, dt):
    a, (Ds, z, bias), h0, _ = scan_inputs(B, T, D, N, G, dt, B + D)
    state = h0.clone()
    y = gdr.selective_scan_step(*a, state, Ds, z, bias, True)
    yw, fw = scan(*(t.double() for t in (*a, Ds, z, bias, h0)))
    check(y, yw, "y")
    check(state, fw, "state")


# ---------------------------------------------------------------- scan: a memory of thousands of tokens

@DT
def test_scan_long_memory(dt):
    """delta |A| about 5e-4: a state remembers some 2,000 tokens.  A step's decay is off by at most 2^-22 (the exponential)
    and 2^-24 (its argument, about 1e-3), the state's update by 2^-24; over the memory these add up to at most
    2000 (2^-22 + 2^-24), twice that where a gradient joins states and their adjoints."""
    more = 2000 * (2.0 ** -22 + 2.0 ** -24)
    a, (Ds, z, bias), h0, randn = scan_inputs(1, 8192, 64, 16, 1, dt, 5, step=-0.43, rate=1e-3)
    bias.zero_()
    dy, ds = randn(1, 8192, 64, dtype=dt), randn(1, 64, 16)
    o = (Ds, z, bias, True, h0)
    y, fin, saved = gdr.selective_scan_fwd(*a, *o, save_for_backward=True)
    grads = gdr.selective_scan_bwd(*a, dy, saved, *o, ds)
    leaves = [f64(t) for t in (*a, Ds, z, bias, h0)]
    yw, fw = scan(*leaves)
    check(y, yw, "y", more)
    check(fin, fw, "final_state", more)
    ((yw * dy.double()).sum() + (fw * ds.double()).sum()).backward()
    for got, leaf, name in zip(grads, leaves, ("x", "dt", "A", "B", "C", "D", "z", "bias", "h0")):
        check(got, leaf.grad, "d" + name, 2 * more)


# ---------------------------------------------------------------- more than 2^31 elements

def room(gb):
    if torch.cuda.mem_get_info()[0] < gb * 1e9:
        pytest.skip("needs about %d GB of free device memory" % gb)


@pytest.mark.parametrize("D", [16384, 16383])
def test_norm_beyond_2_to_31_elements(D):
    room(60)
    R = (1 << 17) + 100
    assert R * D > 2 ** 31
    randn = gen(D)
    x, dy, w = randn(R, D, dtype=BF), randn(R, D, dtype=BF), 1 + 0.1 * randn(D)
    y, _, _ = gdr.rms_norm_fwd(x, w)
    q, _, scale = gdr.rms_norm_fwd(x, w, quant="e4m3", scale_group=128)
    dx, _, dw = gdr.rms_norm_bwd(x, w, dy)
    dw64 = torch.zeros(D, dtype=torch.float64, device="cuda")
    for r0 in range(0, R, 8192):
        s = slice(r0, min(R, r0 + 8192))
        h64, w64 = f64(x[s]), f64(w)
        want = ref.norm(h64, w64, None)[0]
        (want * dy[s].double()).sum().backward()
        dw64 += w64.grad
        if r0 == 0 or s.stop == R:
            check(y[s], want, "y")
            check(dx[s], h64.grad, "dx")
            parts = want.detach().split(128, -1)
            check(scale[s], torch.stack([p.abs().amax(-1) for p in parts], -1) / 448, "scale")
            unit = scale[s].double().repeat_interleave(128, -1)[:, :D]
            assert ((q[s].float().double() * unit - want).abs() <= want.abs() * (2.0 ** -4 + 4e-5) + 2.0 ** -10 * unit).all()
    check(dw, dw64, "dweight")


@pytest.mark.parametrize("D", [8200, 8199])
def test_conv_beyond_2_to_31_elements(D):
    room(60)
    T = (1 << 18) + 9
    assert T * D > 2 ** 31
    randn = gen(D)
    x, dy, w, b, s0 = randn(1, T, D, dtype=BF), randn(1, T, D, dtype=BF), randn(D, 4, scale=0.5), randn(D), randn(1, 3, D, dtype=BF)
    y, fin = gdr.short_conv_fwd(x, w, b, "silu", s0, True)
    grads = gdr.short_conv_bwd(x, w, dy, b, "silu", s0, s0)
    for c in (slice(0, 24), slice(D - 24, D)):  # channels do not mix
        leaves = [f64(t) for t in (x[..., c], w[c], b[c], s0[..., c])]
        yw, fw = conv(*leaves, None)
        check(y[..., c], yw, "y")
        check(fin[..., c], fw, "final_state")
        ((yw * dy[..., c].double()).sum() + (fw * s0[..., c].double()).sum()).backward()
        for got, leaf, name in zip((grads[0][..., c], grads[1][c], grads[2][c], grads[3][..., c]), leaves,
                                   ("dx", "dweight", "dbias", "dinitial_state")):
            check(got, leaf.grad, name)


@pytest.mark.parametrize("D", [8192, 8190])
def test_scan_beyond_2_to_31_elements(D):
    room(100)
    B, T = 4110, 64
    assert B * T * D > 2 ** 31
    a, (Ds, z, bias), h0, randn = scan_inputs(B, T, D, 4, 2, BF, D)
    dy = randn(B, T, D, dtype=BF)
    o = (Ds, z, bias, True, h0)
    y, fin, saved = gdr.selective_scan_fwd(*a, *o, save_for_backward=True)
    grads = gdr.selective_scan_bwd(*a, dy, saved, *o)
    for r in (slice(0, 2), slice(B - 2, B)):  # rows do not mix but in the parameters' gradients
        leaves = [f64(t) for t in (a[0][r], a[1][r], a[2], a[3][r], a[4][r], Ds, z[r], bias, h0[r])]
        yw, fw = scan(*leaves)
        check(y[r], yw, "y")
        check(fin[r], fw, "final_state")
        (yw * dy[r].double()).sum().backward()
        for i, name in ((0, "dx"), (1, "ddt"), (3, "dB"), (4, "dC"), (6, "dz"), (8, "dinitial_state")):
            check(grads[i][r], leaves[i].grad, name)
