"""RMS norm, short causal convolution and selective scan against plain fp64 forms: types, odd sizes, ragged packed
batches with empty sequences, states, strided views, special values, gradients (formula and central differences)."""

import pytest
import torch

import gated_delta_rule_38_gb300 as gdr
import layer_ref as ref

pytestmark = pytest.mark.gpu

BF, FH, F32 = torch.bfloat16, torch.float16, torch.float32
DT = pytest.mark.parametrize("dt", [BF, FH], ids=["bf16", "fp16"])


def gen(seed=0):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape, dtype=F32, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()

    return randn


def cu_of(lens):
    if lens is None:
        return None
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def strided(t, extra=24, off=8):
    """The same values as a slice of a wider projection."""
    wide = torch.zeros(t.shape[:-1] + (t.shape[-1] + extra,), dtype=t.dtype, device=t.device)
    wide[..., off:off + t.shape[-1]] = t
    return wide[..., off:off + t.shape[-1]]


def test_error_word_clear():
    gdr.get_error()


# ---------------------------------------------------------------- RMS norm

NORM_D = [1, 7, 8, 100, 128, 136, 333, 1024, 1031, 4096, 8185, 8186, 8192, 8200, 12289, 16377, 16378, 16383, 16384]


@DT
@pytest.mark.parametrize("res", [None, "same", "fp32"])
@pytest.mark.parametrize("D", NORM_D)
def test_norm_forward_backward(D, res, dt):
    randn = gen(D)
    R = 5 if D > 4096 else 37
    x, dy = randn(R, D, dtype=dt), randn(R, D, dtype=dt)
    w = (1 + 0.1 * randn(D)).to(dt if D % 3 else F32)
    rt = {None: None, "same": dt, "fp32": F32}[res]
    r = None if rt is None else randn(R, D, dtype=rt, scale=2.0)
    y, h, scale = gdr.rms_norm_fwd(x, w, residual=r)
    assert scale is None
    want, hw = ref.norm(ref.f64(x), ref.f64(w), ref.f64(r))
    ref.check(y, want, "y")
    dres = None
    if r is not None:
        assert h.dtype == rt
        ref.check(h, hw, "residual_out")
        dres = randn(R, D, dtype=rt)
    else:
        assert h is None
    at = x if h is None else h
    dx, dr, dw = gdr.rms_norm_bwd(at, w, dy, dresidual=dres)
    h64, w64 = ref.f64(at), ref.f64(w)

    def loss(hh, ww):
        out = (ref.norm(hh, ww, None)[0] * ref.f64(dy, False)).sum()
        return out if dres is None else out + (hh * ref.f64(dres, False)).sum()

    loss(h64, w64).backward()
    ref.check(dx, h64.grad, "dx")
    ref.check(dw, w64.grad, "dweight")
    assert (dr is None) == (rt != F32)
    if dr is not None:
        ref.check(dr, h64.grad, "dresidual")
    for (d, fd), got in zip(ref.directional(loss, [h64.detach(), w64.detach()]), (dx, dw)):
        # the difference's own error is below 1e-8 of the terms; the gradient's rounding is bound() of its norm
        dot = float((got.double().cpu() * d).sum())
        assert abs(dot - fd) <= 4 * ref.bound(got) * float(got.double().norm()) + 1e-6 * abs(fd), (dot, fd)


def quantised(y, group):
    """Scales and e4m3 values of the fp64 y."""
    g = group or y.shape[-1]
    parts = y.split(g, -1)
    scale = torch.stack([p.abs().amax(-1).clamp(min=1e-30) for p in parts], -1) / 448
    return scale, torch.cat([p / scale[..., i:i + 1] for i, p in enumerate(parts)], -1)


@DT
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("D", NORM_D)
def test_norm_e4m3(D, group, dt):
    randn = gen(D + 1)
    R = 3 if D > 4096 else 19
    x, r, w = randn(R, D, dtype=dt), randn(R, D, dtype=dt), 1 + 0.1 * randn(D)
    q, h, scale = gdr.rms_norm_fwd(x, w, residual=r, quant="e4m3", scale_group=group)
    assert q.dtype == torch.float8_e4m3fn
    y, hw = ref.norm(ref.f64(x, False), ref.f64(w, False), ref.f64(r, False))
    sw, v = quantised(y, group)
    ref.check(h, hw, "residual_out")
    ref.check(scale, sw, "scale")
    got = q.float().double().cpu()
    # half a step of e4m3 (4 significant bits: 2^-4 of the value, 2^-10 below the smallest normal 2^-6), and what
    # the scale's own error of 2e-5 moves
    assert ((got - v).abs() <= v.abs() * (2.0 ** -4 + 4e-5) + 2.0 ** -10).all()
    assert got.abs().max() == 448


def test_norm_special_rows():
    D = 256
    x = torch.randn(6, D).cuda().to(BF)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 200] = float("inf")
    x[3] = 1e-30
    w = torch.ones(D, device="cuda")
    q, _, scale = gdr.rms_norm_fwd(x, w, quant="e4m3", scale_group=128)
    y, _, _ = gdr.rms_norm_fwd(x, w)
    assert (y[0] == 0).all() and (q[0].float() == 0).all() and (scale[0] > 0).all()
    assert torch.isnan(y[1].float()).all() and torch.isnan(scale[1]).all() and torch.isnan(q[1].float()).all()
    # an infinity makes the row's norm infinite: it is NaN itself, the others 0
    assert torch.isnan(y[2, 200].float()) and (y[2, :200] == 0).all()
    assert torch.isnan(scale[2, 1]) and not torch.isnan(scale[2, 0]) and (q[2, :128].float() == 0).all()
    assert torch.isfinite(y[3].float()).all() and torch.isfinite(q[3].float()).all()
    ref.check(y[4:], ref.norm(ref.f64(x[4:]), ref.f64(w), None)[0], "y")


@pytest.mark.parametrize("D,off", [(512, 8), (512, 3), (131, 5)])
def test_norm_strided_and_shapes(D, off):
    x = torch.randn(2, 9, D).cuda().to(BF)
    w = torch.rand(D, device="cuda") + 0.5
    a = gdr.rms_norm_fwd(x, w)[0]
    assert torch.equal(a, gdr.rms_norm_fwd(strided(x, 24 if off == 8 else 13, off), w)[0]) or D % 8
    ref.check(gdr.rms_norm_fwd(strided(x, 13, off), w)[0], ref.norm(ref.f64(x), ref.f64(w), None)[0], "y")
    t = x.transpose(0, 1)
    ref.check(gdr.rms_norm_fwd(t, w)[0], ref.norm(ref.f64(t), ref.f64(w), None)[0], "transposed")
    dy = torch.randn(2, 9, D).cuda().to(BF)
    assert torch.equal(gdr.rms_norm_bwd(x, w, dy)[2], gdr.rms_norm_bwd(strided(x, 24, 8), w, dy)[2])


def test_norm_no_rows():
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    y, h, _ = gdr.rms_norm_fwd(x, w, residual=x)
    assert y.shape == x.shape and h.shape == x.shape
    dx, _, dw = gdr.rms_norm_bwd(x, w, x)
    assert dx.shape == x.shape and (dw == 0).all()


@DT
def test_norm_autograd(dt):
    randn = gen(5)
    x, r, w = randn(3, 5, 192, dtype=dt), randn(3, 5, 192), randn(192)
    for t in (x, r, w):
        t.requires_grad_()
    y, h = gdr.rms_norm(x, w, r)
    c1, c2 = randn(3, 5, 192, dtype=dt), randn(3, 5, 192)
    ((y * c1).float().sum() + (h * c2).sum()).backward()
    h64, w64 = ref.f64(h), ref.f64(w)
    ((ref.norm(h64, w64, None)[0] * ref.f64(c1, False)).sum() + (h64 * ref.f64(c2, False)).sum()).backward()
    ref.check(x.grad, h64.grad, "dx")
    ref.check(r.grad, h64.grad, "dresidual")
    ref.check(w.grad, w64.grad, "dweight")
    x.grad = None
    gdr.rms_norm(x, w, r)[1].sum().backward()  # only the stream is used further on
    assert (x.grad == 1).all()


# ---------------------------------------------------------------- short causal convolution

CONV = [  # B, T, D, W, lens, states, bias, silu
    (1, 1, 1, 2, None, True, True, True),
    (2, 2, 5, 4, None, True, True, True),
    (3, 33, 64, 4, None, False, True, True),
    (2, 70, 131, 3, None, True, False, True),
    (1, 150, 264, 4, None, True, True, False),
    (2, 129, 8, 2, None, False, False, False),
    (1, 200, 48, 4, (5, 0, 1, 64, 2, 0, 63, 64, 1), True, True, True),
    (1, 131, 37, 4, (0, 0, 64, 3, 0, 1, 63), True, True, True),
    (1, 70, 40, 3, (70, 0), False, False, True),
    (1, 66, 12, 2, (1,) * 66, True, True, True),
    (1, 300, 4100, 4, (3, 129, 168), True, True, True),
]


@DT
@pytest.mark.parametrize("case", CONV, ids=[str(i) for i in range(len(CONV))])
def test_conv(case, dt):
    B, T, D, W, lens, states, use_bias, silu = case
    randn = gen(T + D)
    n = B if lens is None else len(lens)
    x, dy = randn(B, T, D, dtype=dt), randn(B, T, D, dtype=dt)
    pt = dt if D % 2 else F32
    w = randn(D, W, dtype=pt, scale=W ** -0.5)
    b = randn(D, dtype=pt, scale=0.3) if use_bias else None
    s0 = randn(n, W - 1, D, dtype=dt) if states else None
    ds = randn(n, W - 1, D, dtype=dt) if states else None
    act, cu = "silu" if silu else None, cu_of(lens)
    y, fin = gdr.short_conv_fwd(x, w, b, act, s0, True, cu)
    leaves = [ref.f64(t) for t in (x, w, b, s0)]

    def loss(xx, ww, bb, ss):
        yy, ff = ref.conv(xx, ww, bb, silu, ss, lens)
        out = (yy * ref.f64(dy, False)).sum()
        return out if ds is None else out + (ff * ref.f64(ds, False)).sum()

    yw, fw = ref.conv(*leaves[:3], silu, leaves[3], lens)
    ref.check(y, yw, "y")
    ref.check(fin, fw, "final_state")
    loss(*leaves).backward()
    grads = gdr.short_conv_bwd(x, w, dy, b, act, s0, ds, cu)
    for got, leaf, name in zip(grads, leaves, ("dx", "dweight", "dbias", "dinitial_state")):
        assert (got is None) == (leaf is None)
        if got is not None:
            ref.check(got, leaf.grad, name)
    if T <= 70:
        for pair, got in zip(ref.directional(loss, [None if t is None else t.detach() for t in leaves]), grads):
            if pair is not None:
                dot = float((got.double().cpu() * pair[0]).sum())
                assert abs(dot - pair[1]) <= 4 * ref.bound(got) * float(got.double().norm()) + 1e-6 * abs(pair[1])
    assert gdr.get_error() == 0


@DT
@pytest.mark.parametrize("T", [1, 2, 3, 7])
@pytest.mark.parametrize("B,D,W", [(1, 1, 4), (5, 136, 4), (9, 35, 2), (300, 64, 3)])
def test_conv_step(B, D, W, T, dt):
    randn = gen(B + D + T)
    x, s, w, b = randn(B, T, D, dtype=dt), randn(B, W - 1, D, dtype=dt), randn(D, W, dtype=dt), randn(D, dtype=dt)
    yf, ff = gdr.short_conv_fwd(x, w, b, "silu", s, True)
    state = s.clone()
    y = gdr.short_conv_step(x, state, w, b, "silu")
    assert torch.equal(y, yf) and torch.equal(state, ff)
    yw, fw = ref.conv(*(ref.f64(t, False) for t in (x, w, b)), True, ref.f64(s, False), None)
    ref.check(y, yw, "y")
    ref.check(state, fw, "state")


def test_conv_views_and_no_tokens():
    randn = gen(3)
    for D, extra, off in ((64, 24, 8), (64, 5, 3), (33, 8, 8)):
        x, w, dy = randn(2, 40, D, dtype=BF), randn(D, 4, dtype=BF), randn(2, 40, D, dtype=BF)
        v = strided(x, extra, off)
        for a, b in zip(gdr.short_conv_fwd(x, w, None, "silu", None, True), gdr.short_conv_fwd(v, w, None, "silu", None, True)):
            assert torch.equal(a, b)
        got, want = gdr.short_conv_bwd(v, w, dy, None, "silu"), gdr.short_conv_bwd(x, w, dy, None, "silu")
        assert torch.equal(got[0], want[0])
        ref.check(got[1], want[1].double(), "dweight")
    x = torch.empty(2, 0, 32, dtype=BF, device="cuda")
    s, w = randn(2, 3, 32, dtype=BF), randn(32, 4, dtype=BF)
    y, fin = gdr.short_conv_fwd(x, w, None, None, s, True)
    assert y.shape == x.shape and torch.equal(fin, s)
    dx, dw, _, dsi = gdr.short_conv_bwd(x, w, x, None, None, s, s)
    assert (dw == 0).all() and torch.equal(dsi, s)


# ---------------------------------------------------------------- selective scan

SCAN = [  # B, T, D, N, G, lens, states, D and z and bias, softplus
    (1, 1, 1, 1, 1, None, True, True, True),
    (2, 3, 6, 4, 2, None, True, True, True),
    (1, 17, 40, 16, 1, None, True, True, True),
    (2, 33, 136, 16, 1, None, False, True, True),
    (1, 64, 128, 16, 1, None, True, False, True),
    (2, 50, 30, 5, 3, None, True, True, False),
    (1, 40, 260, 8, 1, None, True, True, True),
    (1, 35, 9, 3, 1, None, True, True, True),
    (1, 30, 70, 32, 1, None, True, True, True),
    (1, 37, 34, 64, 2, None, True, True, True),
    (1, 20, 5, 17, 1, None, True, True, True),
    (1, 1000, 24, 16, 1, None, True, True, True),
    (1, 700, 20, 6, 2, None, True, True, True),
    (1, 90, 24, 16, 1, (5, 0, 1, 16, 2, 0, 31, 32, 3, 0), True, True, True),
    (1, 80, 17, 12, 1, (0, 16, 16, 0, 1, 47), False, True, True),
    (1, 66, 8, 2, 1, (1,) * 66, True, True, True),
    (1, 900, 16, 16, 1, (64, 0, 1, 500, 128, 207), True, True, True),
    (1, 600, 12, 40, 1, (599, 1), True, True, True),
]


def scan_inputs(case, dt):
    B, T, D, N, G, lens, states, rich, softplus = case
    randn = gen(T + 7 * D + N)
    n = B if lens is None else len(lens)
    s = dict(x=randn(B, T, D, dtype=dt), A=-(0.2 + randn(D, N).abs()), B=randn(B, T, G, N, dtype=dt),
             C=randn(B, T, G, N, dtype=dt))
    # steps around a tenth; without softplus they are given as such
    s["dt"] = (randn(B, T, D) - 2.3).to(dt) if softplus else randn(B, T, D).abs().mul(0.1).to(dt)
    s["D"], s["z"], s["bias"] = (randn(D), randn(B, T, D, dtype=dt), randn(D, scale=0.3)) if rich else (None, None, None)
    if rich and not softplus:
        s["bias"] = s["bias"].abs() * 0.1
    s["h0"] = randn(n, D, N) if states else None
    return s, randn, n


@DT
@pytest.mark.parametrize("case", SCAN, ids=[str(i) for i in range(len(SCAN))])
def test_scan(case, dt):
    B, T, D, N, G, lens, states, rich, softplus = case
    s, randn, n = scan_inputs(case, dt)
    dy, ds = randn(B, T, D, dtype=dt), randn(n, D, N) if states else None
    cu = cu_of(lens)
    y, fin, saved = gdr.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], softplus,
                                           s["h0"], True, cu, save_for_backward=True)
    y2, fin2, none = gdr.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], softplus,
                                            s["h0"], True, cu)
    assert none is None and torch.equal(y, y2) and torch.equal(fin, fin2)
    order = ("x", "dt", "A", "B", "C", "D", "z", "bias", "h0")
    leaves = [ref.f64(s[k]) for k in order]

    def outs(x, d, A, Bm, Cm, Ds, z, bias, h0):
        return ref.scan(x, d, A, Bm, Cm, Ds, z, bias, softplus, h0, lens)

    def loss(*a):
        yy, ff = outs(*a)
        out = (yy * ref.f64(dy, False)).sum()
        return out if ds is None else out + (ff * ref.f64(ds, False)).sum()

    yw, fw = outs(*leaves)
    ref.check(y, yw, "y")
    ref.check(fin, fw, "final_state")
    loss(*leaves).backward()
    grads = gdr.selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], dy, saved, s["D"], s["z"], s["bias"],
                                   softplus, s["h0"], ds, cu)
    for got, leaf, name in zip(grads, leaves, order):
        assert (got is None) == (leaf is None), name
        if got is not None:
            ref.check(got, leaf.grad, "d" + name)
    if T <= 40:
        for pair, got in zip(ref.directional(loss, [None if t is None else t.detach() for t in leaves], h=1e-6), grads):
            if pair is not None:
                dot = float((got.double().cpu() * pair[0]).sum())
                assert abs(dot - pair[1]) <= 4 * ref.bound(got) * float(got.double().norm()) + 1e-5 * abs(pair[1])
    assert gdr.get_error() == 0


@DT
@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("B,D,N,G", [(1, 1, 1, 1), (3, 40, 16, 2), (5, 33, 6, 1), (2, 70, 64, 1), (130, 24, 20, 3), (2, 9, 3, 1)])
def test_scan_step(B, D, N, G, T, dt):
    s, _, _ = scan_inputs((B, T, D, N, G, None, True, True, True), dt)
    state = s["h0"].clone()
    y = gdr.selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], state, s["D"], s["z"], s["bias"], True)
    yw, fw = ref.scan(*(ref.f64(s[k], False) for k in ("x", "dt", "A", "B", "C", "D", "z", "bias")), True,
                      ref.f64(s["h0"], False), None)
    ref.check(y, yw, "y")
    ref.check(state, fw, "state")


def test_scan_views():
    s, randn, _ = scan_inputs((2, 40, 64, 16, 1, None, True, True, True), BF)
    dy = randn(2, 40, 64, dtype=BF)

    def call(t):
        a = (t["x"], t["dt"], t["A"], t["B"], t["C"])
        o = (t["D"], t["z"], t["bias"], True, t["h0"])
        y, fin, saved = gdr.selective_scan_fwd(*a, *o, save_for_backward=True)
        return (y, fin) + gdr.selective_scan_bwd(*a, dy, saved, *o)

    want = call(s)
    for extra, off in ((24, 8), (5, 3)):
        v = dict(s)
        for k in ("x", "dt", "z"):
            v[k] = strided(s[k], extra, off)
        for k in ("B", "C"):
            v[k] = strided(s[k].flatten(2), extra, off).unflatten(2, (1, 16))
        for a, b in zip(call(v), want):
            assert torch.equal(a, b)


def test_scan_no_tokens():
    s, randn, _ = scan_inputs((2, 0, 24, 16, 1, None, True, True, True), BF)
    y, fin, saved = gdr.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], True,
                                           s["h0"], save_for_backward=True)
    assert y.shape == (2, 0, 24) and torch.equal(fin, s["h0"])
    g = gdr.selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["x"], saved, s["D"], s["z"], s["bias"], True,
                               s["h0"], s["h0"])
    assert (g[2] == 0).all() and (g[5] == 0).all() and (g[7] == 0).all() and torch.equal(g[8], s["h0"])


def test_scan_reset_and_extremes():
    """A very large step forgets everything (exp(delta A) = 0), a step of zero changes nothing."""
    s, _, _ = scan_inputs((1, 12, 32, 16, 1, None, True, True, False), BF)
    s["dt"][:, 5] = 2000.0
    s["dt"][:, 8] = 0.0
    s["bias"].zero_()
    o = (s["D"], s["z"], s["bias"], False, s["h0"])
    y, fin, _ = gdr.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], *o)
    yw, fw = ref.scan(*(ref.f64(s[k], False) for k in ("x", "dt", "A", "B", "C", "D", "z", "bias")), False,
                      ref.f64(s["h0"], False), None)
    ref.check(y, yw, "y")
    ref.check(fin, fw, "final_state")


# ---------------------------------------------------------------- across the operators

def test_decode_continues_prefill():
    """Convolution and scan over a prompt, then token by token from their states, equal the whole sequence at once."""
    randn = gen(11)
    T, cut, D = 45, 38, 64
    x, w = randn(2, T, D, dtype=BF), randn(D, 4, dtype=BF)
    yc, fc = gdr.short_conv_fwd(x, w, None, "silu", None, True)
    y1, s1 = gdr.short_conv_fwd(x[:, :cut].contiguous(), w, None, "silu", None, True)
    parts = [y1] + [gdr.short_conv_step(x[:, t:t + 1], s1, w, None, "silu") for t in range(cut, T)]
    assert torch.equal(torch.cat(parts, 1), yc) and torch.equal(s1, fc)
    s, _, _ = scan_inputs((2, T, D, 16, 1, None, False, True, True), BF)
    tok = lambda a, b: [s[k][:, a:b] for k in ("x", "dt")] + [s["A"]] + [s[k][:, a:b] for k in ("B", "C")]  # noqa: E731
    opt = lambda a, b: dict(D=s["D"], z=s["z"][:, a:b], dt_bias=s["bias"], dt_softplus=True)  # noqa: E731
    ya, fa, _ = gdr.selective_scan_fwd(*tok(0, T), **opt(0, T))
    y1, st, _ = gdr.selective_scan_fwd(*tok(0, cut), **opt(0, cut))
    parts = [y1] + [gdr.selective_scan_step(*tok(t, t + 1), st, **opt(t, t + 1)) for t in range(cut, T)]
    # two kernels with their own order of fp32 sums: equal to the types' bounds
    ref.check(torch.cat(parts, 1), ya.double(), "y")
    ref.check(st, fa.double(), "state")


def _all_ops(s, w, nw, dy):
    h, res, _ = gdr.rms_norm_fwd(s["x"], nw, residual=s["dt"])
    u, _ = gdr.short_conv_fwd(h, w, None, "silu")
    o = (s["D"], s["z"], s["bias"], True, s["h0"])
    y, fin, saved = gdr.selective_scan_fwd(u, s["dt"], s["A"], s["B"], s["C"], *o, save_for_backward=True)
    g = gdr.selective_scan_bwd(u, s["dt"], s["A"], s["B"], s["C"], dy, saved, *o)
    c = gdr.short_conv_bwd(h, w, g[0], None, "silu")
    n = gdr.rms_norm_bwd(res, nw, c[0])
    return [y, fin, *[t for t in g + c + n if t is not None]]


def _chain_inputs():
    s, randn, _ = scan_inputs((2, 300, 72, 16, 1, None, True, True, True), BF)
    return s, randn(72, 4, dtype=BF), randn(72), randn(2, 300, 72, dtype=BF)


def test_deterministic_and_on_another_stream():
    args = _chain_inputs()
    want = _all_ops(*args)
    for a, b in zip(_all_ops(*args), want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _all_ops(*args)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_graph_capture():
    args = _chain_inputs()
    want = _all_ops(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _all_ops(*args)
    for t in got:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@DT
def test_autograd_chain(dt):
    """The three operators chained under autograd equal the hand-made call sequence."""
    s, w, nw, dy = _chain_inputs()
    leaves = [t.clone().requires_grad_() for t in (s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], s["h0"], w, nw)]
    x, d, A, B, C, Ds, z, bias, h0, cw, cn = leaves
    h, res = gdr.rms_norm(x, cn, d)
    u, _ = gdr.short_conv(h, cw, None, "silu")
    y, _ = gdr.selective_scan(u, s["dt"], A, B, C, Ds, z, bias, True, h0)
    y.backward(dy)
    want = _all_ops(s, w, nw, dy)
    assert torch.equal(y, want[0])
    g = want[2:]
    for leaf, got in zip((A, B, C, Ds, z, bias, h0), g[2:9]):
        assert torch.equal(leaf.grad, got)
    assert torch.equal(cw.grad, g[10]) and torch.equal(x.grad, g[11]) and torch.equal(cn.grad, g[12])


def test_malformed_cu_seqlens_is_latched():
    """Offsets that decrease stay inside the buffers and are reported in the error word."""
    s, randn, _ = scan_inputs((1, 60, 16, 16, 1, (20, 20, 20), True, True, True), BF)
    bad = torch.tensor([0, 40, 20, 60], dtype=torch.int32, device="cuda")
    assert gdr.get_error() == 0
    gdr.short_conv_fwd(s["x"], randn(16, 4, dtype=BF), None, None, randn(3, 3, 16, dtype=BF), True, bad)
    assert gdr.get_error() == 8
    _, _, saved = gdr.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], True, s["h0"],
                                         True, bad, save_for_backward=True)
    assert gdr.get_error() == 8
    gdr.selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["x"], saved, s["D"], s["z"], s["bias"], True,
                           s["h0"], s["h0"], bad)
    assert gdr.get_error() == 8
    gdr.short_conv_bwd(s["x"], randn(16, 4, dtype=BF), s["x"], cu_seqlens=bad)
    assert gdr.get_error() == 8


def test_profiler_names():
    gdr._lib.profile_enable(True)
    _all_ops(*_chain_inputs())
    got = gdr._lib.profile_read()
    gdr._lib.profile_enable(False)
    assert {"norm_fwd", "norm_bwd", "conv_fwd", "conv_bwd", "scan_fwd", "scan_bwd", "reduce"} <= set(got)


def test_refusals():
    """Tensors that do not fit are refused by name before anything is launched."""
    randn = gen(0)
    x, w = randn(2, 6, 32, dtype=BF), randn(32, 4, dtype=BF)
    f = _raises
    nw = randn(32)
    f(gdr.rms_norm_fwd, "x", x.float(), nw)
    f(gdr.rms_norm_fwd, "weight", x, nw[:31])
    f(gdr.rms_norm_fwd, "weight", x, nw.half())
    f(gdr.rms_norm_fwd, "residual", x, nw, residual=x[:1])
    f(gdr.rms_norm_fwd, "quant", x, nw, quant="int8")
    f(gdr.rms_norm_fwd, "scale_group", x, nw, quant="e4m3", scale_group=64)
    f(gdr.rms_norm_fwd, "out", x, nw, out=x.float())
    f(gdr.rms_norm_bwd, "h", x, nw, x[:1])
    f(gdr.rms_norm_bwd, "dtype", x, nw, x, dtype=FH)
    f(gdr.short_conv_fwd, "weight", x, w[:31])
    f(gdr.short_conv_fwd, "weight", x, randn(32, 5, dtype=BF))
    f(gdr.short_conv_fwd, "bias", x, w, randn(32))
    f(gdr.short_conv_fwd, "activation", x, w, activation="relu")
    f(gdr.short_conv_fwd, "initial_state", x, w, initial_state=randn(2, 2, 32, dtype=BF))
    f(gdr.short_conv_fwd, "B = 1", x, w, cu_seqlens=cu_of((3, 3)))
    f(gdr.short_conv_step, "state", x, randn(2, 3, 32), w)
    f(gdr.short_conv_bwd, "dy", x, w, x.transpose(1, 2))
    s, _, _ = scan_inputs((2, 6, 32, 16, 2, None, True, True, True), BF)
    a = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    for i, name in enumerate("x dt A B C".split()):
        bad = list(a)
        bad[i] = bad[i].double()
        f(gdr.selective_scan_fwd, name, *bad)
        bad[i] = None
        f(gdr.selective_scan_fwd, name, *bad)
    f(gdr.selective_scan_fwd, "B", s["x"], s["dt"], s["A"], s["B"][..., :8], s["C"])
    f(gdr.selective_scan_fwd, "initial_state", *a, initial_state=s["h0"].transpose(1, 2))
    f(gdr.selective_scan_step, "state", *a, s["h0"].half())
    f(gdr.selective_scan_bwd, "saved", *a, s["x"], torch.empty(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gdr.GdrError):
        gdr.selective_scan_fwd(s["x"], s["dt"], randn(32, 80), randn(2, 6, 1, 80, dtype=BF), randn(2, 6, 1, 80, dtype=BF))
    with pytest.raises(gdr.GdrError):
        gdr.rms_norm_fwd(randn(2, 16392, dtype=BF), randn(16392))


def _raises(fn, match, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)
