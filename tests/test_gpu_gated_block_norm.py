"""The gated norm and the block norm against their plain fp64 forms: widths, types, gates, residual streams, views, special
rows, gradients (formula and differences), streams and graphs; and a layer made of them with linear attention."""

import pytest
import torch

import gated_delta_rule_38_gb300 as gdr
import layer_ref as lref
import linear_ref as ref

pytestmark = pytest.mark.gpu

BF, FH, F32 = torch.bfloat16, torch.float16, torch.float32
DT = pytest.mark.parametrize("dt", [BF, FH], ids=["bf16", "fp16"])
# one column; short rows that share a block; the ends of whole vectors; more threads a row; the widest
WIDTHS = [1, 2, 7, 8, 9, 100, 128, 333, 505, 512, 513, 1031, 2047, 4096, 4097, 4099, 5121, 8185, 8192, 8193, 8200, 16375, 16376, 16384]


def gen(seed=0):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape, dtype=F32, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()

    return randn


def check(got, want, name):
    """lref.bound: one rounding, or fp32 sums.  At D = 1 every gradient through a norm is what two equal terms leave, which the
    kernels form without the difference; the same bound holds."""
    lref.check(got, want, name)


@DT
@pytest.mark.parametrize("name", ["silu", "sigmoid"])
@pytest.mark.parametrize("D", WIDTHS)
def test_gated(D, name, dt):
    randn = gen(D)
    rows = (7, 3) if D > 2000 else (301, 3)
    x, g, dy = (randn(*rows, D, dtype=dt) for _ in range(3))
    w = (1 + 0.1 * randn(D)).to(dt if D % 3 else F32)
    y = gdr.gated_rms_norm_fwd(x, g, w, activation=name)
    leaves = [lref.f64(t) for t in (x, g, w)]
    out = ref.gated(*leaves, name)
    check(y, out, "y")
    (out * dy.double().cpu()).sum().backward()
    for n, got, leaf in zip(("dx", "dgate", "dweight"), gdr.gated_rms_norm_bwd(x, g, w, dy, activation=name), leaves):
        check(got, leaf.grad, n)


@DT
@pytest.mark.parametrize("res", ["same", "fp32"])
@pytest.mark.parametrize("D", WIDTHS)
def test_block(D, res, dt):
    randn = gen(D)
    R = 11 if D > 2000 else 903
    rt = dt if res == "same" else F32
    post, name = D % 5 != 2, ("sigmoid", None, "silu", "none")[D % 4]
    x, dy = randn(R, D, dtype=dt), randn(R, D, dtype=dt)
    r, dres = randn(R, D, dtype=rt, scale=2.0), randn(R, D, dtype=rt) if D % 3 else None
    wt = dt if D % 2 else F32
    w, pw = (1 + 0.1 * randn(D)).to(wt), (1 + 0.1 * randn(D)).to(wt) if post else None
    g = None if name == "none" else randn(R, D, dtype=dt)
    opt = dict(post_weight=pw, gate=g, gate_activation=None if name == "none" else name, residual_scale=0.25)
    y, h = gdr.block_norm_fwd(x, r, w, **opt)
    assert h.dtype == rt
    xs, ws, ps, gs = (lref.f64(t) for t in (x, w, pw, g))
    hs = ref.block_sum(xs, lref.f64(r, False), ps, gs, name, 0.25)
    check(h, hs, "residual_out")
    check(y, ref.rms(hs, 1e-6) * ws, "y")
    at = lref.f64(h)  # the gradients are those at the stored sum
    total = (ref.rms(at, 1e-6) * ws * dy.double().cpu()).sum()
    if dres is not None:
        total = total + (at * dres.double().cpu()).sum()
    total.backward()
    hs.backward(at.grad)
    got = gdr.block_norm_bwd(x, h, w, dy, dresidual=dres, **opt)
    for n, t, want in zip(("dx", "dresidual", "dweight", "dpost_weight", "dgate"), got,
                          (xs.grad, at.grad, ws.grad, None if ps is None else ps.grad, None if gs is None else gs.grad)):
        assert (t is None) == (want is None), n
        if t is not None:
            check(t, want, n)


def test_differences():
    randn = gen(2)
    x, g, w, dy = randn(40, 96, dtype=FH), randn(40, 96, dtype=FH), 1 + 0.1 * randn(96), randn(40, 96, dtype=FH)
    r, pw = randn(40, 96), 1 + 0.1 * randn(96)
    c = dy.double().cpu()

    def off(got, pairs):
        for (d, fd), t in zip(pairs, got):
            dot = float((t.double().cpu() * d).sum())
            assert abs(dot - fd) <= 4 * lref.bound(t) * float(t.double().norm()) + 1e-6 * abs(fd), (dot, fd)

    args = [lref.f64(t, False) for t in (x, g, w)]
    off(gdr.gated_rms_norm_bwd(x, g, w, dy), lref.directional(lambda a, b, e: (ref.gated(a, b, e, "silu") * c).sum(), args))
    opt = dict(post_weight=pw, gate=g, gate_activation="silu", residual_scale=0.5)
    h = gdr.block_norm_fwd(x, r, w, **opt)[1]  # (fp32: the sum as good as unrounded)

    def loss(a, b, e, p, q):
        return (ref.rms(ref.block_sum(a, b, p, q, "silu", 0.5), 1e-6) * e * c).sum()

    off(gdr.block_norm_bwd(x, h, w, dy, **opt), lref.directional(loss, [lref.f64(t, False) for t in (x, r, w, pw, g)]))


def test_rows_past_the_grid():
    """More rows than the resident blocks take in one round, heads and shifts included."""
    for shape in ((40000, 3, 128), (3001, 2, 1027), (20011, 1, 33)):
        randn = gen(shape[0])
        x, g, dy = (randn(*shape, dtype=BF) for _ in range(3))
        w = 1 + 0.1 * randn(shape[-1])
        leaves = [t.double().requires_grad_() for t in (x, g, w)]
        out = ref.gated(*leaves, "silu")
        (out * dy.double()).sum().backward()
        check(gdr.gated_rms_norm_fwd(x, g, w), out, "y")
        for got, leaf in zip(gdr.gated_rms_norm_bwd(x, g, w, dy), leaves):
            check(got, leaf.grad, "gradient")


def test_special_rows():
    D = 256
    x, g = gen(1)(8, D, dtype=BF), gen(2)(8, D, dtype=BF)
    x[0], x[1, 3], x[3] = 0, float("nan"), 1e-30
    g[4], g[5], g[6, 7], g[7] = 1000.0, -1000.0, float("nan"), float("-inf")
    w = torch.ones(D, device="cuda")
    y = gdr.gated_rms_norm_fwd(x, g, w)
    assert (y[0] == 0).all() and torch.isnan(y[1]).all() and torch.isfinite(y[2:6].float()).all()
    assert torch.isnan(y[6, 7]) and torch.isfinite(y[6, :7].float()).all()
    assert y[5].abs().max() < 1e-30 and y[7].abs().max() < 1e-30  # (silu far below: -g e^g, or what is left of it at -80)
    ref.check(y[4], ref.gated(lref.f64(x[4], False), lref.f64(g[4], False), torch.ones(D, dtype=torch.float64), "silu"), 1.05 * 2.0 ** -8, "y")
    dx, dg, dw = gdr.gated_rms_norm_bwd(x[2:6], g[2:6], w, torch.ones_like(x[2:6]))
    assert all(torch.isfinite(t.float()).all() for t in (dx, dg, dw))
    r = torch.zeros(8, D, device="cuda")
    y, h = gdr.block_norm_fwd(x, r, w, post_weight=w)
    assert (y[0] == 0).all() and (h[0] == 0).all() and torch.isnan(h[1]).all() and torch.isfinite(h[2:]).all()
    big = torch.full((2, D), 6e4, dtype=FH, device="cuda")
    y, h = gdr.block_norm_fwd(big, torch.full((2, D), 1e18, device="cuda"), w)
    assert (y == 1).all()


@pytest.mark.parametrize("D", [64, 67])
def test_views(D):
    """Strided gates and inputs, heads side by side; other views are copied.  The same bits."""
    B, T, H = 2, 19, 3
    randn = gen(D)
    wide = randn(B, T, 2 * H * D + 8, dtype=BF)
    x, g = (wide[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(2))
    dy, w = randn(B, T, H, D, dtype=BF), randn(D)
    args = (x.contiguous(), g.contiguous(), w)
    assert torch.equal(gdr.gated_rms_norm_fwd(x, g, w), gdr.gated_rms_norm_fwd(*args))
    for a, b in zip(gdr.gated_rms_norm_bwd(x, g, w, dy.transpose(0, 1).contiguous().transpose(0, 1)), gdr.gated_rms_norm_bwd(*args, dy)):
        assert torch.equal(a, b)
    xm, gm = x[:, :, 0], g[:, :, 1]  # one head's columns
    r = randn(B, T, D)
    a, b = gdr.block_norm_fwd(xm, r, w, gate=gm), gdr.block_norm_fwd(xm.contiguous(), r, w, gate=gm.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    t = torch.empty(B * T * D + 1, dtype=BF, device="cuda")[1:].view(B, T, D).copy_(xm)
    assert torch.equal(gdr.block_norm_fwd(t, r, w, gate=gm)[0], a[0])
    low = torch.zeros(B * T * D + 4, device="cuda")[4:].view(B, T, D).copy_(r)  # 16 bytes past a sector
    assert torch.equal(gdr.block_norm_fwd(xm, low, w, gate=gm)[1], a[1])


def test_slices_off_16_bytes():
    """Gradients that are slices of a larger one, streams and weights that are slices of flat tensors: copied, the same bits."""
    D, n = 67, 5
    randn = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731

    def at(t):  # the same numbers 2 or 4 bytes past a boundary
        return torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)

    x, g, r, w, pw, dy, dh = randn(n, D).half(), randn(n, D).half(), randn(n, D), randn(D), randn(D), randn(n, D).half(), randn(n, D)
    assert at(dy).data_ptr() % 16 and at(r).data_ptr() % 16 and at(dy).is_contiguous()
    pairs = [(gdr.gated_rms_norm_fwd(x, g, w), gdr.gated_rms_norm_fwd(at(x), at(g), at(w))),
             (gdr.gated_rms_norm_bwd(x, g, w, dy), gdr.gated_rms_norm_bwd(at(x), at(g), at(w), at(dy))),
             (gdr.block_norm_fwd(x, r, w, pw, g), gdr.block_norm_fwd(at(x), at(r), at(w), at(pw), at(g))),
             (gdr.block_norm_bwd(x, r, w, dy, dh, pw, g), gdr.block_norm_bwd(at(x), at(r), at(w), at(dy), at(dh), at(pw), at(g)))]
    for a, b in pairs:
        for s, t in zip(*((z,) if isinstance(z, torch.Tensor) else z for z in (a, b))):
            assert torch.equal(s, t)
    leaf = x.clone().requires_grad_()
    y = torch.cat([gdr.gated_rms_norm(leaf[:3], g[:3], w), gdr.gated_rms_norm(leaf[3:], g[3:], w)])
    y.backward(dy)
    assert torch.equal(leaf.grad, pairs[1][0][0])


def test_neighbours_stay():
    """Rows of odd width are written to their last element and not beyond."""
    D = 131
    buf = torch.full((9 * D + 8,), 7.0, dtype=BF, device="cuda")
    x, w = gen(4)(9, D, dtype=BF), torch.ones(D, device="cuda")
    gdr.gated_rms_norm_fwd(x, x, w, out=buf[:9 * D].view(9, D))
    assert (buf[9 * D:] == 7).all() and torch.equal(buf[:9 * D].view(9, D), gdr.gated_rms_norm_fwd(x, x, w))


def test_no_rows():
    e, w = torch.empty(0, 4, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    assert gdr.gated_rms_norm_fwd(e, e, w).shape == e.shape
    dx, dg, dw = gdr.gated_rms_norm_bwd(e, e, w, e)
    assert dx.shape == dg.shape == e.shape and (dw == 0).all()
    y, h = gdr.block_norm_fwd(e, e, w, post_weight=w)
    assert y.shape == h.shape == e.shape
    got = gdr.block_norm_bwd(e, e, w, e, post_weight=w, gate=e)
    assert (got[2] == 0).all() and (got[3] == 0).all() and got[4].shape == e.shape


def test_same_bits_streams_and_graphs():
    randn = gen(8)
    x, g, dy, r = (randn(700, 515, dtype=BF) for _ in range(4))
    w, pw = randn(515), randn(515)

    def step():
        y, h = gdr.block_norm_fwd(x, r, w, post_weight=pw, gate=g, gate_activation="sigmoid", residual_scale=0.5)
        return y, h, *gdr.block_norm_bwd(x, h, w, dy, r, pw, g, "sigmoid", 0.5), gdr.gated_rms_norm_fwd(x, g, w), *gdr.gated_rms_norm_bwd(x, g, w, dy)

    want = step()
    assert all(torch.equal(a, b) for a, b in zip(want, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(step(), res))


def test_autograd():
    randn = gen(5)
    x, g, w, c = randn(3, 5, 2, 64, dtype=BF), randn(3, 5, 2, 64, dtype=BF), randn(64), randn(3, 5, 2, 64, dtype=BF)
    leaves = [t.clone().requires_grad_() for t in (x, g, w)]
    (gdr.gated_rms_norm(*leaves) * c).float().sum().backward()
    assert all(torch.equal(l.grad, t) for l, t in zip(leaves, gdr.gated_rms_norm_bwd(x, g, w, c)))
    r, pw = randn(3, 5, 2, 64), randn(64)
    leaves = [t.clone().requires_grad_() for t in (x, r, w, pw, g)]
    y, h = gdr.block_norm(*leaves[:3], post_weight=leaves[3], gate=leaves[4], gate_activation="silu", residual_scale=0.5)
    ((y * c).float().sum() + (2 * h).sum()).backward()
    want = gdr.block_norm_bwd(x, h.detach(), w, c, torch.full_like(r, 2.0), pw, g, "silu", 0.5)
    assert all(torch.equal(l.grad, t) for l, t in zip(leaves, want))
    x2 = x.clone().requires_grad_()
    gdr.block_norm(x2, r, w)[1].sum().backward()  # only the stream is used further on
    assert (x2.grad == 1).all()
    x3 = x.clone().requires_grad_()
    (d,) = torch.autograd.grad(gdr.gated_rms_norm(x3, g, w).float().square().sum(), x3, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        d.sum().backward()


def test_offsets_past_31_bits():
    R, D = 540000, 4096
    x = torch.empty(R, D, dtype=BF, device="cuda").normal_()
    w = 1 + 0.1 * gen(1)(D)
    y = gdr.gated_rms_norm_fwd(x, x, w)
    check(y[-5:], ref.gated(lref.f64(x[-5:], False), lref.f64(x[-5:], False), lref.f64(w, False), "silu"), "y")
    h = gdr.block_norm_fwd(y, x, w, post_weight=w, gate=x, gate_activation="sigmoid", residual_scale=0.5)[1]
    tail = [lref.f64(t[-5:], False) for t in (y, x)]
    check(h[-5:], ref.block_sum(tail[0], tail[1], lref.f64(w, False), tail[1], "sigmoid", 0.5), "residual_out")
    dx = gdr.block_norm_bwd(y, h, w, x, post_weight=w)[0]
    xs, hs = lref.f64(y[-5:]), lref.f64(h[-5:])
    (ref.rms(hs, 1e-6) * lref.f64(w, False) * tail[1]).sum().backward()
    ref.block_sum(xs, 0, lref.f64(w, False), None, None, 1.0).backward(hs.grad)
    check(dx[-5:], xs.grad, "dx")


def test_refusals():
    randn = gen(1)
    x, g, w, r = randn(4, 64, dtype=BF), randn(4, 64, dtype=BF), randn(64), randn(4, 64)
    bad = [lambda: gdr.gated_rms_norm_fwd(x, g[:, :32], w), lambda: gdr.gated_rms_norm_fwd(x, g.half(), w),
           lambda: gdr.gated_rms_norm_fwd(x, g, w[:32]), lambda: gdr.gated_rms_norm_fwd(x, g, w.half()),
           lambda: gdr.gated_rms_norm_fwd(x, g, w, activation="relu"), lambda: gdr.gated_rms_norm_fwd(x.float(), g.float(), w),
           lambda: gdr.gated_rms_norm_bwd(x, g, w, r), lambda: gdr.block_norm_fwd(x, r[:2], w),
           lambda: gdr.block_norm_fwd(x, r, w, post_weight=w.bfloat16()), lambda: gdr.block_norm_fwd(x, r, w, gate_activation="silu"),
           lambda: gdr.block_norm_fwd(x, r, w, gate=g, gate_activation="relu"), lambda: gdr.block_norm_fwd(x, r.half(), w),
           lambda: gdr.block_norm_bwd(x, r, w, g, dresidual=g), lambda: gdr.block_norm_fwd(x, r.cpu(), w)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    wide, ww = randn(2, 16377, dtype=BF), randn(16377)
    for call in (lambda: gdr.gated_rms_norm_fwd(x, g, w, out=x), lambda: gdr.block_norm_fwd(x, r, w, out=x),
                 lambda: gdr.gated_rms_norm_fwd(wide, wide, ww), lambda: gdr.block_norm_fwd(wide, wide, ww)):
        with pytest.raises(gdr.GdrError):
            call()


class Layer(torch.nn.Module):
    """A block of linear attention: projection, attention, norm and gate a head, projection, and the norms around the sum."""

    def __init__(self, width=96, heads=4, dim=32):
        super().__init__()
        self.heads, self.dim, self.inner = heads, dim, heads * dim
        lin = lambda i, o: torch.nn.Linear(i, o, bias=False, dtype=BF, device="cuda")  # noqa: E731
        self.qkvg, self.out = lin(width, 4 * self.inner), lin(self.inner, width)
        self.norm, self.post, self.pre = (torch.nn.Parameter(torch.ones(n, device="cuda")) for n in (dim, width, width))
        self.register_buffer("decay", (-torch.exp2(-8.0 * torch.arange(1, heads + 1) / heads)).cuda())

    def forward(self, x, h, cu=None, state=None):
        B, T, _ = x.shape
        q, k, v, g = (t.unflatten(-1, (self.heads, self.dim)) for t in self.qkvg(x).split(self.inner, -1))
        if state is None:
            o, _ = gdr.linear_attention(q, k, v, self.decay, cu_seqlens=cu)
        elif T == 1 and "s" in state:
            o = gdr.linear_attention_step(q, k, v, self.decay, state["s"])
        else:
            o, state["s"] = gdr.linear_attention_fwd(q, k, v, self.decay, initial_state=state.get("s"), output_final_state=True, cu_seqlens=cu)
        y = self.out(gdr.gated_rms_norm(o, g, self.norm).flatten(-2))
        return gdr.block_norm(y, h, self.pre, post_weight=self.post, residual_scale=0.5)


def test_layer():
    """Two layers: their gradients against fp64, and serving (a packed batch of prompts, then token by token) against whole
    sequences."""
    torch.manual_seed(3)
    layers = [Layer(), Layer()]
    h0 = gen(6)(2, 60, 96)
    x0 = gdr.rms_norm_fwd(h0.bfloat16(), torch.ones(96, device="cuda"))[0]
    x, h = x0, h0
    for m in layers:
        x, h = m(x, h)
    c = gen(7)(2, 60, 96)
    (x.float() * c).sum().backward()

    xs, hs = x0.double().cpu(), h0.double().cpu()
    params = []
    for m in layers:
        p = {n: lref.f64(t) for n, t in m.named_parameters()}
        params.append(p)
        q, k, v, g = (t.unflatten(-1, (4, 32)) for t in (xs @ p["qkvg.weight"].T).split(128, -1))
        o, _ = ref.attn(q, k, v, m.decay.double().cpu(), 32 ** -0.5, None, None)
        y = ref.gated(o, g, p["norm"], "silu").flatten(-2) @ p["out.weight"].T
        hs = ref.block_sum(y, hs, p["post"], None, None, 0.5)
        xs = ref.rms(hs, 1e-6) * p["pre"]
    (xs * c.double().cpu()).sum().backward()
    # each layer rounds some ten tensors to bf16 on the way, each to U / sqrt(3) of itself in the mean square, and as many on the
    # way back: sqrt(40) U / sqrt(3) = 1.5e-2 if none is damped or amplified; a factor of two for what amplifies
    ref.check(x, xs, 3e-2, "x")
    for m, p in zip(layers, params):
        for n, t in m.named_parameters():
            ref.check(t.grad, p[n].grad, 3e-2, n)

    lens, new = (33, 1, 26), 6
    cu = torch.tensor([0, 33, 34, 60], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        states = [{} for _ in layers]
        x, h = x0[:1], h0[:1]
        for m, s in zip(layers, states):
            x, h = m(x, h, cu, s)
        tokens = gen(9)(new, 3, 1, 96)
        steps = []
        for t in tokens:
            x, h = gdr.rms_norm_fwd(t.bfloat16(), torch.ones(96, device="cuda"))[0], t
            for m, s in zip(layers, states):
                x, h = m(x, h, None, s)
            steps.append(h)
        at = 0
        for i, n in enumerate(lens):
            hh = torch.cat([h0[0, at:at + n], tokens[:, i, 0]])[None]
            xx = gdr.rms_norm_fwd(hh.bfloat16(), torch.ones(96, device="cuda"))[0]
            for m in layers:
                xx, hh = m(xx, hh)
            got = torch.stack([s[i, 0] for s in steps])
            # the same roundings, but those of P and of the state's copy: 2 U / sqrt(3) a layer, damped by the residual scale
            ref.check(got, hh[0, n:], 1e-2, "row %d" % i)
            at += n


@pytest.mark.parametrize("shape", [(0, 64), (2, 0, 64), (2, 3, 0, 64), (2, 0, 4, 64), (0, 4, 63)], ids=str)
def test_gated_without_rows(shape):
    x, w = torch.empty(*shape, dtype=BF, device="cuda"), torch.ones(shape[-1], device="cuda")
    assert gdr.gated_rms_norm_fwd(x, x, w).shape == x.shape
    dx, dg, dw = gdr.gated_rms_norm_bwd(x, x, w, x)
    assert dx.shape == x.shape and dg.shape == x.shape and (dw == 0).all()


@pytest.mark.parametrize("shape", [(3, 50, 64), (150, 64), (2, 3, 25, 64), (3, 50, 2, 64)], ids=str)
def test_gated_slices_are_read_in_place(shape):
    """Columns of a wider projection, a norm over the whole width or a head: no copy, the same bits."""
    from gated_delta_rule_38_gb300 import layer_ops
    randn = gen(5)
    width = shape[-1] if shape[-2] != 2 else 2 * shape[-1]
    lead = shape[:-1] if shape[-2] != 2 else shape[:-2]
    wide, w = randn(*lead, 2 * width + 16, dtype=BF), 1 + 0.1 * randn(shape[-1])
    x, g = (wide[..., i:i + width].view(*lead, *shape[len(lead):]) for i in (0, width + 8))
    p, xr, gr, _ = layer_ops._gated_problem(x, g, w, 1e-6, "silu")
    assert xr.data_ptr() == x.data_ptr() and gr.data_ptr() == g.data_ptr() and p.x_ld == p.gate_ld == 2 * width + 16
    dy = randn(*shape, dtype=BF)
    want = (gdr.gated_rms_norm_fwd(x.contiguous(), g.contiguous(), w), *gdr.gated_rms_norm_bwd(x.contiguous(), g.contiguous(), w, dy))
    got = (gdr.gated_rms_norm_fwd(x, g, w), *gdr.gated_rms_norm_bwd(x, g, w, dy))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # one of them without gaps, the other a slice
    got = (gdr.gated_rms_norm_fwd(x, g.contiguous(), w), gdr.gated_rms_norm_fwd(x.contiguous(), g, w))
    assert all(torch.equal(a, want[0]) for a in got)
