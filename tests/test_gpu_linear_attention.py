"""Linear attention with one decay a head against its plain fp64 form: head dims, grouped heads, lengths from one token to
cut token axes, ragged packed batches, states, views, gradients, streams and graphs, extreme arguments."""

import pytest
import torch

import gated_delta_rule_38_gb300 as gdr
import layer_ref as lref
import linear_ref as ref

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
    return torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")


def slopes(H):
    return (-torch.exp2(-8.0 * torch.arange(1, H + 1) / H)).cuda()


def make(B, T, Hk, H, K, V, lens=None, states=True, dt=BF, seed=0):
    randn = gen(seed + T + K)
    n = B if lens is None else len(lens)
    x = dict(q=randn(B, T, Hk, K, dtype=dt), k=randn(B, T, Hk, K, dtype=dt), v=randn(B, T, H, V, dtype=dt), do=randn(B, T, H, V, dtype=dt))
    x["s0"] = randn(n, H, K, V) if states else None
    x["ds"] = randn(n, H, K, V) if states else None
    return x


def compare(x, decay, lens, dt, scale=None):
    """Forward and backward against the fp64 form."""
    cu = cu_of(lens)
    sc = x["q"].shape[-1] ** -0.5 if scale is None else scale
    o, fin = gdr.linear_attention_fwd(x["q"], x["k"], x["v"], decay, scale=scale, initial_state=x["s0"], output_final_state=True, cu_seqlens=cu)
    leaves = [lref.f64(x[n]) for n in ("q", "k", "v", "s0")]
    ow, fw = ref.attn(*leaves[:3], decay.double().cpu(), sc, leaves[3], lens)
    ref.check(o, ow, ref.attn_bound(o, dt), "o")
    ref.check(fin, fw, ref.attn_bound(fin, dt), "final_state")
    loss = (ow * x["do"].double().cpu()).sum()
    if x["ds"] is not None:
        loss = loss + (fw * x["ds"].double().cpu()).sum()
    if not loss.requires_grad or x["q"].numel() == 0:
        return
    loss.backward()
    grads = gdr.linear_attention_bwd(x["q"], x["k"], x["v"], decay, x["do"], scale=scale, initial_state=x["s0"], dfinal_state=x["ds"], cu_seqlens=cu)
    for name, got, leaf in zip(("dq", "dk", "dv", "dinitial_state"), grads, leaves):
        assert (got is None) == (leaf is None)
        if got is not None:
            ref.check(got, leaf.grad, ref.attn_bound(got, dt), name)


CASES = [  # B, T, Hk, H, K, V, lens, states
    (1, 1, 1, 1, 128, 128, None, True),
    (3, 2, 2, 4, 128, 128, None, True),
    (2, 17, 1, 3, 64, 128, None, False),
    (1, 127, 2, 2, 128, 64, None, True),
    (2, 128, 2, 2, 128, 128, None, False),
    (2, 129, 2, 2, 128, 128, None, True),
    (1, 300, 2, 6, 8, 8, None, True),
    (1, 257, 2, 2, 16, 24, None, True),
    (2, 200, 3, 3, 72, 120, None, True),
    (1, 401, 2, 4, 96, 40, None, False),
    (1, 1100, 2, 4, 128, 128, None, True),
    (1, 700, 2, 4, 128, 128, (5, 0, 1, 130, 128, 0, 256, 180), True),
    (1, 333, 1, 2, 64, 96, (0, 0, 127, 1, 129, 76, 0), True),
    (1, 64, 2, 2, 128, 128, (1,) * 64, True),
    (1, 260, 2, 2, 56, 128, (260, 0), False),
]


@DT
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_forward_backward(case, dt):
    B, T, Hk, H, K, V, lens, states = case
    compare(make(B, T, Hk, H, K, V, lens, states, dt), slopes(H), lens, dt)
    assert gdr.get_error() == 0


@pytest.mark.parametrize("lens", [None, (3000, 0, 1, 4096, 903), (1024, 2048, 4928)], ids=["one", "ragged", "cuts"])
def test_cut_token_axis(lens):
    """Few heads and many tokens: segments, their windows' states and what is summed up for their starts."""
    T = 8000
    for dt in (BF, FH):
        compare(make(1, T, 1, 2, 128, 64, lens, True, dt), torch.tensor([-0.003, -0.5], device="cuda"), lens, dt)
    x = make(1, T, 2, 2, 40, 128, lens, False, BF)
    compare(x, slopes(2), lens, BF)


def test_many_sequences():
    lens = [1, 2, 0, 3] * 700
    x = make(1, sum(lens), 1, 2, 32, 32, lens, True)
    compare(x, slopes(2), lens, BF)


@pytest.mark.parametrize("decay", [0.0, -1e-5, -0.01, -3.0, -50.0, -200.0, float("-inf")])
def test_decays(decay):
    """From none at all to states that forget at every token; the fp64 form takes -inf as -1e4 (0 times it is 0)."""
    x = make(1, 600, 1, 2, 64, 64)
    d = torch.tensor([decay, -0.1], device="cuda")
    cu, sc = None, 0.125
    o, fin = gdr.linear_attention_fwd(x["q"], x["k"], x["v"], d, initial_state=x["s0"], output_final_state=True, cu_seqlens=cu)
    args = [lref.f64(x[n]) for n in ("q", "k", "v", "s0")]
    dw = d.double().cpu().clamp(min=-1e4)
    ow, fw = ref.attn(*args[:3], dw, sc, args[3], None)
    ref.check(o, ow, ref.attn_bound(o, BF), "o")
    ref.check(fin, fw, ref.attn_bound(fin, BF), "final_state")
    loss = (ow * x["do"].double().cpu()).sum() + (fw * x["ds"].double().cpu()).sum()
    loss.backward()
    for got, leaf in zip(gdr.linear_attention_bwd(x["q"], x["k"], x["v"], d, x["do"], initial_state=x["s0"], dfinal_state=x["ds"]), args):
        ref.check(got, leaf.grad, ref.attn_bound(got, BF), "gradient")


@DT
@pytest.mark.parametrize("decay", [0.0, -1e-4, -0.004, -0.5])
@pytest.mark.parametrize("T", [100, 1100, 9000])
def test_states_are_fp32(T, decay, dt):
    """States that are handed on are as good as fp32 sums, whatever the tokens' type.  Of the keys' numbers: 3 bf16 or 2 fp16
    leave 2^-22 at most, and 2 bf16 (2.5e-6 in the mean square) where the chunk weighs under an eighth, 3.2e-7; the
    accumulator's eight additions of full size, rounded down, 8 x 2^-24 = 4.8e-7; together under 1e-6."""
    x = make(1, T, 1, 2, 128, 128, None, True, dt)
    d = torch.full((2,), decay, device="cuda")
    _, fin = gdr.linear_attention_fwd(x["q"], x["k"], x["v"], d, initial_state=x["s0"], output_final_state=True)
    args = [lref.f64(x[n]) for n in ("q", "k", "v", "s0")]
    ow, fw = ref.attn(*args[:3], d.double().cpu(), 128 ** -0.5, args[3], None)
    ref.check(fin, fw, 1e-6, "final_state")
    ((ow * x["do"].double().cpu()).sum() + (fw * x["ds"].double().cpu()).sum()).backward()
    ds = gdr.linear_attention_bwd(x["q"], x["k"], x["v"], d, x["do"], initial_state=x["s0"], dfinal_state=x["ds"])[3]
    ref.check(ds, args[3].grad, 1e-6, "dinitial_state")


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0 ** -30, 4096.0])
def test_scales(scale):
    """Scales of any size and sign; a scale of zero leaves the states' gradients alone."""
    x = make(1, 300, 1, 2, 64, 64)
    d = torch.tensor([-0.01, -0.3], device="cuda")
    args = [lref.f64(x[n]) for n in ("q", "k", "v", "s0")]
    o, fin = gdr.linear_attention_fwd(x["q"], x["k"], x["v"], d, scale=scale, initial_state=x["s0"], output_final_state=True)
    ow, fw = ref.attn(*args[:3], d.double().cpu(), scale, args[3], None)
    ((ow * x["do"].double().cpu()).sum() + (fw * x["ds"].double().cpu()).sum()).backward()
    grads = gdr.linear_attention_bwd(x["q"], x["k"], x["v"], d, x["do"], scale=scale, initial_state=x["s0"], dfinal_state=x["ds"])
    for got, want in zip((o, fin, *grads), (ow, fw, *(a.grad for a in args))):
        ref.check(got, want, ref.attn_bound(got, BF), "scale")


def test_differences():
    """The gradients against central differences of the fp64 form."""
    x = make(1, 150, 1, 2, 32, 48, dt=FH)
    d = slopes(2)
    grads = gdr.linear_attention_bwd(x["q"], x["k"], x["v"], d, x["do"], initial_state=x["s0"], dfinal_state=x["ds"])
    do, ds, dd = x["do"].double().cpu(), x["ds"].double().cpu(), d.double().cpu()

    def loss(q, k, v, s0):
        o, f = ref.attn(q, k, v, dd, 32 ** -0.5, s0, None)
        return (o * do).sum() + (f * ds).sum()

    args = [lref.f64(x[n], False) for n in ("q", "k", "v", "s0")]
    for (direction, fd), got in zip(lref.directional(loss, args), grads):
        dot = float((got.double().cpu() * direction).sum())
        # the gradient's error is attn_bound of its norm, along a random direction at most four of its standard deviations
        assert abs(dot - fd) <= 4 * ref.attn_bound(got, FH) * float(got.double().norm()) + 1e-6 * abs(fd), (dot, fd)


def test_sequences_do_not_meet():
    """What is not finite in a sequence or in a head stays there, past the ends of tiles too."""
    lens = (100, 200, 77)
    cu, d = cu_of(lens), slopes(2)
    x = make(1, 377, 2, 2, 64, 64, lens)
    y = {n: t.clone() for n, t in x.items()}
    for n in ("q", "k", "v", "do"):
        y[n][0, 100:300, 0] = float("nan")
        y[n][0, 150, 0] = float("inf")
    y["s0"][1, 0], y["ds"][1, 0] = float("nan"), float("inf")
    keep = torch.ones(377, dtype=torch.bool)
    keep[100:300] = False

    def run(z):
        o, f = gdr.linear_attention_fwd(z["q"], z["k"], z["v"], d, initial_state=z["s0"], output_final_state=True, cu_seqlens=cu)
        return o, f, *gdr.linear_attention_bwd(z["q"], z["k"], z["v"], d, z["do"], initial_state=z["s0"], dfinal_state=z["ds"], cu_seqlens=cu)

    for i, (a, b) in enumerate(zip(run(x), run(y))):
        if i in (1, 5):
            assert torch.equal(a[:, 1], b[:, 1]) and torch.equal(a[0::2], b[0::2])
        else:
            assert torch.equal(a[:, :, 1], b[:, :, 1]) and torch.equal(a[:, keep], b[:, keep])


def test_views():
    """Slices of one projection are read in place; other views and misaligned ones are copied: the same bits."""
    B, T, H, D = 2, 150, 2, 64
    wide = gen(3)(B, T, 3 * H * D + 8, dtype=BF)
    q, k, v = (wide[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    d = slopes(H)
    want = gdr.linear_attention_fwd(q.contiguous(), k.contiguous(), v.contiguous(), d)[0]
    assert torch.equal(gdr.linear_attention_fwd(q, k, v, d)[0], want)
    odd = torch.zeros(B * T * H * D + 1, dtype=BF, device="cuda")[1:].view(B, T, H, D).copy_(q)
    assert odd.data_ptr() % 16 and torch.equal(gdr.linear_attention_fwd(odd, k, v, d)[0], want)
    t = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(gdr.linear_attention_fwd(t, k, v, d)[0], want)
    do = torch.randn_like(want)
    a, b = gdr.linear_attention_bwd(q, k, v, d, do), gdr.linear_attention_bwd(q.contiguous(), k.contiguous(), v.contiguous(), d, do)
    assert all(torch.equal(s, t) for s, t in zip(a[:3], b[:3]))
    out = torch.empty(B * T * H * D + 8, dtype=BF, device="cuda")[8:].view(B, T, H, D)  # 16 bytes past a sector
    gdr.linear_attention_fwd(q, k, v, d, out=out)
    assert torch.equal(out, want)
    s = torch.zeros(3 * B, H, D, D, device="cuda")
    x = make(B, 1, H, H, D, D)
    gdr.linear_attention_step(x["q"], x["k"], x["v"], d, s[B:2 * B])
    assert (s[:B] == 0).all() and (s[2 * B:] == 0).all() and (s[B:2 * B] != 0).any()


@DT
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 128, 128), (5, 1, 2, 4, 128, 128), (3, 5, 1, 3, 72, 40), (2, 3, 2, 2, 8, 8), (300, 1, 1, 2, 64, 128)],
                         ids=["one", "gqa", "odd", "narrow", "rows"])
def test_step(case, dt):
    B, T, Hk, H, K, V = case
    x, d = make(*case, dt=dt), slopes(H)
    state = x["s0"].clone()
    o = gdr.linear_attention_step(x["q"], x["k"], x["v"], d, state)
    args = [lref.f64(x[n], False) for n in ("q", "k", "v", "s0")]
    ow, fw = ref.attn(*args[:3], d.double().cpu(), K ** -0.5, args[3], None)
    ref.check(o, ow, 1.05 * lref.U[dt], "o")  # (fp32 throughout: the result's rounding alone)
    ref.check(state, fw, 1e-6, "state")
    again = x["s0"].clone()
    one = [gdr.linear_attention_step(*(x[n][:, t:t + 1] for n in ("q", "k", "v")), d, again) for t in range(T)]
    assert torch.equal(torch.cat(one, 1), o) and torch.equal(again, state)


def test_no_tokens():
    s0, d = gen(1)(2, 2, 64, 64), slopes(2)
    e = torch.empty(2, 0, 2, 64, dtype=BF, device="cuda")
    o, f = gdr.linear_attention_fwd(e, e, e, d, initial_state=s0, output_final_state=True)
    assert o.shape == e.shape and torch.equal(f, s0)
    dq, dk, dv, ds = gdr.linear_attention_bwd(e, e, e, d, e, initial_state=s0, dfinal_state=2 * s0)
    assert dq.shape == e.shape and torch.equal(ds, 2 * s0)
    assert torch.equal(gdr.linear_attention_fwd(e, e, e, d, output_final_state=True)[1], torch.zeros_like(s0))
    gdr.linear_attention_step(e, e, e, d, s0)
    e1, cu = e[:1], torch.zeros(3, dtype=torch.int32, device="cuda")
    assert torch.equal(gdr.linear_attention_fwd(e1, e1, e1, d, initial_state=s0, output_final_state=True, cu_seqlens=cu)[1], s0)
    x = make(1, 130, 1, 1, 64, 64, (0, 130, 0))
    f = gdr.linear_attention_fwd(x["q"], x["k"], x["v"], slopes(1), initial_state=x["s0"], output_final_state=True, cu_seqlens=cu_of((0, 130, 0)))[1]
    assert torch.equal(f[0], x["s0"][0]) and torch.equal(f[2], x["s0"][2])


def test_same_bits_streams_and_graphs():
    x, d = make(1, 3000, 2, 4, 128, 128), slopes(4)

    def step():
        o, f = gdr.linear_attention_fwd(x["q"], x["k"], x["v"], d, initial_state=x["s0"], output_final_state=True)
        return o, f, *gdr.linear_attention_bwd(x["q"], x["k"], x["v"], d, x["do"], initial_state=x["s0"], dfinal_state=x["ds"])

    want = step()
    assert all(torch.equal(a, b) for a, b in zip(want, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step()
        graphs.append((g, res))
    x["v"].mul_(2)  # the captured calls read what lies there when they run
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = step()
    for _, res in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, res))


def test_autograd():
    x, d = make(2, 200, 2, 4, 64, 64), slopes(4)
    leaves = [x[n].clone().requires_grad_() for n in ("q", "k", "v", "s0")]
    o, f = gdr.linear_attention(*leaves[:3], d, initial_state=leaves[3], output_final_state=True)
    ((o * x["do"]).float().sum() + (f * x["ds"]).sum()).backward()
    want = gdr.linear_attention_bwd(x["q"], x["k"], x["v"], d, x["do"], initial_state=x["s0"], dfinal_state=x["ds"])
    assert all(torch.equal(l.grad, w) for l, w in zip(leaves, want))
    for l in leaves:
        l.grad = None
    f = gdr.linear_attention(*leaves[:3], d, initial_state=leaves[3], output_final_state=True)[1]  # only the state is used
    f.sum().backward()
    assert (leaves[0].grad == 0).all() and (leaves[1].grad != 0).any()
    q = x["q"].clone().requires_grad_()
    (g,) = torch.autograd.grad(gdr.linear_attention(q, x["k"], x["v"], d)[0].float().square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        g.sum().backward()


def test_offsets_past_31_bits():
    """Tensors of more than 2^31 elements: the last tokens of the last head."""
    T, H, D = 132000, 128, 128
    q = torch.empty(1, T, H, D, dtype=BF, device="cuda").normal_()
    d = torch.full((H,), -0.5, device="cuda")
    o, fin = gdr.linear_attention_fwd(q, q, q, d, output_final_state=True)
    tail = q[:, -200:, -1:].double().cpu()
    ow, fw = ref.attn(tail, tail, tail, torch.tensor([-0.5], dtype=torch.float64), D ** -0.5, None, None)
    ref.check(o[:, -50:, -1:], ow[:, -50:], ref.attn_bound(o, BF), "o")
    ref.check(fin[:, -1:], fw, ref.attn_bound(fin, BF), "final_state")
    del fin
    dq, dk, dv, _ = gdr.linear_attention_bwd(q, q, q, d, o)
    head = q[:, :200, -1:]
    oh = o[:, :200, -1:].double().cpu()
    leaves = [lref.f64(head) for _ in range(3)]
    (ref.attn(*leaves, torch.tensor([-0.5], dtype=torch.float64), D ** -0.5, None, None)[0] * oh).sum().backward()
    for got, leaf in zip((dq, dk, dv), leaves):
        ref.check(got[:, :50, -1:], leaf.grad[:, :50], ref.attn_bound(got, BF), "gradient")


def test_bad_cu_seqlens():
    x, d = make(1, 300, 1, 1, 64, 64), slopes(1)
    for bad in ([0, 200, 100, 300], [5, 300], [0, 299], [0, 400], [-7, 300], [300, 0]):
        gdr.get_error()
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        gdr.linear_attention_fwd(x["q"], x["k"], x["v"], d, output_final_state=True, cu_seqlens=cu)
        assert gdr.get_error() != 0, bad
    gdr.linear_attention_fwd(x["q"], x["k"], x["v"], d, cu_seqlens=cu_of((300,)))
    assert gdr.get_error() == 0


def test_refusals():
    x, d = make(1, 64, 1, 2, 64, 64), slopes(2)
    q, k, v = x["q"], x["k"], x["v"]
    bad = [lambda: gdr.linear_attention_fwd(q, k, v, d[:1]), lambda: gdr.linear_attention_fwd(q, k, v, d.double()),
           lambda: gdr.linear_attention_fwd(q, k[:, :63], v, d), lambda: gdr.linear_attention_fwd(q.float(), k, v, d),
           lambda: gdr.linear_attention_fwd(q, k, v.half(), d), lambda: gdr.linear_attention_fwd(q[0], k, v, d),
           lambda: gdr.linear_attention_fwd(q, k, v, d, initial_state=x["s0"].half()),
           lambda: gdr.linear_attention_fwd(q, k, v, d, out=v[:, :1]), lambda: gdr.linear_attention_step(q, k, v, d, None),
           lambda: gdr.linear_attention_bwd(q, k, v, d, x["do"][:, :1]), lambda: gdr.linear_attention(q, k, v, d.clone().requires_grad_()),
           lambda: gdr.linear_attention_fwd(q.cpu(), k, v, d)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gdr.linear_attention_fwd(q, k, v, d, out=v), lambda: gdr.linear_attention_step(q, k, v, d, x["s0"], out=v),
                 lambda: gdr.linear_attention_fwd(q[..., :60].contiguous(), k[..., :60].contiguous(), v, d),
                 lambda: gdr.linear_attention_fwd(torch.cat([q, q], 2), torch.cat([k, k], 2), torch.cat([v, v[:, :, :1]], 2), slopes(3))):
        with pytest.raises(gdr.GdrError):
            call()


@DT
@pytest.mark.parametrize("size", [3e-7, 300.0, 2e5, 1e9])
def test_states_past_the_tokens_range(size, dt):
    """States larger and smaller than the tokens' type holds, under a scale that brings the outputs back into it: the copy of a
    state that a query meets has a power of two of its own.  (Keys and values are zeros, so that the states alone show.)"""
    T, H, D = 300, 2, 64
    randn = gen(7)
    q, do = randn(1, T, H, D, dtype=dt), randn(1, T, H, D, dtype=dt)
    zero, s0, d = torch.zeros_like(q), randn(1, H, D, D, scale=size), torch.tensor([0.0, -0.001], device="cuda")
    leaves = [lref.f64(t) for t in (q, zero, zero, s0)]
    ow, fw = ref.attn(*leaves[:3], d.double().cpu(), 1 / size, leaves[3], None)
    (ow * do.double().cpu()).sum().backward()
    o, fin = gdr.linear_attention_fwd(q, zero, zero, d, scale=1 / size, initial_state=s0, output_final_state=True)
    ref.check(o, ow, ref.attn_bound(o, dt), "o")
    ref.check(fin, fw, ref.attn_bound(fin, dt), "final_state")
    dq, dk, dv, ds = gdr.linear_attention_bwd(q, zero, zero, d, do, scale=1 / size, initial_state=s0)
    ref.check(dq, leaves[0].grad, ref.attn_bound(dq, dt), "dq")
    ref.check(ds, leaves[3].grad, ref.attn_bound(ds, dt), "dinitial_state")
    assert (dk == 0).all() and (dv == 0).all()


def test_sums_past_fp16():
    """Tokens of one sign and no decay: the states (backwards: their gradients) pass 65504 on the way, the outputs do not."""
    T, D = 3000, 64
    randn, d = gen(1), torch.zeros(1, device="cuda")
    full = lambda x: torch.full((1, T, 1, D), x, dtype=FH, device="cuda")  # noqa: E731
    q, k, v = randn(1, T, 1, D, dtype=FH, scale=1e-3), full(8.0), full(4.0)
    o, fin = gdr.linear_attention_fwd(q, k, v, d, output_final_state=True)
    ow, fw = ref.attn(*(lref.f64(t, False) for t in (q, k, v)), d.double().cpu(), D ** -0.5, None, None)
    assert float(fw.max()) > 65504 and float(ow.abs().max()) < 6e4
    ref.check(o, ow, ref.attn_bound(o, FH), "o")
    ref.check(fin, fw, ref.attn_bound(fin, FH), "final_state")
    q, do = full(32.0), full(16.0)
    k, v = randn(1, T, 1, D, dtype=FH, scale=1e-3), randn(1, T, 1, D, dtype=FH, scale=1e-3)
    leaves = [lref.f64(t) for t in (q, k, v)]
    (ref.attn(*leaves, d.double().cpu(), D ** -0.5, None, None)[0] * do.double().cpu()).sum().backward()
    for name, got, leaf in zip(("dq", "dk", "dv"), gdr.linear_attention_bwd(q, k, v, d, do), leaves):
        assert float(leaf.grad.abs().max()) < 6e4
        ref.check(got, leaf.grad, ref.attn_bound(got, FH), name)


@DT
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_one_column_that_is_not_finite(value, dt):
    """A value of v that is not finite stays in its column: the others' copy of the state is as good as without it."""
    T, D = 300, 64
    x, d = make(1, T, 1, 1, D, D, None, True, dt), torch.tensor([-0.01], device="cuda")
    args = [lref.f64(x[n], False) for n in ("q", "k", "v", "s0")]
    ow, fw = ref.attn(*args[:3], d.double().cpu(), D ** -0.5, args[3], None)
    x["v"][0, 40, 0, 5] = value
    o, fin = gdr.linear_attention_fwd(x["q"], x["k"], x["v"], d, initial_state=x["s0"], output_final_state=True)
    keep = [c for c in range(D) if c != 5]
    ref.check(o[..., keep], ow[..., keep], ref.attn_bound(o, dt), "o")
    ref.check(fin[..., keep], fw[..., keep], ref.attn_bound(fin, dt), "final_state")
    assert not torch.isfinite(o[0, 128:, 0, 5].float()).any() and not torch.isfinite(fin[..., 5]).any()


@DT
@pytest.mark.parametrize("size", [0.1, 1e-2, 1e-3, 1e-4])
def test_states_of_small_keys(size, dt):
    """As test_states_are_fp32, for keys (backwards: queries) whose second number would be a subnormal one of fp16."""
    x = make(1, 1100, 1, 2, 128, 128, None, False, dt)
    d = torch.full((2,), -0.004, device="cuda")
    q, k = ((x[n].float() * size).to(dt) for n in ("q", "k"))
    s0 = torch.zeros(1, 2, 128, 128, device="cuda")
    _, fin = gdr.linear_attention_fwd(q, k, x["v"], d, initial_state=s0, output_final_state=True)
    args = [lref.f64(t) for t in (q, k, x["v"], s0)]
    ow, fw = ref.attn(*args[:3], d.double().cpu(), 128 ** -0.5, args[3], None)
    ref.check(fin, fw, 1e-6, "final_state")
    (ow * x["do"].double().cpu()).sum().backward()
    ds = gdr.linear_attention_bwd(q, k, x["v"], d, x["do"], initial_state=s0)[3]
    ref.check(ds, args[3].grad, 1e-6, "dinitial_state")


@pytest.mark.parametrize("decay", [0.0, -1e-5, -1e-4, -1e-3, -0.03, -0.49, -0.51, -3.0])
def test_many_steps(decay):
    """States stepped thousands of times stay as good as their own roundings leave them: two a token, each at most 2^-24 of the
    state (which grows, or is forgotten, so that none weighs more at the end), in the mean square 2^-24 sqrt(2 T / 3); what a
    rounded decay would add is T 2^-25 and not random."""
    T, D = 4000, 32
    x, d = make(1, T, 1, 2, D, D), torch.full((2,), decay, device="cuda")
    state = x["s0"].clone()
    gdr.linear_attention_step(x["q"], x["k"], x["v"], d, state)
    fw = ref.attn(*(lref.f64(x[n], False) for n in ("q", "k", "v")), d.double().cpu(), 1.0, lref.f64(x["s0"], False), None)[1]
    ref.check(state, fw, 2.0 ** -24 * (2 * T / 3) ** 0.5, "state")


def test_states_off_16_bytes():
    """States and their gradients that begin anywhere (pieces of a flat buffer, the gradient of a concatenation): copied."""
    x, d = make(2, 200, 2, 2, 64, 64), slopes(2)

    def off(t):
        o = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
        assert o.data_ptr() % 16
        return o

    def both(f):
        o, fin = gdr.linear_attention_fwd(x["q"], x["k"], x["v"], d, initial_state=f(x["s0"]), output_final_state=True)
        return o, fin, *gdr.linear_attention_bwd(x["q"], x["k"], x["v"], d, f(x["do"]), initial_state=f(x["s0"]), dfinal_state=f(x["ds"]))

    assert all(torch.equal(a, b) for a, b in zip(both(lambda t: t), both(off)))
    leaves = [x[n].clone().requires_grad_() for n in ("q", "k", "v", "s0")]
    grads = []
    for flat in (True, False):
        o, fin = gdr.linear_attention(*leaves[:3], d, initial_state=leaves[3], output_final_state=True)
        w = (x["ds"], x["do"].float())
        if flat:  # (the gradient of the states then begins 4 bytes into a buffer)
            both_flat = torch.cat([o.float().sum()[None] * 0, fin.flatten(), o.float().flatten()])
            loss = (both_flat * torch.cat([torch.zeros(1, device="cuda"), *(t.flatten() for t in w)])).sum()
        else:
            loss = (fin * w[0]).sum() + (o.float() * w[1]).sum()
        grads.append(torch.autograd.grad(loss, leaves))
    for a, b in zip(*grads):
        ref.check(a, b, 1e-6, "gradient")
    # what is updated or written in place cannot be copied: refused
    with pytest.raises(gdr.GdrError):
        gdr.linear_attention_step(x["q"][:, :1], x["k"][:, :1], x["v"][:, :1], d, off(x["s0"]))


@pytest.mark.parametrize("case", [(24, 2000, (130, 1000, 0, 870)), (24, 2000, (0, 1999, 1, 0)), (8, 1500, (5, 700, 0, 300, 1, 400, 94)),
                                  (16, 2000, (256, 768, 512, 464)), (16, 1500, (1, 1, 1, 1497))], ids=str)
def test_packed_windows(case):
    """Cut packed batches whose segments have several windows before (backwards: behind) them, in a direction at least, and whose
    sequences begin and end inside windows, on them and on the cuts: every exchanged state in its place."""
    H, T, lens = case
    for dt, K, V in ((BF, 32, 48), (FH, 64, 16)):
        compare(make(1, T, H, H, K, V, lens, True, dt), torch.full((H,), -0.002, device="cuda"), lens, dt)
