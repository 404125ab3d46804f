"""The layer operators at their edges: ties of the 8-bit rounding, widths at the limit of shared memory, calls
from two host threads, values that must not cross from one sequence to another,
extremes of the argument ranges."""

import ctypes
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import gated_delta_rule_38_gb300 as gdr
import layer_ref as ref
from test_gpu_layer_ops import BF, cu_of, gen, scan_inputs

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- RMS norm

@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("shift", [0, 1], ids=["vectors", "ragged"])
def test_e4m3_rounds_the_quotient(group, shift):
    """q = e4m3(y / scale) with the fp32 quotient of the definition, also where it falls beside a tie.  Rows of ones keep
    the norm's factor at 1, so y is the weight itself; an output that starts at an odd byte takes the ragged form."""
    D, R = 1024, 3
    rng = np.random.default_rng(group + 1)
    top = (1 + rng.random(D // 128 if group else 1)).astype(np.float32)  # the largest value of every scale's columns
    scale = (top.astype(np.float64) / 448).astype(np.float32)
    s = np.repeat(scale, D // len(scale))
    tie = (rng.integers(8, 15, D) + 0.5) / 8 * 2.0 ** rng.integers(-5, 8, D)
    w = (tie * s).astype(np.float32)
    w = np.where(rng.random(D) < 0.3, np.nextafter(w, np.float32(9)), np.where(rng.random(D) < 0.3, np.nextafter(w, np.float32(0)), w))
    w[::128] = top
    w *= np.where(rng.random(D) < 0.5, np.float32(-1), np.float32(1))
    want = torch.from_numpy(w / s).to(torch.float8_e4m3fn)
    x = torch.ones(R, D, dtype=BF, device="cuda")
    out = torch.empty(R * D + 1, dtype=torch.float8_e4m3fn, device="cuda")[shift:shift + R * D].view(R, D)
    q, _, got = gdr.rms_norm_fwd(x, torch.from_numpy(w).cuda(), eps=0.0, quant="e4m3", scale_group=group, out=out)
    assert torch.equal(got.cpu(), torch.from_numpy(scale).expand(R, -1))
    assert torch.equal(q.float().cpu(), want.float().expand(R, -1))


@pytest.mark.parametrize("top", [1e-31, 3e-29, 1e-25, 1e-20, 1e30, 3e38])
@pytest.mark.parametrize("shift", [0, 1], ids=["vectors", "ragged"])
def test_e4m3_of_very_small_and_large_rows(shift, top):
    """The quotient holds at both ends of the scales: the least one (of rows below 1e-30), and an infinite one, by which
    what is finite becomes 0.  A quarter of each row is 2, the rest 0, so that the norm's factor is 1 and y twice the
    weight."""
    D = 1024
    rng = np.random.default_rng(3)
    w = (np.exp2(rng.uniform(-11, 0, D)) * top * np.where(rng.random(D) < 0.5, -1, 1)).astype(np.float32)
    w[0] = top
    x = np.zeros(D, dtype=np.float32)
    x[::4] = 2
    with np.errstate(over="ignore", invalid="ignore"):
        y = x * w
        m = np.float32(max(np.abs(y).max(), np.float32(1e-30)))
        scale = np.float32(np.float64(m) / 448) if np.isfinite(m) else m
        want = torch.from_numpy(y / scale).to(torch.float8_e4m3fn).float()
    out = torch.empty(D + 1, dtype=torch.float8_e4m3fn, device="cuda")[shift:shift + D].view(1, D)
    q, _, got = gdr.rms_norm_fwd(torch.from_numpy(x).cuda().to(BF)[None], torch.from_numpy(w).cuda(), eps=0.0, quant="e4m3", out=out)
    assert got.item() == float(scale)
    assert torch.equal(q.float().cpu()[0].nan_to_num(1e4), want.nan_to_num(1e4))


EDGE = '''
import sys
sys.path[:0] = [%r, %r]
import torch, layer_ref as ref, gated_delta_rule_38_gb300 as gdr
g = torch.Generator().manual_seed(0)
randn = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g).to(dtype).cuda()
def fwd(D, dt, rt, quant):
    x, w = randn(3, D, dtype=dt), randn(D)
    r = None if rt is None else randn(3, D, dtype=rt)
    y, h, scale = gdr.rms_norm_fwd(x, w, residual=r, quant="e4m3" if quant else None)
    want = ref.norm(ref.f64(x, False), ref.f64(w, False), ref.f64(r, False))[0]
    if quant:
        ref.check(scale, want.abs().amax(-1, keepdim=True) / 448, "scale at %%d" %% D)
    else:
        ref.check(y, want, "y at %%d" %% D)
def bwd(D, dt, ht, later):
    h, w, dy = randn(3, D, dtype=ht), randn(D), randn(3, D, dtype=dt)
    e = randn(3, D, dtype=ht) if later else None
    dx, dr, dw = gdr.rms_norm_bwd(h, w, dy, dresidual=e)
    h64, w64 = ref.f64(h), ref.f64(w)
    (ref.norm(h64, w64, None)[0] * ref.f64(dy, False)).sum().backward()
    ref.check(dx, h64.grad + (ref.f64(e, False) if later else 0), "dx at %%d" %% D)
    ref.check(dw, w64.grad, "dweight at %%d" %% D)
BF, FH, F32 = torch.bfloat16, torch.float16, torch.float32
%s
print("done")
'''


@pytest.mark.parametrize("calls", [
    # each line's calls are the first of their kernels in the process
    "bwd(1013, BF, BF, True); bwd(4077, FH, FH, True); bwd(4077, BF, F32, False); bwd(1219, FH, F32, True)",
    "bwd(6111, BF, BF, False); bwd(1015, BF, F32, False); bwd(501, FH, FH, True); bwd(2039, FH, F32, False)",
    "fwd(4087, BF, F32, False); fwd(1017, FH, F32, False); fwd(4041, BF, F32, True); fwd(1006, FH, F32, True)",
    "fwd(505, BF, F32, False); fwd(2037, FH, F32, False); fwd(1005, BF, F32, True)",
], ids=["bwd-a", "bwd-b", "fwd-a", "fwd-b"])
def test_norm_rows_that_just_fill_48_kb(calls):
    """Widths whose rows take the last bytes below 48 KB of dynamic shared memory beside the kernels' static part, which
    shares the limit.  In a process of their own: an earlier call of the same kernel may have raised the limit."""
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", EDGE % (os.path.dirname(tests), tests, calls.replace("; ", "\n"))],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr[-2000:]


@pytest.mark.parametrize("R", [1, 37])
def test_norm_backward_without_eps(R):
    """Blocks take several rows at a time; with eps = 0 the places past the last row add nothing to dweight."""
    randn = gen(R)
    h, w, dy = randn(R, 256, dtype=BF), randn(256), randn(R, 256, dtype=BF)
    dx, _, dw = gdr.rms_norm_bwd(h, w, dy, eps=0.0)
    h64, w64 = ref.f64(h), ref.f64(w)
    (ref.norm(h64, w64, None, 0.0)[0] * ref.f64(dy, False)).sum().backward()
    ref.check(dx, h64.grad, "dx")
    ref.check(dw, w64.grad, "dweight")


@pytest.mark.parametrize("D", [256, 259], ids=["vectors", "ragged"])
@pytest.mark.parametrize("size,eps", [(1e15, 1e-6), (1e-15, 0.0)])
def test_norm_backward_of_very_large_and_small_rows(size, eps, D):
    """The gradient does not depend on the cube of the norm's factor staying in range."""
    randn = gen(D)
    h, w, dy = randn(5, D, scale=size), randn(D), randn(5, D, dtype=BF)
    _, dres, dw = gdr.rms_norm_bwd(h, w, dy, eps=eps)
    h64, w64 = ref.f64(h), ref.f64(w)
    (ref.norm(h64, w64, None, eps)[0] * ref.f64(dy, False)).sum().backward()
    ref.check(dres, h64.grad, "dresidual")
    ref.check(dw, w64.grad, "dweight")


# ---------------------------------------------------------------- short convolution

def test_conv_in_place_is_refused():
    """Walks share the tokens between them: an output over the input is refused, strided or not; a step may have it."""
    randn = gen(4)
    x, w = randn(2, 40, 64, dtype=BF), randn(64, 4, dtype=BF)
    before = x.clone()
    with pytest.raises(gdr.GdrError, match="UNSUPPORTED"):
        gdr.short_conv_fwd(x, w, out=x)
    assert torch.equal(x, before)
    one, state = x[:, :1].contiguous(), randn(2, 3, 64, dtype=BF)
    want = gdr.short_conv_step(one, state.clone(), w)
    assert torch.equal(gdr.short_conv_step(one, state, w, out=one), want)


# ---------------------------------------------------------------- selective scan

@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [64, 3000], ids=["one segment", "segments"])
def test_scan_sequences_are_kept_apart(T, value):
    """What is not finite in one sequence of a packed batch stays out of the others, whether or not the token axis is cut
    into segments, forward (a state from before the edge) and backward (a gradient from behind it)."""
    lens = (T // 4, T // 2, 0, T // 4)
    s, randn, _ = scan_inputs((1, T, 40, 16, 1, lens, True, True, True), BF)
    cu, dy, ds = cu_of(lens), randn(1, T, 40, dtype=BF), randn(4, 40, 16)

    def call(x, dy):
        a, o = (x, s["dt"], s["A"], s["B"], s["C"]), (s["D"], s["z"], s["bias"], True, s["h0"])
        y, fin, saved = gdr.selective_scan_fwd(*a, *o, True, cu, save_for_backward=True)
        dx, ddt, _, dB, dC, _, dz, _, dh = gdr.selective_scan_bwd(*a, dy, saved, *o, ds, cu)
        return (y, dx, ddt, dB, dC, dz), (fin, dh)

    want = call(s["x"], dy)
    first, last = T // 4, T // 4 + T // 2  # the middle sequence
    for tensor, at in (("x", first + 3), ("dy", last - 5)):
        bad = {"x": s["x"].clone(), "dy": dy.clone()}
        bad[tensor][0, at] = value
        tokens, states = call(bad["x"], bad["dy"])
        for got, expected in zip(tokens, want[0]):
            assert torch.equal(got[:, :first], expected[:, :first]) and torch.equal(got[:, last:], expected[:, last:])
        for got, expected in zip(states, want[1]):
            assert torch.equal(got[[0, 2, 3]], expected[[0, 2, 3]])


@pytest.mark.parametrize("value", [float("-inf"), -3e38])
@pytest.mark.parametrize("T", [21, 1500], ids=["one segment", "segments"])
def test_scan_states_that_forget_at_once(T, value):
    """A = -inf, or so low that A log2(e) overflows: every step forgets the state before it, and the places past the last
    token of a tile change nothing.  (The gradients' definition multiplies an infinite A by zero; a finite one's hold.)"""
    s, randn, _ = scan_inputs((1, T, 40, 16, 1, None, True, True, True), BF)
    s["A"][:, 3] = value
    dy, ds = randn(1, T, 40, dtype=BF), randn(1, 40, 16)
    a, o = (s["x"], s["dt"], s["A"], s["B"], s["C"]), (s["D"], s["z"], s["bias"], True, s["h0"])
    y, fin, saved = gdr.selective_scan_fwd(*a, *o, save_for_backward=True)
    order = ("x", "dt", "A", "B", "C", "D", "z", "bias", "h0")
    leaves = [ref.f64(s[k]) for k in order]
    yw, fw = ref.scan(*leaves[:8], True, leaves[8], None)
    ref.check(y, yw, "y")
    ref.check(fin, fw, "final_state")
    if value > float("-inf"):
        ((yw * ref.f64(dy, False)).sum() + (fw * ref.f64(ds, False)).sum()).backward()
        for got, leaf, name in zip(gdr.selective_scan_bwd(*a, dy, saved, *o, ds), leaves, order):
            ref.check(got, leaf.grad, "d" + name)
    step = s["h0"].clone()
    one = gdr.selective_scan_step(*(t[:, :1].contiguous() if t.dim() > 2 else t for t in a), step, s["D"], s["z"][:, :1].contiguous(),
                                  s["bias"], True)
    ref.check(one, yw[:, :1], "y of a step")


def test_scan_step_of_rows_beyond_2_to_31_elements():
    """A row's tokens times its channels pass 31 bits; a full group of rows and a partial one."""
    if torch.cuda.mem_get_info()[0] < 80e9:
        pytest.skip("needs about 70 GB of free device memory")
    B, T, D, N = 6, 129, 1 << 24, 4
    x = torch.empty(B, T, D, dtype=BF, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    A = -torch.rand(D, N, device="cuda") - 0.2
    bc = torch.randn(2, B, T, 1, N, device="cuda").to(BF)
    state = torch.randn(B, D, N, device="cuda")
    ends = (slice(0, 24), slice(D - 24, D))
    before = [state[:, c].clone() for c in ends]
    y = gdr.selective_scan_step(x, x, A, bc[0], bc[1], state, dt_softplus=True)  # (the inputs are their own steps)
    for c, h in zip(ends, before):
        xc = ref.f64(x[..., c], False)
        want, fin = ref.scan(xc, xc, ref.f64(A[c], False), ref.f64(bc[0], False), ref.f64(bc[1], False), None, None, None, True,
                             ref.f64(h, False), None)
        ref.check(y[..., c], want, "y")
        ref.check(state[:, c], fin, "state")


# ---------------------------------------------------------------- autograd

def test_second_derivatives_are_refused():
    """The backward passes are not differentiable themselves: asked for second derivatives they say so."""
    randn = gen(9)
    x, w, cw = randn(1, 6, 32, dtype=BF), randn(32), randn(32, 4, dtype=BF)
    s, _, _ = scan_inputs((1, 6, 32, 16, 1, None, False, True, True), BF)
    for f in (lambda t: gdr.rms_norm(t, w)[0], lambda t: gdr.short_conv(t, cw, None, "silu")[0],
              lambda t: gdr.selective_scan(t, s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], True)[0]):
        t = x.clone().requires_grad_()
        # (with a term of its own that has second derivatives, which alone would come back without a word)
        loss = f(t).float().square().sum() + t.float().pow(3).sum()
        (d,) = torch.autograd.grad(loss, t, create_graph=True)
        with pytest.raises(RuntimeError, match="no second derivatives"):
            torch.autograd.grad(d.float().sum(), t, retain_graph=True)
        with pytest.raises(RuntimeError, match="no second derivatives"):
            d.float().sum().backward()
        # the first ones are those of a pass without a graph
        t2 = x.clone().requires_grad_()
        (f(t2).float().square().sum() + t2.float().pow(3).sum()).backward()
        assert torch.equal(t2.grad, d)


# ---------------------------------------------------------------- two host threads

def _in_threads(*calls, rounds=20000):
    """Every C call over and over in a host thread of its own; the statuses that each returned."""
    seen, gate = [set() for _ in calls], threading.Barrier(len(calls))

    def work(call, statuses):
        gate.wait()
        for _ in range(rounds):
            statuses.add(call())

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, seen)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return seen


def _c(fn, p, *tensors):
    """The C call with these buffers, workspace last, on a stream of its own."""
    stream = torch.cuda.Stream()
    ptrs = [None if t is None else t.data_ptr() for t in tensors]

    def call(keep=(stream, p, tensors)):
        return fn(ctypes.byref(p), *ptrs, tensors[-1].numel(), stream.cuda_stream)

    return call


@pytest.mark.parametrize("D", [4096, 4099], ids=["vectors", "ragged"])
def test_norm_backward_of_two_sizes_in_two_threads(D):
    """One kernel at two sizes of shared memory (with and without a later gradient), called by two host threads at once:
    the limit that one sets is not lowered under the other's launch."""
    lib, randn = gdr._lib.load(), gen(2)
    h, w, dy = randn(4, D), randn(D), randn(4, D, dtype=BF)
    want, calls, outs = [], [], []
    for later in (h, None):
        want.append(gdr.rms_norm_bwd(h, w, dy, dresidual=later))
        p = gdr._lib.NormProblem(4, D, D, 0, 2, 2, 0, 0, 1e-6)
        outs.append([torch.empty_like(t) for t in want[-1]])
        calls.append(_c(lib.gdr_norm_bwd, p, h, w, dy, later, *outs[-1], torch.empty(1 << 22, dtype=torch.uint8, device="cuda")))
    assert _in_threads(*calls) == [{0}, {0}]
    for got, expected in zip(outs, want):
        for a, b in zip(got, expected):
            assert torch.equal(a, b)


def test_scan_backward_of_two_sizes_in_two_threads():
    """The same of the scan's backward, by whole vectors and by ragged rows."""
    lib = gdr._lib.load()
    want, calls, outs = [], [], []
    for D in (128, 131):
        s, randn, _ = scan_inputs((1, 16, D, 16, 1, None, True, True, True), BF)
        dy = randn(1, 16, D, dtype=BF)
        a, o = (s["x"], s["dt"], s["A"], s["B"], s["C"]), (s["D"], s["z"], s["bias"], True, s["h0"])
        saved = gdr.selective_scan_fwd(*a, *o, save_for_backward=True)[2]
        want.append(gdr.selective_scan_bwd(*a, dy, saved, *o))
        p = gdr._lib.ScanProblem(1, 16, D, 16, 1, D, D, D, 16, 16, 0, None, 0, 1)
        outs.append([torch.empty_like(t) for t in want[-1]])
        calls.append(_c(lib.gdr_scan_bwd, p, *a, s["D"], s["z"], s["bias"], dy, s["h0"], None, saved, *outs[-1],
                        torch.empty(1 << 22, dtype=torch.uint8, device="cuda")))
    assert _in_threads(*calls, rounds=6000) == [{0}, {0}]
    for got, expected in zip(outs, want):
        for a, b in zip(got, expected):
            assert torch.equal(a, b)
