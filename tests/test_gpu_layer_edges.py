"""The layer operators at their edges: ties of the 8-bit rounding, widths at the limit of shared memory."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_38_gb300 as gdr
from test_gpu_layer_ops import BF

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
