"""The layer operators at their edges: ties of the 8-bit rounding."""

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
