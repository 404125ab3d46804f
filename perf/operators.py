"""The operators of a recurrent mixer layer beside the delta rule, as measured cases: the short causal convolution,
the selective state space scan and the root-mean-square norm with its residual and 8-bit forms.

Every case runs one operator in one direction.  With ``own`` false, ``run`` computes the plain form in elementary
torch operations, in fp32; with ``own`` true it calls the library.  ``exact`` evaluates the definitions in fp64,
token by token."""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one generated token for a serving batch of 256 rows: the convolution over the concatenated q, k, v
        # channels of 32 heads of 128, its cached inputs updated in place
        dict(name="conv step 256x12288", op="conv_step", B=256, T=1, D=12288, W=4, dtype="bf16", bias=False),
        # the same convolution in a training step: forward and every gradient
        dict(name="conv train 2x4096x12288", op="conv_train", B=2, T=4096, D=12288, W=4, dtype="bf16", bias=True,
             states=False, lens=""),
        # a packed batch of ragged prompts that continue from cached inputs; an odd number of channels
        dict(name="conv packed 5311x4099", op="conv_fwd", B=1, T=5311, D=4099, W=4, dtype="fp16", bias=True,
             states=True, lens="512,1024,768,3000,7"),
        # the smallest call: one generated token of one row
        dict(name="scan step 1x2048", op="scan_step", B=1, T=1, D=2048, N=16, G=1, dtype="bf16"),
        # one generated token for a serving batch
        dict(name="scan step 256x4096", op="scan_step", B=256, T=1, D=4096, N=16, G=1, dtype="bf16"),
        # prompts: dense forward with the final states for the cache
        dict(name="scan prompt 2x4096x4096", op="scan_fwd", B=2, T=4096, D=4096, N=16, G=1, dtype="bf16",
             states=False, lens=""),
        # one long prompt, few channels: the token axis has to be split
        dict(name="scan long 1x65536x2048", op="scan_fwd", B=1, T=65536, D=2048, N=16, G=1, dtype="bf16",
             states=True, lens=""),
        # a training step: forward and every gradient
        dict(name="scan train 2x4096x4096", op="scan_train", B=2, T=4096, D=4096, N=16, G=1, dtype="bf16",
             states=False, lens=""),
        # training on a packed ragged batch with states, two groups, an odd number of channels per group
        dict(name="scan packed train 5311x2062", op="scan_train", B=1, T=5311, D=2062, N=10, G=2, dtype="fp16",
             states=True, lens="512,1024,768,3000,7"),
        # the norm before the input projection of a generated token: residual added, 8-bit output per row
        dict(name="norm e4m3 256x4096", op="norm_fwd", R=256, D=4096, dtype="bf16", res="bf16", quant=True, group=0),
        # the same over a prompt batch, scales per 128 columns
        dict(name="norm e4m3 8192x4096", op="norm_fwd", R=8192, D=4096, dtype="bf16", res="fp32", quant=True,
             group=128),
        # training: forward and gradients, residual stream in the token type
        dict(name="norm train 8192x4096", op="norm_train", R=8192, D=4096, dtype="bf16", res="bf16", quant=False,
             group=0),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _lens(rng, T):
    """T tokens cut into a few sequences, some of them empty or of one token."""
    n = rng.randint(1, 12)
    cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))


def draw(rng):
    op = rng.choice(["conv_step", "conv_fwd", "conv_train", "scan_step", "scan_fwd", "scan_train", "norm_fwd",
                     "norm_train"])
    dtype = rng.choice(["bf16", "fp16"])
    if op.startswith("norm"):
        D = _spread(rng, 1, 16384)
        R = min(_spread(rng, 1, 65536), max(1, (1 << 25) // D))
        quant = op == "norm_fwd" and rng.random() < 0.6
        return dict(op=op, R=R, D=D, dtype=dtype, res=rng.choice(["", dtype, "fp32"]), quant=quant,
                    group=rng.choice([0, 128]) if quant else 0)
    if op.endswith("step"):
        B, D = _spread(rng, 1, 512), _spread(rng, 1, 8192)
        if op == "conv_step":
            return dict(op=op, B=B, T=rng.choice([1, 1, 2, 5]), D=D, W=rng.randint(2, 4), dtype=dtype,
                        bias=rng.random() < 0.5)
        G = rng.choice([1, 1, 2, 4])
        N = _spread(rng, 1, 64)
        B = min(B, max(1, (1 << 25) // (D * N)))
        return dict(op=op, B=B, T=rng.choice([1, 1, 2, 5]), D=max(1, D // G) * G, N=N, G=G, dtype=dtype)
    packed = rng.random() < 0.4
    B = 1 if packed else _spread(rng, 1, 8)
    states = rng.random() < 0.5
    if op.startswith("conv"):
        D = _spread(rng, 1, 12288)
        T = min(_spread(rng, 1, 16384), max(1, 90_000_000 // (B * D)))
        return dict(op=op, B=B, T=T, D=D, W=rng.randint(2, 4), dtype=dtype, bias=rng.random() < 0.5, states=states,
                    lens=_lens(rng, T) if packed else "")
    G = rng.choice([1, 1, 2, 4])
    D = max(1, _spread(rng, 1, 6144) // G) * G
    N = rng.choice([16, 16, _spread(rng, 1, 64)])
    cap = 400_000_000 if op == "scan_train" else 1_000_000_000
    T = min(_spread(rng, 1, 16384), max(1, cap // (B * D * N)))
    return dict(op=op, B=B, T=T, D=D, N=N, G=G, dtype=dtype, states=states, lens=_lens(rng, T) if packed else "")


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(seed)
    dt = _DT[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=_DEV) * scale).to(dtype)

    op = case["op"]
    s = dict(case)
    if op.startswith("norm"):
        R, D = case["R"], case["D"]
        s["x"] = randn(R, D)
        s["weight"] = 1 + randn(D, scale=0.1, dtype=torch.float32)
        if case["res"]:
            s["residual"] = randn(R, D, scale=2.0, dtype=torch.float32 if case["res"] == "fp32" else dt)
        if op == "norm_train":
            s["dy"] = randn(R, D)
            if case["res"]:
                s["dres"] = randn(R, D, dtype=s["residual"].dtype)
        return s
    B, T, D = case["B"], case["T"], case["D"]
    lens = [int(n) for n in case["lens"].split(",")] if case.get("lens") else None
    nseq = len(lens) if lens else B
    if lens:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=_DEV)
    s["x"] = randn(B, T, D)
    if op.startswith("conv"):
        W = case["W"]
        s["weight"] = randn(D, W, scale=W ** -0.5)
        if case["bias"]:
            s["b"] = randn(D, scale=0.1)
        if op == "conv_step" or case["states"]:
            s["state"] = randn(nseq, W - 1, D)
        if op == "conv_train":
            s["dy"] = randn(B, T, D)
            if case["states"]:
                s["dstate"] = randn(nseq, W - 1, D)
        return s
    N, G = case["N"], case["G"]
    s["dt"] = randn(B, T, D, scale=0.5)
    # steps between 1e-3 and 1e-1, as such models are initialised: the bias is the inverse softplus
    step = torch.exp(torch.rand(D, generator=g, device=_DEV) * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, N + 1, device=_DEV, dtype=torch.float32) * (
        0.5 + torch.rand(D, N, generator=g, device=_DEV))
    s["Bm"], s["Cm"] = randn(B, T, G, N), randn(B, T, G, N)
    s["Ds"] = 1 + randn(D, scale=0.1, dtype=torch.float32)
    s["z"] = randn(B, T, D)
    if op == "scan_step" or case["states"]:
        s["state"] = randn(nseq, D, N, scale=0.1, dtype=torch.float32)
    if op == "scan_train":
        s["dy"] = randn(B, T, D)
        if case["states"]:
            s["dstate"] = randn(nseq, D, N, scale=0.1, dtype=torch.float32)
    return s


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    import gated_delta_rule_38_gb300 as gdr
    op = s["op"]
    if op == "norm_fwd":
        y, h, scale = gdr.rms_norm_fwd(s["x"], s["weight"], residual=s.get("residual"),
                                       quant="e4m3" if s["quant"] else None, scale_group=s["group"])
        return {"y": y, "residual": h, "scale": scale}
    if op == "norm_train":
        y, h, _ = gdr.rms_norm_fwd(s["x"], s["weight"], residual=s.get("residual"))
        dx, dr, dw = gdr.rms_norm_bwd(s["x"] if h is None else h, s["weight"], s["dy"], dresidual=s.get("dres"),
                                      dtype=s["x"].dtype)
        return {"y": y, "residual": h, "dx": dx, "dresidual": dr, "dweight": dw}
    if op == "conv_step":
        y = gdr.short_conv_step(s["x"], s["state"], s["weight"], bias=s.get("b"), activation="silu")
        return {"y": y, "state": s["state"]}
    if op in ("conv_fwd", "conv_train"):
        y, fin = gdr.short_conv_fwd(s["x"], s["weight"], bias=s.get("b"), activation="silu",
                                    initial_state=s.get("state"), output_final_state=s["states"],
                                    cu_seqlens=s.get("cu"))
        if op == "conv_fwd":
            return {"y": y, "state": fin}
        dx, dw, db, ds = gdr.short_conv_bwd(s["x"], s["weight"], s["dy"], bias=s.get("b"), activation="silu",
                                            initial_state=s.get("state"), dfinal_state=s.get("dstate"),
                                            cu_seqlens=s.get("cu"))
        return {"y": y, "state": fin, "dx": dx, "dweight": dw, "dbias": db, "dstate": ds}
    opt = dict(D=s["Ds"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True)
    if op == "scan_step":
        y = gdr.selective_scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], **opt)
        return {"y": y, "state": s["state"]}
    train = op == "scan_train"
    y, fin, saved = gdr.selective_scan_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], initial_state=s.get("state"),
                                           output_final_state=not train or s["states"], cu_seqlens=s.get("cu"),
                                           save_for_backward=train, **opt)
    if not train:
        return {"y": y, "state": fin}
    grads = gdr.selective_scan_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], saved,
                                   initial_state=s.get("state"), dfinal_state=s.get("dstate"),
                                   cu_seqlens=s.get("cu"), **opt)
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate")
    return {"y": y, "state": fin, **dict(zip(names, grads))}


# ---------------------------------------------------------------- plain forms

def _sequences(s, B, T):
    """(sequence of every token, position in it [B,T]; first and past-the-last flat token of every sequence)."""
    if "cu" in s:
        cu = s["cu"].long()
        t = torch.arange(T, device=cu.device)
        seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        return seq[None], (t - cu[seq])[None], cu[:-1], cu[1:]
    b = torch.arange(B, device=_DEV)
    pos = torch.arange(T, device=_DEV)[None].expand(B, T)
    return b[:, None].expand(B, T), pos, b * T, (b + 1) * T


def _conv_inputs(s, x, state, W):
    """x[t - j] of every token for j = 0 .. W-1 (the cached inputs, or zeros, before a sequence), each [B*T, D]."""
    B, T, D = x.shape
    seq, pos, start, end = _sequences(s, B, T)
    seq, pos, flat = seq.reshape(-1), pos.reshape(-1), x.reshape(B * T, D)
    at = torch.arange(B * T, device=x.device)

    def tap(j):
        v = flat[(at - j).clamp(min=0)]
        before = 0.0 if state is None else state[seq, (W - 1 + pos - j).clamp(0, W - 2)]
        return torch.where((pos >= j)[:, None], v, before)

    return [tap(j) for j in range(W)], pos, start, end


def _conv_final(x, state, start, end, W):
    """The last W-1 inputs of every sequence, reaching back into the cached ones."""
    flat = x.reshape(-1, x.shape[-1])
    i = torch.arange(W - 1, device=x.device)
    p = (end - start)[:, None] - (W - 1) + i
    n = torch.arange(start.numel(), device=x.device)[:, None]
    before = 0.0 if state is None else state[n, (W - 1 + p).clamp(0, W - 2)]
    return torch.where((p >= 0)[..., None], flat[(start[:, None] + p).clamp(0, flat.shape[0] - 1)], before)


def _run_conv(s):
    W, dt = s["W"], s["x"].dtype
    x, w = s["x"].float(), s["weight"].float()
    B, T, D = x.shape
    state = s["state"].float() if "state" in s else None
    taps, pos, start, end = _conv_inputs(s, x, state, W)
    pre = sum(taps[j] * w[:, W - 1 - j] for j in range(W))
    if "b" in s:
        pre = pre + s["b"].float()
    sig = 1 / (1 + torch.exp(-pre))
    y = (pre * sig).view(B, T, D).to(dt)
    if s["op"] == "conv_step":
        s["state"].copy_(_conv_final(x, state, start, end, W))
        return {"y": y, "state": s["state"]}
    fin = _conv_final(x, state, start, end, W).to(dt) if s["states"] else None
    if s["op"] == "conv_fwd":
        return {"y": y, "state": fin}
    dpre = s["dy"].float().reshape(B * T, D) * sig * (1 + pre * (1 - sig))
    at = torch.arange(B * T, device=x.device)

    def ahead(j):  # the gradient that input t gets from token t + j of its sequence
        later = (at + j).clamp(max=B * T - 1)
        same = (at + j < B * T) & (pos[later] >= j) & (pos[later] - j == pos)
        return torch.where(same[:, None], dpre[later] * w[:, W - 1 - j], 0.0)

    dx = sum(ahead(j) for j in range(W))
    dw = torch.stack([(dpre * taps[W - 1 - i]).sum(0) for i in range(W)], 1).to(s["weight"].dtype)
    db = dpre.sum(0).to(s["b"].dtype) if "b" in s else None
    ds = None
    if s["states"]:
        n = torch.arange(start.numel(), device=x.device)
        ln = end - start
        df = s["dstate"].float()
        # the final state's entry i is the input at position ln - (W-1) + i, or the cached input W-1 before it
        p = ln[:, None] - (W - 1) + torch.arange(W - 1, device=x.device)
        inside = (p >= 0)[..., None]
        dx = dx.index_put(((start[:, None] + p).clamp(0, B * T - 1).reshape(-1),),
                          torch.where(inside, df, 0.0).reshape(-1, D), accumulate=True)
        ds = torch.zeros_like(df).index_put((n[:, None].expand_as(p).reshape(-1), (W - 1 + p).clamp(0, W - 2).reshape(-1)),
                                            torch.where(inside, 0.0, df).reshape(-1, D), accumulate=True)

        def cached(i, j):  # cached input i reaches the token at position i - (W-1) + j through tap j
            q = i - (W - 1) + j
            reach = (ln > q)[:, None] if q >= 0 else torch.zeros_like(ln, dtype=torch.bool)[:, None]
            return torch.where(reach, dpre[(start + max(q, 0)).clamp(max=B * T - 1)] * w[:, W - 1 - j], 0.0)

        ds = ds + torch.stack([sum(cached(i, j) for j in range(1, W)) for i in range(W - 1)], 1)
        ds = ds.to(dt)
    return {"y": y, "state": fin, "dx": dx.view(B, T, D).to(dt), "dweight": dw, "dbias": db, "dstate": ds}


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 by doubling; b becomes h, a is used up."""
    step = 1
    while step < a.shape[1]:
        b[:, step:] += a[:, step:] * b[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return b


def _run_scan(s):
    dt = s["x"].dtype
    x = s["x"].float()
    B, T, D = x.shape
    N, G = s["N"], s["G"]
    Dg = D // G
    shape = (B, T, G, Dg, 1)
    raw = s["dt"].float() + s["dt_bias"]
    delta = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    A = s["A"].view(G, Dg, N)
    Bm, Cm = s["Bm"].float().view(B, T, G, 1, N), s["Cm"].float().view(B, T, G, 1, N)
    seq, pos, start, end = _sequences(s, B, T)
    first = (pos == 0).view(B, T, 1, 1, 1)
    a = torch.exp(delta.view(shape) * A)
    b = (delta * x).view(shape) * Bm
    h0 = s["state"].view(-1, G, Dg, N) if "state" in s else None
    if h0 is not None:
        b += torch.where(first, a * h0[seq], 0.0)
    train = s["op"] == "scan_train"
    h = _scan(torch.where(first, 0.0, a), b)
    y = (h * Cm).sum(-1).view(B, T, D) + s["Ds"] * x
    z = s["z"].float()
    sig = 1 / (1 + torch.exp(-z))
    out = (y * z * sig).to(dt)
    fin = None
    if not train or s["states"]:
        fin = h.view(B * T, G, Dg, N)[(end - 1).clamp(min=0)]
        empty = (end == start).view(-1, 1, 1, 1)
        fin = torch.where(empty, h0 if h0 is not None else 0.0, fin).view(-1, D, N)
    if s["op"] == "scan_step":
        s["state"].copy_(fin)
        return {"y": out, "state": s["state"]}
    if not train:
        return {"y": out, "state": fin}
    dy = s["dy"].float()
    dz = dy * y * sig * (1 + z * (1 - sig))
    gy = dy * z * sig
    gh = gy.view(shape) * Cm
    if s["states"]:
        df = s["dstate"].view(-1, G, Dg, N)
        some = (end > start).view(-1, 1, 1, 1)
        gh.view(B * T, G, Dg, N).index_put_(((end - 1).clamp(min=0),), torch.where(some, df, 0.0), accumulate=True)
    after = torch.where(first, 0.0, a)
    after = torch.cat([after[:, 1:], torch.zeros_like(after[:, :1])], 1)
    gh = _scan(after.flip(1), gh.flip(1)).flip(1)
    del after
    prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    prev = torch.where(first, h0[seq] if h0 is not None else 0.0, prev)
    p = gh * a * prev
    del prev
    sb = (gh * Bm).sum(-1).view(B, T, D)
    ddt = x * sb + (p * A).sum(-1).view(B, T, D)
    ddt = ddt / (1 + torch.exp(-raw))
    grads = {
        "dx": (delta * sb + s["Ds"] * gy).to(dt), "ddt": ddt.to(dt),
        "dA": (p * delta.view(shape)).sum((0, 1)).view(D, N),
        "dB": (gh * (delta * x).view(shape)).sum(3).to(dt), "dC": (h * gy.view(shape)).sum(3).to(dt),
        "dD": (gy * x).sum((0, 1)), "dz": dz.to(dt), "ddt_bias": ddt.sum((0, 1)), "dstate": None}
    if s["states"]:
        ds = (gh * a).view(B * T, G, Dg, N)[start.clamp(max=B * T - 1)]
        grads["dstate"] = torch.where(some, ds, df).view(-1, D, N)
    return {"y": out, "state": fin, **grads}


def _run_norm(s):
    x, w = s["x"].float(), s["weight"]
    R, D = x.shape
    dt = s["x"].dtype
    h = x + s["residual"].float() if "residual" in s else x
    hr = h.to(s["residual"].dtype) if "residual" in s else None
    y = h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
    if s["quant"]:
        group = s["group"] or D
        n = -(-D // group)
        yp = torch.nn.functional.pad(y, (0, n * group - D)).view(R, n, group)
        scale = yp.abs().amax(-1).clamp(min=1e-30) / 448.0
        q = (yp / scale[..., None]).clamp(-448.0, 448.0).view(R, -1)[:, :D].to(torch.float8_e4m3fn)
        # the 8-bit output is returned as the float8 values that it holds, and their scales beside it
        return {"y": q, "residual": hr, "scale": scale}
    if s["op"] == "norm_fwd":
        return {"y": y.to(dt), "residual": hr, "scale": None}
    h = x if hr is None else hr.float()
    r = (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    dy = s["dy"].float()
    wd = dy * w
    dh = r * (wd - h * (r * r * (wd * h).mean(-1, keepdim=True)))
    if "dres" in s:
        dh = dh + s["dres"].float()
    return {"y": y.to(dt), "residual": hr, "dx": dh.to(dt),
            "dresidual": dh.to(hr.dtype) if hr is not None and hr.dtype != dt else None, "dweight": (dy * h * r).sum(0)}


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    return _run_norm(state) if op.startswith("norm") else _run_conv(state) if op.startswith("conv") else _run_scan(state)


# ---------------------------------------------------------------- the work that cannot be avoided

def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n, D, R = case["R"] * case["D"], case["D"], case["R"]
        res = {"": 0, "fp32": 4}.get(case["res"], 2)
        if op == "norm_fwd":
            scales = R * (-(-D // case["group"]) if case["group"] else 1) * 4 if case["quant"] else 0
            return {"bytes": n * (2 + 2 * res + (1 if case["quant"] else 2)) + scales + 4 * D, "flops": 6 * n}
        return {"bytes": n * (2 + 2 * res + 2) + n * (2 + (2 * res if res else 0) + (2 if res == 4 else 0) + (0 if res else 2)
                                                    ) + 8 * D, "flops": 18 * n}
    B, T, D = case["B"], case["T"], case["D"]
    n = B * T * D
    seqs = len(case["lens"].split(",")) if case.get("lens") else B
    if op.startswith("conv"):
        W = case["W"]
        st = 4 * seqs * (W - 1) * D if op == "conv_step" or case["states"] else 0
        fwd = {"bytes": 4 * n + st + 2 * D * (W + 1), "flops": n * (2 * W + 4)}
        if op != "conv_train":
            return fwd
        return {"bytes": fwd["bytes"] + 4 * n + st + 2 * D * (W + 1), "flops": n * (8 * W + 14)}
    N, G = case["N"], case["G"]
    st = 8 * seqs * D * N if op == "scan_step" or case["states"] else 4 * seqs * D * N if op == "scan_fwd" else 0
    fwd = {"bytes": 8 * n + 4 * B * T * G * N + st + 4 * D * (N + 2), "flops": n * (7 * N + 14)}
    if op != "scan_train":
        return fwd
    return {"bytes": fwd["bytes"] + 8 * n + 4 * B * T * G * N + st + 4 * D * (N + 2), "flops": n * (24 * N + 30)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _ranges(s, B, T):
    """The sequences as (row, first token, past the last token)."""
    if not s.get("lens"):
        return [(b, 0, T) for b in range(B)]
    out, at = [], 0
    for n in s["lens"].split(","):
        out.append((0, at, at + int(n)))
        at += int(n)
    return out


def _exact_conv(s):
    W = s["W"]
    x, w = s["x"].double(), s["weight"].double()
    B, T, D = x.shape
    train = s["op"] == "conv_train"
    y, dx = torch.empty_like(x), torch.zeros_like(x)
    dw, db = torch.zeros_like(w), torch.zeros(D, dtype=torch.float64, device=x.device)
    fins, dss = [], []
    for n, (b, t0, t1) in enumerate(_ranges(s, B, T)):
        past = s["state"][n].double() if "state" in s else torch.zeros(W - 1, D, dtype=torch.float64, device=x.device)
        ext = torch.cat([past, x[b, t0:t1]])
        L = t1 - t0
        pre = torch.zeros(L, D, dtype=torch.float64, device=x.device)
        for i in range(W):
            pre = pre + ext[i:i + L] * w[:, i]
        if "b" in s:
            pre = pre + s["b"].double()
        sg = torch.sigmoid(pre)
        y[b, t0:t1] = pre * sg
        fins.append(ext[L:])
        if train:
            d = s["dy"][b, t0:t1].double() * (sg + pre * sg * (1 - sg))
            de = torch.zeros_like(ext)
            for i in range(W):
                de[i:i + L] += d * w[:, i]
                dw[:, i] += (d * ext[i:i + L]).sum(0)
            if s["states"]:
                de[L:] += s["dstate"][n].double()
            db += d.sum(0)
            dx[b, t0:t1] = de[W - 1:]
            dss.append(de[:W - 1])
    keep = s["op"] == "conv_step" or s["states"]
    out = {"y": y, "state": torch.stack(fins) if keep else None}
    if train:
        out.update(dx=dx, dweight=dw, dbias=db if "b" in s else None, dstate=torch.stack(dss) if keep else None)
    return out


def _exact_scan(s):
    d64 = torch.float64
    x, z, A = s["x"].double(), s["z"].double(), s["A"].double()
    B, T, D = x.shape
    N, G = s["N"], s["G"]
    raw = s["dt"].double() + s["dt_bias"].double()
    delta = torch.where(raw > 0, raw, 0.0) + torch.log1p(torch.exp(-raw.abs()))
    Bm, Cm = s["Bm"].double(), s["Cm"].double()
    train, packed = s["op"] == "scan_train", bool(s.get("lens"))
    ranges = _ranges(s, B, T)
    init = s["state"].double() if "state" in s else torch.zeros(len(ranges), D, N, dtype=d64, device=x.device)
    fin = init.clone()
    starts = {t0: n for n, (_, t0, t1) in enumerate(ranges) if t1 > t0} if packed else {0: None}
    ends = {t1 - 1: n for n, (_, t0, t1) in enumerate(ranges) if t1 > t0} if packed else {T - 1: None}
    h = None
    hs = torch.empty(T, B, D, N, dtype=d64, device=x.device) if train else None
    y = torch.empty_like(x)

    def wide(m, t):  # [B,G,N] -> [B,D,N]
        return m[:, t].repeat_interleave(D // G, 1)

    def decay(t):
        return torch.exp(delta[:, t, :, None] * A)

    def before(t):
        if t in starts:
            return init if starts[t] is None else init[starts[t]][None]
        return hs[t - 1] if train else h

    for t in range(T):
        h = decay(t) * before(t) + (delta[:, t] * x[:, t])[..., None] * wide(Bm, t)
        y[:, t] = (h * wide(Cm, t)).sum(-1)
        if train:
            hs[t] = h
        if t in ends:
            if ends[t] is None:
                fin = h
            else:
                fin[ends[t]] = h[0]
    yp = y + s["Ds"].double() * x
    sg = torch.sigmoid(z)
    out = {"y": yp * z * sg, "state": fin if not train or s["states"] else None}
    if not train:
        return out
    dy = s["dy"].double()
    gy = dy * z * sg
    dfin = s["dstate"].double() if s["states"] else torch.zeros_like(init)
    dinit = dfin.clone()
    ddelta, dx = torch.empty_like(x), torch.empty_like(x)
    dB, dC = torch.empty_like(Bm), torch.empty_like(Cm)
    dA = torch.zeros_like(A)
    back = torch.zeros(B, D, N, dtype=d64, device=x.device)
    for t in reversed(range(T)):
        if t in ends:
            back = dfin if ends[t] is None else dfin[ends[t]][None]
        gh = back + gy[:, t, :, None] * wide(Cm, t)
        a = decay(t)
        dC[:, t] = (hs[t] * gy[:, t, :, None]).view(B, G, D // G, N).sum(2)
        dB[:, t] = (gh * (delta[:, t] * x[:, t])[..., None]).view(B, G, D // G, N).sum(2)
        through = (gh * wide(Bm, t)).sum(-1)
        back = gh * a
        q = back * before(t)
        dx[:, t] = through * delta[:, t]
        ddelta[:, t] = through * x[:, t] + (q * A).sum(-1)
        dA += (q * delta[:, t, :, None]).sum(0)
        if t in starts:
            if starts[t] is None:
                dinit = back
            else:
                dinit[starts[t]] = back[0]
    draw_ = ddelta * torch.sigmoid(raw)
    out.update(dx=dx + s["Ds"].double() * gy, ddt=draw_, dA=dA, dB=dB, dC=dC, dD=(gy * x).sum((0, 1)),
               dz=dy * yp * sg * (1 + z * (1 - sg)), ddt_bias=draw_.sum((0, 1)),
               dstate=dinit if s["states"] else None)
    return out


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    h = x + s["residual"].double() if "residual" in s else x
    n = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6)
    res = h if "residual" in s else None
    if s["quant"]:
        # the 8-bit values have no value in 64 bits: which one is nearest can hang on the last bit of the scale
        y = n * w
        group = s["group"] or s["D"]
        scale = torch.stack([c.abs().amax(-1) for c in y.split(group, 1)], 1).clamp(min=1e-30) / 448.0
        return {"y": None, "residual": res, "scale": scale}
    out = {"y": n * w, "residual": res, "scale": None}
    if s["op"] == "norm_train":
        h = x if res is None else res.to(s["residual"].dtype).double()  # the gradient is taken at the stored sum
        r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6)
        dy = s["dy"].double()
        dn = dy * w
        dh = r * dn - h * r ** 3 * (dn * h).mean(-1, keepdim=True)
        if "dres" in s:
            dh = dh + s["dres"].double()
        del out["scale"]
        two = res is not None and s["residual"].dtype != s["x"].dtype
        out.update(dx=dh, dresidual=dh if two else None, dweight=(dy * h * r).sum(0))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("scan") and case["T"] > 70000:
        return None
    return _exact_norm(s) if op.startswith("norm") else _exact_conv(s) if op.startswith("conv") else _exact_scan(s)
