"""The operators of a linear attention layer as measured cases: linear attention with one decay a head (whole prompts,
training, single tokens), the norm of its output with its gate, and the norms before and after a block fused with the
block's gate and residual scale.

Every case runs one operator in one direction.  With ``own`` false, ``run`` computes the plain form in elementary
torch operations, in fp32; with ``own`` true it calls the library.  ``exact`` evaluates the definitions in fp64,
the attention token by token."""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: one generated token of one row, its states updated in place
        dict(name="attn step 1x16", op="attn_step", B=1, T=1, Hk=16, H=16, K=128, V=128, dtype="bf16"),
        # one generated token for a serving batch of 256 rows
        dict(name="attn step 256x32", op="attn_step", B=256, T=1, Hk=32, H=32, K=128, V=128, dtype="bf16"),
        # prompts: dense forward with the final states for the cache
        dict(name="attn prompt 2x4096x32", op="attn_fwd", B=2, T=4096, Hk=32, H=32, K=128, V=128, dtype="bf16",
             start=False, lens=""),
        # one long document that continues from a cached state: few heads, the token axis has to be split
        dict(name="attn long 1x65536x16", op="attn_fwd", B=1, T=65536, Hk=16, H=16, K=128, V=128, dtype="bf16",
             start=True, lens=""),
        # a training step: forward and every gradient
        dict(name="attn train 2x4096x32", op="attn_train", B=2, T=4096, Hk=32, H=32, K=128, V=128, dtype="bf16",
             start=False, lens=""),
        # training on a packed ragged batch with states, keys shared by two heads, narrow heads
        dict(name="attn packed train 5311x8", op="attn_train", B=1, T=5311, Hk=4, H=8, K=64, V=96, dtype="fp16",
             start=True, lens="512,1024,768,3000,7"),
        # the mixer's output norm and gate, a head at a time, for one generated token of a serving batch
        dict(name="gated norm 256x32x128", op="gated_fwd", B=256, H=32, D=128, dtype="bf16", act="silu"),
        # the same in a training step: forward and every gradient
        dict(name="gated norm train 8192x32x128", op="gated_train", B=8192, H=32, D=128, dtype="bf16", act="silu"),
        # over the whole width with a sigmoid gate, an odd width
        dict(name="gated norm train 5311x4099", op="gated_train", B=5311, H=1, D=4099, dtype="fp16", act="sigmoid"),
        # between two blocks for one generated token of a serving batch: norm after, residual, norm before
        dict(name="block norm 256x4096", op="block_fwd", R=256, D=4096, dtype="bf16", res="bf16", post=True, gate="",
             rscale=1.0),
        # the same over a prompt batch with a token gate, the residual stream in fp32
        dict(name="block norm 8192x4096", op="block_fwd", R=8192, D=4096, dtype="bf16", res="fp32", post=True,
             gate="sigmoid", rscale=0.25),
        # training: forward and every gradient
        dict(name="block norm train 8192x4096", op="block_train", R=8192, D=4096, dtype="bf16", res="bf16", post=True,
             gate="sigmoid", rscale=0.25),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _lens(rng, T):
    """T tokens cut into a few sequences, some of them empty or of one token."""
    n = rng.randint(1, 12)
    cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))


def draw(rng):
    op = rng.choice(["attn_step", "attn_fwd", "attn_fwd", "attn_train", "attn_train", "gated_fwd", "gated_train",
                     "block_fwd", "block_train"])
    dtype = rng.choice(["bf16", "fp16"])
    if op.startswith("attn"):
        Hk = _spread(rng, 1, 32)
        H = Hk * rng.choice([1, 1, 1, 2, 4])
        K, V = (rng.choice([128, 128, 64, 8 * rng.randint(1, 16)]) for _ in range(2))
        if op == "attn_step":
            B = min(_spread(rng, 1, 512), max(1, 8192 // H))
            return dict(op=op, B=B, T=rng.choice([1, 1, 2, 5]), Hk=Hk, H=H, K=K, V=V, dtype=dtype)
        packed = rng.random() < 0.4
        B = 1 if packed else _spread(rng, 1, 8)
        T = min(_spread(rng, 1, 32768), max(1, (1 << (19 if op == "attn_fwd" else 17)) // (B * H)))
        return dict(op=op, B=B, T=T, Hk=Hk, H=H, K=K, V=V, dtype=dtype, start=rng.random() < 0.5,
                    lens=_lens(rng, T) if packed else "")
    if op.startswith("gated"):
        H = rng.choice([1, _spread(rng, 2, 64)])
        D = _spread(rng, 2, 16384 if H == 1 else 256)
        B = min(_spread(rng, 1, 32768), max(1, (1 << 25) // (D * H)))
        return dict(op=op, B=B, H=H, D=D, dtype=dtype, act=rng.choice(["silu", "sigmoid"]))
    D = _spread(rng, 2, 16384)
    R = min(_spread(rng, 1, 65536), max(1, (1 << 25) // D))
    return dict(op=op, R=R, D=D, dtype=dtype, res=rng.choice([dtype, "fp32"]), post=rng.random() < 0.7,
                gate=rng.choice(["", "raw", "sigmoid", "silu"]), rscale=rng.choice([1.0, 0.25]))


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(seed)
    dt = _DT[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=_DEV) * scale).to(dtype)

    op = case["op"]
    s = dict(case)
    if op.startswith("attn"):
        B, T, Hk, H, K, V = (case[n] for n in ("B", "T", "Hk", "H", "K", "V"))
        s["q"], s["k"], s["v"] = randn(B, T, Hk, K), randn(B, T, Hk, K), randn(B, T, H, V)
        # a geometric ladder of memories, from a token or two to some 256, as such layers fix it
        s["decay"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=_DEV, dtype=torch.float32) / H)
        nseq = B
        if case.get("lens"):
            cu = [0]
            for n in case["lens"].split(","):
                cu.append(cu[-1] + int(n))
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device=_DEV)
            nseq = len(cu) - 1
        if op == "attn_step" or case["start"]:
            s["state"] = randn(nseq, H, K, V, dtype=torch.float32)
        if op == "attn_train":
            s["do"] = randn(B, T, H, V)
            if case["start"]:
                s["dstate"] = randn(nseq, H, K, V, dtype=torch.float32)
        return s
    if op.startswith("gated"):
        shape = (case["B"], case["H"], case["D"])
        s["x"], s["g"] = randn(*shape), randn(*shape)
        s["weight"] = 1 + randn(case["D"], scale=0.1, dtype=torch.float32)
        if op == "gated_train":
            s["dy"] = randn(*shape)
        return s
    R, D, rt = case["R"], case["D"], _DT[case["res"]]
    s["x"], s["residual"] = randn(R, D), randn(R, D, scale=2.0, dtype=rt)
    s["weight"] = 1 + randn(D, scale=0.1, dtype=torch.float32)
    if case["post"]:
        s["post_weight"] = 1 + randn(D, scale=0.1, dtype=torch.float32)
    if case["gate"]:
        s["g"] = randn(R, D)
    if op == "block_train":
        s["dy"], s["dres"] = randn(R, D), randn(R, D, dtype=rt)
    return s


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    import gated_delta_rule_38_gb300 as gdr
    op = s["op"]
    if op == "attn_step":
        return {"o": gdr.linear_attention_step(s["q"], s["k"], s["v"], s["decay"], s["state"]), "state": s["state"]}
    if op.startswith("attn"):
        train = op == "attn_train"
        o, fin = gdr.linear_attention_fwd(s["q"], s["k"], s["v"], s["decay"], initial_state=s.get("state"),
                                          output_final_state=not train or s["start"], cu_seqlens=s.get("cu"))
        if not train:
            return {"o": o, "state": fin}
        dq, dk, dv, ds = gdr.linear_attention_bwd(s["q"], s["k"], s["v"], s["decay"], s["do"],
                                                  initial_state=s.get("state"), dfinal_state=s.get("dstate"),
                                                  cu_seqlens=s.get("cu"))
        return {"o": o, "state": fin, "dq": dq, "dk": dk, "dv": dv, "dstate": ds}
    if op.startswith("gated"):
        y = gdr.gated_rms_norm_fwd(s["x"], s["g"], s["weight"], activation=s["act"])
        if op == "gated_fwd":
            return {"y": y}
        dx, dg, dw = gdr.gated_rms_norm_bwd(s["x"], s["g"], s["weight"], s["dy"], activation=s["act"])
        return {"y": y, "dx": dx, "dgate": dg, "dweight": dw}
    opt = dict(post_weight=s.get("post_weight"), gate=s.get("g"), residual_scale=s["rscale"],
               gate_activation=s["gate"] if s["gate"] in ("sigmoid", "silu") else None)
    y, h = gdr.block_norm_fwd(s["x"], s["residual"], s["weight"], **opt)
    if op == "block_fwd":
        return {"y": y, "residual": h}
    dx, dr, dw, dp, dg = gdr.block_norm_bwd(s["x"], h, s["weight"], s["dy"], dresidual=s["dres"], **opt)
    return {"y": y, "residual": h, "dx": dx, "dresidual": dr, "dweight": dw, "dpost_weight": dp, "dgate": dg}


# ---------------------------------------------------------------- plain forms

def _powers(decay, n):
    """exp(decay n) of every head, [H, ...] for positions n [...]; the exponent in 64 bits."""
    return torch.exp(decay.double().view(-1, *[1] * n.dim()) * n.double()).float()


def _attend(q, k, v, decay, C=128):
    """sum over s <= r of exp(decay (r - s)) (q_r . k_s) v_s for rows [N,H,T,.], in chunks whose states are joined by
    doubling."""
    N, H, T, K = q.shape
    pad = -T % C
    q, k, v = (torch.nn.functional.pad(t, (0, 0, pad, 0)).reshape(N, H, -1, C, t.shape[-1]) for t in (q, k, v))
    i = torch.arange(C, device=q.device)
    d = i[:, None] - i
    gamma = torch.where(d >= 0, _powers(decay, d.clamp(min=0)), 0.0)[None, :, None]
    o = ((q @ k.transpose(-1, -2)) * gamma) @ v
    st = (k * _powers(decay, C - 1 - i)[None, :, None, :, None]).transpose(-1, -2) @ v
    step, nc = 1, st.shape[2]
    while step < nc:
        f = _powers(decay, torch.tensor(C * step, device=q.device)).view(1, H, 1, 1, 1)
        st = torch.cat([st[:, :, :step], st[:, :, step:] + f * st[:, :, :-step]], 2)
        step *= 2
    before = torch.nn.functional.pad(st[:, :, :-1], (0, 0, 0, 0, 1, 0))
    o = o + (q * _powers(decay, i + 1)[None, :, None, :, None]) @ before
    return o.reshape(N, H, -1, v.shape[-1])[:, :, pad:]


def _run_attn(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    B, T, Hk, K = q.shape
    H, V, dt, decay = s["H"], s["V"], s["q"].dtype, s["decay"]
    scale = K ** -0.5
    if "cu" in s:  # each sequence at the end of a row of its own
        cu = s["cu"].long()
        ln = cu[1:] - cu[:-1]
        width = max(int(n) for n in s["lens"].split(","))
        at = torch.arange(width, device=q.device) - (width - ln)[:, None]  # position in its sequence, or negative
        idx = (cu[:-1, None] + at).clamp(0, T - 1)
        live = (at >= 0)
        pos = at.clamp(min=0)
    else:
        idx = torch.arange(B * T, device=q.device).view(B, T)
        live = torch.ones_like(idx, dtype=torch.bool)
        pos = torch.arange(T, device=q.device).expand(B, T)
        ln = torch.full((B,), T, device=q.device)

    def rows(t, heads):  # [B,T,heads,D] -> [N,H,width,D], zeros before a sequence
        t = t.reshape(B * T, heads, -1)[idx] * live[..., None, None]
        return t.transpose(1, 2).repeat_interleave(H // heads, 1)

    def back(t, heads):  # [N,H,width,D] -> [B,T,heads,D], summed over the heads that share one
        t = t.transpose(1, 2)[live]
        return t.reshape(B, T, heads, H // heads, -1).sum(3)

    q, k, v = rows(q, Hk), rows(k, Hk), rows(v, H)
    first = _powers(decay, pos + 1).transpose(0, 1)[..., None]                 # what the start state has decayed by
    last = _powers(decay, ln[:, None] - 1 - pos).transpose(0, 1)[..., None]    # what is left at the sequence's end
    whole = _powers(decay, ln).transpose(0, 1)[..., None, None]
    s0 = s.get("state")
    o = _attend(q, k, v, decay)
    if s0 is not None:
        o = o + (q * first) @ s0
    o = back(scale * o, H).to(dt)
    fin = None
    if s["op"] != "attn_train" or s["start"]:
        fin = (k * last).transpose(-1, -2) @ v
        if s0 is not None:
            fin = fin + whole * s0
    if s["op"] == "attn_step":
        s["state"].copy_(fin)
        return {"o": o, "state": s["state"]}
    if s["op"] == "attn_fwd":
        return {"o": o, "state": fin}
    do = rows(s["do"].float(), H)
    dq = _attend(do, v, k, decay)
    if s0 is not None:
        dq = dq + (do * first) @ s0.transpose(-1, -2)
    # backwards in time the keys are the queries of what follows (rows flipped: sequences then begin them)
    f = [t.flip(2) for t in (q, k, v, do)]
    dk = scale * _attend(f[2], f[3], f[0], decay).flip(2)
    dv = scale * _attend(f[1], f[0], f[3], decay).flip(2)
    ds = None
    if s["start"]:
        df = s["dstate"]
        dk = dk + (v * last) @ df.transpose(-1, -2)
        dv = dv + (k * last) @ df
        ds = scale * ((q * first).transpose(-1, -2) @ do) + whole * df
    return {"o": o, "state": fin, "dq": back(scale * dq, Hk).to(dt), "dk": back(dk, Hk).to(dt),
            "dv": back(dv, H).to(dt), "dstate": ds}


def _gate(act, g):
    """(the gate's factor, its derivative)."""
    if act == "raw":
        return g, torch.ones_like(g)
    sig = 1 / (1 + torch.exp(-g))
    if act == "sigmoid":
        return sig, sig * (1 - sig)
    return g * sig, sig * (1 + g * (1 - sig))


def _run_gated(s):
    x, w, dt = s["x"].float(), s["weight"], s["x"].dtype
    a, da = _gate(s["act"], s["g"].float())
    r = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    n = x * r
    y = (n * w * a).to(dt)
    if s["op"] == "gated_fwd":
        return {"y": y}
    dy = s["dy"].float()
    dn = dy * w * a
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return {"y": y, "dx": dx.to(dt), "dgate": (dy * n * w * da).to(dt), "dweight": (dy * n * a).sum((0, 1))}


def _run_block(s):
    x, dt = s["x"].float(), s["x"].dtype
    rt = s["residual"].dtype
    n = x
    if s["post"]:
        r1 = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        n = x * r1
    b = n * s["post_weight"] if s["post"] else n
    a, da = _gate(s["gate"], s["g"].float()) if s["gate"] else (None, None)
    h = s["residual"].float() + s["rscale"] * (b if a is None else b * a)
    hr = h.to(rt)
    y = (h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * s["weight"]).to(dt)
    if s["op"] == "block_fwd":
        return {"y": y, "residual": hr}
    h = hr.float()
    r2 = (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    dy = s["dy"].float()
    wd = dy * s["weight"]
    dh = r2 * (wd - h * (r2 * r2 * (wd * h).mean(-1, keepdim=True))) + s["dres"].float()
    db = s["rscale"] * dh
    out = {"y": y, "residual": hr, "dresidual": dh.to(rt), "dweight": (dy * h * r2).sum(0), "dgate": None,
           "dpost_weight": None}
    if a is not None:
        out["dgate"] = (db * b * da).to(dt)
        db = db * a
    if s["post"]:
        out["dpost_weight"] = (db * n).sum(0)
        dn = db * s["post_weight"]
        db = r1 * (dn - n * (dn * n).mean(-1, keepdim=True))
    out["dx"] = db.to(dt)
    return out


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    return _run_attn(state) if op.startswith("attn") else _run_gated(state) if op.startswith("gated") else _run_block(state)


# ---------------------------------------------------------------- the work that cannot be avoided

def work(case):
    op = case["op"]
    if op.startswith("attn"):
        B, T, Hk, H, K, V = (case[n] for n in ("B", "T", "Hk", "H", "K", "V"))
        seqs = len(case["lens"].split(",")) if case.get("lens") else B
        qk, vo, st = 2 * B * T * Hk * K, 2 * B * T * H * V, 4 * seqs * H * K * V
        tokens = B * T * H
        if op == "attn_step":
            return {"bytes": 2 * qk + 2 * vo + 2 * st, "flops": 5 * tokens * K * V}
        states = (1 if op == "attn_fwd" else 0) + (1 if case["start"] else 0) * (1 if op == "attn_fwd" else 2)
        fwd = {"bytes": 2 * qk + 2 * vo + states * st, "flops": 4 * tokens * K * V}
        if op == "attn_fwd":
            return fwd
        more = 4 * qk + 3 * vo + (3 * st if case["start"] else 0)
        return {"bytes": fwd["bytes"] + more, "flops": 14 * tokens * K * V}
    if op.startswith("gated"):
        n, D = case["B"] * case["H"] * case["D"], case["D"]
        if op == "gated_fwd":
            return {"bytes": 6 * n + 4 * D, "flops": 10 * n}
        return {"bytes": 16 * n + 12 * D, "flops": 30 * n}
    n, D = case["R"] * case["D"], case["D"]
    rb, gb = (4 if case["res"] == "fp32" else 2), (2 if case["gate"] else 0)
    w = 4 * D * (2 if case["post"] else 1)
    fwd = {"bytes": n * (2 + 2 * rb + gb + 2) + w, "flops": 16 * n}
    if op == "block_fwd":
        return fwd
    return {"bytes": fwd["bytes"] + n * (2 + 3 * rb + 2 * gb + 2 + 2) + 2 * w, "flops": 46 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_attn(s):
    B, T, Hk, K = s["q"].shape
    H, V = s["H"], s["V"]
    scale = K ** -0.5
    lens = [int(n) for n in s["lens"].split(",")] if s.get("lens") else [T] * B
    n, most, dev = len(lens), max(lens), s["q"].device

    def rows(name, heads):  # one row a sequence, zeros behind its end
        flat = s[name].reshape(B * T, heads, -1)
        out = torch.zeros(most, n, heads, flat.shape[-1], dtype=torch.float64, device=dev)
        first = 0
        for i, length in enumerate(lens):
            out[:length, i] = flat[first:first + length].double()
            first += length
        return out.repeat_interleave(H // heads, 2)

    def flat(t, heads):  # [most,n,H,D] -> [B,T,heads,D]
        t = torch.cat([t[:length, i] for i, length in enumerate(lens)])
        return t.view(B, T, heads, H // heads, -1).sum(3)

    q, k, v = rows("q", Hk), rows("k", Hk), rows("v", H)
    lam = torch.exp(s["decay"].double())[None, :, None, None]
    train = s["op"] == "attn_train"
    S = s["state"].double() if "state" in s else torch.zeros(n, H, K, V, dtype=torch.float64, device=dev)
    o = torch.empty_like(v)
    do = rows("do", H) if train else None
    dq = torch.empty_like(q) if train else None
    ended = sorted(set(lens))  # rows of these lengths keep their state from there on
    length = torch.tensor(lens, device=dev).view(n, 1, 1, 1)
    ragged = len(ended) > 1
    for t in range(most):
        new = lam * S + k[t][..., None] * v[t][..., None, :]
        S = torch.where(t < length, new, S) if ragged else new
        o[t] = scale * (q[t][..., None, :] @ S)[..., 0, :]
        if train:
            dq[t] = scale * (S @ do[t][..., None])[..., 0]
    keep = not train or s["start"]
    out = {"o": flat(o, H), "state": S if keep else None}
    if not train:
        return out
    G = s["dstate"].double() if s["start"] else torch.zeros_like(S)
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    for t in reversed(range(most)):
        here = G + scale * q[t][..., None] * do[t][..., None, :]
        dk[t] = (here @ v[t][..., None])[..., 0]
        dv[t] = (k[t][..., None, :] @ here)[..., 0, :]
        G = torch.where(t < length, lam * here, G) if ragged else lam * here
    return {**out, "dq": flat(dq, Hk), "dk": flat(dk, Hk), "dv": flat(dv, H), "dstate": G if s["start"] else None}


def _act64(act, g):
    return g if act == "raw" else torch.sigmoid(g) if act == "sigmoid" else g * torch.sigmoid(g)


def _dact64(act, g):
    p = torch.sigmoid(g)
    return torch.ones_like(g) if act == "raw" else p * (1 - p) if act == "sigmoid" else p + g * p * (1 - p)


def _norm64(x):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)


def _dnorm64(x, d):
    """The gradient at x of sum(d norm(x))."""
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return r * d - x * r ** 3 * (d * x).mean(-1, keepdim=True)


def _exact_gated(s):
    x, g, w = s["x"].double(), s["g"].double(), s["weight"].double()
    a, n = _act64(s["act"], g), _norm64(x)
    out = {"y": n * w * a}
    if s["op"] == "gated_train":
        dy = s["dy"].double()
        out.update(dx=_dnorm64(x, dy * w * a), dgate=dy * n * w * _dact64(s["act"], g),
                   dweight=(dy * n * a).sum((0, 1)))
    return out


def _exact_block(s):
    x, w = s["x"].double(), s["weight"].double()
    b = _norm64(x) * s["post_weight"].double() if s["post"] else x
    a = _act64(s["gate"], s["g"].double()) if s["gate"] else torch.ones_like(x)
    h = s["residual"].double() + s["rscale"] * b * a
    out = {"y": _norm64(h) * w, "residual": h}
    if s["op"] == "block_fwd":
        return out
    h = h.to(s["residual"].dtype).double()  # the gradient is taken at the stored sum
    dy = s["dy"].double()
    dh = _dnorm64(h, dy * w) + s["dres"].double()
    db = s["rscale"] * dh
    out.update(dresidual=dh, dweight=(dy * _norm64(h)).sum(0), dgate=None, dpost_weight=None, dx=db * a)
    if s["gate"]:
        out["dgate"] = db * b * _dact64(s["gate"], s["g"].double())
    if s["post"]:
        out["dpost_weight"] = (db * a * _norm64(x)).sum(0)
        out["dx"] = _dnorm64(x, db * a * s["post_weight"].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_attn(s) if op.startswith("attn") else _exact_gated(s) if op.startswith("gated") else _exact_block(s)
