"""Workloads of the recurrent block's operators: RMS norm (with the residual's addition and an
8-bit output), the short causal convolution and the selective scan, each for prompts, for single
tokens where it has that form, and backward.

Tokens are [B, H, T, d] as everywhere in this package; a block of width D passes H = 1, d = D.
`run` with `own` false computes the plain form (elementary torch operations in fp32, rounded once);
with `own` true it makes the package's calls. `exact` restates the definitions in fp64.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of a few sequences: the residual stream's norm, latency
        dict(name="norm_token", op="norm_fwd", B=8, H=1, T=1, d=2048, dtype="bf16", residual=True, quant=False, per_head=False),
        # a batch of prompts before an 8-bit projection
        dict(name="norm_prompt_8bit", op="norm_fwd", B=4, H=1, T=4096, d=2048, dtype="bf16", residual=True, quant=True, per_head=False),
        # the q/k normalisation of 16 heads of 64 (token-major storage)
        dict(name="norm_heads", op="norm_fwd", B=8, H=16, T=2048, d=64, dtype="bf16", residual=False, quant=False, per_head=True),
        # training: the residual stream's norm, backward
        dict(name="norm_backward", op="norm_bwd", B=4, H=1, T=4096, d=2048, dtype="bf16", residual=True, per_head=False),
        # a batch of prompts through the convolution of an expanded width
        dict(name="conv_prompt", op="conv_fwd", B=4, H=1, T=4096, d=4096, K=4, dtype="bf16", silu=True, state=False, packed=0),
        # ragged prompts packed behind one another, continued from earlier chunks, odd width
        dict(name="conv_packed", op="conv_fwd", B=1, H=3, T=5001, d=203, K=3, dtype="f32", silu=True, state=True, packed=7),
        # training
        dict(name="conv_backward", op="conv_bwd", B=2, H=1, T=4096, d=4096, K=4, dtype="bf16", silu=True, state=False, packed=0),
        # decoding: one token of each sequence
        dict(name="conv_token", op="conv_step", B=64, H=1, d=4096, K=4, dtype="bf16", silu=True, slots=80),
        # a batch of prompts, gated
        dict(name="scan_prompt", op="scan_fwd", B=4, H=1, T=4096, d=4096, N=16, G=1, dtype="bf16", gate=True, state=False, packed=0),
        # ragged packed prompts with states carried in, heads with B and C of their own, odd sizes
        dict(name="scan_packed", op="scan_fwd", B=1, H=3, T=3001, d=203, N=13, G=3, dtype="f32", gate=False, state=True, packed=7),
        # training
        dict(name="scan_backward", op="scan_bwd", B=2, H=1, T=2048, d=2048, N=16, G=1, dtype="bf16", gate=True, state=False, packed=0),
        # decoding: one token of each sequence, states in a pool
        dict(name="scan_token", op="scan_step", B=64, H=1, d=4096, N=16, G=1, dtype="bf16", gate=True, slots=80),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    B, H = _log(rng, 1, 8), rng.choice([1, 1, 2, 3, 8])
    width = _log(rng, 40, 4096)
    d = max(1, width // H)
    if op.startswith("norm"):
        T = max(1, min(_log(rng, 1, 8192), 32_000_000 // (B * H * d)))
        c = dict(op=op, B=B, H=H, T=T, d=d, dtype=dtype, residual=rng.random() < 0.5, per_head=rng.random() < 0.3)
        return dict(c, quant=rng.random() < 0.4) if op == "norm_fwd" else c
    if op == "conv_step":
        B = _log(rng, 1, 128)
        return dict(op=op, B=B, H=H, d=d, K=rng.randint(1, 8), dtype=dtype, silu=rng.random() < 0.8, slots=B + rng.randint(0, 20))
    if op == "scan_step":
        B, G = _log(rng, 1, 128), rng.choice([1, H])
        return dict(op=op, B=B, H=H, d=d, N=rng.choice([1, 5, 8, 13, 16, 16, 24, 32, 64]), G=G, dtype=dtype, gate=rng.random() < 0.7,
                    slots=B + rng.randint(0, 20))
    packed = rng.choice([0, 0, 1, 3, 9, 40])
    B = 1 if packed else B
    if op.startswith("conv"):
        T = max(1, min(_log(rng, 1, 8192), 32_000_000 // (B * H * d)))
        return dict(op=op, B=B, H=H, T=T, d=d, K=rng.randint(1, 8), dtype=dtype, silu=rng.random() < 0.8, state=rng.random() < 0.5, packed=packed)
    N = rng.choice([1, 5, 8, 13, 16, 16, 24, 32, 64])
    cap = (700_000_000 if op == "scan_fwd" else 100_000_000) // (B * H * d * N)
    T = max(1, min(_log(rng, 1, 4096), cap))
    return dict(op=op, B=B, H=H, T=T, d=d, N=N, G=rng.choice([1, H]), dtype=dtype, gate=rng.random() < 0.6, state=rng.random() < 0.5, packed=packed)


# ---- inputs ----------------------------------------------------------------------------------

def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tokens(g, case, T, width, heads=None, scale=1.0):
    """[B, heads, T, width] with token-major storage and rows padded to 16 bytes, as projections leave them."""
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    heads = case["H"] if heads is None else heads
    pad = -(-width // 8) * 8
    x = (_rand(g, case["B"], T, heads, pad) * scale).to(dt)
    return x[..., :width].permute(0, 2, 1, 3)


def _cuts(case, seed):
    """The ends of `packed` sequences in T packed tokens: random, now and then an empty one, and a few tokens behind the last."""
    g = torch.Generator().manual_seed(seed)
    n, T = case["packed"], case["T"]
    last = T - int(torch.randint(0, max(1, T // 20) + 1, (1,), generator=g))
    cuts = torch.randint(0, last + 1, (n - 1,), generator=g).sort().values.tolist()
    if n > 3:
        cuts[1] = cuts[0]
    return [0] + cuts + [last]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, H, d = case["op"], case["H"], case["d"]
    s = dict(case=case)
    if op.startswith("norm"):
        s["x"] = _tokens(g, case, case["T"], d, scale=2.0)
        s["w"] = 1 + 0.1 * _rand(g, *((H, d) if case["per_head"] else (d,)))
        if case["residual"]:
            s["r"] = _tokens(g, case, case["T"], d)
        if op == "norm_bwd":
            s["dy"] = _tokens(g, case, case["T"], d)
        return s
    T = case.get("T", 1)
    s["x"] = _tokens(g, case, T, d)
    if case.get("packed"):
        ends = _cuts(case, seed)
        s["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    S = case["slots"] if "slots" in case else case["packed"] or case["B"]
    if "slots" in case:
        # each row's place in the pool; in a padded batch the last row is nobody's
        s["slots"] = torch.randperm(S, generator=g, device="cuda")[:case["B"]].to(torch.int32)
        if case["B"] > 4:
            s["slots"][-1] = -1
        s["out"] = torch.zeros(case["B"], H, 1, d, dtype=s["x"].dtype, device="cuda")
    if op.startswith("conv"):
        K = case["K"]
        s["w"] = _rand(g, H, d, K) / math.sqrt(K)
        s["bias"] = 0.1 * _rand(g, H, d)
        if case.get("state") or op == "conv_step":
            pad = -(-d // 8) * 8
            s["state"] = _rand(g, S, H, K - 1, pad).to(s["x"].dtype)[..., :d]
        if op == "conv_bwd":
            s["dy"] = _tokens(g, case, T, d)
            if case["state"]:
                s["dstate"] = torch.empty_like(s["state"]).copy_(_rand(g, S, H, K - 1, d))
        return s
    N = case["N"]
    s["dt"] = _tokens(g, case, T, d, scale=0.5)
    # the usual start: A_n = -n, step sizes between 1e-3 and 1e-1 through the bias
    s["A"] = -torch.arange(1, N + 1, device="cuda").float().expand(H, d, N) * (1 + 0.1 * torch.rand(H, d, N, generator=g, device="cuda"))
    step = torch.exp(torch.rand(H, d, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = 1 + 0.1 * _rand(g, H, d)
    s["Bm"] = _tokens(g, case, T, N, case["G"])
    s["Cm"] = _tokens(g, case, T, N, case["G"])
    if case["gate"]:
        s["z"] = _tokens(g, case, T, d)
    if case.get("state") or op == "scan_step":
        s["h0"] = _rand(g, S, H, d, N)
    if op == "scan_bwd":
        s["dy"] = _tokens(g, case, T, d)
        if case["state"]:
            s["dh"] = _rand(g, S, H, d, N)
    return s


# ---- the package's calls ---------------------------------------------------------------------

def _call(s):
    from linear_attention_ttt_b200 import ops
    c, op = s["case"], s["case"]["op"]
    if op == "norm_fwd":
        out, scale, res = ops.rms_norm_fwd(s["x"], s["w"], EPS, residual=s.get("r"), quant=c["quant"])
        return [t for t in (out, scale, res) if t is not None]
    if op == "norm_bwd":
        return list(ops.rms_norm_bwd(s["x"], s["w"], s["dy"], EPS, dres=s.get("r")))
    if op == "conv_fwd":
        return list(ops.causal_conv_fwd(s["x"], s["w"], s["bias"], c["silu"], state0=s.get("state"), cu_seqlens=s.get("cu")))
    if op == "conv_bwd":
        got = ops.causal_conv_bwd(s["x"], s["w"], s["dy"], s["bias"], c["silu"], state0=s.get("state"), dstate_final=s.get("dstate"),
                                  cu_seqlens=s.get("cu"))
        return [t for t in got if t is not None]
    if op == "conv_step":
        return [ops.causal_conv_step(s["x"], s["state"], s["w"], s["bias"], c["silu"], slots=s["slots"], out=s["out"]), s["state"]]
    args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
    kw = dict(D=s["D"], z=s.get("z"), dt_bias=s["dt_bias"], softplus=True)
    if op == "scan_fwd":
        return list(ops.selective_scan_fwd(*args, h0=s.get("h0"), cu_seqlens=s.get("cu"), **kw))
    if op == "scan_bwd":
        got = ops.selective_scan_bwd(*args, s["dy"], h0=s.get("h0"), dh_final=s.get("dh"), cu_seqlens=s.get("cu"), **kw)
        return [t for t in got if t is not None]
    return [ops.selective_scan_step(*args, s["h0"], slots=s["slots"], out=s["out"], **kw), s["h0"]]


# ---- plain forms -----------------------------------------------------------------------------

def _rows(x):
    """[B,H,T,d] -> [B*T, H, d] in fp32: every token of every sequence behind one another."""
    return x.float().permute(0, 2, 1, 3).flatten(0, 1)


def _back(y, like, dtype=None):
    """[B*T, H, d] -> [B,H,T,d], rounded."""
    B, H, T, d = like.shape
    return y.reshape(B, T, H, d).permute(0, 2, 1, 3).to(dtype or like.dtype)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _dsilu(x):
    t = 1 / (1 + torch.exp(-x))
    return t * (1 + x * (1 - t))


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(torch.clamp(x, max=20))))


def _places(s):
    """For every packed row: its sequence, its place in it, whether it is anybody's; and the sequences' ends and lengths."""
    B, _, T, _ = s["x"].shape
    cu = s["cu"].long() if "cu" in s else torch.arange(0, B + 1, device="cuda") * T
    row = torch.arange(B * T, device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True).clamp(max=len(cu) - 2)
    return seq, row - cu[seq], row < cu[-1], cu


def _norm_fwd(s):
    c, x = s["case"], s["x"].float()
    if "r" in s:
        x = x + s["r"].float()
    w = s["w"][:, None, :] if c["per_head"] else s["w"]
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    out = [y.to(s["x"].dtype)]
    if c["quant"]:
        top = y.abs().amax(-1, keepdim=True)
        scale = top / E4M3_MAX
        out = [(y / torch.where(scale > 0, scale, 1.0)).to(torch.float8_e4m3fn), scale[..., 0]]
    return out + ([x.to(s["x"].dtype)] if "r" in s else [])


def _norm_bwd(s):
    h, dy = s["x"].float(), s["dy"].float()
    w = s["w"][:, None, :] if s["case"]["per_head"] else s["w"]
    rs = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n, dn = h * rs, dy * w
    dh = rs * (dn - n * (dn * n).mean(-1, keepdim=True))
    if "r" in s:
        dh = dh + s["r"].float()
    return [dh.to(s["x"].dtype), (dy * n).sum((0, 2) if s["case"]["per_head"] else (0, 1, 2))]


def _taps(s, x):
    """[rows, H, K, d]: the K inputs that each row's output reads, oldest first."""
    K = s["case"]["K"]
    seq, place, live, cu = _places(s)
    back = torch.arange(K - 1, -1, -1, device="cuda")
    at = place[:, None] - back                                             # place of each tap in its sequence
    row = (cu[seq][:, None] + at).clamp(min=0)
    taps = torch.where((at >= 0)[:, :, None, None], x[row], 0.0)
    if "state" in s and K > 1:
        old = s["state"].float().permute(0, 2, 1, 3)                       # [S, K-1, H, d]
        before = old[seq[:, None], (K - 1 + at).clamp(0, K - 2)]
        taps = torch.where((at < 0)[:, :, None, None], before, taps)
    return torch.where(live[:, None, None, None], taps, 0.0), live, seq, at, row


def _last_inputs(s, x):
    """[S, H, K-1, d]: each sequence's last K-1 inputs, with the old state before them."""
    K = s["case"]["K"]
    _, _, _, cu = _places(s)
    n = cu[1:] - cu[:-1]
    at = n[:, None] + torch.arange(-(K - 1), 0, device="cuda")             # place in the sequence
    new = torch.where((at >= 0)[:, :, None, None], x[(cu[:-1, None] + at).clamp(0, len(x) - 1)], 0.0)
    if "state" in s and K > 1:
        old = s["state"].float().permute(0, 2, 1, 3)
        seq = torch.arange(len(n), device="cuda")[:, None]
        new = torch.where((at < 0)[:, :, None, None], old[seq, (K - 1 + at).clamp(0, K - 2)], new)
    return new.permute(0, 2, 1, 3)


def _conv_fwd(s):
    x = _rows(s["x"])
    w = s["w"].permute(2, 0, 1)                                            # [K, H, d]
    taps, live, _, _, _ = _taps(s, x)
    p = (taps * w).sum(1) + s["bias"]
    y = _silu(p) if s["case"]["silu"] else p
    y = torch.where(live[:, None, None], y, 0.0)
    return [_back(y, s["x"]), _last_inputs(s, x).to(s["x"].dtype)]


def _conv_bwd(s):
    x, dy, K = _rows(s["x"]), _rows(s["dy"]), s["case"]["K"]
    w = s["w"].permute(2, 0, 1)
    taps, live, seq, at, row = _taps(s, x)
    p = (taps * w).sum(1) + s["bias"]
    dp = torch.where(live[:, None, None], dy * _dsilu(p) if s["case"]["silu"] else dy, 0.0)
    place = at[:, -1]
    _, _, _, cu = _places(s)
    n = (cu[1:] - cu[:-1])
    ahead = torch.arange(K - 1, -1, -1, device="cuda")                     # tap j of the output `ahead` rows later
    later = torch.arange(len(x), device="cuda")[:, None] + ahead
    inside = (place[:, None] + ahead < n[seq][:, None]) & live[:, None]
    dx = (torch.where(inside[:, :, None, None], dp[later.clamp(max=len(x) - 1)], 0.0) * w).sum(1)
    grads = [(dp[:, None] * taps).sum(0).permute(1, 2, 0), dp.sum(0)]
    if "state" in s:
        # the state's place i (of K-1) is the input at i - (K-1); its taps are those of the first outputs
        i = torch.arange(K - 1, device="cuda")
        out = i[:, None] - (K - 1) + ahead                                 # the output that reads it by tap j
        ok = (out >= 0)[None] & (out[None] < n[:, None, None])
        rows = (cu[:-1, None, None] + out.clamp(min=0)[None]).clamp(max=len(x) - 1)
        ds = (torch.where(ok[..., None, None], dp[rows], 0.0) * w).sum(2)  # [S, K-1, H, d]
        # the last inputs: the final state's gradient goes to the inputs it holds, or to the old state's
        df = s["dstate"].float().permute(0, 2, 1, 3)
        src = n[:, None] + i - (K - 1)                                     # [S, K-1] place it came from
        seqs = torch.arange(len(n), device="cuda")[:, None].expand_as(src)
        held = src >= 0
        dx = dx.index_put(((cu[:-1, None] + src)[held],), df[held], accumulate=True)
        ds = ds.index_put((seqs[~held], (src + K - 1)[~held]), df[~held], accumulate=True)
        grads.append(ds.permute(0, 2, 1, 3).to(s["x"].dtype))
    return [_back(dx, s["x"])] + grads


def _conv_step(s):
    x, live = s["x"].float()[:, :, 0], s["slots"] >= 0
    at = s["slots"].long()[live]
    taps = torch.cat([s["state"][at].float(), x[live][:, :, None]], 2)     # [rows, H, K, d]
    p = (taps * s["w"].transpose(1, 2)).sum(2) + s["bias"]
    s["out"][live] = (_silu(p) if s["case"]["silu"] else p).to(s["x"].dtype)[:, :, None]
    s["state"][at] = taps[:, :, 1:].to(s["state"].dtype)
    return [s["out"], s["state"]]


def _scan(a, b, most):
    """h_t = a_t h_{t-1} + b_t over the first axis, by doubling; a row's reach is at most `most`."""
    step = 1
    while step < most:
        nb = b.clone()
        nb[step:] += a[step:] * b[:-step]
        b = nb
        na = a.clone()
        na[step:] *= a[:-step]
        a = na
        step *= 2
    return b


def _scan_parts(s):
    """dt, the decays and inputs of the recurrence for every packed row: [rows, H, d(, N)], starts cut off with their states put in."""
    c = s["case"]
    seq, place, live, cu = _places(s)
    rep = c["H"] // c["G"]
    mask = live[:, None, None]
    x = torch.where(mask, _rows(s["x"]), 0.0)
    raw = torch.where(mask, _rows(s["dt"]), 0.0) + s["dt_bias"]
    dt = torch.where(mask, _softplus(raw), 0.0)
    Bm = torch.where(mask, _rows(s["Bm"]), 0.0).repeat_interleave(rep, 1)[:, :, None]
    Cm = torch.where(mask, _rows(s["Cm"]), 0.0).repeat_interleave(rep, 1)[:, :, None]
    a = torch.exp(dt[..., None] * s["A"])
    b = (dt * x)[..., None] * Bm
    first = ((place == 0) & live)[:, None, None, None]
    if "h0" in s:
        b = torch.where(first, b + a * s["h0"][seq], b)
    return x, raw, dt, Bm, Cm, a, b, first, seq, live, cu


def _finals(s, h, cu):
    n = cu[1:] - cu[:-1]
    old = s["h0"] if "h0" in s else torch.zeros_like(h[:1])
    return torch.where((n > 0)[:, None, None, None], h[(cu[1:] - 1).clamp(min=0)], old)


def _scan_fwd(s):
    x, _, _, _, Cm, a, b, first, _, live, cu = _scan_parts(s)
    h = _scan(torch.where(first, 0.0, a), b, s["case"]["T"])
    del a, b
    y = (h * Cm).sum(-1) + s["D"] * x
    if "z" in s:
        y = y * _silu(_rows(s["z"]))
    y = torch.where(live[:, None, None], y, 0.0)
    return [_back(y, s["x"]), _finals(s, h, cu)]


def _scan_bwd(s):
    c = s["case"]
    x, raw, dt, Bm, Cm, a, b, first, seq, live, cu = _scan_parts(s)
    h = _scan(torch.where(first, 0.0, a), b, c["T"])
    del b
    mask = live[:, None, None]
    dout = torch.where(mask, _rows(s["dy"]), 0.0)
    y = (h * Cm).sum(-1) + s["D"] * x
    dz = None
    dy = dout
    if "z" in s:
        z = torch.where(mask, _rows(s["z"]), 0.0)
        dz, dy = dout * y * _dsilu(z), dout * _silu(z)
    n = cu[1:] - cu[:-1]
    last = (torch.arange(len(x), device="cuda") == cu[seq + 1] - 1) & live
    g = dy[..., None] * Cm
    if "dh" in s:
        g = torch.where(last[:, None, None, None], g + s["dh"][seq], g)
    after = torch.cat([a[1:], a[:1]])
    after = torch.where(last[:, None, None, None], 0.0, after)
    g = _scan(after.flip(0), g.flip(0), c["T"]).flip(0)
    del after
    was = h - (dt * x)[..., None] * Bm                                     # exp(dt A) h_{t-1}
    ddt = (g * (s["A"] * was + x[..., None] * Bm)).sum(-1)
    dA = (g * was * dt[..., None]).sum(0)
    dB, dC = (g * (dt * x)[..., None]).sum(2), (dy[..., None] * h).sum(2)  # over the head's channels
    dB, dC = (t.unflatten(1, (c["G"], -1)).sum(2) for t in (dB, dC))
    dx = dt * (g * Bm).sum(-1) + s["D"] * dy
    ddt = torch.where(mask, ddt / (1 + torch.exp(-raw)), 0.0)
    out = [_back(dx, s["x"]), _back(ddt, s["x"]), dA, _back(dB, s["Bm"]), _back(dC, s["Bm"]), (dy * x).sum(0)]
    if dz is not None:
        out.append(_back(dz, s["x"]))
    out.append(ddt.sum(0))
    if "h0" in s:
        start = cu[:-1].clamp(max=len(x) - 1)
        out.append(torch.where((n > 0)[:, None, None, None], a[start] * g[start], s["dh"]))
    return out


def _scan_step(s):
    c, live = s["case"], s["slots"] >= 0
    at = s["slots"].long()[live]
    x, raw = s["x"].float()[live, :, 0], s["dt"].float()[live, :, 0] + s["dt_bias"]
    dt, rep = _softplus(raw), c["H"] // c["G"]
    Bm, Cm = (s[k].float()[live, :, 0].repeat_interleave(rep, 1)[:, :, None] for k in ("Bm", "Cm"))
    h = torch.exp(dt[..., None] * s["A"]) * s["h0"][at] + (dt * x)[..., None] * Bm
    y = (h * Cm).sum(-1) + s["D"] * x
    if "z" in s:
        y = y * _silu(s["z"].float()[live, :, 0])
    s["h0"][at] = h
    s["out"][live] = y.to(s["x"].dtype)[:, :, None]
    return [s["out"], s["h0"]]


def run(state):
    if own:
        return _call(state)
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "conv_fwd": _conv_fwd, "conv_bwd": _conv_bwd, "conv_step": _conv_step,
            "scan_fwd": _scan_fwd, "scan_bwd": _scan_bwd, "scan_step": _scan_step}[state["case"]["op"]](state)


# ---- work ------------------------------------------------------------------------------------

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    B, H, T, d = case["B"], case["H"], case.get("T", 1), case["d"]
    n = B * H * T * d
    if op == "norm_fwd":
        out = n + 4 * B * H * T if case["quant"] else n * e
        return dict(bytes=n * e * (3 if case["residual"] else 1) + out + 4 * d, flops=6 * n)
    if op == "norm_bwd":
        return dict(bytes=n * e * (4 if case["residual"] else 3) + 8 * d, flops=12 * n)
    S = case["B"] if "slots" in case else case["packed"] or B
    if op.startswith("conv"):
        K = case["K"]
        state = S * H * (K - 1) * d * e
        if op == "conv_fwd":
            return dict(bytes=2 * n * e + state * (2 if case["state"] else 1) + 4 * H * d * (K + 1), flops=n * (2 * K + 5))
        if op == "conv_bwd":
            return dict(bytes=3 * n * e + state * (3 if case["state"] else 0) + 8 * H * d * (K + 1), flops=n * (6 * K + 8))
        return dict(bytes=2 * n * e + 2 * state + 4 * H * d * (K + 1), flops=n * (2 * K + 5))
    N, G = case["N"], case["G"]
    bc, st = B * G * T * N * e, 4 * S * H * d * N
    par = 4 * H * d * (N + 2)
    if op == "scan_fwd":
        return dict(bytes=n * e * (4 if case["gate"] else 3) + 2 * bc + st * (2 if case["state"] else 1) + par, flops=n * (8 * N + 10))
    if op == "scan_bwd":
        return dict(bytes=n * e * (7 if case["gate"] else 5) + 4 * bc + st * (3 if case["state"] else 0) + 2 * par, flops=n * (26 * N + 30))
    return dict(bytes=n * e * (4 if case["gate"] else 3) + 2 * bc + 2 * st + par, flops=n * (8 * N + 10))


# ---- the definitions in 64 bits --------------------------------------------------------------

def _sequences(s):
    """[(index of its state, batch row, first token, end)] of the sequences."""
    if "cu" in s:
        cu = s["cu"].tolist()
        return [(i, 0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]
    B, _, T, _ = s["x"].shape
    return [(b, b, 0, T) for b in range(B)]


def _norm_exact(s):
    c = s["case"]
    x = s["x"].double().requires_grad_()
    w = s["w"].double().requires_grad_()
    h = x + s["r"].double() if "r" in s and c["op"] == "norm_fwd" else x
    y = h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * (w.unsqueeze(-2) if c["per_head"] else w)
    if c["op"] == "norm_bwd":
        dx, dw = torch.autograd.grad(y, (x, w), s["dy"].double())
        return [dx + s["r"].double() if "r" in s else dx, dw]
    out = [y]
    if c["quant"]:
        scale = y.abs().amax(-1) / 448
        # the nearest of e4m3's values: 3 bits behind the leading one, 2^-9 the smallest step
        v = y / torch.where(scale > 0, scale, 1.0)[..., None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        out = [torch.round(v / step) * step, scale]
    return [t.detach() for t in out + ([h] if "r" in s else [])]


def _conv_exact(s):
    c = s["case"]
    K, x = c["K"], s["x"].double().requires_grad_()
    w, bias = s["w"].double().requires_grad_(), s["bias"].double().requires_grad_()
    S = len(_sequences(s)) if c["op"] != "conv_step" else s["state"].shape[0]
    B, H, T, d = x.shape
    state = (s["state"].double() if "state" in s else torch.zeros(S, H, K - 1, d, dtype=torch.float64, device="cuda")).requires_grad_()
    where = [(int(p), b, 0, 1) for b, p in enumerate(s["slots"].tolist()) if p >= 0] if c["op"] == "conv_step" else _sequences(s)
    y, end = torch.zeros_like(x), state.clone()
    y = y.detach().clone()
    for i, b, lo, hi in where:
        full = torch.cat([state[i], x[b, :, lo:hi]], 1)
        p = bias[:, None] + sum(w[:, None, :, j] * full[:, j:j + hi - lo] for j in range(K))
        y[b, :, lo:hi] = p * torch.sigmoid(p) if c["silu"] else p
        end[i] = full[:, full.shape[1] - (K - 1):]
    if c["op"] != "conv_bwd":
        return [y.detach(), end.detach()]
    live = torch.zeros_like(y)
    for _, b, lo, hi in where:
        live[b, :, lo:hi] = 1
    loss = (y * s["dy"].double() * live).sum()
    if "dstate" in s:
        loss = loss + (end * s["dstate"].double()).sum()
    got = torch.autograd.grad(loss, (x, w, bias, state), allow_unused=True, materialize_grads=True)
    return list(got[:3]) + ([got[3]] if "state" in s else [])


def _scan_exact(s):
    c = s["case"]
    x, A = s["x"].double(), s["A"].double()
    B, H, T, d = x.shape
    N, rep = c["N"], H // c["G"]
    Bm, Cm = (s[k].double().repeat_interleave(rep, 1) for k in ("Bm", "Cm"))
    raw = s["dt"].double() + s["dt_bias"].double()[:, None]
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    if c["op"] == "scan_step":
        where = [(int(p), b, 0, 1) for b, p in enumerate(s["slots"].tolist()) if p >= 0]
    else:
        where = _sequences(s)
    groups = [where] if "cu" not in s else [[q] for q in where]       # sequences of one length go together
    end = s["h0"].double().clone() if "h0" in s else torch.zeros(len(where), H, d, N, dtype=torch.float64, device="cuda")
    out = torch.zeros_like(x)
    back = c["op"] == "scan_bwd"
    if back:
        gate = torch.sigmoid(s["z"].double()) if "z" in s else None
        dout = s["dy"].double()
        dyy = dout * s["z"].double() * gate if "z" in s else dout
        dx, ddt, dz = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
        dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
        dA, dD, dh0 = torch.zeros_like(A), torch.zeros_like(s["D"].double()), torch.zeros_like(end)
    for part in groups:
        i = torch.tensor([q[0] for q in part], device="cuda")
        b = torch.tensor([q[1] for q in part], device="cuda")
        lo, hi = part[0][2], part[0][3]
        h, kept = end[i], []
        for t in range(lo, hi):
            h = torch.exp(dt[b, :, t, :, None] * A) * h + (dt[b, :, t] * x[b, :, t])[..., None] * Bm[b, :, t, None]
            out[b, :, t] = (h * Cm[b, :, t, None]).sum(-1) + s["D"].double() * x[b, :, t]
            if back:
                kept.append(h)
        if not back:
            end[i] = h
            continue
        G = s["dh"].double()[i] if "dh" in s else torch.zeros_like(h)
        for t in range(hi - 1, lo - 1, -1):
            dy, step, u = dyy[b, :, t], dt[b, :, t], x[b, :, t]
            G = G + dy[..., None] * Cm[b, :, t, None]
            dC[b, :, t] = (dy[..., None] * kept[t - lo]).sum(2)
            dB[b, :, t] = (G * (step * u)[..., None]).sum(2)
            inner = (G * Bm[b, :, t, None]).sum(-1)
            dx[b, :, t] = step * inner + s["D"].double() * dy
            a = torch.exp(step[..., None] * A)
            old = a * (kept[t - lo - 1] if t > lo else end[i])
            ddt[b, :, t] = (G * old * A).sum(-1) + u * inner
            dA += (G * old * step[..., None]).sum(0)
            dD += (dy * u).sum(0)
            G = a * G
        dh0[i] = G
    if not back:
        if "z" in s:
            out = out * s["z"].double() * torch.sigmoid(s["z"].double())
        return [out, end]
    ddt = ddt * torch.sigmoid(raw)
    dB, dC = (t.unflatten(1, (c["G"], rep)).sum(2) for t in (dB, dC))
    got = [dx, ddt, dA, dB, dC, dD]
    if "z" in s:
        got.append(dout * out * gate * (1 + s["z"].double() * (1 - gate)))
    live = torch.zeros_like(out)
    for _, b, lo, hi in where:
        live[b, :, lo:hi] = 1
    if "z" in s:
        got[-1] = got[-1] * live
    got.append(ddt.sum((0, 2)))
    return got + ([dh0] if "h0" in s else [])


def exact(case, seed):
    if case["op"].startswith("scan") and case.get("packed") and case["T"] > 20000:
        return None
    s = prepare(case, seed)
    return (_norm_exact if case["op"].startswith("norm") else _conv_exact if case["op"].startswith("conv") else _scan_exact)(s)
