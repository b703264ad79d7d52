"""GPU parity of the recurrent block's operators (RMS norm, causal convolution, selective
scan) with the fp64 oracle (oracle/block_oracle.py).

Bounds are elementwise and derived, not measured: |got - want| <= half |want| + steps * U * mag,
where half is half a step of the output type, mag the same sum over absolute values (the
oracle's mag=True), U = 2^-21 the error allowed to one fp32 operation (a rounding is 2^-24, the
fast exponential and division 2^-22 with their argument's rounding), and `steps` the
operations that a term of the sum passes through: the length of the chain of decays, each with
the rounding of its exponent D_t A relative to 1, the sums over states and channels, and the
activations.
"""
import numpy as np
import pytest
import torch

from linear_attention_ttt_b200 import ops
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -21


def half(dtype):
    return torch.finfo(dtype).eps / 2


def num(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def close(got, want, mag, steps, what=""):
    err = steps * U * mag + 1e-30
    bound = half(got.dtype) * (np.abs(want) + err) + err
    got = num(got)
    assert np.isfinite(got).all(), what
    off = np.abs(got - want) / bound
    assert off.size == 0 or off.max() <= 1, f"{what}: {off.max():.3g} of the bound at {np.unravel_index(off.argmax(), off.shape)}"


def clean():
    torch.cuda.synchronize()
    assert ops.device_status() == 0


def tokens(g, B, H, T, d, dtype, order="thd", scale=1.0):
    """[B,H,T,d] values in one of the storage orders, rows padded to 16 bytes, NaN in the padding."""
    pad = -(-d // 8) * 8
    shape = (B, T, H, pad) if order == "thd" else (B, H, T, pad)
    x = (torch.randn(shape, generator=g) * scale).to(dtype)
    x[..., d:] = float("nan")
    x = x.cuda()[..., :d]
    return x.transpose(1, 2) if order == "thd" else x


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- RMS norm --------------------------------------------------------------------------

WIDTHS = [1, 7, 8, 64, 100, 255, 520, 1024, 1032, 2048, 5000, 16384]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", WIDTHS)
def test_norm(d, dtype):
    g = gen(d)
    B, H, T = (2, 3, 5) if d < 4000 else (1, 2, 3)
    x, r = tokens(g, B, H, T, d, dtype), tokens(g, B, H, T, d, dtype, "htd")
    for per_head in (False, True):
        w = (1 + 0.1 * torch.randn((H, d) if per_head else (d,), generator=g)).cuda()
        wn = num(w)[:, None] if per_head else num(w)
        for res in (None, r):
            y, s, h = ops.rms_norm_fwd(x, w, 1e-5, residual=res)
            sn = num(x) if res is None else num(x) + num(res)
            want = O.rms_norm(sn, wn, 1e-5)
            assert s is None and (h is None) == (res is None)
            # the sum of squares of positive terms: d/2 roundings of 2^-24 at most, as a share of itself
            close(y, want, np.abs(want), 8 + d / 16, "y")
            if res is not None:
                close(h, sn, np.abs(num(x)) + np.abs(num(r)), 1, "sum")
            q, s, h2 = ops.rms_norm_fwd(x, w, 1e-5, residual=res, quant=True)
            top = np.abs(want).max(-1)
            close(s, top / 448, top / 448, 8 + d / 16, "scale")
            # half a step of e4m3 of the value (or half its smallest step), and the value's and scale's own errors
            scale = num(s)[..., None]
            off = np.abs(num(q) * scale - want)
            assert (off <= np.maximum(np.abs(want) * 2.0 ** -4, scale * 2.0 ** -10) + (8 + d / 16) * 3 * U * top[..., None]).all()
            assert h2 is None or torch.equal(h2, h)
    clean()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", WIDTHS)
def test_norm_backward(d, dtype):
    g = gen(d + 1)
    B, H, T = (3, 2, 7) if d < 4000 else (1, 2, 3)
    h, dy, dr = (tokens(g, B, H, T, d, dtype, o) for o in ("thd", "htd", "thd"))
    for per_head in (False, True):
        w = (1 + 0.1 * torch.randn((H, d) if per_head else (d,), generator=g)).cuda()
        wn = num(w)[:, None] if per_head else num(w)
        for res in (None, dr):
            dh, dw = ops.rms_norm_bwd(h, w, dy, 1e-5, dres=res)
            want, rows = O.rms_norm_bwd(num(h), wn, num(dy), 1e-5)
            hn, dn = np.abs(num(h)), np.abs(num(dy) * wn)
            r = 1 / np.sqrt((hn * hn).mean(-1, keepdims=True) + 1e-5)
            mag = r * (dn + hn * r * (dn * hn * r).mean(-1, keepdims=True))
            if res is not None:
                want, mag = want + num(res), mag + np.abs(num(res))
            close(dh, want, mag, 12 + d / 8, "dh")
            axes = (0, 2) if per_head else (0, 1, 2)
            close(dw, rows.sum(axes), np.abs(rows).sum(axes), 12 + d / 16 + B * H * T, "dw")
    clean()


def test_norm_of_many_rows():
    """More rows than the backward has workers: every worker takes several."""
    g = gen(5)
    for d, n in ((64, 60000), (1032, 3000)):
        h, dy = tokens(g, 1, 1, n, d, F32), tokens(g, 1, 1, n, d, F32)
        w = torch.ones(d).cuda()
        dh, dw = ops.rms_norm_bwd(h, w, dy, 1e-5)
        want, rows = O.rms_norm_bwd(num(h), num(w), num(dy), 1e-5)
        assert np.abs(num(dh) - want).max() < 1e-4
        close(dw, rows.sum((0, 1, 2)), np.abs(rows).sum((0, 1, 2)), 200, "dw")
    clean()


def test_norm_rows_that_have_nothing_and_rows_that_are_not_numbers():
    x = torch.randn(1, 1, 4, 64).cuda()
    x[0, 0, 1] = 0
    x[0, 0, 2, 5] = float("nan")
    w = torch.ones(64).cuda()
    for eps in (0.0, 1e-6):
        y, _, _ = ops.rms_norm_fwd(x, w, eps)
        assert (y[0, 0, 1] == 0).all() and torch.isnan(y[0, 0, 2]).all() and torch.isfinite(y[0, 0, [0, 3]]).all()
        q, s, _ = ops.rms_norm_fwd(x, w, eps, quant=True)
        assert s[0, 0, 1] == 0 and (q[0, 0, 1].float() == 0).all()
        assert torch.isnan(s[0, 0, 2]) and torch.isnan(q[0, 0, 2].float()).all() and torch.isfinite(q[0, 0, [0, 3]].float()).all()
    dh, dw = ops.rms_norm_bwd(x[:, :, :2], w, torch.ones_like(x[:, :, :2]), 0.0)
    assert torch.isfinite(dh).all() and (dh[0, 0, 1] == 0).all() and torch.isfinite(dw).all()
    clean()


def test_norm_is_the_l2_norm_that_the_layers_take():
    x = tokens(gen(9), 2, 4, 33, 64, F32)
    y, _, _ = ops.rms_norm_fwd(x, torch.full((64,), 0.125).cuda(), 0.0)
    assert (torch.linalg.vector_norm(y, dim=-1) - 1).abs().max() < 64 * U
    q = y.contiguous()
    out, _ = ops.ttt_linear_fwd(q, q, q, torch.full((2, 4, 33), 0.1).cuda(), torch.zeros(4, 64, 64).cuda(), 16, ops.TTT_LOSS_MSE)
    assert torch.isfinite(out).all()
    clean()


# ---- causal convolution -----------------------------------------------------------------

def conv_case(g, B, H, T, d, K, dtype, S=None, state=True, bias=True):
    S = S or B
    c = dict(x=tokens(g, B, H, T, d, dtype), w=(torch.randn(H, d, K, generator=g) / K ** 0.5).cuda(),
             dy=tokens(g, B, H, T, d, dtype, "htd"))
    c["bias"] = torch.randn(H, d, generator=g).cuda() if bias else None
    c["state"] = tokens(g, S, H, K - 1, d, dtype, "htd") if state else None
    c["dfin"] = tokens(g, S, H, K - 1, d, dtype, "htd") if state else None
    return c


def conv_oracle(c, act, cu=None, mag=False):
    B, H, T, d = c["x"].shape
    K = c["w"].shape[-1]
    x, dy = num(c["x"]), num(c["dy"])
    w = num(c["w"]).reshape(H * d, K)
    b = num(c["bias"]).reshape(-1) if c["bias"] is not None else np.zeros(H * d)
    seqs = O.sequences(B, T, cu)
    S = len(seqs)
    st = num(c["state"]) if c["state"] is not None else np.zeros((S, H, K - 1, d))
    df = num(c["dfin"]) if c["dfin"] is not None else np.zeros((S, H, K - 1, d))
    r = dict(y=np.zeros_like(x), mag=np.zeros_like(x), fin=np.zeros_like(st), dx=np.zeros_like(x), dw=np.zeros_like(w),
             db=np.zeros_like(b), ds=np.zeros_like(st), m={})
    r["m"] = {k: np.zeros_like(r[k]) for k in ("dx", "dw", "db", "ds")}
    for i, bb, lo, hi in seqs:
        xs, s0 = O.flat(x, bb, lo, hi), O.flat(st, i, 0, K - 1)
        y, fin = O.conv(xs, w, b, s0, act)
        p, _ = O.conv(np.abs(xs), np.abs(w), np.abs(b), np.abs(s0), False)
        r["y"][bb, :, lo:hi], r["fin"][i] = O.unflat(y, H), O.unflat(fin, H)
        r["mag"][bb, :, lo:hi] = O.unflat(p, H)          # |silu'| <= 1.1, |silu(p)| <= |p|
        for out, m in ((r, False), (r["m"], True)):
            dx, dw, db, ds = O.conv_bwd(xs, w, b, s0, act, O.flat(dy, bb, lo, hi), O.flat(df, i, 0, K - 1), m)
            if m and act:  # an error of p moves silu'(p) by at most half of it
                e = O.flat(np.abs(dy), bb, lo, hi) * p
                ex = O.conv_bwd(np.abs(xs), np.abs(w), b, np.abs(s0), False, e, np.zeros_like(s0))
                dx, dw, db, ds = dx + ex[0], dw + ex[1], db + ex[2], ds + ex[3]
            out["dx"][bb, :, lo:hi], out["ds"][i] = O.unflat(dx, H), O.unflat(ds, H)
            out["dw"] += dw
            out["db"] += db
    return r


def run_conv(c, act, cu=None):
    B, H, T, d = c["x"].shape
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    r = conv_oracle(c, act, cu)
    K = c["w"].shape[-1]
    y, fin = ops.causal_conv_fwd(c["x"], c["w"], c["bias"], act, state0=c["state"], cu_seqlens=cud)
    close(y, r["y"], r["mag"], K + 8, "y")
    assert np.array_equal(num(fin), r["fin"])
    dx, dw, db, ds = ops.causal_conv_bwd(c["x"], c["w"], c["dy"], c["bias"], act, state0=c["state"], dstate_final=c["dfin"],
                                         cu_seqlens=cud)
    close(dx, r["dx"], r["m"]["dx"], 2 * K + 16, "dx")
    close(dw, r["dw"].reshape(H, d, K), r["m"]["dw"].reshape(H, d, K), 2 * K + 16 + B * T / 4, "dw")
    if db is not None:
        close(db, r["db"].reshape(H, d), r["m"]["db"].reshape(H, d), 2 * K + 16 + B * T / 4, "db")
    if ds is not None:
        close(ds, r["ds"], r["m"]["ds"], 2 * K + 16, "dstate")
    clean()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K", range(1, 9))
def test_conv_taps(K, dtype):
    run_conv(conv_case(gen(K), 2, 2, 21, 12, K, dtype), True)


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d,H", [(1, 8, 1), (2, 1, 3), (7, 30, 1), (8, 64, 2), (9, 5, 2), (130, 33, 3), (257, 200, 1)])
def test_conv_sizes(T, d, H, dtype, act):
    g = gen(T + d)
    run_conv(conv_case(g, 2, H, T, d, 4, dtype), act)
    run_conv(conv_case(g, 1, H, T, d, 3, dtype, state=False, bias=False), act)


CUTS = [[0, 5], [0, 0, 1, 3, 3, 40, 41], [0, 16, 32, 64], [0, 0, 0], [2, 9, 30], [0, 1, 2, 3, 4, 5, 6, 7, 8, 60]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", CUTS, ids=str)
def test_conv_packed(cu, dtype):
    """Ragged sequences, empty ones, and rows before the first and behind the last that hold NaN."""
    g = gen(len(cu))
    T = 64
    c = conv_case(g, 1, 2, T, 20, 4, dtype, S=len(cu) - 1)
    for k in ("x", "dy"):
        c[k][:, :, cu[-1]:] = float("nan")
        c[k][:, :, :cu[0]] = float("nan")
    run_conv(c, True, cu)
    out = torch.full_like(c["x"].contiguous()[..., :16], 7.0)
    x = c["x"].contiguous()[..., :16].contiguous()
    ops.causal_conv_fwd(x, c["w"][:, :16].contiguous(), None, True, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), out=out)
    assert (out[:, :, cu[-1]:] == 7).all() and (out[:, :, :cu[0]] == 7).all()
    clean()


def test_conv_of_no_tokens_keeps_the_state():
    c = conv_case(gen(3), 2, 1, 4, 16, 4, BF16)
    x = c["x"][:, :, :0]
    y, fin = ops.causal_conv_fwd(x, c["w"], c["bias"], True, state0=c["state"])
    assert y.numel() == 0 and torch.equal(fin, c["state"])
    _, fin = ops.causal_conv_fwd(x, c["w"], c["bias"], True)
    assert (fin == 0).all()
    dx, dw, db, ds = ops.causal_conv_bwd(x, c["w"], x, c["bias"], True, state0=c["state"], dstate_final=c["dfin"])
    assert (dw == 0).all() and (db == 0).all() and torch.equal(ds, c["dfin"])
    clean()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K,d", [(1, 8), (4, 33), (4, 256), (8, 40)])
def test_conv_steps_are_the_prompt(K, d, dtype):
    """Tokens one by one through a pool of states, against the same tokens as a prompt: bit for bit."""
    B, H, T, S = 5, 2, 9, 8
    g = gen(K + d)
    c = conv_case(g, B, H, T, d, K, dtype)
    want, fin = ops.causal_conv_fwd(c["x"], c["w"], c["bias"], True, state0=c["state"])
    pool = ops._conv_state(c["x"], S, K).fill_(3.0)
    slots = torch.tensor([6, 0, 3, 7, 1], dtype=torch.int32).cuda()
    pool[slots.long()] = c["state"]
    for t in range(T):
        y = ops.causal_conv_step(c["x"][:, :, t:t + 1], pool, c["w"], c["bias"], True, slots=slots)
        assert torch.equal(y[:, :, 0], want[:, :, t])
    assert torch.equal(pool[slots.long()], fin) and (pool[[2, 4, 5]] == 3).all()
    clean()


# ---- selective scan -----------------------------------------------------------------------

def scan_case(g, B, H, T, d, N, dtype, G=1, S=None, state=True, gate=True, D=True, bias=True, softplus=True):
    S = S or B
    c = dict(x=tokens(g, B, H, T, d, dtype), dt=tokens(g, B, H, T, d, dtype, scale=0.5), Bm=tokens(g, B, G, T, N, dtype),
             Cm=tokens(g, B, G, T, N, dtype, "htd"), dy=tokens(g, B, H, T, d, dtype, "htd"), softplus=softplus)
    if not softplus:
        c["dt"].abs_().mul_(0.3)
    c["A"] = (-torch.rand(H, d, N, generator=g) * N - 0.1).cuda()
    c["z"] = tokens(g, B, H, T, d, dtype, "htd", scale=2.0) if gate else None
    c["D"] = torch.randn(H, d, generator=g).cuda() if D else None
    c["dt_bias"] = (torch.rand(H, d, generator=g) * 4 - 5).cuda() if bias else None
    c["h0"] = torch.randn(S, H, d, N, generator=g).cuda() if state else None
    c["dh"] = torch.randn(S, H, d, N, generator=g).cuda() if state else None
    return c


def scan_args(c):
    return (c["x"], c["dt"], c["A"], c["Bm"], c["Cm"]), dict(D=c["D"], z=c["z"], dt_bias=c["dt_bias"], softplus=c["softplus"])


def scan_oracle(c, cu=None, back=True):
    B, H, T, d = c["x"].shape
    N, G = c["A"].shape[-1], c["Bm"].shape[1]
    A = num(c["A"]).reshape(H * d, N)
    D = num(c["D"]).reshape(-1) if c["D"] is not None else np.zeros(H * d)
    raw = num(c["dt"]) + (num(c["dt_bias"])[None, :, None] if c["dt_bias"] is not None else 0)
    dt = O.softplus(raw) if c["softplus"] else raw
    slope = O.sigmoid(raw) if c["softplus"] else np.ones_like(raw)
    x, dy, Bm, Cm = (num(c[k]) for k in ("x", "dy", "Bm", "Cm"))
    z = num(c["z"]) if c["z"] is not None else None
    seqs = O.sequences(B, T, cu)
    h0 = num(c["h0"]) if c["h0"] is not None else np.zeros((len(seqs), H, d, N))
    dh = num(c["dh"]) if c["dh"] is not None else np.zeros((len(seqs), H, d, N))

    def new():
        return dict(out=np.zeros_like(x), fin=h0.copy() if True else None, dx=np.zeros_like(x), ddt=np.zeros_like(x), dz=np.zeros_like(x),
                    dB=np.zeros_like(Bm), dC=np.zeros_like(Cm), dA=np.zeros_like(A), dD=np.zeros(H * d), dbias=np.zeros(H * d),
                    dh0=dh.copy())
    r, m = new(), new()
    most = 0.0
    for i, b, lo, hi in seqs:
        if hi <= lo:
            continue
        f = lambda v: O.flat(v, b, lo, hi)
        a = (f(x), f(dt), A, O.spread(Bm, b, lo, hi, H, d), O.spread(Cm, b, lo, hi, H, d), D, f(z) if z is not None else None,
             h0[i].reshape(H * d, N))
        most = max(most, np.abs(a[1][:, :, None] * A).max())
        for o, mag in ((r, False), (m, True)):
            y, fin, _ = O.scan(*a, mag=mag)
            o["out"][b, :, lo:hi], o["fin"][i] = O.unflat(y, H), fin.reshape(H, d, N)
            if not back:
                continue
            q = O.scan_bwd(*a, f(dy), dh[i].reshape(H * d, N), mag=mag)
            dd = q["ddt"] * f(slope)
            o["dx"][b, :, lo:hi], o["ddt"][b, :, lo:hi] = O.unflat(q["dx"], H), O.unflat(dd, H)
            if z is not None:
                o["dz"][b, :, lo:hi] = O.unflat(q["dz"], H)
            o["dB"][b, :, lo:hi], o["dC"][b, :, lo:hi] = O.gather(q["dB"], H, G, d), O.gather(q["dC"], H, G, d)
            o["dA"] += q["dA"]
            o["dD"] += q["dD"]
            o["dbias"] += dd.sum(0)
            o["dh0"][i] = q["dh0"].reshape(H, d, N)
    longest = max(hi - lo for _, _, lo, hi in seqs)
    return r, m, longest * (1 + most) + N + 32


def run_scan(c, cu=None, back=True):
    B, H, T, d = c["x"].shape
    N = c["A"].shape[-1]
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    r, m, steps = scan_oracle(c, cu, back)
    a, kw = scan_args(c)
    out, fin = ops.selective_scan_fwd(*a, h0=c["h0"], cu_seqlens=cud, **kw)
    close(out, r["out"], m["out"], steps, "out")
    close(fin, r["fin"], np.abs(m["fin"]), steps, "h_final")
    if back:
        got = ops.selective_scan_bwd(*a, c["dy"], h0=c["h0"], dh_final=c["dh"], cu_seqlens=cud, **kw)
        names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")
        for name, t in zip(names, got):
            if t is None:
                continue
            want, mag = r[name].reshape(t.shape), np.abs(m[name]).reshape(t.shape)
            # forward and backward chains; sums over tokens and channels
            n = 2 * steps + {"dA": B * T / 4, "dD": B * T / 4, "dbias": B * T / 4, "dB": H * d / 4, "dC": H * d / 4}.get(name, 0)
            close(t, want, mag, n, name)
    clean()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [1, 4, 13, 16, 17, 33, 64])
def test_scan_states(N, dtype):
    g = gen(N)
    run_scan(scan_case(g, 2, 2, 70, 9, N, dtype, G=2))
    run_scan(scan_case(g, 1, 3, 37, 40, N, dtype, G=1, gate=False, D=False, bias=False, state=False))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d,H", [(1, 1, 1), (2, 33, 1), (15, 32, 2), (16, 31, 1), (17, 64, 1), (31, 8, 3), (32, 16, 1),
                                   (33, 65, 1), (64, 130, 1), (65, 20, 2), (129, 24, 1), (300, 48, 1)])
def test_scan_sizes(T, d, H, dtype):
    run_scan(scan_case(gen(T + d), 2, H, T, d, 16, dtype))


@pytest.mark.parametrize("gate,D,bias,state,softplus", [(True, False, True, False, True), (False, True, False, True, True),
                                                        (True, True, True, True, False), (False, False, False, False, False)])
def test_scan_optional_inputs(gate, D, bias, state, softplus):
    for dtype in (BF16, F32):
        run_scan(scan_case(gen(3), 1, 2, 75, 20, 12, dtype, G=2, gate=gate, D=D, bias=bias and softplus, state=state, softplus=softplus))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", CUTS + [[0, 100, 130, 130, 280, 297], [0, 300], [0, 64, 128, 256], [3, 290]], ids=str)
def test_scan_packed(cu, dtype):
    g = gen(sum(cu))
    T = 64 if cu[-1] <= 64 else 300
    c = scan_case(g, 1, 2, T, 20, 16, dtype, G=2, S=len(cu) - 1)
    for k in ("x", "dt", "Bm", "Cm", "z", "dy"):
        c[k][:, :, cu[-1]:] = float("nan")
        c[k][:, :, :cu[0]] = float("nan")
    run_scan(c, cu)
    a, kw = scan_args(c)
    out = torch.full((1, 2, T, 24), 7.0, dtype=dtype, device="cuda")[..., :20]
    ops.selective_scan_fwd(*a, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), out=out, **kw)
    assert (out[:, :, cu[-1]:] == 7).all() and (out[:, :, :cu[0]] == 7).all()
    clean()


def test_scan_of_no_tokens_keeps_the_state():
    c = scan_case(gen(3), 2, 1, 4, 16, 8, BF16)
    a = [c[k][:, :, :0] if k != "A" else c[k] for k in ("x", "dt", "A", "Bm", "Cm")]
    y, h = ops.selective_scan_fwd(*a, h0=c["h0"])
    assert y.numel() == 0 and torch.equal(h, c["h0"])
    got = ops.selective_scan_bwd(*a, a[0], D=c["D"], dt_bias=c["dt_bias"], h0=c["h0"], dh_final=c["dh"])
    assert (got[2] == 0).all() and (got[5] == 0).all() and (got[7] == 0).all() and torch.equal(got[8], c["dh"])
    clean()


def test_scan_long_memory():
    """Step sizes of 1e-3 over 3000 tokens: the first input still counts at the end."""
    g = gen(11)
    c = scan_case(g, 1, 1, 3000, 33, 5, F32, bias=False)
    c["dt"].fill_(-6.9)
    c["A"] = -(0.5 + torch.rand(1, 33, 5, generator=g)).cuda()
    run_scan(c, back=False)


def test_scan_steep_and_growing_decays():
    """Decays that underflow to zero, and A > 0 (a state that grows)."""
    g = gen(12)
    c = scan_case(g, 1, 1, 40, 32, 16, F32)
    c["A"][:, :, ::3] = -5000.0
    c["A"][:, :, 1::3] = 0.5
    run_scan(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,d,G", [(16, 96, 1), (5, 33, 2), (64, 10, 2), (1, 70, 1), (24, 40, 1)])
def test_scan_steps_are_the_prompt(N, d, G, dtype):
    B, H, T, S = 5, 2, 7, 9
    c = scan_case(gen(N + d), B, H, T, d, N, dtype, G=G)
    r, m, steps = scan_oracle(c, back=False)
    pool = torch.full((S, H, d, N), 3.0).cuda()
    slots = torch.tensor([6, 0, 3, 7, 1], dtype=torch.int32).cuda()
    pool[slots.long()] = c["h0"]
    one = lambda v, t: None if v is None else v[:, :, t:t + 1]
    for t in range(T):
        y = ops.selective_scan_step(one(c["x"], t), one(c["dt"], t), c["A"], one(c["Bm"], t), one(c["Cm"], t), pool, D=c["D"],
                                    z=one(c["z"], t), dt_bias=c["dt_bias"], slots=slots)
        close(y, r["out"][:, :, t:t + 1], m["out"][:, :, t:t + 1], steps, f"token {t}")
    close(pool[slots.long()], r["fin"], np.abs(m["fin"]), steps, "state")
    assert (pool[[2, 4, 5, 8]] == 3).all()
    clean()


# ---- slots and offsets that are wrong, padded, repeated -------------------------------------

def step_calls(g, B, S, H=2, d=40, N=16, K=4):
    c = scan_case(g, B, H, 1, d, N, BF16)
    cc = conv_case(g, B, H, 1, d, K, BF16)
    pool = torch.randn(S, H, d, N, generator=g).cuda()
    cpool = tokens(g, S, H, K - 1, d, BF16, "htd")
    a, kw = scan_args(c)

    def scan(rows, pool, slots, out):
        return ops.selective_scan_step(a[0][rows], a[1][rows], a[2], a[3][rows], a[4][rows], pool, D=kw["D"], z=kw["z"][rows],
                                       dt_bias=kw["dt_bias"], slots=slots, out=out)

    def conv(rows, pool, slots, out):
        return ops.causal_conv_step(cc["x"][rows], pool, cc["w"], cc["bias"], True, slots=slots, out=out)
    return (scan, pool), (conv, cpool)


def test_padded_rows_and_places_out_of_range():
    B, S = 6, 4
    for call, pool in step_calls(gen(1), B, S):
        slots = torch.tensor([2, -1, 0, 4, -7, 2 ** 31 - 1], dtype=torch.int32).cuda()
        p = pool.clone()
        out = torch.full((B, 2, 1, 40), 5.0, dtype=BF16).cuda()
        call(slice(0, B), p, slots, out)
        assert ops.device_status() == ops.ERR_CODES["TTT_ERR_BOUNDS"] and ops.device_status() == 0
        q = pool.clone()
        want = call(torch.tensor([0, 2]).cuda(), q, slots[[0, 2]], None)
        assert torch.equal(out[[0, 2]], want) and (out[[1, 3, 4, 5]] == 5).all() and torch.equal(p, q)
        slots = torch.full((B,), -1, dtype=torch.int32).cuda()
        call(slice(0, B), p, slots, out)
        assert torch.equal(p, q)
    clean()


def test_rows_of_one_place_are_consecutive_tokens():
    B, S = 7, 3
    for call, pool in step_calls(gen(2), B, S):
        slots = torch.tensor([1, 0, 1, 1, -1, 0, 2], dtype=torch.int32).cuda()
        p, q = pool.clone(), pool.clone()
        out = call(slice(0, B), p, slots, None)
        for i in (0, 1, 2, 3, 5, 6):
            assert torch.equal(out[i:i + 1], call(slice(i, i + 1), q, slots[i:i + 1], None))
        assert torch.equal(p, q)
    clean()


def test_offsets_out_of_order_or_range():
    """Reported by every call, and nothing outside the tensors is touched."""
    g = gen(4)
    for cu in ([0, 20, 10, 40], [-5, 10, 30], [0, 10, 300], [0, 2 ** 31 - 1, -2 ** 31, 64]):
        c, cc = scan_case(g, 1, 1, 64, 16, 8, F32, S=len(cu) - 1), conv_case(g, 1, 1, 64, 16, 4, F32, S=len(cu) - 1)
        cud = torch.tensor(cu, dtype=torch.int32).cuda()
        a, kw = scan_args(c)
        for call in (lambda: ops.selective_scan_fwd(*a, cu_seqlens=cud, want_final=False, **kw),
                     lambda: ops.causal_conv_fwd(cc["x"], cc["w"], cc["bias"], True, cu_seqlens=cud, want_final=False),
                     lambda: ops.selective_scan_bwd(*a, c["dy"], cu_seqlens=cud, **kw),
                     lambda: ops.causal_conv_bwd(cc["x"], cc["w"], cc["dy"], cc["bias"], True, cu_seqlens=cud)):
            call()
            assert ops.device_status() == ops.ERR_CODES["TTT_ERR_BOUNDS"] and ops.device_status() == 0
    clean()


def test_rows_that_start_anywhere():
    """Tensors whose rows are not 16-byte aligned give the same values, element by element."""
    g = gen(41)
    for dtype in (BF16, F32):
        def moved(t):
            """The same values, contiguous, one element behind an aligned address."""
            if t is None:
                return None
            flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            return flat[1:].view(t.shape).copy_(t)
        c, cc = scan_case(g, 2, 2, 45, 17, 12, dtype, G=2), conv_case(g, 2, 2, 45, 17, 4, dtype)
        a, kw = scan_args(c)
        mkw = {k: moved(v) if torch.is_tensor(v) else v for k, v in kw.items()}
        want = ops.selective_scan_fwd(*a, h0=c["h0"], **kw)
        out = moved(want[0]).zero_()
        got = ops.selective_scan_fwd(*map(moved, a), h0=moved(c["h0"]), out=out, **mkw)
        assert same(got, want)
        want = ops.selective_scan_bwd(*a, c["dy"], h0=c["h0"], dh_final=c["dh"], **kw)
        got = ops.selective_scan_bwd(*map(moved, a), moved(c["dy"]), h0=moved(c["h0"]), dh_final=moved(c["dh"]), **mkw)
        assert same(got, want)
        m = {k: moved(v) for k, v in cc.items()}
        want = ops.causal_conv_fwd(cc["x"], cc["w"], cc["bias"], state0=cc["state"])
        assert same(ops.causal_conv_fwd(m["x"], m["w"], m["bias"], state0=m["state"], out=moved(want[0]).zero_()), want)
        want = ops.causal_conv_bwd(cc["x"], cc["w"], cc["dy"], cc["bias"], state0=cc["state"], dstate_final=cc["dfin"])
        assert same(ops.causal_conv_bwd(m["x"], m["w"], m["dy"], m["bias"], state0=m["state"], dstate_final=m["dfin"]), want)
        x, r, w = cc["x"], cc["dy"], torch.randn(17, generator=g).cuda()
        for quant in (False, True):
            want = ops.rms_norm_fwd(x, w, residual=r, quant=quant)
            got = ops.rms_norm_fwd(moved(x), moved(w), residual=moved(r), quant=quant, out=moved(want[0].float()).to(want[0].dtype),
                                   residual_out=moved(want[2]).zero_())
            assert all(torch.equal(p.float(), q.float()) for p, q in zip(got, want) if p is not None)
        assert same(ops.rms_norm_bwd(moved(x), moved(w), moved(r)), ops.rms_norm_bwd(x, w, r))
        one = lambda v: v[:, :, :1]
        pool, cpool = c["h0"].clone(), cc["state"].clone()
        mpool, mcpool = moved(pool), moved(cpool)
        want = ops.selective_scan_step(*(v if v.dim() == 3 else one(v) for v in a), pool, D=kw["D"], dt_bias=kw["dt_bias"])
        got = ops.selective_scan_step(*(moved(v if v.dim() == 3 else one(v)) for v in a), mpool, D=mkw["D"], dt_bias=mkw["dt_bias"],
                                      out=moved(want).zero_())
        assert torch.equal(got, want) and torch.equal(pool, mpool)
        want = ops.causal_conv_step(one(cc["x"]), cpool, cc["w"], cc["bias"])
        got = ops.causal_conv_step(moved(one(cc["x"])), mcpool, m["w"], m["bias"], out=moved(want).zero_())
        assert torch.equal(got, want) and torch.equal(cpool, mcpool)
    clean()


# ---- as they are used -------------------------------------------------------------------------

class Block:
    """norm(+residual) -> projection -> convolution -> scan -> projection, in fp32."""

    def __init__(self, g, D=48, N=8, K=4):
        r = lambda *s: torch.randn(*s, generator=g).cuda()
        self.D, self.N, self.K = D, N, K
        self.norm = 1 + 0.1 * r(D)
        self.w_in, self.w_out = r(D, 2 * D) / D ** 0.5, r(D, D) / D ** 0.5
        self.w_x = r(D, D + 2 * N) / D ** 0.5
        self.conv, self.bias = r(1, D, K) / 2, 0.1 * r(1, D)
        self.A, self.skip = -torch.rand(1, D, N, generator=g).cuda() * 4 - 0.1, 1 + 0.1 * r(1, D)
        self.dt_bias = torch.rand(1, D, generator=g).cuda() * 3 - 4

    def inner(self, u):
        """dt, B, C from the convolved tokens."""
        p = u @ self.w_x
        return p[..., :self.D], p[..., self.D:self.D + self.N], p[..., self.D + self.N:]

    def prompt(self, x, res, state=None, h=None, cu=None):
        y, _, res = ops.rms_norm_fwd(x, self.norm, 1e-5, residual=res)
        xz = y @ self.w_in
        u, state = ops.causal_conv_fwd(xz[..., :self.D], self.conv, self.bias, True, state0=state, cu_seqlens=cu)
        dt, B, C = self.inner(u)
        s, h = ops.selective_scan_fwd(u, dt, self.A, B, C, D=self.skip, z=xz[..., self.D:], dt_bias=self.dt_bias, h0=h, cu_seqlens=cu)
        return s @ self.w_out, res, state, h

    def token(self, x, res, state, h, slots):
        y, _, res = ops.rms_norm_fwd(x, self.norm, 1e-5, residual=res)
        xz = y @ self.w_in
        u = ops.causal_conv_step(xz[..., :self.D], state, self.conv, self.bias, True, slots=slots)
        dt, B, C = self.inner(u)
        s = ops.selective_scan_step(u, dt, self.A, B, C, h, D=self.skip, z=xz[..., self.D:], dt_bias=self.dt_bias, slots=slots)
        return s @ self.w_out, res

    def plain(self, x, res):
        """The whole block in torch (fp64, differentiable), one sequence [T, D]."""
        f = {k: v.double() for k, v in vars(self).items() if torch.is_tensor(v)}
        x = x + res
        y = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * f["norm"]
        xz = y @ f["w_in"]
        u = torch.cat([torch.zeros(self.K - 1, self.D, dtype=torch.float64, device="cuda"), xz[:, :self.D]])
        u = torch.nn.functional.silu(f["bias"][0] + sum(u[j:j + len(x)] * f["conv"][0, :, j] for j in range(self.K)))
        p = u @ f["w_x"]
        dt, B, C = torch.nn.functional.softplus(p[:, :self.D] + f["dt_bias"][0]), p[:, self.D:self.D + self.N], p[:, self.D + self.N:]
        h, out = 0, []
        for t in range(len(x)):
            h = torch.exp(dt[t, :, None] * f["A"][0]) * h + (dt[t] * u[t])[:, None] * B[t]
            out.append((h * C[t]).sum(-1) + f["skip"][0] * u[t])
        return torch.stack(out) * torch.nn.functional.silu(xz[:, self.D:]) @ f["w_out"], x


def test_block_prompts_then_tokens():
    """Three prompts packed, then decoded in a pool of states, against each sequence as one prompt
    in 64 bits. fp32 matmuls in between: 1e-4 of the outputs' size is ten times the bound of a
    chain of some 60 operations and sums of 48 products."""
    b = Block(gen(21))
    lens, more = [37, 1, 70], 5
    xs = [torch.randn(n + more, b.D, generator=gen(n)).cuda() for n in lens]
    rs = [torch.randn(n + more, b.D, generator=gen(n + 1)).cuda() for n in lens]
    cu = torch.tensor([0, 37, 38, 108], dtype=torch.int32).cuda()
    pack = lambda v: torch.cat([t[:n] for t, n in zip(v, lens)])[None, None]
    y, res, state, h = b.prompt(pack(xs), pack(rs), cu=cu)
    slots = torch.tensor([4, 2, 0, -1], dtype=torch.int32).cuda()
    cpool, hpool = torch.zeros(5, 1, b.K - 1, b.D).cuda(), torch.zeros(5, 1, b.D, b.N).cuda()
    cpool[[4, 2, 0]], hpool[[4, 2, 0]] = state, h
    got = [list(y[0, 0].split(lens))[i] for i in range(3)]
    for t in range(more):
        rows = lambda v: torch.stack([v[i][lens[i] + t] for i in range(3)] + [v[0][0]])[:, None, None]
        o, _ = b.token(rows(xs), rows(rs), cpool, hpool, slots)
        got = [torch.cat([got[i], o[i, 0]]) for i in range(3)]
    for i in range(3):
        want, _ = b.plain(xs[i].double(), rs[i].double())
        assert (got[i] - want).abs().max() <= 1e-4 * want.abs().max()
    assert torch.equal(res[0, 0], (pack(xs) + pack(rs))[0, 0])
    clean()


def test_block_gradients():
    """The chain of backward calls against autograd through the whole block in 64 bits, and
    against a difference of the block's own 64-bit form."""
    b = Block(gen(22))
    T = 45
    x, r = torch.randn(T, b.D, generator=gen(1)).cuda(), torch.randn(T, b.D, generator=gen(2)).cuda()
    dy, dres = torch.randn(T, b.D, generator=gen(3)).cuda(), torch.randn(T, b.D, generator=gen(4)).cuda()
    v = lambda t: t[None, None].contiguous()
    y, _, s = ops.rms_norm_fwd(v(x), b.norm, 1e-5, residual=v(r))
    xz = y @ b.w_in
    xi, z = xz[..., :b.D], xz[..., b.D:]
    u, _ = ops.causal_conv_fwd(xi, b.conv, b.bias, True)
    dt, B, C = b.inner(u)
    ds = v(dy) @ b.w_out.T
    du, ddt, dA, dB, dC, dD, dz, dbias, _ = ops.selective_scan_bwd(u, dt, b.A, B, C, ds, D=b.skip, z=z, dt_bias=b.dt_bias)
    du = du + torch.cat([ddt, dB, dC], -1) @ b.w_x.T
    dxi, dconv, dcb, _ = ops.causal_conv_bwd(xi, b.conv, du, b.bias, True)
    dh, dn = ops.rms_norm_bwd(s, b.norm, torch.cat([dxi, dz], -1) @ b.w_in.T, 1e-5, dres=v(dres))
    clean()
    leaves = dict(x=x.double().requires_grad_())
    for k in ("norm", "conv", "bias", "A", "skip", "dt_bias"):
        leaves[k] = getattr(b, k).double().requires_grad_()
    p = Block(gen(22))
    for k, t in leaves.items():
        if k != "x":
            setattr(p, k, t)

    def loss(xx):
        out, res = p.plain(xx, r.double())
        return (out * dy.double()).sum() + (res * dres.double()).sum()
    want = torch.autograd.grad(loss(leaves["x"]), list(leaves.values()))
    for (k, w), got in zip(zip(leaves, want), (dh[0, 0], dn, dconv, dcb, dA, dD, dbias)):
        assert (got.double() - w).abs().max() <= 2e-4 * w.abs().max(), k
    d = torch.randn(T, b.D, generator=gen(6)).double().cuda()
    with torch.no_grad():
        quotient = (loss(x.double() + 1e-6 * d) - loss(x.double() - 1e-6 * d)) / 2e-6
    assert abs(quotient - (dh[0, 0].double() * d).sum()) <= 1e-3 * (dh[0, 0].double() * d).abs().sum()


# ---- streams, graphs, repetition, size ----------------------------------------------------------

def every_call(g):
    """name -> function of no arguments, each on inputs of its own."""
    n = dict(x=tokens(g, 2, 1, 40, 256, BF16), r=tokens(g, 2, 1, 40, 256, BF16), dy=tokens(g, 2, 1, 40, 256, BF16))
    w = torch.ones(256).cuda()
    c, s = conv_case(g, 2, 1, 200, 96, 4, BF16), scan_case(g, 2, 1, 200, 96, 16, BF16)
    a, kw = scan_args(s)
    st = step_calls(g, 4, 6)
    slots = torch.tensor([3, 1, -1, 0], dtype=torch.int32).cuda()
    flat = lambda v: [t for t in v if t is not None]
    calls = dict(
        norm=lambda: flat(ops.rms_norm_fwd(n["x"], w, residual=n["r"], quant=True)),
        norm_bwd=lambda: flat(ops.rms_norm_bwd(n["x"], w, n["dy"], dres=n["r"])),
        conv=lambda: flat(ops.causal_conv_fwd(c["x"], c["w"], c["bias"], state0=c["state"])),
        conv_bwd=lambda: flat(ops.causal_conv_bwd(c["x"], c["w"], c["dy"], c["bias"], state0=c["state"], dstate_final=c["dfin"])),
        scan=lambda: flat(ops.selective_scan_fwd(*a, h0=s["h0"], **kw)),
        scan_bwd=lambda: flat(ops.selective_scan_bwd(*a, s["dy"], h0=s["h0"], dh_final=s["dh"], **kw)))
    for name, (call, pool) in zip(("scan_step", "conv_step"), st):
        calls[name] = lambda call=call, pool=pool: (lambda p: [call(slice(0, 4), p, slots, None), p])(pool.clone())
    inputs = [n["x"], c["x"], s["x"], s["dt"]]
    return calls, inputs


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x.float(), y.float()) for x, y in zip(a, b))


def test_results_do_not_depend_on_the_run():
    calls, _ = every_call(gen(31))
    for name, f in calls.items():
        first = f()
        for _ in range(3):
            assert same(first, f()), name
    clean()


def test_another_stream():
    calls, _ = every_call(gen(32))
    for name, f in calls.items():
        want = f()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [f() for _ in range(2)]
        s.synchronize()
        assert same(got[0], want) and same(got[1], want), name
    clean()


def test_stream_argument():
    """stream= takes a torch stream or a handle; the outputs made by the call are that stream's."""
    x, w = tokens(gen(36), 2, 1, 40, 256, BF16), torch.ones(256).cuda()
    want, _, _ = ops.rms_norm_fwd(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0):
        got, _, _ = ops.rms_norm_fwd(x, w, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    clean()


FIRST_IN_A_GRAPH = """
import torch
from linear_attention_ttt_b200 import ops
x = torch.randn(2, 1, 100, 96, device="cuda")
A, B = -torch.rand(1, 96, 16, device="cuda"), torch.randn(2, 1, 100, 16, device="cuda")
w = torch.randn(1, 96, 4, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y, _, _ = ops.rms_norm_fwd(x, A[0, :, 0].contiguous())
    u, _ = ops.causal_conv_fwd(y, w)
    got = [y, u, *ops.selective_scan_fwd(u, x, A, B, B), *ops.selective_scan_bwd(u, x, A, B, B, x)[:5],
           *ops.causal_conv_bwd(y, w, x)[:2], *ops.rms_norm_bwd(x, A[0, :, 0].contiguous(), x)]
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
y, _, _ = ops.rms_norm_fwd(x, A[0, :, 0].contiguous())
u, _ = ops.causal_conv_fwd(y, w)
want = [y, u, *ops.selective_scan_fwd(u, x, A, B, B), *ops.selective_scan_bwd(u, x, A, B, B, x)[:5],
        *ops.causal_conv_bwd(y, w, x)[:2], *ops.rms_norm_bwd(x, A[0, :, 0].contiguous(), x)]
assert all(torch.equal(p, q) for p, q in zip(got, want)) and ops.device_status() == 0
print("same")
"""


def test_first_calls_of_a_process_inside_a_graph():
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_GRAPH], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_norm_of_no_tokens():
    x, w = torch.zeros(2, 3, 0, 64, device="cuda"), torch.ones(64).cuda()
    y, s, _ = ops.rms_norm_fwd(x, w, quant=True)
    assert y.shape == x.shape and s.shape == (2, 3, 0)
    dh, dw = ops.rms_norm_bwd(x, w, x)
    assert dh.numel() == 0 and (dw == 0).all()
    clean()


def test_two_streams_at_once():
    """Workspaces of calls in flight beside one another are their own."""
    calls, _ = every_call(gen(33))
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for name, f in calls.items():
            for s in streams:
                with torch.cuda.stream(s):
                    got.append((name, f()))
    torch.cuda.synchronize()
    assert all(same(v, want[k]) for k, v in got)
    clean()


def test_captured_and_replayed():
    """Every call in a graph: replayed after its inputs changed, and two graphs in turn."""
    calls, inputs = every_call(gen(34))
    for name, f in calls.items():
        f()
        torch.cuda.synchronize()
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(f())
            graphs.append(g)
        for k in range(3):
            for x in inputs:
                x.mul_(0.9)
            for g in graphs:
                g.replay()
            want = f()
            torch.cuda.synchronize()
            assert same(outs[0], want) and same(outs[1], want), name
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert same(outs[0], want) and same(outs[1], want), name
        del graphs, outs
    clean()


def test_failed_allocations_are_reported():
    calls, _ = every_call(gen(35))
    for name in ("norm_bwd", "conv_bwd", "scan", "scan_bwd"):
        want = calls[name]()
        ops.load().ttt_test_fail_allocations(1)
        try:
            with pytest.raises(ops.TTTError) as e:
                calls[name]()
        finally:
            ops.load().ttt_test_fail_allocations(0)
        assert e.value.code == ops.ERR_CODES["TTT_ERR_ALLOC"]
        assert same(calls[name](), want)
    clean()


def test_offsets_past_32_bits():
    """A token tensor and a pool of states of more than 2^31 elements: their last rows."""
    d, T = 1024, (1 << 21) + 40
    x = torch.empty(1, 1, T, d, dtype=BF16, device="cuda")
    x[:, :, -300:] = torch.randn(300, d, generator=gen(1)).to(BF16).cuda()
    x[:, :, :-300] = 0
    tail = x[:, :, -300:].clone()
    w, b = torch.randn(1, d, 4, generator=gen(2)).cuda(), torch.zeros(1, d).cuda()
    y, _ = ops.causal_conv_fwd(x, w, b)
    want, _ = ops.causal_conv_fwd(tail, w, b)
    assert torch.equal(y[:, :, -300:], want)
    del y, want
    y, _, _ = ops.rms_norm_fwd(x, torch.ones(d).cuda())
    want, _, _ = ops.rms_norm_fwd(tail, torch.ones(d).cuda())
    assert torch.equal(y[:, :, -300:], want)
    del x, y, want, tail
    S = (1 << 31) // (d * 16) + 3
    pool = torch.zeros(S, 1, d, 16, device="cuda")
    c = scan_case(gen(3), 2, 1, 1, d, 16, BF16)
    a, kw = scan_args(c)
    small = torch.randn(2, 1, d, 16, generator=gen(4)).cuda()
    pool[-2:] = small
    slots = torch.tensor([S - 1, S - 2], dtype=torch.int32).cuda()
    got = ops.selective_scan_step(*a, pool, slots=slots, **kw)
    flip = small.flip(0).contiguous()
    want = ops.selective_scan_step(*a, flip, **kw)
    assert torch.equal(got, want) and torch.equal(pool[-2:], flip.flip(0)) and (pool[:-2].amax() == 0)
    clean()
