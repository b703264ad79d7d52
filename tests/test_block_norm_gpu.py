"""RMS norm on the GPU where a rounding decides (8-bit values next to the middle between two) and
where squares leave fp32's range."""
import numpy as np
import pytest
import torch

from linear_attention_ttt_b200 import ops
from oracle import block_oracle as O
from tests.test_parity_block_gpu import BF16, F32, clean, close, gen, num, tokens

pytestmark = pytest.mark.gpu


def to_e4m3(v):
    """Saturating, as the 8-bit output is: a scale among fp32's smallest numbers is rounded by up
    to half of itself, so that the largest quotient leaves 448 (5120 steps / 448 = 11.43 gives a
    scale of 11 and a quotient of 465.5, which torch's conversion alone makes NaN)."""
    return torch.from_numpy(v).clamp(-448, 448).to(torch.float8_e4m3fn)


def quotients_next_to_middles(heads, seed):
    """[heads, d] fp32 rows whose first element is the largest and whose others are, divided by
    the row's scale, within two fp32 steps of the middle between two 8-bit values."""
    values = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    middles = (values[:-1] + values[1:]) / 2
    rng = np.random.default_rng(seed)
    rows = []
    for _ in range(heads):
        top = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-40, 40))
        scale = np.float32(top / np.float32(448))
        at = (middles * np.float64(scale)).astype(np.float32).view(np.int32)
        w = np.concatenate([(at + k).view(np.float32) for k in range(-2, 3)])
        w = np.where(rng.random(len(w)) < 0.5, -w, w)
        rows.append(np.concatenate([[top], w[np.abs(w) < top]])[:600])
    assert all(len(r) == 600 for r in rows)
    return np.stack(rows).astype(np.float32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [600, 2048, 5000])
def test_8_bit_values_are_the_rounded_quotients(d, dtype):
    """A row of +-1 has the mean square 1, so that the norm's fp32 value is the weight itself."""
    H = 40
    w = np.zeros((H, d), np.float32)
    w[:, :600] = quotients_next_to_middles(H, d)
    scale = (np.abs(w).max(-1) / np.float32(448)).astype(np.float32)[:, None]
    want = to_e4m3(w / scale).float()
    by_reciprocal = to_e4m3(w * (np.float32(1) / scale)).float()
    assert (want != by_reciprocal).sum() > 100        # the rows tell the two apart
    sign = torch.where(torch.rand(1, H, 3, d, generator=torch.Generator().manual_seed(d)) < 0.5, -1.0, 1.0)
    x, wd = sign.to(dtype).cuda(), torch.from_numpy(w).cuda()
    if dtype == F32:
        y, _, _ = ops.rms_norm_fwd(x, wd, 0.0)
        assert torch.equal(y.cpu(), sign * torch.from_numpy(w)[None, :, None])
    q, s, _ = ops.rms_norm_fwd(x, wd, 0.0, quant=True)
    assert torch.equal(s.cpu(), torch.from_numpy(scale[:, 0])[None, :, None].expand(1, H, 3))
    assert torch.equal(q.float().cpu(), sign * want[None, :, None])
    clean()


def test_8_bit_values_of_small_and_infinite_rows():
    """Scales down to fp32's smallest, and one that is infinite: the division itself."""
    w = np.zeros((40, 64), np.float32)
    w[:, 0] = np.ldexp(np.float32(1.25), np.arange(-143, -143 + 80, 2)).astype(np.float32)
    w[:, 1:] = w[:, :1] * np.linspace(-1, 1, 63, dtype=np.float32)
    w[39, 0] = np.inf
    with np.errstate(all="ignore"):
        scale = (np.abs(w).max(-1) / np.float32(448)).astype(np.float32)[:, None]
        want = to_e4m3(np.where(scale > 0, w / np.where(scale > 0, scale, 1), w).astype(np.float32)).float()
    x = torch.ones(1, 40, 1, 64).cuda()
    q, s, _ = ops.rms_norm_fwd(x, torch.from_numpy(w).cuda(), 0.0, quant=True)
    assert torch.equal(s.cpu()[0, :, 0], torch.from_numpy(scale[:, 0]))
    got = q.float().cpu()[0, :, 0]
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(1), want.nan_to_num(1))
    clean()


# ---- rows whose squares fp32 does not hold ------------------------------------------------------

SIZES = [-140, -126, -100, -75, -64, -55, -45, -20, 0, 50, 58, 62, 64, 90, 120]  # powers of two


def sized_rows(g, d, dtype):
    """A token of every size, beside one another: rows of both kinds share a warp."""
    x = tokens(g, 2, 2, len(SIZES), d, dtype)
    return x.mul_(torch.tensor([2.0 ** e for e in SIZES]).cuda().to(dtype)[:, None])


@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-28, 1e-6, 1e30])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [7, 64, 256, 1024, 2048, 2056, 9000])
def test_rows_of_every_size(d, dtype, eps):
    """x / rms(x) does not depend on x's size, as long as x is representable. The bounds are
    those of rows of an ordinary size: a power of two in front changes no rounding."""
    g = gen(d)
    x = sized_rows(g, d, dtype)
    w = (1 + 0.1 * torch.randn(2, d, generator=g)).cuda()
    want = O.rms_norm(num(x), num(w)[:, None], eps)
    y, _, _ = ops.rms_norm_fwd(x, w, eps)
    close(y, want, np.abs(want), 8 + d / 16, "y")
    q, s, _ = ops.rms_norm_fwd(x, w, eps, quant=True)
    top = np.abs(want).max(-1)
    close(s, top / 448, top / 448, 8 + d / 16, "scale")
    # the largest row's size bounds e4m3's own errors, the scale's and the value's
    off = np.abs(num(q) * num(s)[..., None] - want) / np.maximum(top, 1e-30)[..., None]
    assert (off <= 2.0 ** -4 + (8 + d / 16) * 3 * 2.0 ** -21 + 1e-9).all()
    clean()


@pytest.mark.parametrize("eps", [0.0, 1e-28, 1e-6])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [7, 64, 256, 1024, 2056, 9000])
def test_gradients_of_rows_of_every_size(d, dtype, eps):
    g = gen(d + 1)
    h = sized_rows(g, d, dtype)[:, :, 1:]  # not the denormal ones
    dy = tokens(g, 2, 2, len(SIZES) - 1, d, dtype, "htd")
    dy.mul_(torch.tensor([2.0 ** (e / 2) for e in SIZES[1:]]).cuda().to(dtype)[:, None])
    for w in ((1 + 0.1 * torch.randn(2, d, generator=g)).cuda(), (1 + 0.1 * torch.randn(d, generator=g)).cuda()):
        wn = num(w)[:, None] if w.dim() == 2 else num(w)
        dh, dw = ops.rms_norm_bwd(h, w, dy, eps)
        want, rows = O.rms_norm_bwd(num(h), wn, num(dy), eps)
        hn, dn = np.abs(num(h)), np.abs(num(dy) * wn)
        r = 1 / np.sqrt((hn * hn).mean(-1, keepdims=True) + eps)
        mag = r * (dn + hn * r * (dn * hn * r).mean(-1, keepdims=True))
        close(dh, want, mag, 12 + d / 8, "dh")
        axes = (0, 2) if w.dim() == 2 else (0, 1, 2)
        close(dw, rows.sum(axes), np.abs(rows).sum(axes), 12 + d / 16 + 4 * len(SIZES), "dw")
    clean()


def test_infinite_and_empty_rows_among_sized_ones():
    x = sized_rows(gen(1), 64, F32)
    x[0, 0, 3] = 0
    x[0, 1, 4, 7] = float("inf")
    x[1, 0, 5, 9] = float("nan")
    y, _, _ = ops.rms_norm_fwd(x, torch.ones(64).cuda(), 0.0)
    assert (y[0, 0, 3] == 0).all()
    assert torch.isnan(y[0, 1, 4, 7]) and (y[0, 1, 4, :7] == 0).all()      # a finite value over an infinite one
    assert torch.isnan(y[1, 0, 5]).all()
    x[0, 1, 4], x[1, 0, 5] = 0, 0
    rest, _, _ = ops.rms_norm_fwd(x, torch.ones(64).cuda(), 0.0)
    keep = torch.ones(2, 2, len(SIZES), dtype=torch.bool).cuda()
    keep[0, 1, 4] = keep[1, 0, 5] = False
    assert torch.equal(y[keep], rest[keep])
    clean()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [2, 9, 63, 1023, 2049, 4099, 8195, 16383])
def test_aligned_rows_of_any_length(d, dtype):
    """Rows that 4 does not divide move 16 bytes at a time but for their last elements: NaN lies
    behind every row, in the inputs and in what an output's row has behind its end."""
    g = gen(d)
    B, H, T = 1, 2, 5
    x, r, dy = (tokens(g, B, H, T, d, dtype, o) for o in ("thd", "htd", "thd"))
    w = (1 + 0.1 * torch.randn(H, d, generator=g)).cuda()
    wn, sn = num(w)[:, None], num(x) + num(r)
    want = O.rms_norm(sn, wn, 1e-5)
    pad = -(-d // 16) * 16
    for quant in (False, True):
        out = torch.full((B, H, T, pad), 3.0, device="cuda").to(torch.float8_e4m3fn if quant else dtype)
        got, s, h = ops.rms_norm_fwd(x, w, 1e-5, residual=r, quant=quant, out=out[..., :d])
        assert (out[..., d:].float() == 3).all()
        close(h, sn, np.abs(num(x)) + np.abs(num(r)), 1, "sum")
        if not quant:
            close(got, want, np.abs(want), 8 + d / 16, "y")
        else:
            top, scale = np.abs(want).max(-1)[..., None], num(s)[..., None]
            off = np.abs(num(got) * scale - want)
            assert (off <= np.maximum(np.abs(want) * 2.0 ** -4, scale * 2.0 ** -10) + (8 + d / 16) * 3 * 2.0 ** -21 * top).all()
    dh, dw = ops.rms_norm_bwd(x, w, dy, 1e-5)
    want, rows = O.rms_norm_bwd(num(x), wn, num(dy), 1e-5)
    hn, dn = np.abs(num(x)), np.abs(num(dy) * wn)
    rs = 1 / np.sqrt((hn * hn).mean(-1, keepdims=True) + 1e-5)
    close(dh, want, rs * (dn + hn * rs * (dn * hn * rs).mean(-1, keepdims=True)), 12 + d / 8, "dh")
    close(dw, rows.sum((0, 2)), np.abs(rows).sum((0, 2)), 12 + d / 16 + B * T, "dw")
    clean()
