"""RMS norm on the GPU where a rounding decides: 8-bit values next to the middle between two."""
import numpy as np
import pytest
import torch

from linear_attention_ttt_b200 import ops
from tests.test_parity_block_gpu import BF16, F32, clean

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
