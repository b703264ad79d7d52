"""Packed sequences of the recurrent block's operators on the GPU: sequences that begin and end
next to the borders of the parts (32 tokens) and chunks (64 and more) that the scan works in,
and the packed calls repeated, on other streams, beside one another and in graphs.

Bounds are those of test_parity_block_gpu.py. Results of repeated calls are compared bit for
bit: the operators' sums have a fixed order.
"""
import pytest
import torch

from linear_attention_ttt_b200 import ops
from tests.test_parity_block_gpu import BF16, F32, clean, gen, run_scan, same, scan_args, scan_case

pytestmark = pytest.mark.gpu

# Tokens 300, H 3, d 203: the forward pass has five chunks of two parts. Sequences begin with the
# last tokens of a chunk's first part (28 .. 31 of 32), on both sides of borders, and the last one
# ends in a chunk that is not the last.
LATE = [[0, 31, 95, 159, 223, 290], [0, 28, 31, 95, 100], [0, 29, 94, 95, 158, 159, 160, 222, 224, 300],
        [0, 32, 64, 96, 128, 160, 192, 224, 256, 288, 300], [5, 31, 63, 127, 191, 192, 250]]


def packed(cu, dtype, N=16, H=3, d=203, T=300, far=True):
    """A scan whose sequences start from states that are far apart."""
    S = len(cu) - 1
    c = scan_case(gen(sum(cu) + N), 1, H, T, d, N, dtype, G=H, S=S)
    if far:
        c["h0"] += 10 * torch.arange(S, dtype=torch.float32).view(S, 1, 1, 1).cuda()
    for k in ("x", "dt", "Bm", "Cm", "z", "dy"):
        if c[k] is not None:
            c[k][:, :, cu[-1]:] = float("nan")
            c[k][:, :, :cu[0]] = float("nan")
    return c


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", LATE, ids=str)
def test_sequences_that_begin_late_in_a_part(cu, dtype):
    run_scan(packed(cu, dtype), cu)


@pytest.mark.parametrize("N", [16, 13, 24, 40])
@pytest.mark.parametrize("cu", LATE[:2], ids=str)
def test_packed_states_are_the_same_every_time(cu, N):
    """Each sequence's start state is its own however the warps of a block run."""
    c = packed(cu, F32, N=N)
    a, kw = scan_args(c)
    cud = torch.tensor(cu, dtype=torch.int32).cuda()
    first = ops.selective_scan_fwd(*a, h0=c["h0"], cu_seqlens=cud, **kw)
    for _ in range(200):
        assert same(first, ops.selective_scan_fwd(*a, h0=c["h0"], cu_seqlens=cud, **kw))
    clean()
