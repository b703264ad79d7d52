"""Packed sequences of the recurrent block's operators on the GPU: sequences that begin and end
next to the borders of the parts (32 tokens) and chunks (64 and more) that the scan works in,
and the packed calls repeated, on other streams, beside one another and in graphs.

Bounds are those of test_parity_block_gpu.py. Results of repeated calls are compared bit for
bit: the operators' sums have a fixed order.
"""
import subprocess
import sys

import pytest
import torch

from linear_attention_ttt_b200 import ops
from tests.test_parity_block_gpu import (BF16, F32, clean, conv_case, gen, run_scan, same, scan_args, scan_case,
                                         step_calls)

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


# ---- streams, graphs, repetition ------------------------------------------------------------------

CUTS = [[0, 31, 95, 95, 223, 290], [3, 64, 100, 170, 171, 300], [0, 0, 300, 300, 300, 300], [10, 10, 40, 47, 48, 48]]


def packed_calls(cud, dtype=BF16):
    """name -> function of no arguments: the packed calls, with states, on the offsets that cud
    holds; and tensors that they read."""
    g = gen(41)
    c, s = conv_case(g, 1, 3, 300, 203, 4, dtype, S=5), scan_case(g, 1, 3, 300, 203, 16, dtype, G=3, S=5)
    a, kw = scan_args(s)
    flat = lambda v: [t for t in v if t is not None]
    calls = dict(
        conv=lambda: flat(ops.causal_conv_fwd(c["x"], c["w"], c["bias"], state0=c["state"], cu_seqlens=cud)),
        conv_bwd=lambda: flat(ops.causal_conv_bwd(c["x"], c["w"], c["dy"], c["bias"], state0=c["state"],
                                                  dstate_final=c["dfin"], cu_seqlens=cud)),
        scan=lambda: flat(ops.selective_scan_fwd(*a, h0=s["h0"], cu_seqlens=cud, **kw)),
        scan_bwd=lambda: flat(ops.selective_scan_bwd(*a, s["dy"], h0=s["h0"], dh_final=s["dh"], cu_seqlens=cud, **kw)))
    return calls, [c["x"], s["x"], s["dt"], s["h0"]]


def offsets(cu):
    return torch.tensor(cu, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", CUTS, ids=str)
def test_packed_calls_do_not_depend_on_the_run(cu, dtype):
    for name, f in packed_calls(offsets(cu), dtype)[0].items():
        first = f()
        for _ in range(20):
            assert same(first, f()), name
    clean()


def test_packed_calls_on_two_streams_at_once():
    calls, _ = packed_calls(offsets(CUTS[0]))
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(6):
        for name, f in calls.items():
            for s in streams:
                with torch.cuda.stream(s):
                    got.append((name, f()))
    torch.cuda.synchronize()
    assert all(same(v, want[k]) for k, v in got)
    clean()


def test_packed_calls_captured_and_replayed():
    """Two graphs of every call, replayed after the inputs and the offsets changed in place."""
    cud = offsets(CUTS[0])
    calls, inputs = packed_calls(cud)
    for name, f in calls.items():
        f()
        torch.cuda.synchronize()
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(f())
            graphs.append(g)
        for cu in CUTS[1:] + CUTS[:1]:
            cud.copy_(offsets(cu))
            for x in inputs:
                x.mul_(0.9)
            for g in graphs:
                g.replay()
            want = f()
            torch.cuda.synchronize()
            assert same(outs[0], want) and same(outs[1], want), (name, cu)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert same(outs[0], want) and same(outs[1], want), name
        del graphs, outs
    clean()


FIRST_STEPS_IN_A_GRAPH = """
import torch
from linear_attention_ttt_b200 import ops
x = torch.randn(2, 1, 1, 96, device="cuda")
A, B = -torch.rand(1, 96, 16, device="cuda"), torch.randn(2, 1, 1, 16, device="cuda")
w, b = torch.randn(1, 96, 4, device="cuda"), torch.randn(1, 96, device="cuda")
conv, scan = torch.randn(5, 1, 3, 96, device="cuda"), torch.randn(5, 1, 96, 16, device="cuda")
slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
def token(conv, scan):
    u = ops.causal_conv_step(x, conv, w, b, slots=slots)
    return [u, ops.selective_scan_step(u, x, A, B, B, scan, z=x, slots=slots), conv, scan]
c1, s1, c2, s2 = conv.clone(), scan.clone(), conv.clone(), scan.clone()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = token(c1, s1)
for _ in range(3):
    g.replay()
    want = token(c2, s2)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
assert ops.device_status() == 0
print("same")
"""


def test_first_steps_of_a_process_inside_a_graph():
    r = subprocess.run([sys.executable, "-c", FIRST_STEPS_IN_A_GRAPH], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_steps_beside_one_another():
    """Steps on pools of their own, two streams at once, with rows of one place among them."""
    slots = torch.tensor([3, 1, 3, -1], dtype=torch.int32).cuda()
    for call, pool in step_calls(gen(42), 4, 6):
        p = pool.clone()
        want = [call(slice(0, 4), p, slots, None), p]
        torch.cuda.synchronize()
        streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
        for _ in range(6):
            for s in streams:
                with torch.cuda.stream(s):
                    q = pool.clone()
                    got.append([call(slice(0, 4), q, slots, None), q])
        torch.cuda.synchronize()
        assert all(same(v, want) for v in got)
    clean()
