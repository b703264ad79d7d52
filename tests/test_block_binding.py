"""The Python half of the recurrent block's calls, without a GPU: what reaches the native
binding, and what comes back from it."""
import contextlib
import inspect
import os
import subprocess
import sys

import pytest
import torch

from linear_attention_ttt_b200 import build as B
from linear_attention_ttt_b200 import ops

ROOT = os.path.dirname(B.PKG)


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def run(code):
    """A process of its own: one that ends takes no test with it."""
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)


WITHOUT_MEMORY = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from linear_attention_ttt_b200 import ops

def call(x):
    try:
        ops._block_call("rms_norm_fwd", (x[None, None], None, torch.empty(8, device="cuda"), x[None, None], None, None), 3, 1e-6)
    except RuntimeError as e:
        print("raised", e)
    return x

with FakeTensorMode():  # a CUDA tensor that needs no GPU
    torch.func.vmap(call)(torch.empty(3, 4, 8, device="cuda"))
print("alive")
"""


def test_a_tensor_without_memory_raises():
    """Inside torch.func's transforms a tensor has no address. The exception that torch throws
    for it would end the process if it passed through the interpreter."""
    r = run(WITHOUT_MEMORY)
    assert r.returncode == 0 and "raised" in r.stdout and "alive" in r.stdout, (r.returncode, r.stderr[-500:])


def test_tokens_of_ragged_sizes_raise():
    t = torch.nested.nested_tensor([torch.zeros(2, 3, 8), torch.zeros(1, 3, 8)])
    with pytest.raises(RuntimeError):
        ops._like_tokens(t, 8, torch.float32)


NEGATED = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from linear_attention_ttt_b200 import ops
with FakeTensorMode():
    x, w = torch.empty(1, 1, 4, 8, device="cuda"), torch.empty(8, device="cuda")
    n = torch.empty(1, 1, 4, 8, 1, dtype=torch.complex64, device="cuda").conj().imag[..., 0]
    assert n.is_neg()
    for t in ((n, None, w, x, None, None), (x, None, w, n, None, None)):
        try:
            ops._block_call("rms_norm_fwd", t, 3, 1e-6)
        except ValueError as e:
            print("refused", e)
"""


def test_a_negated_view_is_refused():
    """The imaginary part of a conjugate is a view of memory that holds its values with the
    other sign."""
    r = run(NEGATED)
    assert r.returncode == 0 and r.stdout.count("refused") == 2, (r.stdout, r.stderr[-500:])


# ---- arguments by name ----------------------------------------------------------------------

def arguments(T=4, B=2, H=2, d=8, N=4, K=4):
    """op -> its required arguments by name."""
    x, s = torch.zeros(B, H, T, d), torch.zeros(B, H, 1, d)
    bc, bc1 = torch.zeros(B, 1, T, N), torch.zeros(B, 1, 1, N)
    A, w = torch.zeros(H, d, N), torch.zeros(H, d, K)
    return dict(rms_norm_fwd=dict(x=x, weight=x[0, 0, 0]), rms_norm_bwd=dict(h=x, weight=x[0, 0, 0], dy=x),
                causal_conv_fwd=dict(x=x, weight=w), causal_conv_bwd=dict(x=x, weight=w, dy=x),
                causal_conv_step=dict(x=s, state=torch.zeros(B, H, K - 1, d), weight=w),
                selective_scan_fwd=dict(x=x, dt=x, A=A, Bm=bc, Cm=bc),
                selective_scan_bwd=dict(x=x, dt=x, A=A, Bm=bc, Cm=bc, dy=x),
                selective_scan_step=dict(x=s, dt=s, A=A, Bm=bc1, Cm=bc1, state=torch.zeros(B, H, d, N)))


@pytest.fixture
def reached(monkeypatch):
    """The calls that reach the library, in place of making them."""
    got = []
    monkeypatch.setattr(ops, "_block_call", lambda name, tensors, split, scalar: got.append((name, tensors)))
    return got


@pytest.mark.parametrize("name", arguments())
def test_arguments_may_be_named(name, reached):
    op, kw = getattr(ops, name), arguments()[name]
    required = [k for k, p in inspect.signature(op).parameters.items() if p.default is p.empty]
    assert required == list(kw)
    op(*kw.values())
    op(**kw)
    op(**dict(reversed(kw.items())))
    assert [r[0] for r in reached] == [name] * 3
    for _, tensors in reached[1:]:
        assert [t.data_ptr() for t in tensors if any(t is v for v in kw.values())] == \
               [t.data_ptr() for t in reached[0][1] if any(t is v for v in kw.values())]
    with pytest.raises(TypeError):
        op(**kw, no_such_argument=1)
    with pytest.raises(TypeError):
        op(**{("x" if k == "h" else "h" if k == "x" else k): v for k, v in kw.items()})


@pytest.mark.parametrize("name", arguments())
def test_a_stream_and_named_arguments(name, reached, monkeypatch):
    used = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: used.append(s) or contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: (handle, device))
    cpu = torch.device("cpu")
    for handle in (0, 7):
        getattr(ops, name)(**arguments()[name], stream=handle)
    assert used == [("default", cpu), (7, cpu)] and len(reached) == 2


@pytest.mark.parametrize("name", arguments())
def test_a_stream_of_another_device_is_refused(name, reached, monkeypatch):
    """The call would run on the tensors' device, on a stream that is not the one given."""
    class Stream:
        cuda_stream, device = 7, torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    with pytest.raises(ValueError, match="stream"):
        getattr(ops, name)(**arguments()[name], stream=Stream())
    assert not reached


@pytest.mark.parametrize("name", arguments())
def test_a_stream_and_no_tensor(name, reached):
    with pytest.raises(TypeError):
        getattr(ops, name)(stream=7)
    assert not reached


# ---- first calls ------------------------------------------------------------------------------

FIRST_CALLS = """
import threading, time, torch
import linear_attention_ttt_b200 as package
from linear_attention_ttt_b200 import _binding as real, ops

class Slow:  # a function of the native half that takes its time to say its name
    def __init__(self, f):
        self.f = f
    @property
    def __name__(self):
        time.sleep(0.05)
        return self.f.__name__
    def __call__(self, *args):
        return self.f(*args)

class Module:
    built_for = real.built_for
    call, like_tokens, zeros_like_tokens = Slow(real.call), Slow(real.like_tokens), Slow(real.zeros_like_tokens)

package._binding = Module
x, failed = torch.zeros(1, 1, 4, 8), []

def first(i):
    time.sleep(0.02 * i)
    try:
        ops._like_tokens(x)
    except Exception as e:
        failed.append(repr(e))

threads = [threading.Thread(target=first, args=(i,)) for i in range(10)]
[t.start() for t in threads], [t.join() for t in threads]
assert not failed, failed
"""


def test_first_calls_of_two_threads():
    r = run(FIRST_CALLS)
    assert r.returncode == 0, r.stderr[-500:]


# ---- what the native half is built against ------------------------------------------------------

def test_the_binding_is_built_again_for_another_torch(tmp_path, monkeypatch):
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_binding.so"))
    compiled = []

    def compile_it(cmd, **_):
        compiled.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(B.subprocess, "run", compile_it)
    B.build_binding()
    B.build_binding()
    assert len(compiled) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    B.build_binding()
    B.build_binding()
    assert len(compiled) == 2 and any("0.0.0" in c for c in compiled[1])
    os.remove(tmp_path / "_binding.so")
    B.build_binding()
    assert len(compiled) == 3
    B.build_binding(force=True)
    assert len(compiled) == 4
    monkeypatch.setattr(B.subprocess, "run", lambda cmd, **_: subprocess.CompletedProcess(cmd, 1, "", ""))
    with pytest.raises(RuntimeError):
        B.build_binding(force=True)
    monkeypatch.setattr(B.subprocess, "run", compile_it)
    B.build_binding()  # what a failed build left behind is not taken for whole
    assert len(compiled) == 5


def test_a_binding_built_for_another_torch_is_refused(monkeypatch):
    monkeypatch.setattr(ops, "_NATIVE", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(OSError, match="0.0.0"):
        ops._like_tokens(torch.zeros(1, 1, 4, 8))
