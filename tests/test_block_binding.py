"""The Python half of the recurrent block's calls, without a GPU: what reaches the native
binding, and what comes back from it."""
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
