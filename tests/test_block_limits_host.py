"""Sizes that the recurrent block's entry points refuse, from both sides (no GPU needed;
descriptors carry fake, never dereferenced pointers)."""
import pytest
import torch

from linear_attention_ttt_b200 import build as B
from linear_attention_ttt_b200 import ops
from tests.test_abi_host import ERR, dense, tok
from tests.test_block_host import CALLS, FAKE, GAP, ConvFwd, ConvStep, ScanFwd, ScanStep, i32

# on a GPU a call that passes the checks would launch on the fake pointers
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: host checks are run without a GPU")

PASSED = (ERR["TTT_ERR_CUDA"], ERR["TTT_ERR_ALLOC"])  # without a GPU the first thing behind the checks fails


@pytest.fixture(scope="module")
def lib():
    B.build()
    return ops.load()


def status(lib, call, gap=GAP, **tensors):
    c = call()
    c.t.update(tensors)
    for i, t in enumerate(c.t.values()):
        if t is not None:
            t.data = FAKE + i * gap
    return c(lib)


@pytest.mark.parametrize("rows,ok", [(65535, True), (65536, False)])
def test_rows_of_a_single_token_call(lib, rows, ok):
    for call, new in ((ConvStep, dict(x=tok(rows, 1, 1, 8), state=tok(7, 1, 3, 8), slots=i32(rows, 0),
                                      weight=dense((1, 8, 4), 0), bias=dense((1, 8), 0), out=tok(rows, 1, 1, 8))),
                      (ScanStep, dict(x=tok(rows, 1, 1, 8), dt=tok(rows, 1, 1, 8), z=tok(rows, 1, 1, 8),
                                      A=dense((1, 8, 4), 0), B=tok(rows, 1, 1, 4), C=tok(rows, 1, 1, 4),
                                      D=dense((1, 8), 0), dt_bias=dense((1, 8), 0), state=dense((7, 1, 8, 4), 0),
                                      slots=i32(rows, 0), out=tok(rows, 1, 1, 8)))):
        st = status(lib, call, **new)
        assert st in PASSED if ok else st == ERR["TTT_ERR_UNSUPPORTED"], call.name


@pytest.mark.parametrize("slots,ok", [(1 << 24, True), ((1 << 24) + 1, False)])
def test_states_of_a_pool(lib, slots, ok):
    """S*H: heads 1."""
    st = status(lib, ConvStep, gap=1 << 34, x=tok(2, 1, 1, 8), state=tok(slots, 1, 3, 8), slots=i32(2, 0),
                weight=dense((1, 8, 4), 0), bias=dense((1, 8), 0), out=tok(2, 1, 1, 8))
    assert st in PASSED if ok else st == ERR["TTT_ERR_UNSUPPORTED"]


@pytest.mark.parametrize("sequences,ok", [(1 << 24, True), ((1 << 24) + 1, False)])
def test_sequences_of_a_packed_call(lib, sequences, ok):
    st = status(lib, ConvFwd, gap=1 << 34, x=tok(1, 1, 50, 8), out=tok(1, 1, 50, 8), weight=dense((1, 8, 4), 0),
                bias=dense((1, 8), 0), state0=None, state_final=None, cu=i32(sequences + 1, 0))
    assert st in PASSED if ok else st == ERR["TTT_ERR_UNSUPPORTED"]


@pytest.mark.parametrize("heads,width,ok", [(1, 1 << 20, True), (1, (1 << 20) + 1, False), (512, 1 << 20, True),
                                            (513, 1 << 20, False)])
def test_widths(lib, heads, width, ok):
    """d, and the channel tiles H*ceil(d/32)."""
    st = status(lib, ScanFwd, gap=1 << 40, x=tok(1, heads, 2, width), dt=tok(1, heads, 2, width), z=tok(1, heads, 2, width),
                out=tok(1, heads, 2, width), A=dense((heads, width, 4), 0), B=tok(1, 1, 2, 4), C=tok(1, 1, 2, 4),
                D=dense((heads, width), 0), dt_bias=dense((heads, width), 0), h0=None, h_final=None, cu=None)
    assert st in PASSED if ok else st == ERR["TTT_ERR_UNSUPPORTED"]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.name)
def test_no_rows_are_refused(lib, call):
    c = call()
    first = c.order[0]
    c.t[first].shape[0] = 0
    assert c(lib) == ERR["TTT_ERR_SHAPE"]
