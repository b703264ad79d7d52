"""Host-side checks of the recurrent block's entry points (no GPU needed): arguments
are refused before any CUDA call. Descriptors carry fake, never dereferenced pointers."""
import ctypes

import pytest
import torch

from linear_attention_ttt_b200 import build as B
from linear_attention_ttt_b200 import ops
from tests.test_abi_host import ERR, FAKE, dense, tok

GAP = 1 << 28

# on a GPU a call that passes the checks would launch on the fake pointers
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: host checks are run without a GPU")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return ops.load()


def i32(n, base):
    return dense((n,), base, ops.TTT_I32)


class Call:
    """A valid call; tests break one field at a time. None passes NULL."""
    name, order, scalar_at, scalar = "", (), 0, 0

    def __init__(self):
        self.t = {}
        for i, (k, v) in enumerate(self.tensors().items()):
            if v is not None:
                v.data = FAKE + i * GAP
            self.t[k] = v

    def __call__(self, lib, scalar=None, **changes):
        t = dict(self.t)
        for k, v in changes.items():
            if callable(v):
                v(t[k])
            else:
                t[k] = v
        args = [ctypes.byref(t[k]) if t[k] is not None else None for k in self.order]
        args.insert(self.scalar_at, self.scalar if scalar is None else scalar)
        return getattr(lib, self.name)(*args, None)


class NormFwd(Call):
    name, scalar_at, scalar = "rms_norm_fwd", 3, 1e-6
    order = ("x", "residual", "weight", "out", "scale", "residual_out")

    def tensors(self):
        return dict(x=tok(2, 3, 5, 64), residual=tok(2, 3, 5, 64), weight=dense((64,), 0), out=tok(2, 3, 5, 64),
                    scale=None, residual_out=tok(2, 3, 5, 64))


class NormBwd(Call):
    name, scalar_at, scalar = "rms_norm_bwd", 4, 1e-6
    order = ("h", "weight", "dy", "dres", "dh", "dweight")

    def tensors(self):
        return dict(h=tok(2, 3, 5, 64), weight=dense((3, 64), 0), dy=tok(2, 3, 5, 64), dres=tok(2, 3, 5, 64),
                    dh=tok(2, 3, 5, 64), dweight=dense((3, 64), 0))


class ConvFwd(Call):
    name, scalar_at, scalar = "causal_conv_fwd", 5, 1
    order = ("x", "weight", "bias", "state0", "cu", "out", "state_final")

    def tensors(self):
        return dict(x=tok(1, 3, 50, 64), weight=dense((3, 64, 4), 0), bias=dense((3, 64), 0), state0=tok(4, 3, 3, 64),
                    cu=i32(5, 0), out=tok(1, 3, 50, 64), state_final=tok(4, 3, 3, 64))


class ConvBwd(Call):
    name, scalar_at, scalar = "causal_conv_bwd", 5, 1
    order = ("x", "weight", "bias", "state0", "cu", "dy", "dstate_final", "dx", "dweight", "dbias", "dstate0")

    def tensors(self):
        return dict(x=tok(1, 3, 50, 64), weight=dense((3, 64, 4), 0), bias=dense((3, 64), 0), state0=tok(4, 3, 3, 64),
                    cu=i32(5, 0), dy=tok(1, 3, 50, 64), dstate_final=tok(4, 3, 3, 64), dx=tok(1, 3, 50, 64),
                    dweight=dense((3, 64, 4), 0), dbias=dense((3, 64), 0), dstate0=tok(4, 3, 3, 64))


class ConvStep(Call):
    name, scalar_at, scalar = "causal_conv_step", 5, 1
    order = ("x", "state", "slots", "weight", "bias", "out")

    def tensors(self):
        return dict(x=tok(2, 3, 1, 64), state=tok(7, 3, 3, 64), slots=i32(2, 0), weight=dense((3, 64, 4), 0),
                    bias=dense((3, 64), 0), out=tok(2, 3, 1, 64))


class ScanFwd(Call):
    name, scalar_at, scalar = "selective_scan_fwd", 10, 1
    order = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0", "cu", "out", "h_final")

    def tensors(self):
        x = dict(x=tok(1, 4, 50, 64), dt=tok(1, 4, 50, 64), A=dense((4, 64, 16), 0), B=tok(1, 2, 50, 16),
                 C=tok(1, 2, 50, 16), D=dense((4, 64), 0), z=tok(1, 4, 50, 64), dt_bias=dense((4, 64), 0),
                 h0=dense((3, 4, 64, 16), 0), cu=i32(4, 0))
        return dict(x, out=tok(1, 4, 50, 64), h_final=dense((3, 4, 64, 16), 0))


class ScanBwd(ScanFwd):
    name = "selective_scan_bwd"
    order = ScanFwd.order[:10] + ("dy", "dh_final", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")

    def tensors(self):
        x = super().tensors()
        x.pop("out"), x.pop("h_final")
        return dict(x, dy=tok(1, 4, 50, 64), dh_final=dense((3, 4, 64, 16), 0), dx=tok(1, 4, 50, 64),
                    ddt=tok(1, 4, 50, 64), dA=dense((4, 64, 16), 0), dB=tok(1, 2, 50, 16), dC=tok(1, 2, 50, 16),
                    dD=dense((4, 64), 0), dz=tok(1, 4, 50, 64), ddt_bias=dense((4, 64), 0),
                    dh0=dense((3, 4, 64, 16), 0))


class ScanStep(Call):
    name, scalar_at, scalar = "selective_scan_step", 10, 1
    order = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state", "slots", "out")

    def tensors(self):
        return dict(x=tok(2, 4, 1, 64), dt=tok(2, 4, 1, 64), A=dense((4, 64, 16), 0), B=tok(2, 2, 1, 16),
                    C=tok(2, 2, 1, 16), D=dense((4, 64), 0), z=tok(2, 4, 1, 64), dt_bias=dense((4, 64), 0),
                    state=dense((9, 4, 64, 16), 0), slots=i32(2, 0), out=tok(2, 4, 1, 64))


CALLS = [NormFwd, NormBwd, ConvFwd, ConvBwd, ConvStep, ScanFwd, ScanBwd, ScanStep]
OPTIONAL = dict(rms_norm_fwd={"residual_out"}, rms_norm_bwd={"dres"}, causal_conv_fwd={"state0", "cu", "state_final"},
                causal_conv_bwd={"dstate_final", "dstate0"}, causal_conv_step={"bias"},
                selective_scan_fwd={"D", "z", "dt_bias", "h0", "h_final"}, selective_scan_bwd={"dh_final", "dh0"},
                selective_scan_step={"D", "z", "dt_bias"})


def put(**fields):
    def change(t):
        for k, v in fields.items():
            if k in ("shape", "stride"):
                for i, x in v.items():
                    getattr(t, k)[i] = x
            else:
                setattr(t, k, v)
    return change


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.name)
def test_valid_calls_pass_every_check(lib, call):
    """Without a GPU the first thing behind the checks fails: an allocation or a CUDA call."""
    assert call()(lib) in (ERR["TTT_ERR_CUDA"], ERR["TTT_ERR_ALLOC"])
    for k in OPTIONAL[call.name]:
        if not (k == "cu" or (k == "h0" and call is ScanBwd)):
            assert call()(lib, **{k: None}) in (ERR["TTT_ERR_CUDA"], ERR["TTT_ERR_ALLOC"]), k


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.name)
def test_every_tensor_is_checked(lib, call):
    for k, t in call().t.items():
        if t is None:
            continue
        last = t.ndim - 1
        assert call()(lib, **{k: put(ndim=t.ndim % 4 + 1)}) == ERR["TTT_ERR_SHAPE"] or k == "weight", k
        assert call()(lib, **{k: put(shape={last: t.shape[last] + 1})}) < 0, k
        assert call()(lib, **{k: put(dtype=ops.TTT_E4M3)}) in (ERR["TTT_ERR_DTYPE"], ERR["TTT_ERR_NULL"]), k
        assert call()(lib, **{k: put(data=FAKE + 60 * GAP + 1)}) == ERR["TTT_ERR_LAYOUT"], k
        assert call()(lib, **{k: put(data=0)}) == ERR["TTT_ERR_NULL"], k
        assert call()(lib, **{k: put(stride={last: 2})}) == ERR["TTT_ERR_LAYOUT"], k
        if k not in OPTIONAL[call.name] and k not in ("cu", "slots", "bias", "dbias", "residual", "D", "z", "dt_bias",
                                                      "h0", "state0"):
            assert call()(lib, **{k: None}) == ERR["TTT_ERR_NULL"], k


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.name)
def test_outputs_may_not_overlap(lib, call):
    c = call()
    outs = [k for k in c.order if k in ("out", "dx", "dh", "dz", "ddt", "residual_out")]
    for o in outs:
        for k, t in c.t.items():
            if t is not None and k != o:
                d = call()
                d.t[o].data = d.t[k].data
                assert d(lib) == ERR["TTT_ERR_ARG"], (o, k)


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.name)
def test_outputs_need_addresses_of_their_own(lib, call):
    """A stride of 0 broadcasts an input; an output would be written by several at once."""
    for o in ("out", "dx", "dh"):
        c = call()
        if o in c.t:
            assert c(lib, **{o: put(stride={1: 0})}) == ERR["TTT_ERR_LAYOUT"]


def test_broadcast_inputs_are_taken(lib):
    assert ConvFwd()(lib, x=put(stride={1: 0})) in (ERR["TTT_ERR_CUDA"], ERR["TTT_ERR_ALLOC"])


def test_scalars(lib):
    for eps in (float("nan"), float("inf"), -1.0):
        assert NormFwd()(lib, scalar=eps) == ERR["TTT_ERR_ARG"]
        assert NormBwd()(lib, scalar=eps) == ERR["TTT_ERR_ARG"]
    for call in CALLS[2:]:
        assert call()(lib, scalar=2) == ERR["TTT_ERR_ARG"]


def test_norm_output_kinds(lib):
    e4m3 = put(dtype=ops.TTT_E4M3)
    assert NormFwd()(lib, out=e4m3) == ERR["TTT_ERR_NULL"]                     # 8 bits need scales
    assert NormFwd()(lib, scale=dense((2, 3, 5), FAKE + 30 * GAP)) == ERR["TTT_ERR_ARG"]
    assert NormFwd()(lib, out=e4m3, scale=dense((2, 3, 6), FAKE + 30 * GAP)) == ERR["TTT_ERR_SHAPE"]
    assert NormFwd()(lib, residual=None) == ERR["TTT_ERR_ARG"]                 # a sum of one
    assert NormBwd()(lib, dweight=dense((64,), FAKE + 30 * GAP)) == ERR["TTT_ERR_SHAPE"]


def test_sizes_without_a_kernel(lib):
    t = lambda d: tok(2, 3, 5, d)
    c = NormFwd()
    for k in ("x", "residual", "out", "residual_out"):
        c.t[k] = t(16392)
    assert c(lib) == ERR["TTT_ERR_UNSUPPORTED"]
    assert ConvFwd()(lib, weight=dense((3, 64, 9), FAKE + GAP)) == ERR["TTT_ERR_UNSUPPORTED"]
    assert ScanFwd()(lib, A=dense((4, 64, 65), FAKE + 2 * GAP)) == ERR["TTT_ERR_UNSUPPORTED"]
    for call in CALLS:
        c = call()
        first = c.order[0]
        assert c(lib, **{first: put(shape={2: (1 << 30) + 1})}) == ERR["TTT_ERR_UNSUPPORTED"]
        c = call()
        assert c(lib, **{first: put(shape={0: 1 << 20, 1: 1 << 20})}) == ERR["TTT_ERR_UNSUPPORTED"]


def test_sequences_and_slots(lib):
    for call in (ConvFwd, ConvBwd, ScanFwd, ScanBwd):
        assert call()(lib, cu=i32(1, FAKE + 40 * GAP)) == ERR["TTT_ERR_SHAPE"]     # no sequence
        assert call()(lib, cu=i32(3, FAKE + 40 * GAP)) == ERR["TTT_ERR_SHAPE"]     # not the states' number
        assert call()(lib, cu=None) == ERR["TTT_ERR_SHAPE"]                        # B = 1, states of several
        assert call()(lib, cu=dense((4,), FAKE + 40 * GAP)) == ERR["TTT_ERR_DTYPE"]
    c = ConvFwd()
    c.t.update(x=tok(2, 3, 50, 64), out=tok(2, 3, 50, 64, base=FAKE + 41 * GAP))   # packed rows have no batch
    assert c(lib) == ERR["TTT_ERR_SHAPE"]
    for call in (ConvStep, ScanStep):
        assert call()(lib, slots=i32(3, FAKE + 40 * GAP)) == ERR["TTT_ERR_SHAPE"]
        assert call()(lib, slots=None) == ERR["TTT_ERR_SHAPE"]                     # 2 rows, a pool of more
    c = ScanStep()
    for k in ("x", "dt", "z", "out"):
        c.t[k] = tok(2, 4, 2, 64, base=c.t[k].data)
    for k in ("B", "C"):
        c.t[k] = tok(2, 2, 2, 16, base=c.t[k].data)
    assert c(lib) == ERR["TTT_ERR_SHAPE"]                                          # one token a row


def test_groups_divide_the_heads(lib):
    c = ScanFwd()
    c.t.update(B=tok(1, 3, 50, 16, base=c.t["B"].data), C=tok(1, 3, 50, 16, base=c.t["C"].data))
    assert c(lib) == ERR["TTT_ERR_SHAPE"]


def test_gradients_belong_to_inputs(lib):
    for k, g in (("D", "dD"), ("z", "dz"), ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        assert ScanBwd()(lib, **{k: None}) == ERR["TTT_ERR_ARG"], k
        if g != "dh0":
            assert ScanBwd()(lib, **{g: None}) == ERR["TTT_ERR_NULL"], g
    assert ConvBwd()(lib, bias=None) == ERR["TTT_ERR_ARG"]
    assert ConvBwd()(lib, dbias=None) == ERR["TTT_ERR_NULL"]
    assert ConvBwd()(lib, state0=None) == ERR["TTT_ERR_ARG"]


def test_wrappers_refuse_what_is_not_on_a_gpu():
    """A host pointer would fault in a kernel: it never reaches the library."""
    x = torch.zeros(1, 1, 4, 8)
    with pytest.raises(ValueError):
        ops.rms_norm_fwd(x, torch.ones(8))
    with pytest.raises(ValueError):
        ops.causal_conv_fwd(x, torch.ones(1, 8, 4))
    with pytest.raises(ValueError):
        ops.selective_scan_step(x[:, :, :1], x[:, :, :1], torch.ones(1, 8, 4), x[:, :, :1, :4], x[:, :, :1, :4],
                                torch.zeros(1, 1, 8, 4))


def test_new_token_tensors_have_aligned_rows():
    x = torch.zeros(2, 5, 3, 10, dtype=torch.bfloat16).permute(0, 2, 1, 3)
    y = ops._like_tokens(x)
    assert y.shape == x.shape and all(s * 2 % 16 == 0 for s in y.stride()[:3]) and y.stride(1) < y.stride(2)
    q = ops._like_tokens(x, dtype=torch.float8_e4m3fn)
    assert all(s % 16 == 0 for s in q.stride()[:3])


@pytest.mark.parametrize("heads,shared,ok", [(65535, False, True), (65536, False, False), (65536, True, True)])
def test_norm_backward_heads_of_a_weight(lib, heads, shared, ok):
    """A weight per head takes a row of blocks per head, of which a launch has 65535 at
    most; a shared weight has no such limit."""
    w = (8,) if shared else (heads, 8)
    new = dict(h=tok(1, heads, 1, 8), weight=dense(w, 0), dy=tok(1, heads, 1, 8), dres=tok(1, heads, 1, 8),
               dh=tok(1, heads, 1, 8), dweight=dense(w, 0))
    for i, t in enumerate(new.values()):
        t.data = FAKE + i * GAP
    st = NormBwd()(lib, **new)
    if ok:
        assert st in (ERR["TTT_ERR_CUDA"], ERR["TTT_ERR_ALLOC"])
    else:
        assert st == ERR["TTT_ERR_UNSUPPORTED"]
