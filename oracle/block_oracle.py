"""fp64 oracle of the recurrent block's operators: RMS norm, short causal
convolution, selective scan, each forward and backward, one sequence at a time.

Test infrastructure only. Channels are flattened ([T, C] tokens); `sequences`
and the functions behind it run the packed and padded-batch [B,H,T,d] layouts
of include/ttt.h over it. Everything is written from the definitions: token by
token, no chunks. With `mag=True` the same sums run over absolute values: the
size that an elementwise rounding bound is relative to.
"""
import numpy as np


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def silu(x):
    return x * sigmoid(x)


def dsilu(x, mag=False):
    s = sigmoid(x)
    return s * (1 + (np.abs(x) if mag else x) * (1 - s))


def softplus(x):
    return np.logaddexp(0.0, x)


# ---- RMS norm ------------------------------------------------------------------

def rms_norm(x, w, eps):
    m = np.mean(x * x, -1, keepdims=True) + eps
    return np.where(m > 0, x / np.sqrt(np.where(m > 0, m, 1.0)), 0.0) * w


def rms_norm_bwd(h, w, dy, eps):
    """(dh, dweight per row): the caller sums the latter over the rows that share w."""
    m = np.mean(h * h, -1, keepdims=True) + eps
    r = np.where(m > 0, 1 / np.sqrt(np.where(m > 0, m, 1.0)), 0.0)
    n, dn = h * r, dy * w
    return r * (dn - n * np.mean(dn * n, -1, keepdims=True)), dy * n


def e4m3_round(v):
    """The nearest of e4m3's values (ties to even): 3 bits behind the leading one,
    steps of 2^-9 below 2^-6, saturating at 448."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    return np.clip(np.round(v / step) * step, -448, 448)


# ---- causal convolution ----------------------------------------------------------

def conv(x, w, b, state, act):
    """x [T,C], w [C,K], b [C], state [K-1,C] -> (out, final state)."""
    T, K = len(x), w.shape[1]
    full = np.concatenate([state, x])
    p = b + sum((full[j:j + T] * w[:, j] for j in range(K)), np.zeros_like(x))
    return (silu(p) if act else p), full[T:]


def conv_bwd(x, w, b, state, act, dy, dfin, mag=False):
    """-> (dx, dw, db, dstate). mag: bounds (p itself stays signed)."""
    T, K = len(x), w.shape[1]
    full = np.concatenate([state, x])
    p = b + sum((full[j:j + T] * w[:, j] for j in range(K)), np.zeros_like(x))
    if mag:
        full, w, dy, dfin = np.abs(full), np.abs(w), np.abs(dy), np.abs(dfin)
    dp = dy * np.abs(dsilu(p, mag)) if act and mag else dy * dsilu(p) if act else dy
    dfull = np.zeros_like(full)
    dfull[T:] += dfin
    dw = np.zeros_like(w)
    for j in range(K):
        dfull[j:j + T] += dp * w[:, j]
        dw[:, j] = (dp * full[j:j + T]).sum(0)
    return dfull[K - 1:], dw, dp.sum(0), dfull[:K - 1]


# ---- selective scan ---------------------------------------------------------------

def scan(x, dt, A, B, C, D, z, h0, mag=False):
    """x [T,C], dt [T,C] (step sizes), A [C,N], B, C [T,C,N], D [C], z [T,C] or None,
    h0 [C,N] -> (out, final state, states [T,C,N])."""
    if mag:
        x, B, C, D, h0, dt_u = np.abs(x), np.abs(B), np.abs(C), np.abs(D), np.abs(h0), np.abs(dt)
    else:
        dt_u = dt
    h, out, states = h0, np.zeros_like(x), np.zeros((len(x),) + h0.shape)
    for t in range(len(x)):
        h = np.exp(dt[t][:, None] * A) * h + (dt_u[t] * x[t])[:, None] * B[t]
        states[t] = h
        out[t] = (C[t] * h).sum(-1) + D * x[t]
    if z is not None:
        out = out * (np.abs(silu(z)) if mag else silu(z))
    return out, h, states


def scan_bwd(x, dt, A, B, C, D, z, h0, dy, dfin, mag=False):
    """-> dict of dx, ddt (of the step sizes), dA, dB, dC [T,C,N] (per channel), dD, dz, dh0."""
    ungated, _, states = scan(x, dt, A, B, C, D, None, h0, mag)
    dz = None
    if mag:
        x, B, C, D, h0, dy, dfin = (np.abs(v) for v in (x, B, C, D, h0, dy, dfin))
    u_dt, rate = (np.abs(dt), np.abs(A)) if mag else (dt, A)
    if z is not None:
        dz = dy * ungated * (np.abs(dsilu(z, True)) if mag else dsilu(z))
        dy = dy * (np.abs(silu(z)) if mag else silu(z))
    T = len(x)
    out = dict(dx=np.zeros_like(x), ddt=np.zeros_like(x), dA=np.zeros_like(A), dB=np.zeros(B.shape),
               dC=np.zeros(C.shape), dz=dz, dD=(dy * x).sum(0))
    g = dfin
    for t in range(T - 1, -1, -1):
        g = g + dy[t][:, None] * C[t]
        dec = np.exp(dt[t][:, None] * A)
        old = dec * (states[t - 1] if t else h0)
        inner = (g * B[t]).sum(-1)
        out["dC"][t] = dy[t][:, None] * states[t]
        out["dB"][t] = g * (u_dt[t] * x[t])[:, None]
        out["dx"][t] = u_dt[t] * inner + D * dy[t]
        out["ddt"][t] = (g * old * rate).sum(-1) + x[t] * inner
        out["dA"] += g * old * u_dt[t][:, None]
        g = dec * g
    out["dh0"] = g
    return out


# ---- layouts ------------------------------------------------------------------------

def sequences(B, T, cu=None):
    """[(index of its state, batch row, first token, end)]."""
    if cu is None:
        return [(b, b, 0, T) for b in range(B)]
    return [(i, 0, int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


def flat(x, b, lo, hi):
    """Tokens [lo,hi) of batch row b of [B,H,T,d] as [T, H*d]."""
    return x[b, :, lo:hi].transpose(1, 0, 2).reshape(hi - lo, x.shape[1] * x.shape[3])


def unflat(y, H):
    """[T, H*d] -> [H,T,d]."""
    return y.reshape(len(y), H, y.shape[1] // H).transpose(1, 0, 2)


def spread(Bm, b, lo, hi, H, d):
    """Group rows [B,G,T,N] as every channel sees them: [T, H*d, N]."""
    g = np.repeat(Bm[b, :, lo:hi], H // Bm.shape[1], 0)      # [H, T, N]
    return np.repeat(g.transpose(1, 0, 2), d, 1)


def gather(dB, H, G, d):
    """Per-channel gradients [T, H*d, N] summed over the channels of a group: [G,T,N]."""
    T, _, N = dB.shape
    return dB.reshape(T, G, H // G * d, N).sum(2).transpose(1, 0, 2)
