"""fp64 definitions of the state space layer's operators -- TEST INFRASTRUCTURE ONLY.

Plain numpy, token by token and element by element as the operators are defined (include/gdn.h),
with no code of the CUDA library.  Inputs are widened exactly from what the GPU sees.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def _f64(t):
    if t is None:
        return None
    return t.detach().to("cpu").double().numpy() if hasattr(t, "detach") else np.asarray(t, np.float64)


def softplus(v):
    with np.errstate(over="ignore"):
        return np.where(v > 20.0, v, np.log1p(np.exp(v)))


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def ssm_scan(x, dt, Bm, Cm, A_log, dt_bias, D=None, z=None, h0=None, cu_seqlens=None):
    """(y, hT, mag): the scan over [B,T,...] inputs, and per output the sum of the magnitudes of
    the terms it is made of (what a rounding of each term is relative to)."""
    x, dt, Bm, Cm, A_log, dt_bias, D, z, h0 = map(_f64, (x, dt, Bm, Cm, A_log, dt_bias, D, z, h0))
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    grp = np.arange(H) // (H // G)
    if cu_seqlens is None:
        seqs = [(b * T, (b + 1) * T) for b in range(B)]
    else:
        cu = [int(v) for v in cu_seqlens]
        seqs = list(zip(cu[:-1], cu[1:]))
    xf, dtf, Bf, Cf = (t.reshape(B * T, *t.shape[2:]) for t in (x, dt, Bm, Cm))
    y, mag = np.zeros((B * T, H, P)), np.zeros((B * T, H, P))
    hT = np.zeros((len(seqs), H, N, P))
    A = -np.exp(A_log)
    for i, (r0, r1) in enumerate(seqs):
        h = h0[i].copy() if h0 is not None else np.zeros((H, N, P))
        ha = np.abs(h)
        for t in range(r0, r1):
            d = softplus(dtf[t] + dt_bias)
            a = np.exp(A * d)[:, None, None]
            add = (d[:, None, None] * Bf[t][grp][:, :, None]) * xf[t][:, None, :]
            h = a * h + add
            ha = a * ha + np.abs(add)
            c = Cf[t][grp][:, :, None]
            y[t] = (h * c).sum(1)
            mag[t] = (ha * np.abs(c)).sum(1)
        hT[i] = h
    if D is not None:
        y = y + D[:, None] * xf
        mag = mag + np.abs(D[:, None] * xf)
    if z is not None:
        gate = silu(z.reshape(B * T, H, P))
        y, mag = y * gate, mag * np.abs(gate)
    return y.reshape(B, T, H, P), hT, mag.reshape(B, T, H, P)


def ssm_decode_step(row, dt, conv_w, conv_state, A_log, dt_bias, state, H, G, P, N, D=None, z=None,
                    conv_bias=None, activation=True, state_indices=None):
    """(y, state, conv_state, y's magnitude, state's magnitude) after one token.  A magnitude is the
    same expression on the magnitudes of its terms, from the convolution's on (|silu(v)| <= |v| <=
    the sum of its taps' magnitudes): what a rounding of any term is relative to."""
    row, dt, conv_w, cs, A_log, dt_bias, st, D, z, conv_bias = map(
        _f64, (row, dt, conv_w, conv_state, A_log, dt_bias, state, D, z, conv_bias))
    cs, st = cs.copy(), st.copy()
    n = row.shape[0]
    y, ymag, smag = np.zeros((n, H, P)), np.zeros((n, H, P)), np.abs(st)
    grp = np.arange(H) // (H // G)
    cut = lambda v: (v[:H * P].reshape(H, P), v[H * P:H * P + G * N].reshape(G, N), v[H * P + G * N:].reshape(G, N))
    for r in range(n):
        s = r if state_indices is None else int(state_indices[r])
        if s < 0 or s >= st.shape[0]:
            continue
        win = np.concatenate([cs[s], row[r][:, None]], 1)
        v = (conv_w * win).sum(1) + (0.0 if conv_bias is None else conv_bias)
        if activation:
            v = silu(v)
        x, b, c = cut(v)
        xm, bm, cm = cut((np.abs(conv_w * win)).sum(1) + (0.0 if conv_bias is None else np.abs(conv_bias)))
        d = softplus(dt[r] + dt_bias)
        a = np.exp(-np.exp(A_log) * d)
        st[s] = a[:, None, None] * st[s] + d[:, None, None] * b[grp][:, :, None] * x[:, None, :]
        smag[s] = a[:, None, None] * smag[s] + d[:, None, None] * bm[grp][:, :, None] * xm[:, None, :]
        y[r] = (st[s] * c[grp][:, :, None]).sum(1)
        ymag[r] = (smag[s] * cm[grp][:, :, None]).sum(1)
        if D is not None:
            y[r] += D[:, None] * x
            ymag[r] += np.abs(D[:, None]) * xm
        if z is not None:
            gate = silu(z[r].reshape(H, P))
            y[r] *= gate
            ymag[r] *= np.abs(gate)
        cs[s] = win[:, 1:]
    return y, st, cs, ymag, smag


def rmsnorm(x, weight, residual=None, eps=1e-6):
    """(s, y, scales): the sum behind the residual, the normed row, and max|y| / 448 per block."""
    x, weight, residual = map(_f64, (x, weight, residual))
    s = x if residual is None else x + residual
    y = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * weight
    D = y.shape[-1]
    top = np.stack([np.abs(y[..., j:j + 128]).max(-1) for j in range(0, D, 128)], -1)
    return s, y, np.where(top > 0, top / E4M3_MAX, 1.0)


def fp8_matmul(a, a_scales, w, w_scales):
    """(out, mag): the scaled product, and the sum of its terms' magnitudes."""
    a, a_scales, w, w_scales = map(_f64, (a, a_scales, w, w_scales))
    K = a.shape[1]
    ak = a * np.repeat(a_scales, 128, 1)[:, :K]
    wk = w * np.repeat(np.repeat(w_scales, 128, 0), 128, 1)[:w.shape[0], :K]
    return ak @ wk.T, np.abs(ak) @ np.abs(wk).T
