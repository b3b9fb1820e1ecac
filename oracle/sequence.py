"""Sequence operators in numpy float64, written position by position.

The plain counterpart of causal_conv, state_scan and block_norm: the tests
compare the GPU kernels with these, and these with differences.  Every function
also gives, as ``S``, its outputs' sums with every term taken by magnitude, the
scale that rounding errors of the sums are measured on.
"""
from __future__ import annotations

import numpy as np


def _f64(*arrays):
    return [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]


def _lengths(lengths, B, L):
    if lengths is None:
        return [L] * B
    return [min(max(int(n), 0), L) for n in lengths]


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def softplus(v):
    return np.logaddexp(v, 0.0)


def causal_conv(x, w, bias=None, silu=True, state=None, lengths=None):
    """(y, new_state, S of the sum before SiLU)."""
    x, w, bias, state = _f64(x, w, bias, state)
    B, D, L = x.shape
    K = w.shape[1]
    y, S = np.zeros((B, D, L)), np.zeros((B, D, L))
    new = np.zeros((B, D, K - 1))
    for b, n in enumerate(_lengths(lengths, B, L)):
        full = np.zeros((D, K - 1 + n))
        if state is not None:
            full[:, :K - 1] = state[b]
        full[:, K - 1:] = x[b, :, :n]
        for t in range(n):
            terms = w * full[:, t:t + K]
            p = terms.sum(1) + (0 if bias is None else bias)
            S[b, :, t] = np.abs(terms).sum(1) + (0 if bias is None else np.abs(bias))
            y[b, :, t] = p * sigmoid(p) if silu else p
        new[b] = full[:, n:n + K - 1]
    return y, new, S


def causal_conv_grads(gy, x, w, bias=None, silu=True, lengths=None):
    """{dx, dw, db} and {"S" + name}."""
    gy, x, w, bias = _f64(gy, x, w, bias)
    B, D, L = x.shape
    K = w.shape[1]
    out = {"dx": np.zeros_like(x), "dw": np.zeros_like(w), "db": np.zeros(D)}
    out.update({"S" + k: np.zeros_like(v) for k, v in out.items()})
    for b, n in enumerate(_lengths(lengths, B, L)):
        full = np.concatenate([np.zeros((D, K - 1)), x[b, :, :n]], 1)
        for t in range(n):
            seen = full[:, t:t + K]
            dp = gy[b, :, t].copy()
            if silu:
                p = (w * seen).sum(1) + (0 if bias is None else bias)
                s = sigmoid(p)
                dp *= s * (1 + p * (1 - s))
            out["db"] += dp
            out["Sdb"] += np.abs(dp)
            out["dw"] += dp[:, None] * seen
            out["Sdw"] += np.abs(dp[:, None] * seen)
            for k in range(K):
                at = t - (K - 1) + k
                if at >= 0:
                    out["dx"][b, :, at] += dp * w[:, k]
                    out["Sdx"][b, :, at] += np.abs(dp * w[:, k])
    return out


def _per_channel(m, D):
    """[B, G, N, L] as [B, D, N, L]."""
    return np.repeat(m, D // m.shape[1], axis=1)


def state_scan(x, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, soft=True, state=None,
               lengths=None, every=0):
    """(y, new_state, S of y, S of the state[, states before every `every`-th position])."""
    x, dt, A, Bm, Cm, skip, z, dt_bias, state = _f64(x, dt, A, Bm, Cm, skip, z, dt_bias, state)
    B, D, L = x.shape
    N = A.shape[1]
    Bd, Cd = _per_channel(Bm, D), _per_channel(Cm, D)
    y, S = np.zeros((B, D, L)), np.zeros((B, D, L))
    h = np.zeros((B, D, N)) if state is None else state.copy()
    H = np.abs(h)
    marks = []
    ns = np.array(_lengths(lengths, B, L))
    for t in range(L):
        if every and t % every == 0:
            marks.append(h.copy())
        for b in np.nonzero(t < ns)[0]:
            raw = dt[b, :, t] + (0 if dt_bias is None else dt_bias)
            s = softplus(raw) if soft else raw
            a = np.exp(s[:, None] * A)
            into = (s * x[b, :, t])[:, None] * Bd[b, :, :, t]
            h[b] = a * h[b] + into
            H[b] = a * H[b] + np.abs(into)
            v = (h[b] * Cd[b, :, :, t]).sum(1)
            V = (H[b] * np.abs(Cd[b, :, :, t])).sum(1)
            if skip is not None:
                v, V = v + skip * x[b, :, t], V + np.abs(skip * x[b, :, t])
            if z is not None:
                f = z[b, :, t] * sigmoid(z[b, :, t])
                v, V = v * f, V * np.abs(f)
            y[b, :, t], S[b, :, t] = v, V
    return (y, h, S, H, np.stack(marks, 2)) if every else (y, h, S, H)


def state_scan_grads(gout, x, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, soft=True, state=None,
                     lengths=None, gstate=None):
    """{dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dstate} and {"S" + name}."""
    gout, x, dt, A, Bm, Cm, skip, z, dt_bias, state, gstate = _f64(
        gout, x, dt, A, Bm, Cm, skip, z, dt_bias, state, gstate)
    B, D, L = x.shape
    N, G = A.shape[1], Bm.shape[1]
    of = np.arange(D) // (D // G)
    o = {"dx": np.zeros_like(x), "ddt": np.zeros_like(x), "dA": np.zeros_like(A),
         "dB": np.zeros_like(Bm), "dC": np.zeros_like(Cm), "dD": np.zeros(D),
         "dz": np.zeros_like(x), "ddt_bias": np.zeros(D), "dstate": np.zeros((B, D, N))}
    o.update({"S" + k: np.zeros_like(v) for k, v in o.items()})

    def put(name, at, value, size):
        o[name][at] += value
        o["S" + name][at] += size

    for b, n in enumerate(_lengths(lengths, B, L)):
        raw = dt[b, :, :n] + (0 if dt_bias is None else dt_bias[:, None])
        s = softplus(raw) if soft else raw
        hs, Hs = np.zeros((n + 1, D, N)), np.zeros((n + 1, D, N))
        if state is not None:
            hs[0], Hs[0] = state[b], np.abs(state[b])
        for t in range(n):
            a = np.exp(s[:, t, None] * A)
            into = (s[:, t] * x[b, :, t])[:, None] * Bm[b, of, :, t]
            hs[t + 1] = a * hs[t] + into
            Hs[t + 1] = a * Hs[t] + np.abs(into)
        back = np.zeros((D, N)) if gstate is None else gstate[b].copy()
        Back = np.abs(back)
        for t in range(n - 1, -1, -1):
            xt, st = x[b, :, t], s[:, t]
            gy, y = gout[b, :, t].copy(), (hs[t + 1] * Cm[b, of, :, t]).sum(1)
            Y = (Hs[t + 1] * np.abs(Cm[b, of, :, t])).sum(1)
            if skip is not None:
                y, Y = y + skip * xt, Y + np.abs(skip * xt)
            if z is not None:
                sg = sigmoid(z[b, :, t])
                slope = sg * (1 + z[b, :, t] * (1 - sg))
                put("dz", (b, slice(None), t), gy * y * slope,
                    np.abs(gy) * sg * (1 + np.abs(z[b, :, t]) * (1 - sg)) * Y)
                gy *= z[b, :, t] * sg
            q = back + Cm[b, of, :, t] * gy[:, None]
            Q = Back + np.abs(Cm[b, of, :, t] * gy[:, None])
            a = np.exp(st[:, None] * A)
            for g in range(G):
                rows = of == g
                put("dB", (b, g, slice(None), t), (q * (st * xt)[:, None])[rows].sum(0),
                    (Q * np.abs(st * xt)[:, None])[rows].sum(0))
                put("dC", (b, g, slice(None), t), (hs[t + 1] * gy[:, None])[rows].sum(0),
                    (Hs[t + 1] * np.abs(gy)[:, None])[rows].sum(0))
            qB = (q * Bm[b, of, :, t]).sum(1)
            QB = (Q * np.abs(Bm[b, of, :, t])).sum(1)
            put("dx", (b, slice(None), t), st * qB + (0 if skip is None else skip * gy),
                st * QB + (0 if skip is None else np.abs(skip * gy)))
            if skip is not None:
                put("dD", slice(None), gy * xt, np.abs(gy * xt))
            through = q * a * hs[t]
            Through = Q * a * Hs[t]
            put("dA", slice(None), through * st[:, None], Through * np.abs(st)[:, None])
            ds = (through * A).sum(1) + xt * qB
            Ds = (Through * np.abs(A)).sum(1) + np.abs(xt) * QB
            if soft:
                ds, Ds = ds * sigmoid(raw[:, t]), Ds * sigmoid(raw[:, t])
            put("ddt", (b, slice(None), t), ds, Ds)
            put("ddt_bias", slice(None), ds, Ds)
            back, Back = a * q, a * Q
        put("dstate", b, back, Back)
    return o


def _norm_parts(y, w_post, gate, scale, eps):
    f = (np.ones(y.shape[1]) if scale is None else scale)[:, None]
    open_ = np.ones_like(y) if gate is None else sigmoid(gate)
    if w_post is None:
        return f, open_, y, None
    i_post = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
    return f, open_, y * i_post * w_post[:, None], i_post


def block_norm(y, r, w_post=None, w_pre=None, gate=None, scale=None, eps=1e-6, lengths=None):
    """(new residual, u or None, S of the residual, S of u or None)."""
    y, r, w_post, w_pre, gate, scale = _f64(y, r, w_post, w_pre, gate, scale)
    B, D, L = y.shape
    y, r, gate = y.copy(), r.copy(), None if gate is None else gate.copy()
    for b, m in enumerate(_lengths(lengths, B, L)):
        for v in (y, r) if gate is None else (y, r, gate):
            v[b, :, m:] = 0
    f, open_, n, _ = _norm_parts(y, w_post, gate, scale, eps)
    out, S = r + f * open_ * n, np.abs(r) + np.abs(f * open_ * n)
    if w_pre is None:
        return out, None, S, None
    i_pre = 1 / np.sqrt((out * out).mean(1, keepdims=True) + eps)
    return out, out * i_pre * w_pre[:, None], S, S * i_pre * np.abs(w_pre)[:, None]


def block_norm_grads(gr, gu, y, r_out, w_post=None, w_pre=None, gate=None, scale=None, eps=1e-6,
                     lengths=None):
    """{dy, dresidual, dgate, dscale, dweight_post, dweight_pre} and {"S" + name},
    from the new residual."""
    gr, gu, y, r_out, w_post, w_pre, gate, scale = _f64(gr, gu, y, r_out, w_post, w_pre, gate, scale)
    B, D, L = y.shape
    gr = np.zeros_like(y) if gr is None else gr.copy()
    gu = np.zeros_like(y) if gu is None else gu.copy()
    y, r_out, gate = y.copy(), r_out.copy(), None if gate is None else gate.copy()
    for b, m in enumerate(_lengths(lengths, B, L)):
        for v in (gr, gu, y, r_out) + (() if gate is None else (gate,)):
            v[b, :, m:] = 0
    f, open_, n, i_post = _norm_parts(y, w_post, gate, scale, eps)
    i_pre = 1 / np.sqrt((r_out * r_out).mean(1, keepdims=True) + eps)
    o = {}
    dr, Sdr = gr, np.abs(gr)
    if w_pre is not None:
        v = gu * w_pre[:, None]
        dr = gr + i_pre * v - r_out * i_pre ** 3 * (v * r_out).mean(1, keepdims=True)
        Sdr = (Sdr + i_pre * np.abs(v)
               + np.abs(r_out) * i_pre ** 3 * np.abs(v * r_out).mean(1, keepdims=True))
        o["dweight_pre"] = (gu * r_out * i_pre).sum((0, 2))
        o["Sdweight_pre"] = np.abs(gu * r_out * i_pre).sum((0, 2))
    dn, Sdn = dr * f * open_, Sdr * np.abs(f) * open_
    if w_post is None:
        o["dy"], o["Sdy"] = dn, Sdn
    else:
        v, V = dn * w_post[:, None], Sdn * np.abs(w_post)[:, None]
        o["dy"] = i_post * v - y * i_post ** 3 * (v * y).mean(1, keepdims=True)
        o["Sdy"] = i_post * V + np.abs(y) * i_post ** 3 * (V * np.abs(y)).mean(1, keepdims=True)
        o["dweight_post"] = (dn * y * i_post).sum((0, 2))
        o["Sdweight_post"] = (Sdn * np.abs(y) * i_post).sum((0, 2))
    o["dresidual"], o["Sdresidual"] = dr, Sdr
    if gate is not None:
        o["dgate"], o["Sdgate"] = dn * n * (1 - open_), Sdn * np.abs(n)
    if scale is not None:
        o["dscale"] = (dr * open_ * n).sum((0, 2))
        o["Sdscale"] = (Sdr * open_ * np.abs(n)).sum((0, 2))
    return o
