"""The selective state space operators and the block norm in 64 bits on the CPU,
token by token from their definitions, with the magnitudes that error bounds need."""
from __future__ import annotations

import torch

F64 = torch.float64


def d(t):
    return None if t is None else t.detach().cpu().to(F64)


def silu(v):
    return v * torch.sigmoid(v)


def softplus(v):
    return torch.logaddexp(v, torch.zeros((), dtype=F64))


def bounds(cu, n_rows):
    return [0, n_rows] if cu is None else [int(v) for v in cu]


def conv(x, w, bias, hist, cu, slots, has, y0, activation=1):
    """(y, hist after, magnitude of the sums)."""
    x, w, bias, y = d(x), d(w), d(bias), d(y0).clone()
    hist = None if hist is None else d(hist).clone()
    k, ch = w.shape[1], x.shape[1]
    mag = torch.zeros_like(y)
    cu = bounds(cu, x.shape[0])
    for i in range(len(cu) - 1):
        b, e = cu[i], cu[i + 1]
        if b == e:
            continue
        slot = i if slots is None else int(slots[i])
        ok = hist is not None and 0 <= slot < hist.shape[0]
        old = hist[slot] if ok and (has is None or bool(has[i])) else torch.zeros(k - 1, ch, dtype=F64)
        ext = torch.cat([old, x[b:e]])
        acc = torch.zeros(e - b, ch, dtype=F64) if bias is None else bias.expand(e - b, ch).clone()
        m = acc.abs()
        for j in range(k):
            acc += w[:, j] * ext[j:j + e - b]
            m += (w[:, j] * ext[j:j + e - b]).abs()
        y[b:e] = silu(acc) if activation else acc
        mag[b:e] = m
        if ok:
            hist[slot] = ext[-(k - 1):]
    return y, hist, mag


def scan(x, a, B, C, A_log, dt_bias, states, D, z, cu, slots, has, y0, mags=None):
    """(y, states after, magnitude of y's sums, magnitude of the states' sums).  `mags`:
    magnitudes of x, B and C themselves where those are sums (their values otherwise)."""
    xm, bm, cm = (t.detach().cpu().to(F64).abs() for t in (mags or (x, B, C)))
    x, a, B, C, A_log, dt_bias, D, z = (d(t) for t in (x, a, B, C, A_log, dt_bias, D, z))
    y = d(y0).clone()
    T, H, P = x.shape
    G, N = B.shape[1:]
    of = torch.arange(H) % G
    states = None if states is None else d(states).clone()
    mag, smag = torch.zeros_like(y), None if states is None else states.abs()
    cu = bounds(cu, T)
    for i in range(len(cu) - 1):
        b, e = cu[i], cu[i + 1]
        if b == e:
            continue
        slot = i if slots is None else int(slots[i])
        ok = states is not None and 0 <= slot < states.shape[0]
        S = states[slot].clone() if ok and (has is None or bool(has[i])) else torch.zeros(H, N, P, dtype=F64)
        M = S.abs()
        for t in range(b, e):
            dt = softplus(a[t] + dt_bias)
            keep = torch.exp(-torch.exp(A_log) * dt)[:, None, None]
            new = (dt[:, None] * B[t][of])[:, :, None] * x[t][:, None, :]
            S = keep * S + new
            M = keep * M + (dt[:, None] * bm[t][of])[:, :, None] * xm[t][:, None, :]
            o = torch.einsum("hnp,hn->hp", S, C[t][of])
            m = torch.einsum("hnp,hn->hp", M, cm[t][of])
            if D is not None:
                o = o + D[:, None] * x[t]
                m = m + D.abs()[:, None] * xm[t]
            if z is not None:
                o = o * silu(z[t])
                m = m * silu(z[t]).abs()
            y[t], mag[t] = o, m
        if ok:
            states[slot], smag[slot] = S, M
    return y, states, mag, smag


def step(xbc, a, conv_w, conv_bias, A_log, dt_bias, hist, states, D, z, slots, y0, activation=1):
    """(y, hist after, states after, magnitude of y, magnitude of the states)."""
    n, cw = xbc.shape
    _, H, N, P = states.shape
    G = (cw - H * P) // (2 * N)
    y, hist, states = d(y0).clone(), d(hist).clone(), d(states).clone()
    mag, smag = torch.zeros_like(y), states.abs()
    for i in range(n):
        slot = i if slots is None else int(slots[i])
        if not 0 <= slot < states.shape[0]:
            continue
        u, h2, um = conv(xbc[i:i + 1], conv_w, conv_bias, hist[slot:slot + 1], None, None, None, torch.zeros(1, cw),
                        activation)
        hist[slot] = h2[0]
        x, B, C = (v.view(1, -1, q) for v, q in zip(u.split([H * P, G * N, G * N], dim=1), (P, N, N)))
        mags = [v.view(1, -1, q) for v, q in zip(um.split([H * P, G * N, G * N], dim=1), (P, N, N))]
        o, s2, m, sm = scan(x, a[i:i + 1], B, C, A_log, dt_bias, states[slot:slot + 1], D,
                            None if z is None else z[i:i + 1], None, None, None, torch.zeros(1, H, P), mags)
        y[i], states[slot], mag[i], smag[slot] = o[0], s2[0], m[0], sm[0]
    return y, hist, states, mag, smag


def block_norm(b, r, w_pre, w_post, gate, gate_sigmoid, scale, eps):
    """(residual, y, magnitude of the residual's sum)."""
    b, r, w_pre, w_post, gate = (d(t) for t in (b, r, w_pre, w_post, gate))
    u = b
    if w_post is not None:
        u = u / torch.sqrt(u.square().mean(-1, keepdim=True) + eps) * w_post
    if gate is not None:
        u = u * (torch.sigmoid(gate) if gate_sigmoid else gate)
    out = r + scale * u
    mag = r.abs() + (scale * u).abs()
    return out, out / torch.sqrt(out.square().mean(-1, keepdim=True) + eps) * w_pre, mag
