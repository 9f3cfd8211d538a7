"""fp64 reference of the gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per
(sequence, head, channel), token by token, and of its gradients."""
from __future__ import annotations

import numpy as np


def _f64(x):
    if x is None:
        return None
    return (x.detach().double().cpu().numpy() if hasattr(x, "detach")
            else np.asarray(x, np.float64))


def forward(x, g, initial_state=None, lens=None):
    """x, g [total, H, d]; lens: the sequences' lengths (default: one).  Returns
    (h [total, H, d], final_state [N, H, d])."""
    x, g, h0 = _f64(x), _f64(g), _f64(initial_state)
    lens = [x.shape[0]] if lens is None else lens
    h, final = np.empty_like(x), np.zeros((len(lens), *x.shape[1:]))
    t = 0
    for n, length in enumerate(lens):
        s = np.zeros(x.shape[1:]) if h0 is None else h0[n].copy()
        for _ in range(length):
            s = np.exp(g[t]) * s + x[t]
            h[t] = s
            t += 1
        final[n] = s
    return h, final


def backward(x, g, dout, initial_state=None, dfinal_state=None, lens=None):
    """Gradients of sum(h * dout) + sum(final_state * dfinal_state): (dx, dg,
    dinitial_state)."""
    x, g, dout, h0, dfin = map(_f64, (x, g, dout, initial_state, dfinal_state))
    lens = [x.shape[0]] if lens is None else lens
    h, _ = forward(x, g, h0, lens)
    dx, dg = np.empty_like(x), np.empty_like(x)
    dh0 = np.zeros((len(lens), *x.shape[1:]))
    end = 0
    for n, length in enumerate(lens):
        begin, end = end, end + length
        e = np.zeros(x.shape[1:]) if dfin is None else dfin[n].copy()
        for t in range(end - 1, begin - 1, -1):
            if t > begin:
                before = h[t - 1]
            else:
                before = 0.0 if h0 is None else h0[n]
            dx[t] = dout[t] + e
            e = np.exp(g[t]) * dx[t]
            dg[t] = e * before
        dh0[n] = e
    return dx, dg, dh0
