"""fp64 reference of linear attention with one decay a head and of the query/key
norm with rotation (numpy, token by token) -- TEST INFRASTRUCTURE ONLY.

    S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   a_t = exp(max(log_alpha_t, -100))

Arrays are token-major as in :mod:`oracle`: q, k ``[n, H, dk]``, v ``[n, H, dv]``,
log_alpha ``[n, H]``; sequences are ranges of ``seq_start``; states ``[N, H, dk, dv]``.
The norm takes x ``[n, H, d]``.
"""
from __future__ import annotations

import numpy as np

FLOOR = -100.0


def _alpha(log_alpha):
    return np.exp(np.maximum(np.asarray(log_alpha, np.float64), FLOOR))


def forward(q, k, v, log_alpha, seq_start, init_state=None):
    """(o, final_state) of the recurrence."""
    a = _alpha(log_alpha)
    H, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    N = len(seq_start) - 1
    o = np.zeros(v.shape)
    final = np.zeros((N, H, dk, dv)) if init_state is None else np.array(init_state, np.float64)
    for n in range(N):
        s = final[n]
        for t in range(int(seq_start[n]), int(seq_start[n + 1])):
            s = a[t][:, None, None] * s + k[t][:, :, None] * v[t][:, None, :]
            o[t] = (q[t][:, None, :] @ s)[:, 0]
        final[n] = s
    return o, final


def backward(q, k, v, log_alpha, seq_start, d_o, d_final_state=None, init_state=None):
    """Gradients (dict) of sum(d_o o) + sum(d_final_state final_state)."""
    a = _alpha(log_alpha)
    H, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    N = len(seq_start) - 1
    g = dict(dq=np.zeros(q.shape), dk=np.zeros(q.shape), dv=np.zeros(v.shape), dlog_alpha=np.zeros(a.shape),
             d_init_state=np.zeros((N, H, dk, dv)))
    for n in range(N):
        t0, t1 = int(seq_start[n]), int(seq_start[n + 1])
        states = [np.zeros((H, dk, dv)) if init_state is None else np.asarray(init_state[n], np.float64)]
        for t in range(t0, t1):
            states.append(a[t][:, None, None] * states[-1] + k[t][:, :, None] * v[t][:, None, :])
        ds = np.zeros((H, dk, dv)) if d_final_state is None else np.array(d_final_state[n], np.float64)
        for t in reversed(range(t0, t1)):
            ds = ds + q[t][:, :, None] * d_o[t][:, None, :]
            g["dq"][t] = (states[t - t0 + 1] @ d_o[t][:, :, None])[..., 0]
            g["dk"][t] = (ds @ v[t][:, :, None])[..., 0]
            g["dv"][t] = (k[t][:, None, :] @ ds)[:, 0]
            g["dlog_alpha"][t] = a[t] * (ds * states[t - t0]).sum((1, 2))
            ds = a[t][:, None, None] * ds
        g["d_init_state"][n] = ds
    g["dlog_alpha"][np.asarray(log_alpha, np.float64) < FLOOR] = 0.0
    return g


def decode_step(q, k, v, log_alpha, state):
    """(o, state) after one token of every sequence; q ``[N, H, dk]``, log_alpha ``[N, H]``."""
    s = _alpha(log_alpha)[..., None, None] * state + k[..., :, None] * v[..., None, :]
    return (q[..., None, :] @ s)[..., 0, :], s


def _turn(y, positions, inv_freq, interleaved, sign):
    rot = 2 * len(inv_freq)
    t = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(t)[:, None], sign * np.sin(t)[:, None]
    out = np.array(y)
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = y[..., first], y[..., second]
    out[..., first] = a * c - b * s
    out[..., second] = b * c + a * s
    return out


def _inv_rms(x, eps):
    m = (x ** 2).mean(-1, keepdims=True) + eps
    return np.where(m > 0, 1.0 / np.sqrt(np.where(m > 0, m, 1.0)), 0.0)


def norm_rope(x, w, positions, inv_freq, eps, interleaved):
    """The normed and turned rows of x ``[n, H, d]`` (w ``[d]`` or None)."""
    y = x * _inv_rms(x, eps) * (1.0 if w is None else w)
    return _turn(y, positions, inv_freq, interleaved, 1.0)


def norm_rope_backward(x, w, positions, inv_freq, eps, interleaved, d_y):
    """(dx, dw) of sum(d_y norm_rope(x))."""
    g = _turn(np.asarray(d_y, np.float64), positions, inv_freq, interleaved, -1.0)
    r = _inv_rms(x, eps)
    h = g if w is None else g * w
    return r * h - x * r ** 3 * (h * x).mean(-1, keepdims=True), (g * x * r).sum((0, 1))
