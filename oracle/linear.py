"""Linear attention with one decay per head, and the norms around a block, in
fp64 NumPy from their definitions (test infrastructure; nothing on the product
path imports it).

  S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = S_t^T (scale q_t)

q, k [T, Hk, dk]; v [T, H, dv]; g [T, H] or [H]; head h reads q, k of head
h // (H // Hk).  cu: offsets of the packed sequences.
"""
from __future__ import annotations

import numpy as np


def _heads(q, k, v, g):
    q, k, v, g = (np.asarray(x, np.float64) for x in (q, k, v, g))
    rep = v.shape[1] // q.shape[1]
    return (np.repeat(q, rep, 1), np.repeat(k, rep, 1), v,
            np.broadcast_to(g, v.shape[:2]), rep)


def forward(q, k, v, g, cu, *, scale=1.0, initial_state=None):
    """(o [T, H, dv], final states [N, H, dk, dv])."""
    q, k, v, g, _ = _heads(q, k, v, g)
    N, (T, H, dv), dk = len(cu) - 1, v.shape, q.shape[2]
    o = np.zeros((T, H, dv))
    fin = np.zeros((N, H, dk, dv))
    for n in range(N):
        S = np.zeros((H, dk, dv)) if initial_state is None else np.array(initial_state[n], np.float64)
        for t in range(cu[n], cu[n + 1]):
            S = np.exp(g[t])[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = np.einsum("hk,hkv->hv", scale * q[t], S)
        fin[n] = S
    return o, fin


def backward(q, k, v, g, cu, dy, *, scale=1.0, initial_state=None, d_final_state=None):
    """Gradients of sum(dy * o) + sum(d_final_state * final): dict of dq, dk
    [T, Hk, dk], dv [T, H, dv], dg (the shape of g), ds0 [N, H, dk, dv], and
    dg_tokens [T, H], whose sum over the tokens is dg when g is per head."""
    per_head, Hk = np.asarray(g).ndim == 1, np.asarray(q).shape[1]
    q, k, v, g, rep = _heads(q, k, v, g)
    dy = np.asarray(dy, np.float64)
    N, (T, H, dv), dk = len(cu) - 1, v.shape, q.shape[2]
    out = dict(dq=np.zeros((T, H, dk)), dk=np.zeros((T, H, dk)), dv=np.zeros((T, H, dv)),
               dg=np.zeros((T, H)), ds0=np.zeros((N, H, dk, dv)))
    for n in range(N):
        S = np.zeros((H, dk, dv)) if initial_state is None else np.array(initial_state[n], np.float64)
        states = []
        for t in range(cu[n], cu[n + 1]):
            states.append(S)
            S = np.exp(g[t])[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            out["dq"][t] = scale * np.einsum("hkv,hv->hk", S, dy[t])
        B = np.zeros((H, dk, dv)) if d_final_state is None else np.array(d_final_state[n], np.float64)
        for t in reversed(range(cu[n], cu[n + 1])):
            B = B + scale * q[t][:, :, None] * dy[t][:, None, :]
            out["dk"][t] = np.einsum("hkv,hv->hk", B, v[t])
            out["dv"][t] = np.einsum("hkv,hk->hv", B, k[t])
            a = np.exp(g[t])
            out["dg"][t] = a * np.einsum("hkv,hkv->h", states[t - cu[n]], B)
            B = a[:, None, None] * B
        out["ds0"][n] = B
    for x in ("dq", "dk"):
        out[x] = out[x].reshape(T, Hk, rep, dk).sum(2)
    out["dg_tokens"] = out["dg"]
    if per_head:
        out["dg"] = out["dg"].sum(0)
    return out


def _act(z, kind):
    s = 1.0 / (1.0 + np.exp(-z))
    if kind == "given":
        return z, np.ones_like(z)
    return (s, s * (1 - s)) if kind == "logits" else (z * s, s * (1 + z * (1 - s)))


def block_norm(y, *, post_norm=True, post_weight=None, gate=None, act="given", residual=None,
               res_scale=1.0, pre_norm=False, pre_weight=None, eps=1e-6):
    """(out, normed or None) over the rows of y [R, D]."""
    y = np.asarray(y, np.float64)
    u = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) if post_norm else y
    if post_weight is not None:
        u = u * np.asarray(post_weight, np.float64)
    if gate is not None:
        u = u * _act(np.asarray(gate, np.float64), act)[0]
    r = res_scale * u + (0.0 if residual is None else np.asarray(residual, np.float64))
    if not pre_norm:
        return r, None
    h = r / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return r, h if pre_weight is None else h * np.asarray(pre_weight, np.float64)


def block_norm_backward(dout, dnormed, y, *, post_norm=True, post_weight=None, gate=None, act="given",
                        residual=None, res_scale=1.0, pre_norm=False, pre_weight=None, eps=1e-6):
    """Gradients of sum(dout * out) + sum(dnormed * normed) as a dict."""
    f = lambda x, d=None: d if x is None else np.asarray(x, np.float64)  # noqa: E731
    y, wp, wn = f(y), f(post_weight, 1.0), f(pre_weight, 1.0)
    r, _ = block_norm(y, post_norm=post_norm, post_weight=post_weight, gate=gate, act=act, residual=residual,
                      res_scale=res_scale, eps=eps)
    got = {}
    d = np.zeros_like(y) + f(dout, 0.0)
    got["dpre_weight"] = None
    if pre_norm and dnormed is not None:
        ir = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
        m, rn = f(dnormed) * wn, r * ir
        d = d + ir * (m - rn * (m * rn).mean(-1, keepdims=True))
        got["dpre_weight"] = (f(dnormed) * rn).sum(0)
    got["dresidual"] = d
    du = res_scale * d
    iy = 1.0 / np.sqrt((y * y).mean(-1, keepdims=True) + eps) if post_norm else 1.0
    yn = y * iy
    a = 1.0
    got["dgate"] = None
    if gate is not None:
        a, slope = _act(f(gate), act)
        got["dgate"] = du * yn * wp * slope
    got["dpost_weight"] = (du * a * yn).sum(0)
    m = du * a * wp
    got["dy"] = iy * (m - yn * (m * yn).mean(-1, keepdims=True)) if post_norm else m
    got["dy_term"] = iy * m  # the larger of the two terms dy is the difference of
    return got
