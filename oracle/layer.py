"""The operators around the mixer in fp64 (NumPy).

TEST INFRASTRUCTURE ONLY (see the package docstring).

* ``step_slots``: the recurrence token by token over a pool of state slots
  ("Decoding Hybrid Linear Attention Architectures", section 6, and the step
  order of section 3 item 6: decay, erase along k, write).
* ``slot_map``: offsets, start slots and kept slots of a batch from its
  request lengths, as plain loops.
* ``group_norm`` / ``group_norm_grad``: each group of channels of each token
  by its own mean square (or variance), with an activation, and its gradient.
* ``prologue_grad``: the gradient of ``oracle.prologue.prologue`` with key
  heads shared by several value heads.
"""
from __future__ import annotations

import numpy as np

from .prologue import EPS, l2_normalise, log_decay, sigmoid, softplus


def step_slots(q, k, v, g, beta, pool, src, dst=None, cu=None, gate_scale=None, norm_q=False,
               norm_k=False, o=None):
    """(o, pool) after the call; the inputs fp64, nothing modified.  g, beta are
    logits where gate_scale is given.  Rows no request covers come from ``o``."""
    total, H, dv = v.shape
    share = H // q.shape[1]
    o = np.zeros(v.shape) if o is None else np.array(o, dtype=np.float64)
    pool = np.array(pool, dtype=np.float64)
    start = pool.copy()
    q = l2_normalise(q) if norm_q else q
    k = l2_normalise(k) if norm_k else k
    if gate_scale is not None:
        g = log_decay(g[None], gate_scale)[0]
        beta = sigmoid(beta)
    alpha = np.exp(g if g.ndim == 3 else g[..., None])
    for r, s in enumerate(src):
        lo, hi = (r, r + 1) if cu is None else (int(cu[r]), int(cu[r + 1]))
        if lo == hi or s < -1 or s >= len(pool):
            continue
        for h in range(H):
            S = start[s, h].copy() if s >= 0 else np.zeros(pool.shape[2:])
            for t in range(lo, hi):
                kt = k[t, h // share]
                S = S * alpha[t, h]
                S = S + np.outer(beta[t, h] * (v[t, h] - S @ kt), kt)
                o[t, h] = S @ q[t, h // share]
                d = dst[t] if dst is not None else (s if t == hi - 1 else -1)
                if 0 <= d < len(pool):
                    pool[d, h] = S
    return o, pool


def slot_map(lens, kept, table, slots, max_tokens, keep_all):
    """(cu, src, request, dst, bad): int32 arrays, and whether a request was refused."""
    R, W = table.shape
    cu, src = np.zeros(R + 1, np.int32), np.full(R, -2, np.int32)
    request, dst = np.full(max_tokens, -1, np.int32), np.full(max_tokens, -1, np.int32)
    at, bad = 0, False
    for r in range(R):
        n = max(int(lens[r]), 0)
        bad = bad or lens[r] < 0
        uses = n if keep_all else 1
        end = at + n
        if n:
            good = 0 <= kept[r] <= W and uses <= W and end <= max_tokens
            if good:
                named = [int(table[r, j]) for j in range(uses)]
                first = int(table[r, kept[r] - 1]) if kept[r] else -1
                good = all(0 <= s < slots for s in named) and (not kept[r] or 0 <= first < slots)
            if good:
                src[r] = first
                for j in range(n):
                    dst[at + j] = named[j] if keep_all else (named[0] if j == n - 1 else -1)
            bad = bad or not good
        request[min(at, max_tokens):min(end, max_tokens)] = r
        cu[r + 1] = min(end, max_tokens)
        at = end
    return cu, src, request, dst, bad


def _act(name, u):
    """(value, slope)"""
    if name == "none":
        return u, np.ones_like(u)
    s = sigmoid(u)
    if name == "silu":
        return u * s, s * (1 + u * (1 - s))
    return s, s * (1 - s)


def _normalised(x, weight, bias, center, eps):
    d = x - x.mean(-1, keepdims=True) if center else x
    rstd = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    n = d * rstd
    lin = n if weight is None else n * weight
    return n, rstd, lin if bias is None else lin + bias


def group_norm(x, z=None, weight=None, bias=None, act="silu", center=False, eps=1e-5):
    """x, z [rows, G, D] fp64; weight, bias [D] or [G, D] or None."""
    _, _, lin = _normalised(x, weight, bias, center, eps)
    return _act(act, lin)[0] if z is None else _act(act, z)[0] * lin


def group_norm_grad(dy, x, z=None, weight=None, bias=None, act="silu", center=False, eps=1e-5):
    """dict dx, dz, dweight, dbias (None where there is no such input)."""
    n, rstd, lin = _normalised(x, weight, bias, center, eps)
    f, df = _act(act, lin if z is None else z)
    dlin = dy * df if z is None else dy * f
    out = {"dz": None if z is None else dy * lin * df}
    for name, p, term in (("dweight", weight, dlin * n), ("dbias", bias, dlin)):
        out[name] = None if p is None else term.sum((0, 1) if p.ndim == 1 else 0)
    h = dlin if weight is None else dlin * weight
    dx = h - n * (h * n).mean(-1, keepdims=True)
    out["dx"] = rstd * (dx - h.mean(-1, keepdims=True) if center else dx)
    return out


def prologue_grad(q, k, a, b, gate_scale, dq, dk, dg, dbeta, norm_q=True, norm_k=True):
    """q, k [tokens, Hk, d]; a [tokens, H(, d)]; b [tokens, H]; dq, dk [tokens, H, d].
    Returns dict dq, dk, da, db, dgate_scale."""
    share = b.shape[1] // q.shape[1]
    out = {}
    for name, x, d, norm in (("dq", q, dq, norm_q), ("dk", k, dk, norm_k)):
        d = d.reshape(x.shape[0], x.shape[1], share, x.shape[2]).sum(2)
        if norm:
            r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) + EPS)
            d = r * d - x * r**3 * (x * d).sum(-1, keepdims=True)
        out[name] = d
    s = np.asarray(gate_scale).reshape(1, -1, *[1] * (a.ndim - 2))
    out["da"] = -s * sigmoid(a) * dg
    beta = sigmoid(b)
    out["db"] = beta * (1 - beta) * dbeta
    out["dgate_scale"] = -(dg * softplus(a)).sum(tuple(i for i in range(a.ndim) if i != 1))
    return out
