"""Plain float64 definition of attention over packed sequences (test infrastructure only; see
the package docstring for who may import it).

Sequence i owns q_lens[i] query rows, one behind the other, and the key rows
[k_starts[i], k_starts[i] + k_lens[i]); its queries are its last rows, so causal query t sees
the keys j <= k_lens[i] - q_lens[i] + t.  Query head h reads k/v head h // (heads / kv_heads).
"""
from __future__ import annotations

import numpy as np

from .dualparal import as_f64


def packed_attention(q, k, v, q_lens, k_lens, k_starts=None, causal=True, scale=None):
    """(out, lse, weight): out [rows][heads][d], lse [rows][heads] of the sequences' query rows,
    and weight = sum_j p_j |v_j|, the size that errors of the softmax weights are relative to.
    Queries that see no key: out 0, lse -inf."""
    q, k, v = as_f64(q), as_f64(k), as_f64(v)
    heads, d = q.shape[1], q.shape[2]
    group = heads // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    rows = sum(q_lens)
    out, weight = np.zeros((rows, heads, d)), np.zeros((rows, heads, d))
    lse = np.full((rows, heads), -np.inf)
    at, nk = 0, 0
    for i, (ql, kl) in enumerate(zip(q_lens, k_lens)):
        ks = nk if k_starts is None else k_starts[i]
        for h in range(heads):
            s = q[at:at + ql, h] @ k[ks:ks + kl, h // group].T * scale
            if causal:
                t, j = np.arange(ql)[:, None], np.arange(kl)[None]
                s = np.where(j <= kl - ql + t, s, -np.inf)
            see = np.isfinite(s).any(axis=1) if kl else np.zeros(ql, dtype=bool)
            if not see.any():
                continue
            s = s[see]
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(axis=1, keepdims=True)
            p /= total
            r = at + np.nonzero(see)[0]
            out[r, h] = p @ v[ks:ks + kl, h // group]
            weight[r, h] = p @ np.abs(v[ks:ks + kl, h // group])
            lse[r, h] = (top + np.log(total))[:, 0]
        at += ql
        nk += kl
    return out, lse, weight
