"""fp64 CPU oracle of the check of drafted tokens. Plain numpy from the
definitions in include/q4dec_rollout.h; shares no code with the HIP path."""
from __future__ import annotations

import numpy as np


def distribution(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, cap=30.0):
    """(probabilities [V], border): what a row's filters leave, all zero if no token may be drawn; border: the
    distance of the top-p border to the nearest running sum it is compared with, as a share of the whole."""
    z = np.asarray(z, dtype=np.float64)
    out = np.zeros(len(z))
    live = np.nonzero(z > -np.inf)[0]
    if not live.size:
        return out, 1.0
    order = live[np.argsort(-z[live], kind="stable")]
    if not temperature > 0:
        out[order[0]] = 1.0
        return out, 1.0
    x = cap * np.tanh(z[order] / cap) if cap > 0 else z[order]
    if np.isfinite(x[0]):
        w = np.where(z[order] == z[order[0]], 1.0, np.exp((x - x[0]) / temperature))
    else:
        w = (z[order] == z[order[0]]).astype(np.float64)
    if 0 < top_k < len(z):
        order, w = order[:top_k], w[:top_k]
    stay, border = np.ones(len(w), bool), 1.0
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        stay = before < max(top_p, 0.0) * w.sum()
        if len(w) > 1:
            border = np.abs(before[1:] - top_p * w.sum()).min() / w.sum()
    if min_p > 0:
        stay &= w >= min(min_p, 1.0)
    stay[0] = True
    out[order[stay]] = w[stay] / w[stay].sum()
    return out, border


def check(logits, draft_logits, drafts, u, u_draw, cap=30.0, draft_cap=30.0, **filters):
    """One sequence: logits [n, V], drafts [n] (the last one not looked at), draft_logits [n, V] or None.
    Returns (tokens, probabilities of them, border): the drafts that stay and the new token (-1, NaN where none
    may be drawn); border: the least distance of a decision to its other outcome: of u q(x) and p(x) relative to
    p(x), of a running sum and what it is compared with as a probability."""
    n, tokens, probs, border = len(logits), [], [], 1.0
    unit = lambda v: min(float(v), 1 - 2.0 ** -24) if v > 0 else 0.0  # noqa: E731
    for i in range(n):
        p, edge = distribution(logits[i], cap=cap, **filters)
        border = min(border, edge)
        rest = p
        if i < n - 1:
            x = int(drafts[i])
            there = 0 <= x < len(p)
            q = np.zeros(len(p))
            if draft_logits is not None:
                q, edge = distribution(draft_logits[i], cap=draft_cap, **filters)
                border = min(border, edge)
            elif there:
                q[x] = 1.0
            px, qx = (p[x], q[x]) if there else (0.0, 0.0)
            if px > 0:
                border = min(border, abs(unit(u[i]) * qx - px) / px)
            if there and unit(u[i]) * qx < px:
                tokens.append(x)
                probs.append(px)
                continue
            rest = np.maximum(p - q, 0.0)
            if not rest.sum() > 0:
                rest = p
            else:  # a rest of about the rounding of p and q may as well be none
                border = min(border, rest.sum())
        if not p.any():
            return tokens + [-1], probs + [np.nan], border
        run = np.cumsum(rest)
        at = (unit(u_draw) if not u_draw >= 1 else 1.0) * run[-1]
        new = min(int(np.searchsorted(run, at, side="right")), int(np.nonzero(rest)[0][-1]))
        if np.count_nonzero(rest) > 1 and not u_draw >= 1:
            inner = run[run < run[-1]]
            border = min(border, np.abs(inner - at).min() if len(inner) else 1.0)
        return tokens + [new], probs + [p[new]], border
    return tokens, probs, border
