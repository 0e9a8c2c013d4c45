"""Verification of drafted tokens in float64, row by row (test infrastructure only)."""
from __future__ import annotations

import numpy as np

LOWEST = -float(np.finfo(np.float32).max)


def softmax(row, temperature):
    """Probabilities, and the scaled logits; None where nothing has any."""
    by = float(np.float32(1) / np.float32(temperature)) if temperature > 0 else 1.0
    x = np.where(np.isnan(row), LOWEST, np.clip(np.asarray(row, np.float64) * min(by, -LOWEST), LOWEST, -LOWEST))
    if x.max() <= LOWEST:
        return None, x
    e = np.exp(x - x.max())
    return e / e.sum(), x


def verify(start, logits, draft, u_accept, u_token, temperature, draft_logits=None):
    """For each sequence a dict: accepted and token; `near`: how near the closest of its decisions about acceptance was
    (|u q / p - 1|); for a drawn token the weights, their sum's target, and the size of p and q they come from."""
    out = []
    prob = np.full(len(logits), np.nan)
    for i in range(len(start) - 1):
        r0, r1 = int(start[i]), int(start[i + 1])
        if r0 == r1:
            out.append(dict(accepted=0, token=-1, near=np.inf))
            continue
        t = float(temperature[i])
        greedy = not t > 0
        near, accepted, refused = np.inf, 0, False
        for r in range(r0, r1 - 1):
            d = int(draft[r])
            p, x = softmax(logits[r], t)
            inside = 0 <= d < logits.shape[1]
            prob[r] = p[d] if p is not None and inside else 0.0
            if refused:
                continue
            if greedy:
                yes = p is not None and d == int(np.argmax(x))
            else:
                qd = 1.0
                if draft_logits is not None:
                    q, _ = softmax(draft_logits[r], t)
                    qd = q[d] if q is not None and inside else 0.0
                a, b = float(u_accept[r]) * qd, prob[r]
                yes = a < b
                near = min(near, abs(a - b) / max(a, b, 1e-300))
            if yes:
                accepted += 1
            else:
                refused = True
        r = r0 + accepted
        p, x = softmax(logits[r], t)
        one = dict(accepted=accepted, near=near, token=-1)
        if p is not None and greedy:
            one["token"] = int(np.argmax(x))
        elif p is not None:
            w, size = p.copy(), p.sum()
            if refused and draft_logits is None:
                if 0 <= int(draft[r]) < len(w):
                    w[int(draft[r])] = 0
            elif refused:
                q, _ = softmax(draft_logits[r], t)
                if q is not None:
                    w, size = np.maximum(p - q, 0), 2.0
            if w.sum() <= 0:
                w = p.copy()
            c = np.cumsum(w)
            one.update(weights=w, cum=c, target=float(u_token[i]) * c[-1], size=size, reach=float(np.abs(x).max()))
            one["token"] = int(np.flatnonzero(c > one["target"])[0]) if (c > one["target"]).any() else int(np.flatnonzero(w)[-1])
        out.append(one)
    return out, prob


def probabilities(row, temperature):
    """Probabilities in 64 bits of the fp32 products that the call defines, and those products; temperature > 0."""
    with np.errstate(over="ignore"):
        by = min(np.float32(1) / np.float32(temperature), np.float32(-LOWEST))
        x = np.asarray(row, np.float32) * by
    x = np.where(np.isnan(x), LOWEST, np.clip(x.astype(np.float64), LOWEST, -LOWEST))
    e = np.exp(x - x.max())
    return e / e.sum(), x
