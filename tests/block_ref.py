"""Plain references of the operators around the experts, in 64 bits on the CPU
(NumPy; shared by the tests, not collected by pytest)."""
from __future__ import annotations

import numpy as np
import torch

LOWEST = np.float32(-3.4028234663852886e38)
U = 2.0 ** -24        # float32 rounding unit


def f64(t):
    """A tensor's values in float64 (bf16 included)."""
    return t.detach().cpu().double().numpy()


def bf16_rne(a):
    """float32 values -> the nearest bf16's value, by torch's conversion."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).double().numpy()


def norm(x, r, w, eps):
    """h, y in float64 and bf16(h) (one float32 sum, rounded once)."""
    h = f64(x) if r is None else f64(x) + f64(r)
    hb = f64(x) if r is None else f64((x.cpu().float() + r.cpu().float()).to(torch.bfloat16))
    with np.errstate(all="ignore"):
        y = h * f64(w) / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h, y, hb


def norm_rel(H):
    """Relative error of the float32 y: each thread adds up to 32 squares, then 6 steps across
    the wavefront and at most 16 wavefronts' sums, all of positive terms (halved by the root); the
    bf16 inputs' sum, product, quotient, root and two products round once each."""
    return (0.5 * (32 + 6 + 16) + 6) * U


def quant_int8(x32):
    """The definition in float32: codes and scales of finite rows."""
    amax = np.abs(x32).max(1).astype(np.float32)
    s = np.maximum(amax / np.float32(127.0), np.float32(2.0 ** -126)).astype(np.float32)
    inv = (np.float32(1.0) / s).astype(np.float32)
    q = np.clip(np.rint((x32 * inv[:, None]).astype(np.float32)), -127, 127)
    return q.astype(np.int8), s


def int8_matmul(q, sx, w, sw):
    """Exact sums (whole numbers far below 2^53), then the three factors in float32."""
    s = q.astype(np.float64) @ w.astype(np.float64).T
    return (s.astype(np.float32) * sx.astype(np.float32)[:, None]) * sw.astype(np.float32)


def route(logits, bias, K, G, KG, score, group, renorm, scaling):
    """Token by token, expert by expert."""
    T, E = logits.shape
    per = E // G
    idx = np.full((T, K), -1, np.int32)
    wt = np.zeros((T, K), np.float64)
    for t in range(T):
        l = logits[t].astype(np.float64)
        masked = logits[t] <= LOWEST
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-l))
            else:
                live = l[~masked]
                top = np.fmax.reduce(live) if live.size else 0.0
                e = np.where(masked, 0.0, np.exp(l - top))
                s = e / e[~masked].sum() if live.size else e
            s = s.astype(np.float32)
            key = s + bias if bias is not None else s.copy()
        masked = masked | (key == -np.inf)

        def ranked(items):   # (value, index): NaN last, larger first, lower index first
            return sorted(items, key=lambda i: (np.isnan(i[0]), 0.0 if np.isnan(i[0]) else -i[0],
                                                i[1]))

        live_groups = []
        for g in range(G):
            best = ranked([(key[e], e) for e in range(g * per, (g + 1) * per) if not masked[e]])
            if best:
                w = best[0][0]
                if group == "top2" and len(best) > 1:
                    with np.errstate(all="ignore"):
                        w = np.float32(w + best[1][0])
                live_groups.append((w, g))
        keep = {g for _, g in ranked(live_groups)[:KG]}
        chosen = ranked([(key[e], e) for e in range(E) if not masked[e] and e // per in keep])[:K]
        ids = [e for _, e in chosen]
        idx[t, :len(ids)] = ids
        w = s[ids].astype(np.float64)
        if renorm:
            total = 0.0
            for v in w:
                total += v
            w = w * 0.0 if total == 0.0 else w / total
        wt[t, :len(ids)] = w * np.float64(np.float32(scaling))
    return idx, wt
