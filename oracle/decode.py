"""Plain 64-bit forms of the decode-step operators, written from their formulas (numpy).

Every function returns the value and a bound on what fp32 arithmetic may add to the one
rounding of the output type: sums of n terms t_i are allowed (n + 8) 2^-24 sum |t_i|.
"""

import numpy as np

E32 = 2.0 ** -24


def add_rms_norm(x, delta, weight, eps):
    """(y, s) and the relative bound of y."""
    s = x + delta if delta is not None else x
    mean = (s * s).sum(axis=1, keepdims=True) / s.shape[1]
    return s / np.sqrt(mean + eps) * weight, s


def rotate(x, positions, inv_freq, sections, interleaved):
    """x [tokens][heads][d] with its leading pairs turned; the bound of each element."""
    y, err = x.copy(), np.zeros_like(x)
    half = len(inv_freq)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = (positions[axis[i]].astype(np.float64) * float(inv_freq[i]))[:, None]
        c, s = np.cos(angle), np.sin(angle)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        # sine and cosine to 2^-21 (the reduced angle, up to pi, is rounded to fp32)
        err[..., a] = err[..., b] = (abs(x[..., a]) + abs(x[..., b])) * 2.0 ** -20
    return y, err


def paged_attention(q, k_cache, v_cache, table, lens, scale, window=0, softcap=0.0, keep=None,
                    bad=None):
    """q [batch][q_heads][d]; caches [page][slot][kv_head][d] (scales applied).  Returns out,
    lse and the bounds of both before the output's rounding."""
    batch, q_heads, d = q.shape
    pages, page_size, kv_heads = k_cache.shape[:3]
    per = q_heads // kv_heads
    out, out_err = np.zeros_like(q), np.zeros_like(q)
    lse, lse_err = np.full((batch, q_heads), -np.inf), np.zeros((batch, q_heads))
    for b in range(batch):
        live = []
        for j in range(max(0, lens[b] - window) if window else 0, lens[b]):
            page = table[b][j // page_size]
            if 0 <= page < pages and (keep is None or keep[b][j]):
                live.append((page, j % page_size))
        if not live:
            continue
        at = tuple(np.array(live).T)
        k, v = k_cache[at], v_cache[at]  # [n][kv_heads][d]
        for h in range(q_heads):
            kh, vh = k[:, h // per], v[:, h // per]
            s = kh @ q[b, h] * scale
            s_err = (np.abs(kh) @ np.abs(q[b, h])) * abs(scale) * (d + 8) * E32
            s_err = s_err + np.abs(s) * 8 * E32
            if softcap:
                s = softcap * np.tanh(s / softcap)
                # tanh is right to its own size, and its last product to the cap's
                s_err = s_err + np.minimum(np.abs(s) * 12, softcap * 8) * E32
            s_err = s_err.max() + np.abs(s).max() * 8 * E32  # to base 2 and back
            p = np.exp(s - s.max())
            total = p.sum()
            lse[b, h] = np.log(total) + s.max()
            lse_err[b, h] = s_err + (len(live) / 32 + 16) * E32 * (1 + abs(lse[b, h]))
            out[b, h] = p @ vh / total
            # p is off by its score's error and keeps 16 bits
            rel = 2 * s_err + 2.0 ** -16 + (len(live) + 8) * E32
            out_err[b, h] = rel * (p @ np.abs(vh)) / total
    return out, lse, out_err, lse_err


def moe_layer(x, router, gate, up, down, top_k, renormalize, scale, residual, half_step):
    """x [tokens][hidden], weights [expert][k][n].  Returns y, ids, weights and the bound of y
    before its rounding; half_step: half the relative step of the type of the activation
    between the products."""
    tokens = x.shape[0]
    logits = x @ router.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    e = np.exp(logits - logits.max(axis=1, keepdims=True))
    w = np.take_along_axis(e, ids, 1)
    w = scale * w / (w.sum(axis=1, keepdims=True) if renormalize else e.sum(axis=1, keepdims=True))
    y = np.zeros_like(x) if residual is None else residual.copy()
    err = np.abs(y) * E32
    k1, k2 = gate.shape[1], down.shape[1]
    for t in range(tokens):
        for j in range(top_k):
            i = ids[t, j]
            g, u = x[t] @ gate[i], x[t] @ up[i]
            dg = (np.abs(x[t]) @ np.abs(gate[i])) * (k1 + 8) * E32
            du = (np.abs(x[t]) @ np.abs(up[i])) * (k1 + 8) * E32
            silu = g / (1 + np.exp(-g))
            h = silu * u
            # |silu'| <= 1.1; the hardware exp and reciprocal are good to a few units
            dh = 1.1 * np.abs(u) * dg + np.abs(silu) * du + np.abs(h) * (half_step + 16 * E32)
            dh = dh + 2.0 ** -25  # fp16's smallest steps
            y[t] += w[t, j] * (h @ down[i])
            err[t] += w[t, j] * ((dh + np.abs(h) * (k2 + 16) * E32) @ np.abs(down[i]))
    return y, ids, w, err
