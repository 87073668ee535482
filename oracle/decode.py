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
                    bad=None, k_terms=None, v_terms=None, q_step=0.0):
    """q [batch][q_heads][d]; caches [page][slot][kv_head][d] (scales applied).  Returns out,
    lse and the bounds of both before the output's rounding.  k_terms, v_terms: the sum of the sizes
    of the terms that make up each element (its own size where it is one term).  q_step: how far each
    element of q may be off, relative to its head's largest."""
    k_terms = np.abs(k_cache) if k_terms is None else k_terms
    v_terms = np.abs(v_cache) if v_terms is None else v_terms
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
        k_size, v_size = k_terms[at], v_terms[at]
        for h in range(q_heads):
            kh, vh = k[:, h // per], v[:, h // per]
            s = kh @ q[b, h] * scale
            s_err = (k_size[:, h // per] @ np.abs(q[b, h])) * abs(scale) * (d + 8) * E32
            s_err = s_err + np.abs(s) * 8 * E32
            s_err = s_err + q_step * np.abs(q[b, h]).max() * k_size[:, h // per].sum(1) * abs(scale)
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
            out_err[b, h] = rel * (p @ v_size[:, h // per]) / total
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


def head_norm(x, weight, eps):
    """x [tokens][heads][d] with each head normed, and the bound of each element."""
    d = x.shape[-1]
    y = x / np.sqrt((x * x).sum(axis=-1, keepdims=True) / d + eps) * weight
    # half of the mean's relative error, a root, a quotient and three products
    return y, np.abs(y) * ((d + 8) / 2 + 8) * E32


def spread(err, half, interleaved):
    """What a rotation makes of its input's bounds."""
    out = err.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        out[..., a] = out[..., b] = err[..., a] + err[..., b]
    return out


def unpack4(codes):
    """[...][d] codes from bytes [...][d / 2], the even element in the low half."""
    return np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)


def values4(codes, pairs):
    """What bytes [...][d / 2] and pairs [...][groups][2] stand for, in 64 bits."""
    c = unpack4(codes).astype(np.float64)
    c = c.reshape(*c.shape[:-1], pairs.shape[-2], -1)
    with np.errstate(invalid="ignore"):
        return (pairs[..., 1:] + pairs[..., :1] * c).reshape(*codes.shape[:-1], -1)


def terms4(codes, pairs, shift=16):
    """The sizes of the terms of values4's elements as the attention adds them: V's code is taken
    16 larger, and 16 scales off again; K's as it is, with a shift of 0."""
    c = unpack4(codes).astype(np.float64)
    c = c.reshape(*c.shape[:-1], pairs.shape[-2], -1)
    p = np.abs(pairs)
    return (p[..., 1:] + p[..., :1] * (c + 2 * shift)).reshape(*codes.shape[:-1], -1)


def e4m3(x):
    """The nearest numbers with four significant bits, ties to even, of multiples of 2^-9 up to 448."""
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.rint(x / step) * step


def held4(q, pieces):
    """What the 4-bit attention's products take of the elements q [...][n] of a query head's group, in
    so many pieces of four bits."""
    top = np.abs(q).max(axis=-1, keepdims=True) * (256 / 248)
    unit = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(top, 2.0 ** -140))) - 7, -110)
    held, left = np.zeros_like(q), q / unit
    for i in range(pieces):
        piece = e4m3(np.rint(left * 8) / 8)
        held, left = held + piece * 16.0 ** -i, (left - piece) * 16
    return held * unit


def paged_attention4(q, k, v, table, lens, scale, window=0, softcap=0.0, keep=None, pieces=3):
    """paged_attention over a 4-bit cache, k and v pairs of (codes, pairs): the formula's out and lse
    for the q that the products take (held4), and the bounds of fp32 arithmetic on both."""
    (kc, kp), (vc, vp) = ((unpack4(c).astype(np.float64), p) for c, p in (k, v))
    groups = kp.shape[-2]
    k_size, v_size = terms4(*k, shift=0), terms4(*v)
    values = values4(*v)
    batch, q_heads, d = q.shape
    pages, page_size, kv_heads = kc.shape[:3]
    per = q_heads // kv_heads
    out, out_err = np.zeros_like(q), np.zeros_like(q)
    lse, lse_err = np.full((batch, q_heads), -np.inf), np.zeros((batch, q_heads))
    for b in range(batch):
        j = np.arange(max(0, lens[b] - window) if window else 0, lens[b])
        if keep is not None:
            j = j[keep[b][j] != 0]
        page = table[b][j // page_size]
        at = page[(page >= 0) & (page < pages)], (j % page_size)[(page >= 0) & (page < pages)]
        n = len(at[0])
        if n == 0:
            continue
        for h in range(q_heads):
            kh = h // per
            parts = q[b, h].reshape(groups, -1)
            dots = np.einsum("jge,ge->jg", kc[at][:, kh].reshape(n, groups, -1), held4(parts, pieces))
            pair = kp[at][:, kh]
            s = (pair[..., 0] * dots + pair[..., 1] * parts.sum(axis=1)).sum(axis=1) * scale
            # The codes' products are whole; a lane adds a quarter of a head's q in turn.
            s_err = (k_size[at][:, kh] @ np.abs(q[b, h])) * abs(scale) * (d / 4 + 12) * E32
            s_err = s_err + np.abs(s) * 8 * E32
            if softcap:
                s = softcap * np.tanh(s / softcap)
                s_err = s_err + np.minimum(np.abs(s) * 12, softcap * 8) * E32
            s_err = s_err.max() + np.abs(s).max() * 8 * E32  # to base 2 and back
            p = np.exp(s - s.max())
            total = p.sum()
            lse[b, h] = np.log(total) + s.max()
            lse_err[b, h] = s_err + (n / 32 + 16) * E32 * (1 + abs(lse[b, h]))
            out[b, h] = p @ values[at][:, kh] / total
            # p is off by its score's error; p times the scale keeps 16 bits where it meets 16 + code
            cut = (vp[at][:, kh][..., :1] * (vc[at][:, kh].reshape(n, groups, -1) + 16)).reshape(n, d)
            out_err[b, h] = ((2 * s_err + (n + 8) * E32) * (p @ v_size[at][:, kh])
                             + 2.0 ** -16 * (p @ np.abs(cut))) / total
    return out, lse, out_err, lse_err


def check_quantized4(x, err, codes, pairs, half_step, tiny):
    """Whether bytes and pairs are what x [...][d], known to err, may be stored as: the offset its
    group's smallest value and the scale a fifteenth of its range, each within a rounding, and
    every code the nearest one by the pair that is stored.  half_step, tiny: of the pairs' type."""
    groups = pairs.shape[-2]
    x = x.reshape(*x.shape[:-1], groups, -1)
    err = np.broadcast_to(err, codes.shape[:-1] + (codes.shape[-1] * 2,)).reshape(x.shape)
    code = unpack4(codes).reshape(x.shape).astype(np.float64)
    scale, offset = pairs[..., :1], pairs[..., 1:]
    low, high, e = (f(v, axis=-1, keepdims=True) for f, v in ((np.min, x), (np.max, x),
                                                              (np.max, err)))
    e = e + tiny
    assert (np.abs(offset - low) <= np.abs(low) * half_step * 1.01 + e).all()
    span = (high - low) / 15
    # the quotient's own rounding, and both ends' errors
    assert (np.abs(scale - span) <= span * (half_step * 1.01 + 4 * E32) + e).all()
    off = x - (offset + scale * code)
    # half a step, the errors of x, its difference and quotient (a code of up to 16 in fp32)
    room = scale * (0.5 + 64 * E32) + err + (np.abs(x) + np.abs(offset)) * 2 * E32
    fine = (np.abs(off) <= room) | ((code == 0) & (off < 0)) | ((code == 15) & (off > 0))
    assert (fine | (scale == 0)).all() and (code[np.broadcast_to(scale == 0, code.shape)] == 0).all()


def sample(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The token of one row of logits (64 bits), the log of its share, whether the token is certain,
    and how far the share may be off, relative to itself.

    n values of p, each off by half a step of 2^-44, make sums that are off by n 2^-45 of the largest p
    at worst, which the whole holds at least once; a share of the whole is off by twice that, and
    2^-40 is left for p's own error and that of the sums here."""
    n = len(z)
    eps = n * 2.0 ** -44 + 2.0 ** -40
    if np.isnan(z).any() or z.max() == -np.inf:
        return -1, np.nan, True, 0.0
    order = np.lexsort((np.arange(n), -z))
    if not temperature > 0:
        return int(order[0]), 0.0, True, 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        x = np.where(z == z.max(), 0.0, (z - z.max()) / temperature)
    x[z == -np.inf] = -np.inf
    p = np.exp(x)
    keep, slack = order, 8 * eps * p.sum()
    if 0 < top_k < n:
        keep = keep[:top_k]
    if top_p < 1:
        upto = np.cumsum(p[keep])
        want, off = max(top_p, 0.0) * upto[-1], eps * upto[-1] if top_p > 0 else 0.0
        low, count, high = (min(int(np.searchsorted(upto, w)) + 1, len(keep))
                            for w in (want - off, want, want + off))
        slack += upto[high - 1] - upto[low - 1]  # tokens that may stay or not
        keep = keep[:count]
    if min_p > 0:
        keep = keep[(p[keep] >= min_p) | (np.arange(len(keep)) == 0)]  # the first in any case
    keep = np.sort(keep[p[keep] > 0])
    upto = np.cumsum(p[keep])
    want = min(max(u, 0.0), 1 - 2.0 ** -53) * upto[-1]
    i = min(int(np.searchsorted(upto, want, side="right")), len(keep) - 1)
    certain = len(keep) == 1 or np.abs(upto[:-1] - want).min() > slack
    return int(keep[i]), float(x[keep[i]] - np.log(upto[-1])), bool(certain), slack / upto[-1]
