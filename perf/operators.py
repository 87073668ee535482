"""What is measured of the decode-step operators: RMS norm with a residual add, rotary
positions with the paged cache write, single-token attention over that cache, and the
mixture-of-experts layer of a few tokens on quantized weights.

`run` computes an operator in plain torch operations, or, where `own` is set, through
weight_only_quantized_gemm_amd.decode.  `exact` gives the definition's value in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
EPS = 1e-5


def listed():
    return [
        # one user's first answer token after a short prompt: pure latency
        dict(name="attn_short", op="attn", type="fp16", cache="same", batch=1, hq=32, hkv=8, d=128,
             page=16, max_len=128, ragged=False, window=0, softcap=0.0, keep=False, order="hnd"),
        # a serving batch of ordinary chats, four query heads to a KV head
        dict(name="attn_batch", op="attn", type="bf16", cache="same", batch=16, hq=32, hkv=8, d=128,
             page=16, max_len=4096, ragged=True, window=0, softcap=0.0, keep=False, order="hnd"),
        # one long document: few rows, the work has to be split over the length
        dict(name="attn_long", op="attn", type="bf16", cache="same", batch=1, hq=32, hkv=8, d=128,
             page=64, max_len=131072, ragged=False, window=0, softcap=0.0, keep=False, order="nhd"),
        # a full batch on an E4M3 cache with evicted positions
        dict(name="attn_full_e4m3", op="attn", type="bf16", cache="e4m3", batch=64, hq=64, hkv=8,
             d=128, page=32, max_len=8192, ragged=True, window=0, softcap=0.0, keep=True, order="hnd"),
        # one query head to a KV head, odd sizes, a sliding window and capped scores
        dict(name="attn_odd", op="attn", type="fp16", cache="same", batch=7, hq=12, hkv=12, d=80,
             page=24, max_len=3001, ragged=True, window=1000, softcap=30.0, keep=False, order="nhd"),
        # the append of one decoded token
        dict(name="append_token", op="append", type="bf16", cache="same", tokens=1, hq=32, hkv=8,
             d=128, rot=128, page=16, axes=1, interleaved=False, order="hnd"),
        # a prompt chunk with image positions (three axes) into an E4M3 cache
        dict(name="append_chunk", op="append", type="fp16", cache="e4m3", tokens=2048, hq=32, hkv=8,
             d=128, rot=128, page=32, axes=3, interleaved=False, order="hnd"),
        # the norm before a decode product, with the residual add
        dict(name="norm_token", op="norm", type="fp16", rows=1, n=4096, delta=True),
        # the norm of a long prefill
        dict(name="norm_prefill", op="norm", type="bf16", rows=8192, n=8192, delta=True),
        # one token through two of eight large experts
        dict(name="moe_one", op="moe", type="fp16", weights="u4b8", tokens=1, experts=8, top_k=2,
             hidden=4096, inter=14336, group=128, renorm=True, residual=True),
        # a few users' tokens, zero points
        dict(name="moe_few", op="moe", type="bf16", weights="u4", tokens=4, experts=8, top_k=2,
             hidden=4096, inter=14336, group=128, renorm=True, residual=True),
        # sixteen tokens over many small experts
        dict(name="moe_fine", op="moe", type="fp16", weights="u4b8", tokens=16, experts=64, top_k=8,
             hidden=2048, inter=1024, group=64, renorm=False, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "norm", "moe", "moe"])
    ty = rng.choice(["fp16", "bf16"])
    if op == "attn":
        hkv = rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([64, 72, 96, 128, 128, 192, 256])
        batch = _log(rng, 1, 64)
        room = 64 * 8192 * 8 * 128 // (4 * batch * hkv * d)  # a quarter of the largest listed cache
        return dict(op=op, type=ty, cache=rng.choice(["same", "e4m3"]), batch=batch,
                    hq=hkv * rng.choice([1, 2, 3, 4, 5, 8, 16]), hkv=hkv, d=d,
                    page=rng.choice([1, 8, 16, 24, 32, 64, 128]),
                    max_len=_log(rng, 1, min(100000, room)), ragged=rng.random() < 0.7,
                    window=rng.choice([0, 0, 0, 777]), softcap=rng.choice([0.0, 0.0, 25.0]),
                    keep=rng.random() < 0.3, order=rng.choice(["hnd", "nhd"]))
    if op == "append":
        hkv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 80, 128, 256])
        return dict(op=op, type=ty, cache=rng.choice(["same", "e4m3"]),
                    tokens=_log(rng, 1, min(2048, 3500000 // (hkv * d))),
                    hq=hkv * rng.choice([1, 4, 7]), hkv=hkv, d=d,
                    rot=rng.choice([d, d // 2, 0]), page=rng.choice([1, 16, 24, 64]),
                    axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.4,
                    order=rng.choice(["hnd", "nhd"]))
    if op == "norm":
        return dict(op=op, type=ty, rows=_log(rng, 1, 8192), n=8 * _log(rng, 1, 1024),
                    delta=rng.random() < 0.7)
    weights = rng.choice(["u4b8", "u4", "e4m3"])
    experts, hidden = rng.choice([1, 5, 8, 32, 64]), 256 * rng.randint(1, 8)
    blocks = min(16, 64 * 2048 * 8 // (experts * hidden))  # at most the listed many-expert layer
    return dict(op=op, type=ty, weights=weights, tokens=rng.randint(1, 16),
                experts=experts, top_k=min(experts, rng.choice([1, 2, 3, 6, 8])),
                hidden=hidden, inter=128 * _log(rng, 1, blocks),
                group=128 if weights == "e4m3" else rng.choice([32, 64, 128]),
                renorm=rng.random() < 0.5, residual=rng.random() < 0.7)


# ---- inputs ------------------------------------------------------------------------------


def _normal(g, shape, dtype, sd=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * sd).to(dtype)


def _pages(s, storage):
    """The logical [page][slot][head][d] view of a cache stored head-major or slot-major."""
    return storage.transpose(1, 2) if s["order"] == "hnd" else storage


def _bytes(x):
    """E4M3 tensors as bytes (copied and indexed as they are), others unchanged."""
    return x.view(torch.uint8) if x.dtype == E4M3 else x


def _cache(g, s, pages):
    """K and V storage for `pages` pages, and the scale per KV head of an E4M3 cache."""
    shape = ((pages, s["hkv"], s["page"], s["d"]) if s["order"] == "hnd"
             else (pages, s["page"], s["hkv"], s["d"]))
    s["k_scale"] = s["v_scale"] = None
    k, v = _normal(g, shape, TYPES[s["type"]]), _normal(g, shape, TYPES[s["type"]])
    if s["cache"] == "e4m3":
        s["k_scale"] = torch.rand(s["hkv"], generator=g, device=DEV) * 0.02 + 0.005
        s["v_scale"] = torch.rand(s["hkv"], generator=g, device=DEV) * 0.02 + 0.005
        k, v = (k.float() * 60).to(E4M3), (v.float() * 60).to(E4M3)
    s["k_cache"], s["v_cache"] = _pages(s, k), _pages(s, v)


def _inputs_attn(s, g):
    b, page, top = s["batch"], s["page"], s["max_len"]
    lens = torch.full((b,), top, dtype=torch.int64, device=DEV)
    if s["ragged"]:
        lens = torch.randint(0, top + 1, (b,), generator=g, device=DEV)
        lens[-1] = 1
        lens[0] = top
    per = -(-top // page)
    # every sequence's pages lie anywhere in the pool; one page more than is used
    order = torch.randperm(b * per + 1, generator=g, device=DEV)[: b * per]
    s["table"] = order.view(b, per).to(torch.int32)
    _cache(g, s, b * per + 1)
    # what lies behind a sequence's end is whatever was there: here NaN, on the last page
    last = s["table"].long().gather(1, ((lens - 1).clamp(min=0) // page)[:, None]).flatten()
    behind = (torch.arange(page, device=DEV) > ((lens - 1) % page)[:, None]) & (lens > 0)[:, None]
    for name in ("k_cache", "v_cache"):
        one = _bytes(s[name])[last]
        one[behind] = 0x7F if s[name].dtype == E4M3 else float("nan")
        _bytes(s[name])[last] = one
    s["lens"] = lens.to(torch.int32)
    s["q"] = _normal(g, (b, s["hq"], s["d"]), TYPES[s["type"]])
    s["scale"] = 1.0 / math.sqrt(s["d"])
    s["mask"] = None
    if s["keep"]:
        s["mask"] = (torch.rand((b, top), generator=g, device=DEV) > 0.3).to(torch.uint8)


def _inputs_append(s, g):
    t, d, ty = s["tokens"], s["d"], TYPES[s["type"]]
    qkv = _normal(g, (t, (s["hq"] + 2 * s["hkv"]) * d), ty)  # one fused projection's rows
    q, k, v = qkv.split([s["hq"] * d, s["hkv"] * d, s["hkv"] * d], dim=1)
    s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in (q, k, v))
    pages = -(-t // s["page"]) + 3
    _cache(g, s, pages)
    slots = torch.randperm(pages * s["page"], generator=g, device=DEV)[:t]
    if t > 4:
        slots[t // 2] = -1  # a padding token
    s["slots"] = slots
    base = torch.randint(0, 200000, (s["axes"], 1), generator=g, device=DEV)
    s["positions"] = (base + torch.randint(0, 4096, (s["axes"], t), generator=g,
                                           device=DEV)).to(torch.int32)
    half = s["rot"] // 2
    s["inv_freq"] = (torch.exp(torch.arange(half, device=DEV, dtype=torch.float64)
                               * (-math.log(500000.0) / max(1, half)))).float()
    cut = [half * i // s["axes"] for i in range(s["axes"] + 1)]
    s["sections"] = [cut[i + 1] - cut[i] for i in range(s["axes"])]
    s["q_out"] = torch.empty((t, s["hq"], d), dtype=ty, device=DEV)


def _inputs_norm(s, g):
    ty = TYPES[s["type"]]
    s["x"] = _normal(g, (s["rows"], s["n"]), ty, 3.0)
    s["w"] = _normal(g, (s["n"],), ty, 0.2) + 1
    s["d"] = _normal(g, (s["rows"], s["n"]), ty) if s["delta"] else None


def _bank(s, g, k, n):
    """Quantized weights [experts] of k x n: words, scales, zero-point words."""
    e, ty, fp8 = s["experts"], TYPES[s["type"]], s["weights"] == "e4m3"
    per = 4 if fp8 else 8
    words = torch.randint(-2**31, 2**31, (e, k // per, n), generator=g, device=DEV,
                          dtype=torch.int64).to(torch.int32)
    if fp8:
        words &= ~0x08080808  # finite codes, at most 240
        scales = torch.rand((e, k // s["group"], n), generator=g, device=DEV) * 5e-4 + 1e-4
    else:
        scales = torch.rand((e, k // s["group"], n), generator=g, device=DEV) * 0.015 + 0.005
    zeros = None
    if s["weights"] == "u4":
        zeros = torch.randint(-2**31, 2**31, (e, k // s["group"], n // 8), generator=g, device=DEV,
                              dtype=torch.int64).to(torch.int32)
    return dict(words=words, scales=scales.to(ty), zeros=zeros)


def _inputs_moe(s, g):
    ty, h, i = TYPES[s["type"]], s["hidden"], s["inter"]
    s["x"] = _normal(g, (s["tokens"], h), ty)
    s["router"] = _normal(g, (s["experts"], h), ty, 1.5 / math.sqrt(h))
    s["gate"], s["up"], s["down"] = _bank(s, g, h, i), _bank(s, g, h, i), _bank(s, g, i, h)
    s["res"] = _normal(g, (s["tokens"], h), ty, 20.0) if s["residual"] else None


def _inputs(case, seed):
    s = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    dict(attn=_inputs_attn, append=_inputs_append, norm=_inputs_norm, moe=_inputs_moe)[s["op"]](s, g)
    return s


def _own_bank(torch_ops, s, names):
    def one(b, e):
        zeros = None if b["zeros"] is None else b["zeros"][e]
        return dict(qweight=b["words"][e], scales=b["scales"][e], zeros=zeros, group_size=s["group"])
    experts = []
    for e in range(s["experts"]):
        w = [one(s[n], e) for n in names]
        experts.append(w[0] if len(w) == 1 else dict(gate=w[0], up=w[1], group_size=s["group"]))
    return torch_ops.ExpertBank(experts, device=DEV, bf16=s["type"] == "bf16",
                                fp8=s["weights"] == "e4m3")


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from weight_only_quantized_gemm_amd import decode, torch_ops
    s["decode"] = decode
    if s["op"] in ("attn", "append"):
        s["paged"] = decode.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if s["op"] == "attn":
        s["plan"] = decode.PagedAttention(s["paged"], s["batch"], s["hq"], s["max_len"],
                                          dtype=TYPES[s["type"]], scale=s["scale"],
                                          window=s["window"], softcap=s["softcap"])
    if s["op"] == "moe":
        s["layer"] = decode.MoELayer(_own_bank(torch_ops, s, ("gate", "up")),
                                     _own_bank(torch_ops, s, ("down",)), s["router"], s["top_k"],
                                     renormalize=s["renorm"])
    return s


# ---- the plain forms -----------------------------------------------------------------------


def _plain_attn(s):
    b, hq, hkv, d, top = s["batch"], s["hq"], s["hkv"], s["d"], s["max_len"]
    idx = s["table"].long()
    k, v = (_bytes(s[n])[idx].view(s[n].dtype).flatten(1, 2)[:, :top].float()
            .permute(0, 2, 1, 3).contiguous() for n in ("k_cache", "v_cache"))
    if s["k_scale"] is not None:
        k = k * s["k_scale"][:, None, None]
        v = v * s["v_scale"][:, None, None]
    at = torch.arange(top, device=DEV)
    live = at < s["lens"][:, None]
    if s["window"]:
        live = live & (at >= (s["lens"] - s["window"])[:, None])
    if s["mask"] is not None:
        live = live & (s["mask"] != 0)
    q = s["q"].float().view(b, hkv, hq // hkv, d)
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    if s["softcap"]:
        scores = torch.tanh(scores / s["softcap"]) * s["softcap"]
    scores = torch.where(live[:, None, None, :], scores, float("-inf"))
    high = scores.amax(dim=3, keepdim=True)
    high = torch.where(high == float("-inf"), 0.0, high)
    p = torch.exp(scores - high)
    total = p.sum(dim=3, keepdim=True)
    v = torch.where(live[:, None, :, None], v, 0.0)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = (torch.log(total) + high).view(b, hq)
    return o.view(b, hq, d).to(TYPES[s["type"]]), lse


def _angles(s):
    axis = torch.repeat_interleave(torch.arange(s["axes"], device=DEV),
                                   torch.tensor(s["sections"], device=DEV),
                                   output_size=s["rot"] // 2)
    return s["positions"].double()[axis].t() * s["inv_freq"].double()  # [tokens][rot / 2]


def _rotated(x, s, cos, sin):
    x, half = x.float(), s["rot"] // 2
    turn, rest = x[..., : s["rot"]], x[..., s["rot"]:]
    if s["interleaved"]:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = turn[..., :half], turn[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _stored(x, scale, dtype):
    if scale is None:
        return x.to(dtype)
    return (x / scale[:, None]).clamp(-448.0, 448.0).to(E4M3)


def _plain_append(s):
    angles = _angles(s)
    cos, sin = angles.cos().float()[:, None], angles.sin().float()[:, None]
    q = _rotated(s["q"], s, cos, sin).to(s["q"].dtype)
    k = _stored(_rotated(s["k"], s, cos, sin), s["k_scale"], s["k"].dtype)
    v = _stored(s["v"].float(), s["v_scale"], s["v"].dtype)
    page, slot = s["slots"] // s["page"], s["slots"] % s["page"]
    real = s["slots"] >= 0
    _bytes(s["k_cache"])[page[real], slot[real]] = _bytes(k)[real]
    _bytes(s["v_cache"])[page[real], slot[real]] = _bytes(v)[real]
    return q, s["k_cache"], s["v_cache"]


def _plain_norm(s):
    x = s["x"].float()
    if s["d"] is not None:
        x = x + s["d"].float()
    y = x * torch.rsqrt(x.square().mean(dim=1, keepdim=True) + EPS) * s["w"].float()
    return y.to(s["x"].dtype), x.to(s["x"].dtype)


def _e4m3_value(byte):
    sign = 1.0 - 2.0 * (byte >> 7).float()
    e, m = ((byte >> 3) & 15).float(), (byte & 7).float()
    return sign * torch.where(e == 0, m * 2.0**-9, (8.0 + m) * torch.exp2(e - 10.0))


def _plain_weight(bank, s):
    """The dequantized weights [experts][k][n] in 32 bits."""
    words = bank["words"]
    e, rows, n = words.shape
    bits, count = (8, 4) if s["weights"] == "e4m3" else (4, 8)
    shift = torch.arange(count, device=DEV, dtype=torch.int32) * bits
    code = ((words[:, :, None, :] >> shift[:, None]) & (2**bits - 1)).view(e, rows * count, n)
    scale = bank["scales"].float()[:, :, None, :]
    if s["weights"] == "e4m3":
        w = _e4m3_value(code)
    elif bank["zeros"] is None:
        w = code.float() - 8
    else:
        z = (bank["zeros"][..., None] >> (torch.arange(8, device=DEV, dtype=torch.int32) * 4)) & 15
        w = (code.view(e, -1, s["group"], n) - z.flatten(2)[:, :, None, :]).float()
    return (w.view(e, -1, s["group"], n) * scale).view(e, rows * count, n)


def _plain_moe(s):
    # the logits in 64 bits: their order decides which experts run
    logits = torch.matmul(s["x"].double(), s["router"].double().t().contiguous())
    p = torch.softmax(logits, dim=1)
    order = torch.sort(p, dim=1, descending=True, stable=True)
    ids, w = order.indices[:, : s["top_k"]], order.values[:, : s["top_k"]]
    if s["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w.float()
    dense = torch.zeros_like(logits, dtype=torch.float32).scatter(1, ids, w)  # [tokens][experts]
    x = s["x"].float()
    g = torch.matmul(x, _plain_weight(s["gate"], s))
    u = torch.matmul(x, _plain_weight(s["up"], s))
    h = g / (1 + torch.exp(-g)) * u  # [experts][tokens][inter]
    y = (torch.matmul(h, _plain_weight(s["down"], s)) * dense.t()[:, :, None]).sum(dim=0)
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(s["x"].dtype), ids.to(torch.int32), w


# ---- one pass -------------------------------------------------------------------------------


def _own_attn(s):
    return s["plan"](s["q"], s["table"], s["lens"], keep=s["mask"], lse=True)


def _own_append(s):
    s["decode"].rope_append(s["q"], s["k"], s["v"], s["paged"], s["slots"],
                            positions=s["positions"], inv_freq=s["inv_freq"],
                            sections=s["sections"], interleaved=s["interleaved"],
                            q_out=s["q_out"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_norm(s):
    return s["decode"].add_rms_norm(s["x"], s["w"], EPS, delta=s["d"])


def _own_moe(s):
    y = s["layer"](s["x"], residual=s["res"])
    return y, s["layer"].ids[: s["tokens"]], s["layer"].weights[: s["tokens"]]


def run(state):
    if own:
        f = dict(attn=_own_attn, append=_own_append, norm=_own_norm, moe=_own_moe)
    else:
        f = dict(attn=_plain_attn, append=_plain_append, norm=_plain_norm, moe=_plain_moe)
    return f[state["op"]](state)


# ---- the least work ---------------------------------------------------------------------------


def _work_attn(c):
    mean = c["max_len"]
    if c["ragged"] and c["batch"] > 2:
        mean = (c["max_len"] * (1 + (c["batch"] - 2) / 2) + 1) / c["batch"]
    elif c["ragged"]:
        mean = 1 if c["batch"] == 1 else (c["max_len"] + 1) / 2
    if c["window"]:
        mean = min(mean, c["window"])
    if c["keep"]:
        mean *= 0.7
    size = 1 if c["cache"] == "e4m3" else 2
    live = mean * c["batch"]
    return dict(bytes=live * 2 * c["hkv"] * c["d"] * size + c["batch"] * c["hq"] * (4 * c["d"] + 4),
                flops=live * 4 * c["hq"] * c["d"])


def _work_append(c):
    size = 1 if c["cache"] == "e4m3" else 2
    return dict(bytes=c["tokens"] * c["d"] * (4 * c["hq"] + 2 * c["hkv"] * (2 + size)),
                flops=c["tokens"] * 3 * c["rot"] * (c["hq"] + c["hkv"]))


def _work_norm(c):
    n = c["rows"] * c["n"]
    return dict(bytes=n * 2 * (4 if c["delta"] else 2) + 2 * c["n"], flops=5 * n)


def _work_moe(c):
    active = c["experts"] * (1 - (1 - c["top_k"] / c["experts"]) ** c["tokens"])  # expected
    weights = 3 * c["hidden"] * c["inter"]
    size = 1.0 if c["weights"] == "e4m3" else 0.5
    extra = (2 + (0.5 if c["weights"] == "u4" else 0)) / c["group"]
    return dict(bytes=active * weights * (size + extra) + 2 * c["experts"] * c["hidden"]
                + c["tokens"] * c["hidden"] * (6 if c["residual"] else 4),
                flops=2 * c["tokens"] * c["top_k"] * weights)


def work(case):
    f = dict(attn=_work_attn, append=_work_append, norm=_work_norm, moe=_work_moe)
    return f[case["op"]](case)


# ---- the definition in 64 bits ------------------------------------------------------------------


def _exact_attn(s):
    out = torch.zeros((s["batch"], s["hq"], s["d"]), dtype=torch.float64, device=DEV)
    lse = torch.full((s["batch"], s["hq"]), float("-inf"), dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    for b in range(s["batch"]):
        pos = torch.arange(max(0, lens[b] - s["window"]) if s["window"] else 0, lens[b], device=DEV)
        if s["mask"] is not None:
            pos = pos[s["mask"][b, pos] != 0]
        if not len(pos):
            continue
        page = s["table"][b, pos // s["page"]].long()
        k, v = (_bytes(s[n])[page, pos % s["page"]].view(s[n].dtype).double()  # [len][hkv][d]
                for n in ("k_cache", "v_cache"))
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
        per = s["hq"] // s["hkv"]
        for h in range(s["hq"]):
            z = k[:, h // per] @ s["q"][b, h].double() * s["scale"]
            if s["softcap"]:
                z = s["softcap"] * torch.tanh(z / s["softcap"])
            lse[b, h] = torch.logsumexp(z, 0)
            out[b, h] = torch.exp(z - lse[b, h]) @ v[:, h // per]
    return out, lse


def _exact_append(s):
    half, t = s["rot"] // 2, s["tokens"]
    axis = [a for a in range(s["axes"]) for _ in range(s["sections"][a])]
    pair = [(2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half) for i in range(half)]
    q, k = s["q"].double(), s["k"].double().clone()
    q = q.clone()
    for x in (q, k):
        for i, (a, b) in enumerate(pair):
            angle = (s["positions"][axis[i]].double() * s["inv_freq"][i].double())[:, None]
            re, im = x[..., a].clone(), x[..., b].clone()
            x[..., a] = re * torch.cos(angle) - im * torch.sin(angle)
            x[..., b] = re * torch.sin(angle) + im * torch.cos(angle)
    v = s["v"].double()
    if s["k_scale"] is not None:
        k = (k / s["k_scale"].double()[:, None]).clamp(-448, 448)
        v = (v / s["v_scale"].double()[:, None]).clamp(-448, 448)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for i, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            kc[slot // s["page"], slot % s["page"]] = k[i]
            vc[slot // s["page"], slot % s["page"]] = v[i]
    return q, kc, vc


def _exact_norm(s):
    x = s["x"].double() if s["d"] is None else s["x"].double() + s["d"].double()
    return x / torch.sqrt((x * x).sum(1, keepdim=True) / s["n"] + EPS) * s["w"].double(), x


def _exact_product(x, bank, e, s):
    """x @ W_e in 64 bits, one row of packed words' lanes at a time."""
    words, scales = bank["words"][e].long(), bank["scales"][e].double()
    count = 4 if s["weights"] == "e4m3" else 8
    y = torch.zeros((x.shape[0], words.shape[1]), dtype=torch.float64, device=DEV)
    for i in range(count):
        rows = torch.arange(words.shape[0], device=DEV) * count + i
        group = rows // s["group"]
        if count == 4:
            w = ((words >> (8 * i)) & 255).to(torch.uint8).view(E4M3).double()
        else:
            w = ((words >> (4 * i)) & 15).double()
            if bank["zeros"] is None:
                w -= 8
            else:
                col = torch.arange(words.shape[1], device=DEV)
                z = (bank["zeros"][e].long()[:, col // 8] >> (4 * (col % 8))) & 15
                w -= z.double()[group]
        y += x[:, rows] @ (w * scales[group])
    return y


def _exact_moe(s):
    x = s["x"].double()
    logits = x @ s["router"].double().T
    y = torch.zeros_like(x) if s["res"] is None else s["res"].double()
    weights = torch.zeros((s["tokens"], s["top_k"]), dtype=torch.float64, device=DEV)
    pairs = {}
    for t, row in enumerate(logits.tolist()):
        top = max(row)
        e = [math.exp(r - top) for r in row]
        chosen = sorted(range(len(row)), key=lambda i: (-row[i], i))[: s["top_k"]]
        total = sum(e[i] for i in chosen) if s["renorm"] else sum(e)
        for j, i in enumerate(chosen):
            weights[t, j] = e[i] / total
            pairs.setdefault(i, []).append((t, e[i] / total))
    for e, rows in pairs.items():
        at = torch.tensor([t for t, _ in rows], device=DEV)
        g, u = _exact_product(x[at], s["gate"], e, s), _exact_product(x[at], s["up"], e, s)
        part = _exact_product(g * torch.sigmoid(g) * u, s["down"], e, s)
        y[at] += part * torch.tensor([w for _, w in rows], dtype=torch.float64, device=DEV)[:, None]
    return y, None, weights


def exact(case, seed):
    s = _inputs(case, seed)
    f = dict(attn=_exact_attn, append=_exact_append, norm=_exact_norm, moe=_exact_moe)
    return f[case["op"]](s)
