"""What is measured of a decode step on a 4-bit cache: the rotary append with the norms of each
query and key head, single-token attention over keys and values held in 4 bits, and the choice of
the next token from its logits.

`run` computes an operator in plain torch operations, or, where `own` is set, through
weight_only_quantized_gemm_amd.decode.  `exact` gives the definition's value in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # the append of one decoded token, heads normed, to a 4-bit cache: pure latency
        dict(name="append4_token", op="append", type="bf16", cache="int4", group=64, tokens=1, hq=32,
             hkv=8, d=128, rot=128, page=16, norm=True, axes=1, interleaved=False, order="hnd"),
        # a prompt chunk into a 4-bit cache of the finest groups
        dict(name="append4_chunk", op="append", type="fp16", cache="int4", group=32, tokens=2048,
             hq=32, hkv=8, d=128, rot=128, page=32, norm=True, axes=1, interleaved=False, order="hnd"),
        # odd sizes: a few hundred tokens, heads of 80 turned in part, normed, to an E4M3 cache
        dict(name="append_norm_e4m3", op="append", type="bf16", cache="e4m3", group=0, tokens=333,
             hq=21, hkv=3, d=80, rot=40, page=24, norm=True, axes=2, interleaved=True, order="nhd"),
        # one user's first answer token after a short prompt: pure latency
        dict(name="attn4_short", op="attn", type="fp16", group=64, batch=1, hq=32, hkv=8, d=128,
             page=16, max_len=128, ragged=False, window=0, softcap=0.0, keep=False, order="hnd"),
        # a serving batch of ordinary chats, four query heads to a KV head
        dict(name="attn4_batch", op="attn", type="bf16", group=64, batch=16, hq=32, hkv=8, d=128,
             page=16, max_len=4096, ragged=True, window=0, softcap=0.0, keep=False, order="hnd"),
        # one long document: few rows, the work has to be split over the length
        dict(name="attn4_long", op="attn", type="bf16", group=64, batch=1, hq=32, hkv=8, d=128,
             page=64, max_len=131072, ragged=False, window=0, softcap=0.0, keep=False, order="nhd"),
        # a full batch with evicted positions, fine groups, eight query heads to a KV head
        dict(name="attn4_full", op="attn", type="bf16", group=32, batch=64, hq=64, hkv=8, d=128,
             page=32, max_len=8192, ragged=True, window=0, softcap=0.0, keep=True, order="hnd"),
        # one query head to a KV head, odd sizes, a group a head, a window and capped scores
        dict(name="attn4_odd", op="attn", type="fp16", group=80, batch=7, hq=12, hkv=12, d=80,
             page=24, max_len=3001, ragged=True, window=1000, softcap=30.0, keep=False, order="nhd"),
        # one user's next token: nucleus sampling from one row of logits
        dict(name="sample_one", op="sample", type="bf16", rows=1, vocab=128000, style="nucleus"),
        # a few users, the most likely tokens only, an odd vocabulary
        dict(name="sample_few", op="sample", type="fp16", rows=7, vocab=50001, style="top"),
        # a serving batch in which every request has settings of its own
        dict(name="sample_batch", op="sample", type="fp32", rows=64, vocab=128000, style="mixed"),
        # the largest batch
        dict(name="sample_full", op="sample", type="bf16", rows=256, vocab=128000, style="mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _groups(d):
    return [g for g in (32, 64, 128) if d % g == 0 and g < d] + [d]


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "sample"])
    ty = rng.choice(["fp16", "bf16"])
    if op == "attn":
        hkv = rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([64, 72, 96, 128, 128, 192, 256])
        batch = _log(rng, 1, 64)
        room = 64 * 8192 * 8 * 128 // (4 * batch * hkv * d)  # a quarter of the largest listed cache
        return dict(op=op, type=ty, group=rng.choice(_groups(d)), batch=batch,
                    hq=hkv * rng.choice([1, 2, 3, 4, 5, 8, 16]), hkv=hkv, d=d,
                    page=rng.choice([1, 8, 16, 24, 32, 64, 128]),
                    max_len=_log(rng, 1, min(100000, room)), ragged=rng.random() < 0.7,
                    window=rng.choice([0, 0, 0, 777]), softcap=rng.choice([0.0, 0.0, 25.0]),
                    keep=rng.random() < 0.3, order=rng.choice(["hnd", "nhd"]))
    if op == "append":
        hkv = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 80, 128, 256])
        cache = rng.choice(["same", "e4m3", "int4", "int4"])
        return dict(op=op, type=ty, cache=cache, group=rng.choice(_groups(d)) if cache == "int4" else 0,
                    tokens=_log(rng, 1, min(2048, 2000000 // (hkv * d))),
                    hq=hkv * rng.choice([1, 4, 7]), hkv=hkv, d=d, rot=rng.choice([d, d // 2, 0]),
                    page=rng.choice([1, 16, 24, 64]), norm=cache != "int4" or rng.random() < 0.7,
                    axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.4,
                    order=rng.choice(["hnd", "nhd"]))
    rows = _log(rng, 1, 256)
    return dict(op=op, type=rng.choice(["fp16", "bf16", "fp32"]), rows=rows,
                vocab=_log(rng, 100, min(260000, 256 * 128000 // (2 * rows))),
                style=rng.choice(["plain", "top", "nucleus", "mixed"]))


# ---- inputs ------------------------------------------------------------------------------


def _normal(g, shape, dtype, sd=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * sd).to(dtype)


def _logical(s, storage):
    """The [page][slot][head]... view of a tensor stored head-major or slot-major."""
    return storage.transpose(1, 2) if s["order"] == "hnd" else storage


def _bytes(x):
    """E4M3 tensors as bytes (copied and indexed as they are), others unchanged."""
    return x.view(torch.uint8) if x.dtype == E4M3 else x


def _cache(g, s, pages):
    """K and V of `pages` pages: 16-bit or E4M3 values (with a scale per KV head), or 4-bit codes,
    two to a byte, with a scale and an offset for each group of a head."""
    shape = (pages, s["hkv"], s["page"]) if s["order"] == "hnd" else (pages, s["page"], s["hkv"])
    ty, d = TYPES[s["type"]], s["d"]
    s["k_scale"] = s["v_scale"] = None
    for x in ("k", "v"):
        if s.get("cache", "int4") == "int4":
            codes = torch.randint(0, 256, (*shape, d // 2), generator=g, device=DEV, dtype=torch.uint8)
            step = torch.rand((*shape, d // s["group"]), generator=g, device=DEV) * 0.2 + 0.2
            low = step * -7.5 + 0.3 * torch.randn(step.shape, generator=g, device=DEV)
            s[x + "_pairs"] = _logical(s, torch.stack([step, low], dim=-1).to(ty))
            s[x + "_cache"] = _logical(s, codes)
            continue
        value = _normal(g, (*shape, d), ty)
        if s["cache"] == "e4m3":
            s[x + "_scale"] = torch.rand(s["hkv"], generator=g, device=DEV) * 0.02 + 0.005
            value = (value.float() * 60).to(E4M3)
        s[x + "_cache"] = _logical(s, value)


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
    for name in ("k_pairs", "v_pairs"):
        one = s[name][last]
        one[behind] = float("nan")
        s[name][last] = one
    s["lens"] = lens.to(torch.int32)
    s["q"] = _normal(g, (b, s["hq"], s["d"]), TYPES[s["type"]])
    s["scale"] = 1.0 / math.sqrt(s["d"])
    s["mask"] = None
    if s["keep"]:
        s["mask"] = (torch.rand((b, top), generator=g, device=DEV) > 0.3).to(torch.uint8)


def _inputs_append(s, g):
    t, d, ty = s["tokens"], s["d"], TYPES[s["type"]]
    qkv = _normal(g, (t, (s["hq"] + 2 * s["hkv"]) * d), ty, 1.5)  # one fused projection's rows
    q, k, v = qkv.split([s["hq"] * d, s["hkv"] * d, s["hkv"] * d], dim=1)
    s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in (q, k, v))
    s["q_norm"] = s["k_norm"] = None
    if s["norm"]:
        s["q_norm"], s["k_norm"] = (1 + _normal(g, (d,), ty, 0.1) for _ in range(2))
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


def _inputs_sample(s, g):
    rows, vocab = s["rows"], s["vocab"]
    logits = torch.randn((rows, vocab), generator=g, device=DEV) * 2
    # some tokens stand out of the rest, as a trained model's do; a few are banned
    at = torch.randint(0, vocab, (rows, 60), generator=g, device=DEV)
    logits.scatter_add_(1, at, 14 * torch.rand((rows, 60), generator=g, device=DEV))
    ban = torch.randint(0, vocab, (rows, 3), generator=g, device=DEV)
    logits.scatter_(1, ban, float("-inf"))
    s["logits"] = logits.to(TYPES[s["type"]])

    def pick(*values):
        i = torch.randint(0, len(values), (rows,), generator=g, device=DEV)
        return torch.tensor(values, device=DEV, dtype=torch.float32)[i]

    style = s["style"]
    s["temperature"] = pick(0.6, 0.7, 1.0, 1.3) if style != "mixed" else pick(0.0, 0.7, 1.0, 1.0, 1.5)
    s["top_k"] = s["top_p"] = s["min_p"] = None  # a setting that nobody uses is left out
    if style == "top":
        s["top_k"], s["min_p"] = pick(1, 20, 40, 50).int(), pick(0.0, 0.05)
    if style == "nucleus":
        s["top_p"] = pick(0.8, 0.9, 0.95)
    if style == "mixed":
        s["top_k"] = pick(0, 0, 0, 20, 50, 1000).int()  # 0: all
        s["top_p"], s["min_p"] = pick(1.0, 1.0, 0.9, 0.95), pick(0.0, 0.0, 0.02, 0.1)
    s["u"] = torch.rand(rows, generator=g, device=DEV)


def _inputs(case, seed):
    s = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 23)
    dict(attn=_inputs_attn, append=_inputs_append, sample=_inputs_sample)[s["op"]](s, g)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from weight_only_quantized_gemm_amd import decode
    s["decode"] = decode
    if s["op"] == "sample":
        s["plan"] = decode.Sampler(s["rows"], s["vocab"], dtype=TYPES[s["type"]], device=DEV)
    elif s.get("cache", "int4") == "int4":
        s["paged"] = decode.PagedCache4(s["k_cache"], s["v_cache"], s["k_pairs"], s["v_pairs"])
    else:
        s["paged"] = decode.PagedCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if s["op"] == "attn":
        s["plan"] = decode.PagedAttention(s["paged"], s["batch"], s["hq"], s["max_len"],
                                          dtype=TYPES[s["type"]], scale=s["scale"],
                                          window=s["window"], softcap=s["softcap"])
    return s


# ---- the plain forms -----------------------------------------------------------------------


def _values(codes, pairs):
    """[...][d] from codes [...][d / 2] and pairs [...][groups][2]: offset + scale * code."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float()
    c = c.unflatten(-1, (pairs.shape[-2], -1))
    p = pairs.float()
    return (p[..., 1:] + p[..., :1] * c).flatten(-2)


def _plain_attn(s):
    b, hq, hkv, d, top = s["batch"], s["hq"], s["hkv"], s["d"], s["max_len"]
    idx = s["table"].long()
    k, v = (_values(s[n + "_cache"][idx].flatten(1, 2)[:, :top], s[n + "_pairs"][idx].flatten(1, 2)[:, :top])
            .permute(0, 2, 1, 3).contiguous() for n in ("k", "v"))
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


def _normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * weight.float()


def _angles(s):
    axis = torch.repeat_interleave(torch.arange(s["axes"], device=DEV),
                                   torch.tensor(s["sections"], device=DEV),
                                   output_size=s["rot"] // 2)
    return s["positions"].double()[axis].t() * s["inv_freq"].double()  # [tokens][rot / 2]


def _rotated(x, s, cos, sin):
    half = s["rot"] // 2
    turn, rest = x[..., : s["rot"]], x[..., s["rot"]:]
    if s["interleaved"]:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = turn[..., :half], turn[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _quantized(x, group, dtype):
    """Codes and pairs of [...][d]: the offset is the group's smallest value, the scale a
    fifteenth of its range, both rounded to the type; the code nearest by what they became (ties:
    the even one)."""
    x = x.unflatten(-1, (-1, group))
    low, high = x.amin(dim=-1, keepdim=True), x.amax(dim=-1, keepdim=True)
    pairs = torch.cat([(high - low) / 15, low], dim=-1).to(dtype)
    scale, low = pairs[..., :1].float(), pairs[..., 1:].float()
    code = torch.where(scale > 0, torch.round((x - low) / scale), 0.0).clamp(0, 15).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, pairs


def _stored(x, scale, dtype):
    if scale is None:
        return x.to(dtype)
    return (x / scale[:, None]).clamp(-448.0, 448.0).to(E4M3)


def _plain_append(s):
    angles = _angles(s)
    cos, sin = angles.cos().float()[:, None], angles.sin().float()[:, None]
    ty = TYPES[s["type"]]
    q = _rotated(_normed(s["q"], s["q_norm"]), s, cos, sin).to(ty)
    k, v = _rotated(_normed(s["k"], s["k_norm"]), s, cos, sin), s["v"].float()
    real = s["slots"] >= 0
    page, slot = (s["slots"] // s["page"])[real], (s["slots"] % s["page"])[real]
    if s["cache"] != "int4":
        _bytes(s["k_cache"])[page, slot] = _bytes(_stored(k, s["k_scale"], ty))[real]
        _bytes(s["v_cache"])[page, slot] = _bytes(_stored(v, s["v_scale"], ty))[real]
        return q, s["k_cache"], s["v_cache"]
    outs = [q]
    for name, x in (("k", k), ("v", v)):
        codes, pairs = _quantized(x, s["group"], ty)
        s[name + "_cache"][page, slot] = codes[real]
        s[name + "_pairs"][page, slot] = pairs[real]
        # what the tokens' slots now stand for; a padding token's none is zero
        value = _values(s[name + "_cache"][page, slot], s[name + "_pairs"][page, slot])
        out = torch.zeros((s["tokens"], s["hkv"], s["d"]), dtype=ty, device=DEV)
        out[real] = value.to(ty)
        outs.append(out)
    return tuple(outs)


def _plain_sample(s):
    z, vocab = s["logits"].double(), s["vocab"]  # sums and cuts next to a border: 64 bits
    t = s["temperature"].double()[:, None]
    top = z.amax(dim=1, keepdim=True)
    w = torch.exp((z - top) / torch.where(t > 0, t, 1.0))
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    ranked = w.gather(1, order)
    keep = torch.ones_like(ranked, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep = torch.arange(vocab, device=DEV) < torch.where(k > 0, k, vocab)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        mass = torch.where(keep, ranked, 0.0)
        before = mass.cumsum(dim=1) - mass
        keep = keep & ((before < p * mass.sum(dim=1, keepdim=True)) | (p >= 1))
    if s["min_p"] is not None:
        keep = keep & (ranked >= s["min_p"].double()[:, None])
    kept = torch.where(torch.zeros_like(keep).scatter(1, order, keep), w, 0.0)
    upto = kept.cumsum(dim=1)
    total = upto[:, -1:]
    ids = (upto <= s["u"].double()[:, None] * total).sum(dim=1, keepdim=True)
    ids = torch.where(t > 0, ids.clamp(max=vocab - 1), order[:, :1])
    logprob = torch.where(t > 0, torch.log(kept.gather(1, ids) / total), 0.0)
    return ids.flatten().to(torch.int32), logprob.flatten().float()


# ---- one pass -------------------------------------------------------------------------------


def _own_attn(s):
    return s["plan"](s["q"], s["table"], s["lens"], keep=s["mask"], lse=True)


def _own_append(s):
    s["decode"].rope_append(s["q"], s["k"], s["v"], s["paged"], s["slots"],
                            positions=s["positions"], inv_freq=s["inv_freq"],
                            sections=s["sections"], interleaved=s["interleaved"],
                            q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, q_out=s["q_out"])
    if s["cache"] != "int4":
        return s["q_out"], s["k_cache"], s["v_cache"]
    return (s["q_out"], *s["paged"].read(s["slots"]))


def _own_sample(s):
    return s["plan"](s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                     top_p=s["top_p"], min_p=s["min_p"], logprob=True)


def run(state):
    if own:
        f = dict(attn=_own_attn, append=_own_append, sample=_own_sample)
    else:
        f = dict(attn=_plain_attn, append=_plain_append, sample=_plain_sample)
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
    live = mean * c["batch"]
    row = c["d"] // 2 + 4 * (c["d"] // c["group"])
    return dict(bytes=live * 2 * c["hkv"] * row + c["batch"] * c["hq"] * (4 * c["d"] + 4),
                flops=live * 4 * c["hq"] * c["d"])


def _work_append(c):
    size = dict(same=2, e4m3=1, int4=0)[c["cache"]]
    if c["cache"] == "int4":
        size = 0.5 + 4 / c["group"] + 2  # codes, pairs and the values that are read back
    return dict(bytes=c["tokens"] * c["d"] * (4 * c["hq"] + 2 * c["hkv"] * (2 + size)),
                flops=c["tokens"] * (3 * c["rot"] + 4 * c["d"] * c["norm"]) * (c["hq"] + c["hkv"]))


def _work_sample(c):
    size = 4 if c["type"] == "fp32" else 2
    return dict(bytes=c["rows"] * (c["vocab"] * size + 28), flops=c["rows"] * c["vocab"] * 4)


def work(case):
    return dict(attn=_work_attn, append=_work_append, sample=_work_sample)[case["op"]](case)


# ---- the definition in 64 bits ------------------------------------------------------------------


def _exact_values(codes, pairs):
    out = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.float64, device=DEV)
    group = out.shape[-1] // pairs.shape[-2]
    for i in range(out.shape[-1]):
        code = (codes[..., i // 2].int() >> (4 * (i % 2))) & 15
        pair = pairs[..., i // group, :].double()
        out[..., i] = pair[..., 1] + pair[..., 0] * code
    return out


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
        at = s["table"][b, pos // s["page"]].long(), pos % s["page"]
        k, v = (_exact_values(s[n + "_cache"][at], s[n + "_pairs"][at]) for n in ("k", "v"))
        per = s["hq"] // s["hkv"]
        for h in range(s["hq"]):
            z = k[:, h // per] @ s["q"][b, h].double() * s["scale"]
            if s["softcap"]:
                z = s["softcap"] * torch.tanh(z / s["softcap"])
            lse[b, h] = torch.logsumexp(z, 0)
            out[b, h] = torch.exp(z - lse[b, h]) @ v[:, h // per]
    return out, lse


def _exact_append(s):
    half, d, ty = s["rot"] // 2, s["d"], TYPES[s["type"]]
    axis = [a for a in range(s["axes"]) for _ in range(s["sections"][a])]
    pair = [(2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half) for i in range(half)]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if s["norm"]:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) / d + EPS) * s["q_norm"].double()
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) / d + EPS) * s["k_norm"].double()
    q, k = q.clone(), k.clone()
    for x in (q, k):
        for i, (a, b) in enumerate(pair):
            angle = (s["positions"][axis[i]].double() * s["inv_freq"][i].double())[:, None]
            re, im = x[..., a].clone(), x[..., b].clone()
            x[..., a] = re * torch.cos(angle) - im * torch.sin(angle)
            x[..., b] = re * torch.sin(angle) + im * torch.cos(angle)
    if s["cache"] == "int4":
        outs = [q]
        for x in (k, v):
            y = torch.zeros_like(x)
            for g in range(0, d, s["group"]):
                part = x[..., g: g + s["group"]]
                low, high = part.min(-1, keepdim=True).values, part.max(-1, keepdim=True).values
                step = ((high - low) / 15).to(ty).double()
                low = low.to(ty).double()
                code = ((part - low) / step).round().clamp(0, 15)  # ties to even codes
                y[..., g: g + s["group"]] = low + step * code
            y[s["slots"] < 0] = 0
            outs.append(y)
        return tuple(outs)
    if s["cache"] == "e4m3":
        k = (k / s["k_scale"].double()[:, None]).clamp(-448, 448)
        v = (v / s["v_scale"].double()[:, None]).clamp(-448, 448)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for i, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            kc[slot // s["page"], slot % s["page"]] = k[i]
            vc[slot // s["page"], slot % s["page"]] = v[i]
    return q, kc, vc


def _exact_sample(s):
    logprob = torch.zeros(s["rows"], dtype=torch.float64, device=DEV)
    setting = {n: None if s[n] is None else s[n].double().tolist()
               for n in ("temperature", "top_k", "top_p", "min_p", "u")}
    for r in range(s["rows"]):
        t = setting["temperature"][r]
        if t == 0:
            continue  # the largest, for certain
        z = s["logits"][r].double()
        values, ids = torch.sort(z, descending=True, stable=True)
        p = torch.exp((values - values[0]) / t)
        n = s["vocab"]
        if s["top_k"] is not None and setting["top_k"][r] > 0:
            n = min(n, int(setting["top_k"][r]))
        if s["top_p"] is not None and setting["top_p"][r] < 1:
            upto = torch.cumsum(p[:n], 0)
            n = 1 + int(torch.searchsorted(upto, setting["top_p"][r] * upto[-1]))
        if s["min_p"] is not None:
            n = min(n, int((p >= setting["min_p"][r]).sum()))
        chosen, at = torch.sort(ids[:n])
        upto = torch.cumsum(p[:n][at], 0)
        i = int(torch.searchsorted(upto, setting["u"][r] * upto[-1], right=True))
        logprob[r] = torch.log(p[at[min(i, n - 1)]] / upto[-1])
    return None, logprob


def exact(case, seed):
    s = _inputs(case, seed)
    return dict(attn=_exact_attn, append=_exact_append, sample=_exact_sample)[case["op"]](s)
