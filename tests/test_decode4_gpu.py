"""The decode-step operators on a 4-bit cache, and the norms of query and key heads, on the GPU
against their 64-bit forms (oracle/decode.py).

Tolerances: half a step of the output type relative to the value (finfo.eps / 2), plus the
bound the oracle derives for fp32 arithmetic, plus half of fp16's smallest step."""

import math

import numpy as np
import pytest

from oracle import decode as ref

torch = pytest.importorskip("torch")
wq = pytest.importorskip("weight_only_quantized_gemm_amd")
from weight_only_quantized_gemm_amd import decode  # noqa: E402

from test_decode_gpu import BF16, E4M3, F16, check, half_step, normal, np64, paged, rng_of  # noqa: E402

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -25  # half of fp16's smallest step


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def paged4(dev, pages, page, heads, d, group, dtype, order, g=None):
    """A 4-bit cache of random codes and pairs, of the given storage order."""
    g = g or rng_of(dev, 1)
    shape = (pages, heads, page) if order == "hnd" else (pages, page, heads)
    parts = []
    for _ in range(2):
        parts.append(torch.randint(0, 256, (*shape, d // 2), generator=g, device=dev,
                                   dtype=torch.uint8))
    for _ in range(2):
        step = torch.rand((*shape, d // group), generator=g, device=dev) * 0.2 + 0.2
        low = step * -7.5 + 0.3 * torch.randn(step.shape, generator=g, device=dev)
        parts.append(torch.stack([step, low], dim=-1).to(dtype))
    return decode.PagedCache4(*(x.transpose(1, 2) if order == "hnd" else x for x in parts))


# ---- norms, rotary positions and the cache write -------------------------------------------------

def append_case(dev, t, hq, hkv, d, rot, page, axes, kind, order, dtype, group=None, seed=0):
    g = rng_of(dev, seed + 11 + t + d)
    qkv = normal(g, (t, (hq + 2 * hkv) * d), dtype, 2.0)
    q, k, v = (x.unflatten(1, (-1, d)) if x.shape[1] else None
               for x in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
    scales = None
    if kind == "e4m3":
        scales = [torch.rand(hkv, generator=g, device=dev) * 0.02 + 0.004 for _ in range(2)]
    pages = -(-t // page) + 2
    if kind == "int4":
        cache = paged4(dev, pages, page, hkv, d, group, dtype, order, g)
    else:
        cache = paged(dev, pages, page, hkv, d, E4M3 if kind == "e4m3" else dtype, order, scales, g)
    slots = torch.randperm(pages * page, generator=g, device=dev)[:t]
    if t > 4:
        slots[1], slots[3] = -1, pages * page  # padding, and a slot past the cache
    half = rot // 2
    inv = (10000.0 ** (-torch.arange(half, device=dev).double() / max(1, half))).float()
    pos = torch.randint(0, 1 << 20, (axes, t), generator=g, device=dev).to(torch.int32)
    cut = [half * i // axes for i in range(axes + 1)]
    sections = [cut[i + 1] - cut[i] for i in range(axes)]
    weights = [1 + normal(g, (d,), dtype, 0.3) for _ in range(2)]
    return dict(q=q, k=k, v=v, cache=cache, slots=slots, half=half, inv=inv, pos=pos, g=g,
                sections=sections, weights=weights, scales=scales, kind=kind, dtype=dtype)


def turned(x, weight, c, inter, eps):
    """The 64-bit value of normed and rotated heads, and its bound."""
    x, err = np64(x), 0.0
    if weight is not None:
        x, err = ref.head_norm(x, np64(weight), eps)
    y, turn_err = ref.rotate(x, c["pos"].cpu().numpy(), c["inv"].cpu().numpy(), c["sections"], inter)
    return y, turn_err + (ref.spread(err, c["half"], inter) if weight is not None else 0.0)


def append_check(c, inter, q_norm, k_norm, eps=1e-5):
    cache, slots = c["cache"], c["slots"].tolist()
    stored = ["k", "v"] + (["k_pairs", "v_pairs"] if c["kind"] == "int4" else [])
    before = {n: getattr(cache, n).clone() for n in stored}
    qn, kn = (w if use else None for w, use in zip(c["weights"], (q_norm, k_norm)))
    got = decode.rope_append(c["q"], c["k"], c["v"], cache, c["slots"],
                             positions=c["pos"] if c["half"] else None, inv_freq=c["inv"],
                             sections=c["sections"], interleaved=inter,
                             q_norm=qn if c["q"] is not None else None, k_norm=kn, eps=eps)
    if c["q"] is not None:
        check(got, *turned(c["q"], qn, c, inter, eps), "q")
    kw, kerr = turned(c["k"], kn, c, inter, eps)
    vw, verr = np64(c["v"]), np.zeros_like(np64(c["v"]))
    real = [i for i, s in enumerate(slots) if 0 <= s < cache.num_pages * cache.page_size]
    at = tuple(np.array([divmod(slots[i], cache.page_size) for i in real]).T.reshape(2, -1))
    for i, (name, want, err) in enumerate((("k", kw, kerr), ("v", vw, verr))):
        tensor, was = getattr(cache, name), before[name]
        if c["kind"] == "int4":
            codes, pairs = tensor.cpu().numpy(), np64(getattr(cache, name + "_pairs"))
            ref.check_quantized4(want[real], err[real], codes[at], pairs[at], half_step(c["dtype"]),
                                 TINY)
            for now, old in ((tensor, was), (getattr(cache, name + "_pairs"), before[name + "_pairs"])):
                old = old.clone()
                old[at] = now[at]  # nothing else has changed
                assert torch.equal(now, old), name
            continue
        full = np64(was)
        full_err = np.zeros_like(full)
        if c["scales"] is not None:
            s = np64(c["scales"][i])[:, None]
            want = np.clip(want / s, -448, 448)
            # the quotient is fp32; E4M3's smallest half step is 2^-10
            err = err / s + np.abs(want) * 2 * ref.E32 + 2.0 ** -10
        full[at], full_err[at] = want[real], err[real]
        check(tensor, full, full_err, name)


APPENDS = [
    # tokens, q heads, kv heads, d, rot, page, axes, interleaved, order, type, groups
    (1, 4, 2, 128, 128, 16, 1, False, "hnd", F16, (32, 64, 128)),
    (1, 0, 1, 64, 64, 16, 1, True, "nhd", BF16, (32, 64)),
    (37, 7, 1, 80, 40, 24, 2, False, "hnd", F16, (80,)),
    (37, 7, 1, 80, 40, 24, 2, True, "nhd", BF16, (80,)),
    (5, 3, 3, 16, 8, 1, 1, False, "nhd", BF16, (16,)),
    (130, 8, 2, 256, 256, 7, 3, False, "nhd", BF16, (32, 128, 256)),
    (130, 8, 2, 256, 128, 7, 4, True, "hnd", F16, (64, 256)),
    (9, 2, 2, 72, 0, 8, 1, False, "hnd", BF16, (72,)),
    (33, 5, 5, 96, 96, 8, 1, False, "nhd", F16, (32, 96)),
    (20, 3, 3, 192, 64, 16, 1, True, "hnd", BF16, (32, 64, 192)),
    (3, 1, 1, 24, 24, 4, 1, False, "hnd", F16, (24,)),
    (4200, 1, 1, 64, 64, 64, 1, False, "hnd", F16, (32,)),
    (600, 32, 8, 128, 128, 16, 3, False, "hnd", BF16, (64,)),
    (1100, 24, 8, 128, 64, 16, 1, True, "nhd", F16, (128,)),
]


@pytest.mark.parametrize("case", APPENDS)
@pytest.mark.parametrize("q_norm,k_norm", [(True, True), (False, True), (True, False), (False, False)])
def test_append_to_a_4_bit_cache(dev, case, q_norm, k_norm):
    t, hq, hkv, d, rot, page, axes, inter, order, dtype, groups = case
    for group in groups if q_norm == k_norm else groups[:1]:
        c = append_case(dev, t, hq, hkv, d, rot, page, axes, "int4", order, dtype, group)
        append_check(c, inter, q_norm, k_norm)


@pytest.mark.parametrize("case", APPENDS)
@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_append_with_norms(dev, case, kind):
    t, hq, hkv, d, rot, page, axes, inter, order, dtype, _ = case
    for q_norm, k_norm in ((True, True), (False, True), (True, False)):
        c = append_case(dev, t, hq, hkv, d, rot, page, axes, kind, order, dtype)
        append_check(c, inter, q_norm, k_norm)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_append_in_place_and_over_strided_rows(dev, dtype, inter):
    g = rng_of(dev, 4)
    wide = normal(g, (37, 9 * 64), dtype)
    q = wide[:, 64:320].unflatten(1, (4, 64))
    k = normal(g, (37, 1, 64), dtype)
    cache = paged4(dev, 5, 8, 1, 64, 32, dtype, "nhd")
    args = k, k, cache, torch.arange(37, device=dev)
    w = 1 + normal(g, (64,), dtype, 0.2)
    kw = dict(positions=torch.arange(37, device=dev, dtype=torch.int32) * 999, interleaved=inter,
              inv_freq=torch.rand(32, generator=g, device=dev), q_norm=w, k_norm=w)
    rest = wide[:, 320:].clone()
    want = decode.rope_append(q, *args, **kw)
    assert not torch.equal(want, q)
    got = decode.rope_append(q, *args, q_out=q, **kw)
    assert torch.equal(got, want) and torch.equal(wide[:, 320:], rest)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_append_special_groups(dev, dtype):
    """Constant groups, NaN, infinities, a range past the type, tiny ranges; their neighbours."""
    v = torch.zeros((9, 1, 64), dtype=dtype, device=dev)
    v[:, :, 32:] = torch.linspace(-3, 3, 32, device=dev).to(dtype)
    v[0, 0, :32] = 5.0
    v[1, 0, 3], v[2, 0, 31], v[3, 0, 0] = math.nan, math.inf, -math.inf
    v[4, 0, :32] = torch.linspace(-1, 1, 32, device=dev).to(dtype) * (2.0 ** -13 if dtype is F16 else 1e-30)
    v[5, 0, 0], v[5, 0, 1] = torch.finfo(dtype).max, torch.finfo(dtype).min  # range past fp32, or not
    v[6, 0, :32] = -0.0
    v[7, 0, 4] = 2.0 ** -24 if dtype is F16 else 1e-38  # a scale below the type's steps
    v[8, 0, :32] = torch.finfo(dtype).max
    cache = paged4(dev, 3, 4, 1, 64, 32, dtype, "hnd")
    slots = torch.arange(9, device=dev)
    decode.rope_append(None, v, v, cache, slots)
    for x in cache.read(slots):
        nan = x.isnan()
        broken = [1, 2, 3] + ([5] if dtype is BF16 else [])
        assert all(bool(nan[i, 0, :32].all()) for i in broken) and int(nan.sum()) == 32 * len(broken)
        for i in (0, 6, 7, 8):
            want = v[i, 0, :32] if i != 7 else torch.zeros_like(v[i, 0, :32])
            if i == 7 and dtype is BF16:
                want = v[i, 0, :32]
                assert float((x[i, 0, :32].double() - want.double()).abs().max()) <= 1e-39
                continue
            assert torch.equal(x[i, 0, :32], want), i
        step = float((v[4, 0, 31].double() - v[4, 0, 0].double()) / 15)
        # half a step, and the roundings of scale (times 15) and offset to the type
        slack = step * (0.5 + 16 * half_step(dtype)) + float(v[4, 0, 31]) * 2 * half_step(dtype) + 16 * TINY
        assert float((x[4, 0, :32].double() - v[4, 0, :32].double()).abs().max()) <= slack
        if dtype is F16:
            # 131008 / 15 becomes 8736 in fp16, and 15 * 8736 - 65504 = 65536 rounds to inf there
            assert bool(x[5, 0, 0] == math.inf) and bool(x[5, 0, 1:32].isfinite().all())
        assert all(torch.equal(x[i, 0, 32:], x[0, 0, 32:]) for i in range(9))


def test_append_norm_extremes(dev):
    """Squares past fp32 give 0, NaN reaches its own head only, a zero head stays zero."""
    q = torch.ones((4, 3, 64), dtype=BF16, device=dev)
    q[0, 1] = 3e38
    q[1, 1, 5] = math.nan
    q[2, 1] = 0
    q[3, 1] = 1e-30
    k = q[:, :1].contiguous()
    w = torch.ones(64, dtype=BF16, device=dev)
    cache = paged(dev, 2, 4, 1, 64, BF16, "hnd")
    y = decode.rope_append(q, k, k, cache, torch.arange(4, device=dev), q_norm=w, eps=1e-6)
    assert bool((y[0, 1] == 0).all()) and bool(y[1, 1].isnan().all()) and bool((y[2, 1] == 0).all())
    assert bool(y[3, 1].isfinite().all()) and bool((y[:, [0, 2]] == 1).all())


# ---- what a 4-bit cache holds --------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,group,heads,order", [(16, 16, 1, "hnd"), (80, 80, 3, "nhd"), (128, 32, 8, "hnd"),
                                                 (128, 128, 2, "nhd"), (192, 64, 5, "hnd"), (256, 32, 1, "nhd")])
def test_read(dev, dtype, d, group, heads, order):
    cache = paged4(dev, 7, 6, heads, d, group, dtype, order)
    slots = torch.tensor([41, 0, 41, -1, 42, 13, -2 ** 40, 2 ** 40, 5], device=dev)
    k, v = cache.read(slots)
    s = [x for x in slots.tolist()]
    for got, codes, pairs in ((k, cache.k, cache.k_pairs), (v, cache.v, cache.v_pairs)):
        full = ref.values4(codes.cpu().numpy(), np64(pairs)).reshape(42, heads, d)
        want = np.stack([full[x] if 0 <= x < 42 else np.zeros((heads, d)) for x in s])
        check(got, want, np.abs(want) * 2 * ref.E32, "read")
        assert bool((got[[3, 4, 6, 7]] == 0).all())
    wide = torch.full((9, 2, heads, d), 7.0, dtype=dtype, device=dev)
    k2, v2 = cache.read(slots, k_out=wide[:, 1])
    assert torch.equal(k2, k) and torch.equal(v2, v) and bool((wide[:, 0] == 7).all())
    assert cache.read(slots[:0])[0].shape == (0, heads, d)


# ---- attention ------------------------------------------------------------------------------

def attn_case(dev, lens, hq, hkv, d, group, page, dtype, order="hnd", window=0, softcap=0.0,
              keep=False, max_len=None, seed=0, spare=3, poison=True):
    g = rng_of(dev, seed + 31 * d + hq)
    b = len(lens)
    top = max_len or max(1, max(lens))
    per = -(-top // page)
    cache = paged4(dev, b * per + spare, page, hkv, d, group, dtype, order, g)
    order_ = torch.randperm(b * per + spare, generator=g, device=dev)[: b * per]
    table = order_.view(b, per).to(torch.int32).contiguous()
    lens_t = torch.tensor(lens, dtype=torch.int32, device=dev)
    q = normal(g, (b, hq, d), dtype)
    mask = None
    if keep:
        mask = (torch.rand((b, top + 5), generator=g, device=dev) > 0.4).to(torch.uint8)
        mask[0] = 0
    if poison:  # NaN wherever no live position lies
        live = torch.zeros(cache.k.shape[:2], dtype=torch.bool, device=dev)
        for i, n in enumerate(lens):
            j = torch.arange(max(0, n - window) if window else 0, n, device=dev)
            if mask is not None:
                j = j[mask[i, j] != 0]
            live[table[i, j // page].long(), j % page] = True
        for x in (cache.k_pairs, cache.v_pairs):
            x.masked_fill_((~live)[:, :, None, None, None], math.nan)
    return dict(cache=cache, table=table, lens=lens_t, q=q, keep=mask, top=top, window=window,
                softcap=softcap, hq=hq, dtype=dtype, scale=1 / math.sqrt(d))


def attn_run(c, cut=False, **kw):
    """cut: planned for sequences far longer than the table's pages (the rest are no pages of the
    cache), so that they are cut into ranges."""
    if cut:
        c = dict(c, top=c["top"] + (1 << 20) // c["cache"].head_dim)
        pages = -(-c["top"] // c["cache"].page_size)
        c["table"] = torch.nn.functional.pad(c["table"], (0, pages - c["table"].shape[1]), value=-1)
        if c["keep"] is not None:
            c["keep"] = torch.nn.functional.pad(c["keep"], (0, c["top"] - c["keep"].shape[1]),
                                                value=1)
    plan = decode.PagedAttention(c["cache"], len(c["lens"]), c["hq"], c["top"], dtype=c["dtype"],
                                 scale=c["scale"], window=c["window"], softcap=c["softcap"])
    assert not cut or c["window"] or plan.workspace.numel()
    plan.workspace.fill_(0xFF)  # its contents need no initialization
    return plan(c["q"], c["table"], c["lens"], keep=c["keep"], lse=True, **kw)


# q is cut into two E4M3 pieces at least (fp16: three) below 2^8 times a power of two, multiples of 2^-3 and 2^-7
# (and 2^-11) that meet K's codes without loss; what they leave is half of the last at most, beside a
# largest element of 124 at least (half of 248, past which a piece would round up to 2^8): 2^-8 / 124 <
# 2^-14.95 (2^-12 / 124 < 2^-18.95).
Q_STEP = {BF16: 2.0 ** -14.95, F16: 2.0 ** -18.95}


def attn_check(c, out, lse, label=""):
    cache = c["cache"]
    parts = [(x.cpu().numpy(), np64(y)) for x, y in ((cache.k, cache.k_pairs), (cache.v, cache.v_pairs))]
    want, want_lse, err, lse_err = ref.paged_attention(
        np64(c["q"]), *(ref.values4(*x) for x in parts), c["table"].cpu().numpy(),
        c["lens"].cpu().numpy(), c["scale"], c["window"], c["softcap"],
        None if c["keep"] is None else c["keep"].cpu().numpy(), None,
        *(ref.terms4(*x) for x in parts), Q_STEP[c["dtype"]])
    check(out, want, err, label + " out")
    check(lse, want_lse, lse_err, label + " lse")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,group,hq,hkv,page,order", [
    (16, 16, 1, 1, 1, "hnd"), (24, 24, 2, 2, 4, "nhd"), (64, 32, 4, 4, 16, "nhd"), (64, 64, 4, 1, 16, "hnd"),
    (72, 72, 6, 2, 5, "hnd"), (80, 80, 3, 3, 24, "nhd"), (96, 32, 20, 1, 16, "hnd"),
    (96, 96, 5, 5, 16, "nhd"), (120, 120, 4, 2, 16, "hnd"),
    (128, 32, 8, 1, 16, "hnd"), (128, 64, 8, 2, 16, "nhd"), (128, 128, 40, 2, 64, "nhd"),
    (128, 64, 40, 2, 64, "hnd"), (128, 32, 9, 3, 7, "nhd"),
    (136, 136, 2, 1, 32, "hnd"), (160, 32, 4, 2, 16, "hnd"), (184, 184, 2, 1, 16, "nhd"),
    (192, 32, 16, 1, 7, "nhd"), (192, 64, 3, 3, 16, "hnd"), (192, 192, 4, 1, 16, "nhd"),
    (200, 200, 3, 1, 9, "hnd"), (224, 32, 5, 1, 16, "hnd"),
    (256, 32, 5, 1, 16, "hnd"), (256, 64, 4, 4, 16, "nhd"), (256, 128, 17, 1, 16, "hnd"),
    (256, 256, 8, 2, 16, "nhd")])
def test_attention_heads(dev, dtype, d, group, hq, hkv, page, order):
    c = attn_case(dev, [0, 1, 15, 31, 32, 33, 64, 65, 127, 300, 600], hq, hkv, d, group, page, dtype, order)
    for cut in (False, True):
        attn_check(c, *attn_run(c, cut), f"cut {cut}")


@pytest.mark.parametrize("lens,kw", [
    ([1], {}), ([0], {}), ([2, 0, 0], {}),
    ([255, 256, 257, 129], dict(max_len=1000)),
    ([5000, 17], {}), ([12345], dict(hkv=1, hq=2)), ([4097] * 3, dict(window=100)),
    ([700, 33, 1], dict(window=1)), ([700, 33, 1], dict(window=64)), ([700, 33], dict(window=4000)),
    ([513, 64], dict(softcap=20.0)), ([900, 300, 40], dict(keep=True)),
    ([3000, 1], dict(keep=True, window=1500, softcap=5.0)),
    ([700, 33, 1], dict(hq=40, hkv=2)), ([0, 3, 64, 129] * 5, dict(hq=34)),
    ([9000, 40, 6000], dict(window=5000)), ([7000, 1], dict(keep=True, window=6500, softcap=5.0)),
])
@pytest.mark.parametrize("group", [32, 64])
def test_attention_lengths_and_masks(dev, lens, kw, group):
    kw = dict(dict(hq=8, hkv=2), **kw)
    c = attn_case(dev, lens, d=64, group=group, page=16, dtype=BF16, seed=sum(lens), **kw)
    for cut in (False, True):
        attn_check(c, *attn_run(c, cut), f"cut {cut}")


@pytest.mark.parametrize("batch,longest,hq,hkv", [(65, 700, 2, 1), (130, 3000, 2, 1),
                                                  (200, 140, 4, 4), (64, 1500, 16, 8)])
def test_attention_many_sequences(dev, batch, longest, hq, hkv):
    """More sequences than a wave has lanes; one much longer than the rest; all alike."""
    g = np.random.default_rng(batch)
    lens = g.integers(0, 60, batch)
    lens[batch // 2] = longest
    lens[-1] = longest // 2
    for n in (lens.tolist(), [130] * batch):
        c = attn_case(dev, n, hq, hkv, 64, 32, 16, BF16, max_len=longest, seed=batch)
        for cut in (False, True):
            attn_check(c, *attn_run(c, cut), f"cut {cut}")


@pytest.mark.parametrize("hq,hkv,d,group,order", [(96, 96, 64, 32, "hnd"), (520, 520, 128, 128, "nhd"),
                                                  (780, 20, 72, 72, "nhd"), (300, 10, 128, 32, "hnd")])
def test_attention_of_many_units(dev, hq, hkv, d, group, order):
    """Few ranges, or one, because a range has nearly as many work-groups as a launch, or more; with
    and without the grid that is rounded up to eight ranges."""
    c = attn_case(dev, [300, 0, 41], hq, hkv, d, group, 16, BF16, order)
    for cut in (False, True):
        attn_check(c, *attn_run(c, cut), f"cut {cut}")


@pytest.mark.parametrize("kw", [{}, dict(keep=True)])
def test_attention_several_short_sequences_in_a_range(dev, kw):
    """Waves with no, one, two and more tiles of a sequence, in every order."""
    g = np.random.default_rng(7)
    sizes = np.array([0, 1, 31, 63, 64, 65, 96, 127, 128, 129, 200, 256, 257, 300, 511, 513, 700])
    lens = sizes[g.integers(0, len(sizes), 260)]
    c = attn_case(dev, lens.tolist(), 8, 8, 64, 32, 16, F16, **kw)
    attn_check(c, *attn_run(c, True))


def test_attention_a_split_without_kept_positions(dev):
    """Whole splits masked away, the first and one between others."""
    c = attn_case(dev, [9000, 5000], 4, 1, 64, 64, 16, F16, keep=True, poison=False)
    c["keep"][:] = 1
    c["keep"][0, :3000] = 0
    c["keep"][1, 1500:4000] = 0
    attn_check(c, *attn_run(c, True))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_live_nan(dev, dtype):
    """A NaN group of K reaches its sequence's heads, one of V its elements, and nothing else."""
    c = attn_case(dev, [300, 300, 300], 2, 1, 64, 32, 16, dtype)
    at = [(c["table"][i, 5].long(), 3) for i in range(3)]
    c["cache"].v_pairs[at[0][0], at[0][1], 0, 1, 0] = math.nan
    c["cache"].k_pairs[at[1][0], at[1][1], 0, 0, 1] = math.nan
    for cut in (False, True):
        out, lse = attn_run(c, cut)
        assert bool(out[0, :, 32:].isnan().all()) and bool(out[0, :, :32].isfinite().all())
        assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
        assert bool(out[2].isfinite().all()) and bool(lse[[0, 2]].isfinite().all())


def test_attention_empty_rows_are_zero(dev):
    c = attn_case(dev, [600, 0, 40], 4, 2, 128, 64, 16, F16, keep=True)
    c["keep"][2] = 0
    for cut in (False, True):  # keep[0] is all zero
        out, lse = attn_run(c, cut)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_attention_page_numbers_outside_the_cache_are_left_out(dev):
    c = attn_case(dev, [200, 64, 40], 4, 2, 64, 32, 16, BF16, poison=False)
    c["table"][0, 3], c["table"][0, 7] = -1, c["cache"].num_pages
    c["table"][1, :] = 2 ** 31 - 1
    c["table"][2, 0] = -2 ** 31
    k, v = (ref.values4(x.cpu().numpy(), np64(y)) for x, y in
            ((c["cache"].k, c["cache"].k_pairs), (c["cache"].v, c["cache"].v_pairs)))
    assert np.isfinite(k).all() and np.isfinite(v).all()
    for cut in (False, True):
        attn_check(c, *attn_run(c, cut), f"cut {cut}")


def test_attention_lens_are_taken_into_range(dev):
    c = attn_case(dev, [100, 100], 2, 1, 64, 32, 16, F16)
    want = attn_run(c)
    c["lens"] = torch.tensor([1000000, -5], dtype=torch.int32, device=dev)
    out, lse = attn_run(c)
    assert torch.equal(out[0], want[0][0]) and bool((out[1] == 0).all())
    assert lse[1].tolist() == [-math.inf] * 2


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("cap", [0.3, 30.0, 1e4, 1e30])
def test_attention_caps(dev, dtype, cap):
    c = attn_case(dev, [700, 33, 1], 4, 2, 64, 32, 16, dtype, softcap=cap)
    c["q"] *= 4
    for cut in (False, True):
        attn_check(c, *attn_run(c, cut), f"cut {cut}")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_scales_and_offsets_of_every_size(dev, dtype):
    """Large offsets over small scales, zero scales, and groups far apart in size."""
    c = attn_case(dev, [500, 77], 4, 2, 128, 32, 16, dtype, poison=False)
    k, v = c["cache"].k_pairs, c["cache"].v_pairs
    k[..., 0, 1] = 8.0                  # an outlying group of every key
    k[..., 0, 0] = 0.01
    k[..., 1, :] = 0
    v[..., 0, 0] = 0                    # constant groups
    v[..., 1, :] *= 1000
    v[..., 2, :] *= 2.0 ** -10
    for cut in (False, True):
        attn_check(c, *attn_run(c, cut), f"cut {cut}")


def test_attention_small_positions_beside_a_large_one(dev):
    """In every tile one position leads the others by 17.5 and holds V = 0: the output is what
    the others, at 2^-25.2 of it, hold."""
    c = attn_case(dev, [4000], 1, 1, 64, 32, 32, F16, poison=False)
    cache = c["cache"]
    for x in (cache.k, cache.v):
        x.zero_()
    cache.k_pairs.zero_()
    cache.v_pairs[..., 0], cache.v_pairs[..., 1] = 0, 60000.0
    cache.k_pairs[:, 5, :, :, 1] = 1.0
    cache.v_pairs[:, 5] = 0.0
    c["q"].fill_(17.5 / 8)
    attn_check(c, *attn_run(c))


def test_attention_strided_rows_and_given_outputs(dev):
    c = attn_case(dev, [77, 300], 4, 2, 64, 32, 16, BF16)
    want, want_lse = attn_run(c)
    wide = torch.zeros((2, 10 * 64), dtype=BF16, device=dev)
    wide[:, 128:384] = c["q"].flatten(1)
    c["q"] = wide[:, 128:384].unflatten(1, (4, 64))
    dest = torch.full((2, 6, 64), 9.0, dtype=BF16, device=dev)
    lse = torch.zeros((2, 4), device=dev)
    plan = decode.PagedAttention(c["cache"], 2, 4, c["top"], dtype=BF16)
    got = plan(c["q"], c["table"], c["lens"], out=dest[:, 1:5], lse=lse)
    assert torch.equal(got[0], want) and torch.equal(lse, want_lse)
    assert bool((dest[:, 0] == 9).all()) and bool((dest[:, 5] == 9).all())
    assert torch.equal(plan(c["q"], c["table"], c["lens"]), want)


def test_attention_strides_of_a_larger_pool(dev):
    """Codes and pairs as slices of wider tensors: rows 4 bytes apart from any 16."""
    g = rng_of(dev, 12)
    codes = [torch.randint(0, 256, (5, 16, 3, 36), generator=g, device=dev, dtype=torch.uint8)
             for _ in range(2)]
    pairs = [torch.rand((5, 16, 3, 3, 2), generator=g, device=dev).to(F16) for _ in range(2)]
    cache = decode.PagedCache4(*(x[..., :32] for x in codes), *(x[:, :, :, 1:] for x in pairs))
    c = dict(cache=cache, q=normal(g, (2, 6, 64), F16), scale=0.125, window=0, softcap=0.0, keep=None,
             table=torch.tensor([[3, 0], [4, 1]], dtype=torch.int32, device=dev), top=32, hq=6, dtype=F16,
             lens=torch.tensor([29, 17], dtype=torch.int32, device=dev))
    attn_check(c, *attn_run(c))


def test_attention_offsets_past_32_bits(dev):
    """Pages beyond 4 GiB of codes: element and byte offsets need 64 bits."""
    pages, page, hkv, d, group = (1 << 21) + 64, 16, 2, 128, 128  # 2048 bytes a page
    kv = [torch.empty((pages, hkv, page, d // 2), dtype=torch.uint8, device=dev) for _ in range(2)]
    pr = [torch.empty((pages, hkv, page, 1, 2), dtype=BF16, device=dev) for _ in range(2)]
    g = rng_of(dev, 9)
    table = torch.tensor([[pages - 1, 3, pages - 40, (1 << 20) + 5]], dtype=torch.int32, device=dev)
    near = paged4(dev, 4, page, hkv, d, group, BF16, "hnd", g)
    for x, s in zip(kv + pr, (near.k, near.v, near.k_pairs, near.v_pairs)):
        x[table[0].long()] = s.transpose(1, 2)
    far = decode.PagedCache4(*(x.transpose(1, 2) for x in kv + pr))
    q, lens = normal(g, (1, 4, d), BF16), torch.tensor([61], dtype=torch.int32, device=dev)
    a = decode.PagedAttention(far, 1, 4, 64, dtype=BF16)(q, table, lens)
    order = torch.arange(4, dtype=torch.int32, device=dev)[None]
    assert torch.equal(a, decode.PagedAttention(near, 1, 4, 64, dtype=BF16)(q, order, lens))
    k = normal(g, (1, hkv, d), BF16)
    slot = torch.tensor([pages * page - 3], device=dev)
    decode.rope_append(None, k, k, far, slot)
    decode.rope_append(None, k, k, near, torch.tensor([61], device=dev))
    assert torch.equal(far.k[pages - 1, 13], near.k[3, 13])
    assert torch.equal(far.v_pairs[pages - 1, 13], near.v_pairs[3, 13])
    assert torch.equal(far.read(slot)[0], near.read(torch.tensor([61], device=dev))[0])


def test_attention_is_deterministic(dev):
    c = attn_case(dev, [9000, 100, 4000], 8, 2, 128, 64, 16, BF16)
    first = attn_run(c)
    for _ in range(3):
        again = attn_run(c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
