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
