"""The decode-step operators on the GPU against their 64-bit forms (oracle/decode.py).

Tolerances: half a step of the output type relative to the value (finfo.eps / 2), plus the
bound the oracle derives for fp32 sums, plus half of fp16's smallest step."""

import math

import numpy as np
import pytest

from oracle import decode as ref

torch = pytest.importorskip("torch")
wq = pytest.importorskip("weight_only_quantized_gemm_amd")
from weight_only_quantized_gemm_amd import decode, torch_ops  # noqa: E402

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def np64(t):
    return t.double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(got, want, err, label):
    """|got - want| within one rounding of got's type and err; infinities and NaN in place."""
    half = half_step(got.dtype)
    got = np64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), label
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), label
    fine = np.isfinite(want)
    got, want, err = got[fine], want[fine], np.broadcast_to(err, want.shape)[fine]
    off = np.abs(got - want) - (np.abs(want) * half * 1.01 + err * 1.01 + 2.0 ** -25)
    assert off.max(initial=0) <= 0, (label, float(off.max()))


def rng_of(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def normal(g, shape, dtype, sd=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * sd).to(dtype)


# ---- RMS norm ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,n", [(1, 8), (3, 512), (1, 520), (5, 2048), (2, 4096), (7, 4104),
                                    (1, 8192), (3, 8200), (2, 16384), (1, 16392), (2, 32768),
                                    (1, 32776), (1, 65536), (300, 4096), (1000, 136)])
def test_add_rms_norm(dev, dtype, rows, n):
    g = rng_of(dev, n + rows)
    x, d = normal(g, (rows, n), dtype, 3.0), normal(g, (rows, n), dtype)
    w = normal(g, (n,), dtype)
    eps = 1e-5
    for delta in (None, d):
        y, s = decode.add_rms_norm(x, w, eps, delta=delta)
        want_y, want_s = ref.add_rms_norm(np64(x), None if delta is None else np64(d), np64(w), eps)
        check(s, want_s, np.abs(want_s) * 2 * ref.E32, "sum")
        check(y, want_y, np.abs(want_y) * 128 * ref.E32, "norm")


def test_add_rms_norm_strides_and_aliases(dev):
    g = rng_of(dev, 5)
    wide = normal(g, (9, 3 * 640), F16)
    x, d = wide[:, 640:1280], wide[:, 1280:]
    w = normal(g, (640,), F16)
    y0, s0 = decode.add_rms_norm(x.contiguous(), w, delta=d.contiguous())
    out = torch.full((9, 1280), 7.0, dtype=F16, device=dev)
    y1, _ = decode.add_rms_norm(x, w, delta=d, sum_out=x, out=out[:, 640:])  # sum over x
    assert torch.equal(y1, y0) and torch.equal(wide[:, 640:1280], s0)
    assert bool((out[:, :640] == 7).all())
    y2, s2 = decode.add_rms_norm(s0, w, out=d)  # norm over another operand's rows
    assert s2 is s0 and torch.equal(wide[:, 1280:], y2)


def test_add_rms_norm_extremes(dev):
    x = torch.zeros((4, 64), dtype=BF16, device=dev)
    x[1] = 3e38          # its square overflows fp32: the norm is 0, as in the formula's fp32
    x[2, 5] = float("nan")
    x[3] = 1e-30
    w = torch.ones(64, dtype=BF16, device=dev)
    y, _ = decode.add_rms_norm(x, w, 1e-6)
    assert bool((y[0] == 0).all()) and bool(y[2].isnan().all())
    assert bool(y[3].isfinite().all())


@pytest.mark.parametrize("delta", [False, True])
def test_add_rms_norm_of_squares_past_fp32_and_below_it(dev, delta):
    """Squares past fp32 give 0; squares below it leave eps alone under the root."""
    x = torch.full((2, 520), 3e38, dtype=BF16, device=dev)
    x[1] = 1e-30
    x[:, 1::2] *= -1
    d = torch.zeros_like(x) if delta else None
    w = torch.linspace(0.5, 2, 520, device=dev).to(BF16)
    y, s = decode.add_rms_norm(x, w, 1e-6, delta=d)
    assert bool((y[0] == 0).all()) and torch.equal(s, x)
    want = np64(x[1]) * np64(w) / math.sqrt(float(np.float32(1e-6)))
    assert (np.abs(np64(y[1]) - want) <= np.abs(want) * (half_step(BF16) + 8 * ref.E32)).all()


# ---- rotary positions and the cache write -----------------------------------------------------

def paged(dev, pages, page, heads, d, dtype, order, scales=None, g=None):
    """A cache of the given storage order, filled with random values."""
    shape = (pages, heads, page, d) if order == "hnd" else (pages, page, heads, d)
    g = g or rng_of(dev, 1)
    kv = [torch.randn(shape, generator=g, device=dev) for _ in range(2)]
    kv = [(x * (60 if dtype is E4M3 else 1)).to(dtype) for x in kv]
    kv = [x.transpose(1, 2) if order == "hnd" else x for x in kv]
    return decode.PagedCache(kv[0], kv[1], *(scales or (None, None)))


@pytest.mark.parametrize("case", [
    # tokens, q heads, kv heads, d, rot, page, axes, interleaved, cache, order, type
    (1, 4, 2, 128, 128, 16, 1, False, "same", "hnd", F16),
    (1, 0, 1, 64, 64, 16, 1, True, "same", "nhd", BF16),
    (37, 7, 1, 80, 40, 24, 2, False, "e4m3", "hnd", F16),
    (37, 7, 1, 80, 40, 24, 2, True, "e4m3", "nhd", BF16),
    (5, 3, 3, 16, 8, 1, 1, False, "same", "nhd", BF16),
    (130, 8, 2, 256, 256, 7, 3, False, "e4m3", "nhd", BF16),
    (130, 8, 2, 256, 128, 7, 4, True, "same", "hnd", F16),
    (9, 2, 2, 72, 0, 8, 1, False, "e4m3", "hnd", BF16),
    (4200, 1, 1, 64, 64, 64, 1, False, "same", "hnd", F16),
    (600, 32, 8, 128, 128, 16, 3, False, "e4m3", "hnd", BF16),
    (1100, 24, 8, 128, 64, 16, 1, True, "same", "nhd", F16),
])
def test_rope_append(dev, case):
    t, hq, hkv, d, rot, page, axes, inter, kind, order, dtype = case
    g = rng_of(dev, 11 + t + d)
    qkv = normal(g, (t, (hq + 2 * hkv) * d), dtype)
    q, k, v = (x.unflatten(1, (-1, d)) if x.shape[1] else None
               for x in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
    scales = None
    if kind == "e4m3":
        scales = [torch.rand(hkv, generator=g, device=dev) * 0.02 + 0.004 for _ in range(2)]
    pages = -(-t // page) + 2
    cache = paged(dev, pages, page, hkv, d, E4M3 if kind == "e4m3" else dtype, order, scales, g)
    slots = torch.randperm(pages * page, generator=g, device=dev)[:t]
    if t > 4:
        slots[1], slots[3] = -1, pages * page  # padding, and a slot past the cache
    before = np64(cache.k), np64(cache.v)
    half = rot // 2
    inv = (10000.0 ** (-torch.arange(half, device=dev).double() / max(1, half))).float()
    pos = torch.randint(0, 1 << 20, (axes, t), generator=g, device=dev).to(torch.int32)
    cut = [half * i // axes for i in range(axes + 1)]
    sections = [cut[i + 1] - cut[i] for i in range(axes)]
    got = decode.rope_append(q, k, v, cache, slots, positions=pos if half else None,
                             inv_freq=inv, sections=sections, interleaved=inter)
    posn, invn = pos.cpu().numpy(), inv.cpu().numpy()
    if q is not None:
        want, err = ref.rotate(np64(q), posn, invn, sections, inter)
        check(got, want, err, "q")
    kw, kerr = ref.rotate(np64(k), posn, invn, sections, inter)
    vw, verr = np64(v), np.zeros_like(np64(v))
    for name, tensor, was, want, err, sc in (
            ("k", cache.k, before[0], kw, kerr, 0), ("v", cache.v, before[1], vw, verr, 1)):
        full, full_err = was.copy(), np.zeros_like(was)
        if scales is not None:
            s = np64(scales[sc])[:, None]
            # the quotient is fp32; E4M3's smallest half step is 2^-10
            want = np.clip(want / s, -448, 448)
            err = err / s + np.abs(want) * 2 * ref.E32 + 2.0 ** -10
        for i, slot in enumerate(slots.tolist()):
            if 0 <= slot < pages * page:
                full[slot // page, slot % page] = want[i]
                full_err[slot // page, slot % page] = err[i]
        check(tensor, full, full_err, name)


def test_rope_append_in_place_and_special_values(dev):
    """q may be rotated over itself; NaN and infinities reach an E4M3 cache as NaN and 448."""
    g = rng_of(dev, 3)
    q = normal(g, (6, 4, 64), F16)
    k, v = normal(g, (6, 1, 64), F16), normal(g, (6, 1, 64), F16)
    v[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 449.0])
    cache = paged(dev, 2, 4, 1, 64, E4M3, "hnd")
    slots = torch.arange(6, device=dev)
    pos = torch.arange(6, device=dev, dtype=torch.int32)
    inv = torch.rand(32, generator=g, device=dev)
    want = decode.rope_append(q, k, v, cache, slots, positions=pos, inv_freq=inv)
    got = decode.rope_append(q, k, v, cache, slots, positions=pos, inv_freq=inv, q_out=q)
    assert got is q and torch.equal(got, want)
    head = cache.v[0, 0, 0, :4].float()
    assert bool(head[0].isnan()) and head[1:].tolist() == [448.0, -448.0, 448.0]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rot", [64, 40])
def test_rope_append_interleaved_in_place(dev, dtype, rot):
    g = rng_of(dev, 4)
    wide = normal(g, (37, 9 * 64), dtype)
    q = wide[:, 64:320].unflatten(1, (4, 64))
    k = normal(g, (37, 1, 64), dtype)
    cache = paged(dev, 5, 8, 1, 64, dtype, "nhd")
    args = k, k, cache, torch.arange(37, device=dev)
    kw = dict(positions=torch.arange(37, device=dev, dtype=torch.int32) * 999, interleaved=True,
              inv_freq=torch.rand(rot // 2, generator=g, device=dev))
    rest = wide[:, 320:].clone()
    want = decode.rope_append(q, *args, **kw)
    assert not torch.equal(want, q)
    got = decode.rope_append(q, *args, q_out=q, **kw)
    assert torch.equal(got, want) and torch.equal(wide[:, 320:], rest)


# ---- attention ------------------------------------------------------------------------------

def attn_case(dev, lens, hq, hkv, d, page, dtype, kind="same", order="hnd", window=0, softcap=0.0,
              keep=False, max_len=None, seed=0, spare=3, poison=True):
    g = rng_of(dev, seed + 31 * d + hq)
    b = len(lens)
    top = max_len or max(1, max(lens))
    per = -(-top // page)
    scales = None
    if kind == "e4m3":
        scales = [torch.rand(hkv, generator=g, device=dev) * 0.02 + 0.005 for _ in range(2)]
    cache = paged(dev, b * per + spare, page, hkv, d, E4M3 if kind == "e4m3" else dtype, order,
                  scales, g)
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
        dead = (~live)[:, :, None, None]
        for x in (cache.k, cache.v):
            if kind == "e4m3":
                x.view(torch.uint8).masked_fill_(dead, 0x7F)
            else:
                x.masked_fill_(dead, float("nan"))
    return dict(cache=cache, table=table, lens=lens_t, q=q, keep=mask, top=top, window=window,
                softcap=softcap, hq=hq, dtype=dtype, scale=1 / math.sqrt(d))


def attn_run(c, cut=False, **kw):
    """cut: planned for sequences far longer than the table's pages (the rest are no pages of the
    cache), so that they are cut into ranges."""
    if cut:
        c = dict(c, top=c["top"] + (1 << 18) // c["cache"].head_dim)
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


def attn_check(c, out, lse, label=""):
    cache = c["cache"]
    k, v = np64(cache.k), np64(cache.v)
    if cache.k_scale is not None:
        k, v = k * np64(cache.k_scale)[:, None], v * np64(cache.v_scale)[:, None]
    want, want_lse, err, lse_err = ref.paged_attention(
        np64(c["q"]), k, v, c["table"].cpu().numpy(), c["lens"].cpu().numpy(), c["scale"],
        c["window"], c["softcap"], None if c["keep"] is None else c["keep"].cpu().numpy())
    check(out, want, err, label + " out")
    check(lse, want_lse, lse_err, label + " lse")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("d,hq,hkv,page,order", [
    (16, 1, 1, 1, "hnd"), (64, 4, 4, 16, "nhd"), (72, 6, 2, 5, "hnd"), (80, 3, 3, 24, "nhd"),
    (96, 20, 1, 16, "hnd"), (128, 8, 1, 16, "hnd"), (128, 40, 2, 64, "nhd"), (136, 2, 1, 32, "hnd"),
    (160, 4, 2, 16, "hnd"), (184, 2, 1, 16, "nhd"), (192, 16, 1, 7, "nhd"), (200, 3, 1, 9, "hnd"),
    (256, 5, 1, 16, "hnd")])
def test_attention_heads(dev, dtype, kind, d, hq, hkv, page, order):
    c = attn_case(dev, [0, 1, 15, 31, 32, 33, 127, 300], hq, hkv, d, page, dtype, kind, order)
    for cut in (False, True):
        attn_check(c, *attn_run(c, cut), f"cut {cut}")


@pytest.mark.parametrize("lens,kw", [
    ([1], {}), ([0], {}), ([2, 0, 0], {}),
    ([255, 256, 257, 129], dict(max_len=1000)),
    ([5000, 17], {}), ([12345], dict(hkv=1, hq=2)), ([4097] * 3, dict(window=100)),
    ([700, 33, 1], dict(window=1)), ([700, 33, 1], dict(window=32)), ([700, 33], dict(window=4000)),
    ([513, 64], dict(softcap=20.0)), ([900, 300, 40], dict(keep=True)),
    ([3000, 1], dict(keep=True, window=1500, softcap=5.0)),
    ([700, 33, 1], dict(hq=40, hkv=2)), ([0, 3, 64, 129] * 5, dict(hq=34)),
    ([9000, 40, 6000], dict(window=5000)), ([7000, 1], dict(keep=True, window=6500, softcap=5.0)),
])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_attention_lengths_and_masks(dev, lens, kw, kind):
    kw = dict(dict(hq=8, hkv=2), **kw)
    c = attn_case(dev, lens, d=64, page=16, dtype=BF16, kind=kind, seed=sum(lens), **kw)
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
        c = attn_case(dev, n, hq, hkv, 64, 16, BF16, max_len=longest, seed=batch)
        for cut in (False, True):
            attn_check(c, *attn_run(c, cut), f"cut {cut}")


@pytest.mark.parametrize("hq,hkv,d,order", [(96, 96, 64, "hnd"), (520, 520, 136, "hnd"),
                                            (600, 600, 72, "nhd"), (780, 20, 72, "nhd")])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_attention_of_many_units(dev, hq, hkv, d, order, kind):
    """Few ranges, or one, because a range has nearly as many work-groups as a launch, or more; with
    and without the grid that is rounded up to eight ranges."""
    c = attn_case(dev, [300, 0, 41], hq, hkv, d, 16, BF16, kind, order)
    for cut in (False, True):
        attn_check(c, *attn_run(c, cut), f"cut {cut}")


@pytest.mark.parametrize("kw", [{}, dict(kind="e4m3"), dict(keep=True)])
def test_attention_several_short_sequences_in_a_range(dev, kw):
    """Waves with no, one, two and more tiles of a sequence, in every order."""
    g = np.random.default_rng(7)
    sizes = np.array([0, 1, 31, 32, 33, 64, 96, 127, 128, 129, 160, 200, 256, 257, 300, 390])
    lens = sizes[g.integers(0, len(sizes), 260)]
    c = attn_case(dev, lens.tolist(), 8, 8, 64, 16, F16, **kw)
    attn_check(c, *attn_run(c, True))


def test_attention_a_split_without_kept_positions(dev):
    """Whole splits masked away, the first and one between others."""
    c = attn_case(dev, [6000, 5000], 4, 1, 64, 16, F16, keep=True, poison=False)
    c["keep"][:] = 1
    c["keep"][0, :2000] = 0
    c["keep"][1, 1500:4000] = 0
    attn_check(c, *attn_run(c))


def test_attention_live_infinities_and_nan(dev):
    """What live positions hold takes part: infinite values and NaN keys reach the output."""
    c = attn_case(dev, [300, 300, 300], 2, 1, 64, 16, BF16)
    at = [(c["table"][i, 5].long(), 3) for i in range(3)]
    c["cache"].v[at[0][0], at[0][1], 0, 7] = float("inf")
    c["cache"].k[at[1][0], at[1][1], 0, 0] = float("nan")
    for cut in (False, True):
        out, lse = attn_run(c, cut)
        assert bool(out[0, :, 7].isinf().all()) and int(out[0].isinf().sum()) == 2
        assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
        assert bool(out[2].isfinite().all()) and bool(lse[0].isfinite().all())


@pytest.mark.parametrize("kind,dtype", [("same", F16), ("e4m3", F16), ("e4m3", BF16)])
def test_attention_live_infinities_and_nan_of_other_types(dev, kind, dtype):
    """fp16's parts of p are cut at another place than bf16's; an E4M3 cache holds NaN only."""
    c = attn_case(dev, [300, 300, 300, 300], 2, 1, 64, 16, dtype, kind)
    k, v = c["cache"].k, c["cache"].v
    page = [c["table"][i, 5].long() for i in range(4)]
    if kind == "same":
        v[page[0], 3, 0, 7], v[page[1], 3, 0, 9] = float("inf"), float("-inf")
        k[page[2], 3, 0, 0] = float("nan")
    else:
        v.view(torch.uint8)[page[0], 3, 0, 7] = v.view(torch.uint8)[page[1], 3, 0, 9] = 0x7F
        k.view(torch.uint8)[page[2], 3, 0, 0] = 0xFF
    for cut in (False, True):
        out, lse = attn_run(c, cut)
        hit = [out[0, :, 7], out[1, :, 9]]
        if kind == "same":
            assert bool((hit[0] == math.inf).all()) and bool((hit[1] == -math.inf).all())
        else:
            assert all(bool(x.isnan().all()) for x in hit)
        assert [int((~out[i].isfinite()).sum()) for i in range(4)] == [2, 2, 128, 0]
        assert bool(out[2].isnan().all()) and bool(lse[2].isnan().all())
        assert bool(lse[[0, 1, 3]].isfinite().all())


def test_attention_scores_of_minus_infinity(dev):
    """They count for nothing, beside others and alone."""
    c = attn_case(dev, [300, 40], 2, 1, 64, 16, BF16, poison=False)
    c["q"].abs_()
    cut_off = c["table"][0, 2:9].long()
    c["cache"].k[cut_off] = 0
    c["cache"].k[cut_off, :, 0, 0] = float("-inf")
    c["cache"].k[c["table"][1, :3].long()] = 0
    c["cache"].k[c["table"][1, :3].long(), :, 0, 0] = float("-inf")
    kept = dict(c, keep=torch.ones((2, 300), dtype=torch.uint8, device=dev))
    kept["keep"][0, 32:144] = 0
    kept["keep"][1] = 0
    for cut in (False, True):
        out, lse = attn_run(c, cut)
        want, want_lse = attn_run(kept, cut)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())


def test_an_e4m3_cache_without_scales(dev):
    g = rng_of(dev, 21)
    cache = decode.PagedCache.empty(8, 16, 2, 64, E4M3, dev)
    k, v = normal(g, (100, 2, 64), F16), normal(g, (100, 2, 64), F16)
    decode.rope_append(None, k, v, cache, torch.arange(100, device=dev))
    q = normal(g, (1, 4, 64), F16)
    table = torch.arange(8, dtype=torch.int32, device=dev)[None]
    lens = torch.tensor([100], dtype=torch.int32, device=dev)
    c = dict(cache=cache, q=q, table=table, lens=lens, scale=0.125, window=0, softcap=0.0,
             keep=None, top=128, hq=4, dtype=F16)
    attn_check(c, *attn_run(c))


def test_attention_empty_rows_are_zero(dev):
    c = attn_case(dev, [600, 0, 40], 4, 2, 128, 16, F16, keep=True)
    c["keep"][2] = 0
    for cut in (False, True):  # keep[0] is all zero
        out, lse = attn_run(c, cut)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_attention_page_numbers_outside_the_cache_are_left_out(dev):
    c = attn_case(dev, [200, 64, 40], 4, 2, 64, 16, BF16, poison=False)
    c["table"][0, 3], c["table"][0, 7] = -1, c["cache"].num_pages
    c["table"][1, :] = 2 ** 31 - 1
    c["table"][2, 0] = -2 ** 31
    for cut in (False, True):
        attn_check(c, *attn_run(c, cut), f"cut {cut}")


def test_attention_lens_are_taken_into_range(dev):
    c = attn_case(dev, [100, 100], 2, 1, 64, 16, F16)
    want = attn_run(c)
    c["lens"] = torch.tensor([1000000, -5], dtype=torch.int32, device=dev)
    out, lse = attn_run(c)
    assert torch.equal(out[0], want[0][0]) and bool((out[1] == 0).all())
    assert lse[1].tolist() == [-math.inf] * 2


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("cap", [0.3, 30.0, 1e3, 1e4, 1e6, 1e30])
def test_attention_caps(dev, dtype, kind, cap):
    """From caps that flatten every score to caps that leave them as they are."""
    c = attn_case(dev, [700, 33, 1], 4, 2, 64, 16, dtype, kind, softcap=cap)
    c["q"] *= 4
    for cut in (False, True):
        out, lse = attn_run(c, cut)
        attn_check(c, out, lse, f"cut {cut}")
        if cap > 1e7:  # s / c is past the last bit: the same scores
            plain, plain_lse = attn_run(dict(c, softcap=0.0), cut)
            assert torch.allclose(lse, plain_lse, rtol=2.0 ** -20, atol=2.0 ** -20)
            # three roundings of a score of 20 at most, twice, of V up to 5; and an output step
            assert torch.allclose(out, plain, rtol=2 * torch.finfo(dtype).eps, atol=2.0 ** -12)


def test_attention_extreme_scores(dev):
    """Equal huge scores, one dominating score, and scores that fp16 p could not hold."""
    c = attn_case(dev, [400], 2, 1, 64, 16, F16, poison=False)
    c["cache"].k.fill_(20.0)
    c["q"].fill_(30.0)
    attn_check(c, *attn_run(c), "huge")
    c["cache"].k.zero_()
    c["cache"].k[c["table"][0, 0].long(), 3] = 1.0
    c["q"].fill_(2.0)  # position 3 leads by 16: the rest are exp(-16) of it
    attn_check(c, *attn_run(c), "tail")


def test_attention_small_tail_counts_in_fp16(dev):
    """40000 positions at 2^-25.2 of the largest hold 1/1000 of the sum: V is 1000 there."""
    c = attn_case(dev, [40000], 1, 1, 64, 64, F16, poison=False)
    c["cache"].k.zero_()
    c["cache"].v.fill_(1000.0)
    first = c["table"][0, 0].long()
    c["cache"].k[first, 0] = 1.0
    c["cache"].v[first, 0] = 0.0
    c["q"].fill_(17.5 / 8)  # 64 * q * scale = 17.5
    attn_check(c, *attn_run(c))


def test_attention_small_positions_beside_a_large_one(dev):
    """In every tile one position leads the others by 17.5 and holds V = 0: the output is what
    the others, at 2^-25.2 of it, hold."""
    c = attn_case(dev, [4000], 1, 1, 64, 32, F16, poison=False)
    c["cache"].k.zero_()
    c["cache"].v.fill_(60000.0)
    c["cache"].k[:, 5] = 1.0
    c["cache"].v[:, 5] = 0.0
    c["q"].fill_(17.5 / 8)
    attn_check(c, *attn_run(c))


def test_attention_strided_rows_and_given_outputs(dev):
    c = attn_case(dev, [77, 300], 4, 2, 64, 16, BF16)
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


def test_attention_offsets_past_32_bits(dev):
    """Pages beyond 4 GiB of an E4M3 cache: element and byte offsets need 64 bits."""
    pages, page, hkv, d = (1 << 20) + 64, 16, 2, 128  # 4096 bytes a page
    kv = [torch.empty((pages, hkv, page, d), dtype=torch.uint8, device=dev) for _ in range(2)]
    g = rng_of(dev, 9)
    table = torch.tensor([[pages - 1, 3, pages - 40, (1 << 19) + 5]], dtype=torch.int32, device=dev)
    small = [(torch.randn((4, hkv, page, d), generator=g, device=dev) * 50).to(E4M3)
             for _ in range(2)]
    for x, s in zip(kv, small):
        x[table[0].long()] = s.view(torch.uint8)
    far = decode.PagedCache(*(x.view(E4M3).transpose(1, 2) for x in kv))
    near = decode.PagedCache(*(x.transpose(1, 2) for x in small))
    q, lens = normal(g, (1, 4, d), BF16, 0.02), torch.tensor([61], dtype=torch.int32, device=dev)
    a = decode.PagedAttention(far, 1, 4, 64, dtype=BF16)(q, table, lens)
    order = torch.arange(4, dtype=torch.int32, device=dev)[None]
    assert torch.equal(a, decode.PagedAttention(near, 1, 4, 64, dtype=BF16)(q, order, lens))
    k = normal(g, (1, hkv, d), BF16)
    slot = torch.tensor([pages * page - 3], device=dev)
    decode.rope_append(None, k, k, far, slot)
    assert torch.equal(far.k[pages - 1, 13].float(), k[0].to(E4M3).float())


def test_attention_is_deterministic(dev):
    c = attn_case(dev, [9000, 100, 4000], 8, 2, 128, 16, BF16)
    first = attn_run(c)
    for _ in range(3):
        again = attn_run(c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ---- the mixture-of-experts layer ---------------------------------------------------------------

def moe_case(dev, tokens, experts, top_k, hidden, inter, dtype, kind="u4b8", group=128, seed=0,
             **kw):
    g = rng_of(dev, seed + 7 * tokens + experts + inter)

    def bank(k, n):
        per = 4 if kind == "e4m3" else 8
        words = torch.randint(-2 ** 31, 2 ** 31, (experts, k // per, n), generator=g, device=dev,
                              dtype=torch.int64).to(torch.int32)
        if kind == "e4m3":
            words &= ~0x08080808
        rows = 1 if group == -1 else k // group
        s = torch.rand((experts, rows, n), generator=g, device=dev)
        s = (s * 5e-4 + 1e-4 if kind == "e4m3" else s * 0.015 + 0.005).to(dtype)
        z = None
        if kind == "u4":
            z = torch.randint(-2 ** 31, 2 ** 31, (experts, rows, n // 8), generator=g, device=dev,
                              dtype=torch.int64).to(torch.int32)
        return dict(words=words, s=s, z=z)

    gate, up, down = bank(hidden, inter), bank(hidden, inter), bank(inter, hidden)

    def one(b, e):
        return dict(qweight=b["words"][e], scales=b["s"][e],
                    zeros=None if b["z"] is None else b["z"][e], group_size=group)

    pairs = [dict(gate=one(gate, e), up=one(up, e), group_size=group) for e in range(experts)]
    banks = [torch_ops.ExpertBank(x, device=dev, bf16=dtype is BF16, fp8=kind == "e4m3")
             for x in (pairs, [one(down, e) for e in range(experts)])]
    router = normal(g, (experts, hidden), dtype, 1.5 / math.sqrt(hidden))
    x = normal(g, (tokens, hidden), dtype)
    return dict(banks=banks, router=router, x=x, raw=(gate, up, down), kind=kind, group=group,
                top_k=top_k, dtype=dtype, g=g, **kw)


def dequant(b, kind, group):
    w = b["words"].cpu().numpy()
    e, r, n = w.shape
    per, bits = (4, 8) if kind == "e4m3" else (8, 4)
    code = np.stack([(w >> (bits * i)) & (2 ** bits - 1) for i in range(per)], 2).reshape(e, r * per, n)
    rows = r * per if group == -1 else group
    if kind == "e4m3":
        v = np64(torch.from_numpy(code.astype(np.uint8)).view(E4M3))
    else:
        zero = np.full((e, r * per // rows, n), 8.0)
        if b["z"] is not None:
            zw = b["z"].cpu().numpy()
            zero = np.stack([(zw >> (4 * i)) & 15 for i in range(8)], 3).reshape(e, -1, n)
        v = code - np.repeat(zero, rows, 1)
    return v * np.repeat(np64(b["s"]), rows, 1)


def moe_check(c, residual=None, renormalize=True, scale=1.0, **kw):
    layer = decode.MoELayer(*c["banks"], c["router"], c["top_k"], renormalize=renormalize,
                            routed_scale=scale)
    x = c["x"]
    layer.workspace.fill_(0xFF)  # its contents need no initialization
    y = layer(x, residual=residual, **kw)
    n = x.shape[0]
    w = [dequant(b, c["kind"], c["group"]) for b in c["raw"]]
    want, ids, weights, err = ref.moe_layer(np64(x), np64(c["router"]), *w, c["top_k"], renormalize,
                                            scale, None if residual is None else np64(residual),
                                            half_step(c["dtype"]))
    assert np.array_equal(layer.ids[:n].cpu().numpy(), ids)
    check(layer.weights[:n], weights, weights * 32 * ref.E32, "weights")
    # the routing weights' own error is relative to every term
    check(y, want, err * (1 + 64 * ref.E32) + np.abs(want) * 64 * ref.E32, "y")
    return layer, y


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind,group", [("u4b8", 128), ("u4b8", 64), ("u4b8", 32), ("u4b8", 16),
                                        ("u4b8", -1), ("u4", 128), ("u4", 64), ("u4", 32),
                                        ("u4", 16), ("e4m3", 128), ("e4m3", -1)])
@pytest.mark.parametrize("hidden,inter", [(512, 384), (1024, 896)])  # few launches, and more
def test_moe_weights(dev, dtype, kind, group, hidden, inter):
    c = moe_case(dev, 5, 6, 2, hidden, inter, dtype, kind, group)
    moe_check(c, residual=normal(c["g"], (5, hidden), dtype))


@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter,renorm", [
    (1, 1, 1, 256, 128, True), (1, 8, 2, 512, 256, False), (2, 8, 2, 256, 1408, True),
    (16, 4, 4, 256, 128, False), (16, 64, 8, 256, 128, True), (7, 256, 16, 256, 128, False),
    (13, 65, 3, 768, 128, True), (16, 1, 1, 1280, 640, True), (3, 100, 1, 256, 256, False),
    (9, 5, 3, 512, 768, True), (1, 16, 4, 512, 1024, True), (4, 3, 2, 2560, 256, False),
    (16, 2, 1, 1024, 2048, True), (1, 1, 1, 8192, 128, True), (1, 3, 2, 1280, 512, True),
    (1, 16, 16, 2048, 128, False), (1, 17, 2, 256, 256, True), (1, 8, 2, 4352, 128, True), (2, 20, 16, 256, 256, True),
])
def test_moe_shapes(dev, tokens, experts, top_k, hidden, inter, renorm):
    c = moe_case(dev, tokens, experts, top_k, hidden, inter, BF16)
    moe_check(c, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("experts", [12, 40, 70])
def test_moe_ties_take_the_lowest_expert(dev, experts):
    c = moe_case(dev, 4, experts, 5, 256, 128, F16)
    c["router"][:] = 0
    equal = [3, experts // 2 + 1, experts - 2]
    c["router"][equal] = c["router"].new_ones(256) * 0.5  # equal logits, either sign
    layer, _ = moe_check(c)
    for t in range(4):
        up = float(c["x"][t].double().sum()) > 0
        assert layer.ids[t].tolist() == (equal + [0, 1] if up else [0, 1, 2, 4, 5])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind,group", [("u4b8", 128), ("u4b8", 64), ("u4b8", 32), ("u4b8", 16),
                                        ("u4b8", -1), ("u4", 128), ("u4", 64), ("u4", 32),
                                        ("u4", 16), ("e4m3", 128), ("e4m3", -1)])
@pytest.mark.parametrize("tokens,experts,inter", [(1, 8, 1024), (16, 5, 384), (16, 17, 128),
                                                  (3, 4, 512), (8, 1, 2048), (9, 2, 2176)])
def test_moe_weights_of_small_layers(dev, dtype, kind, group, tokens, experts, inter):
    """On both sides of the border of the down projections in one launch, 16 groups of K: whole and
    half rows of work, one expert's rows up to all tokens."""
    c = moe_case(dev, tokens, experts, min(2, experts), 512, inter, dtype, kind, group)
    moe_check(c, residual=normal(c["g"], (tokens, 512), dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,experts,hidden", [(1, 8, 512), (1, 16, 2048), (1, 17, 512),
                                                   (4, 8, 512), (16, 8, 512), (16, 40, 512),
                                                   (3, 70, 512)])
@pytest.mark.parametrize("top_k", [1, 3])
def test_moe_logits_closer_than_an_fp32_step(dev, dtype, tokens, experts, hidden, top_k):
    """Two experts lead by far and differ by 2^-26 of logits near 16, the higher one ahead: the
    router's products, sums and order keep fp64 on every route (one token, a few, many; counted
    or in rounds)."""
    c = moe_case(dev, tokens, experts, top_k, hidden, 128, dtype)
    low, high = 1, experts - 2
    x, r = c["x"], c["router"]
    x[:, 0], x[:, 7], x[:, 8], x[:, 300] = 1, 2.0 ** -13, 64, 64
    r[high] = r[low]
    r[:, [8, 300]] = 0
    r[[low, high], 0], r[low, 7], r[high, 7] = 16, 0, 2.0 ** -13
    want = [high, low][:top_k]
    for cancelling in (0, 64):  # the lower one's products 4096 and -4096
        r[low, 8], r[low, 300] = cancelling, -cancelling
        layer, _ = moe_check(c)
        assert all(layer.ids[t].tolist()[:2] == want for t in range(tokens))


def test_moe_logits_past_fp32(dev):
    """bf16 products and logits beyond fp32's range are ordered, and their weights those of fp64."""
    c = moe_case(dev, 3, 8, 2, 512, 128, BF16)
    c["x"][:, 4] = 2.0 ** 60
    c["router"][:, 4] = 0
    c["router"][5, 4], c["router"][2, 4] = 2.0 ** 80, 2.0 ** 79
    layer = decode.MoELayer(*c["banks"], c["router"], 2)
    layer(c["x"])
    assert layer.ids[:3].tolist() == [[5, 2]] * 3 and layer.weights[:3].tolist() == [[1, 0]] * 3


def test_moe_strides_aliases_and_nan_rows(dev):
    c = moe_case(dev, 6, 8, 2, 512, 256, BF16)
    _, want = moe_check(c, residual=c["x"])
    layer = decode.MoELayer(*c["banks"], c["router"], 2)
    wide = torch.zeros((6, 2048), dtype=BF16, device=dev)
    wide[:, 512:1024] = c["x"]
    view = wide[:, 512:1024]
    got = layer(view, residual=view, out=view)  # over its own input
    assert torch.equal(got, want) and bool((wide[:, :512] == 0).all())
    x = c["x"].clone()
    x[2, 7] = float("nan")
    y = layer(x, residual=x)
    rest = [0, 1, 3, 4, 5]
    assert torch.equal(y[rest], want[rest]) and bool(y[2].isnan().all())
    assert bool(layer.weights[2].isnan().all())


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_moe_over_its_residual_or_input(dev, dtype):
    """The launches of a larger layer: an output over the residual, and over the input."""
    c = moe_case(dev, 6, 8, 2, 512, 1280, dtype)
    res = normal(c["g"], (6, 512), dtype)
    layer, want = moe_check(c, residual=res)
    x = c["x"].clone()
    over = torch.cat([x, res], dim=1)
    got = layer(over[:, :512], residual=over[:, 512:], out=over[:, 512:])
    assert torch.equal(got, want) and torch.equal(over[:, :512], x)
    got = layer(x, residual=res, out=x)
    assert got is x and torch.equal(x, want)
    both = c["x"].clone()
    want = layer(c["x"], residual=c["x"])
    assert torch.equal(layer(both, residual=both, out=both), want)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,experts,top_k,inter", [
    (1, 8, 3, 128), (1, 8, 2, 128), (1, 40, 2, 128), (4, 8, 3, 128), (4, 8, 3, 1280),
    (4, 40, 2, 128), (4, 70, 3, 128)])
@pytest.mark.parametrize("some", [False, True])
def test_moe_infinite_logits(dev, dtype, tokens, experts, top_k, inter, some):
    """A row whose logits are infinite (one +inf before -inf, or -inf alone) is NaN, its experts
    are in order, and the other rows are what they are without it."""
    c = moe_case(dev, tokens, experts, top_k, 512, inter, dtype)
    c["router"][:, 3] = -1
    if some:
        c["router"][experts - 3, 3] = 1
    c["x"][0, 3] = math.inf
    layer = decode.MoELayer(*c["banks"], c["router"], top_k)
    y = layer(c["x"])
    want = ([experts - 3, 0, 1] if some else [0, 1, 2])[:top_k]
    assert layer.ids[0].tolist() == want
    assert bool(layer.weights[0].isnan().all()) and bool(y[0].isnan().all())
    if tokens > 1:
        w = [dequant(b, c["kind"], c["group"]) for b in c["raw"]]
        want, ids, weights, err = ref.moe_layer(np64(c["x"][1:]), np64(c["router"]), *w, top_k, True,
                                                1.0, None, 2.0 ** -16)
        assert np.array_equal(layer.ids[1:tokens].cpu().numpy(), ids)
        check(y[1:], want, err * (1 + 64 * ref.E32) + np.abs(want) * 64 * ref.E32, "y")


@pytest.mark.parametrize("inter", [256, 1280])
@pytest.mark.parametrize("kind", ["u4b8", "e4m3"])
def test_moe_an_expert_s_values_reach_only_its_own_tokens(dev, inter, kind):
    """Infinite scales of one expert: the other tokens' rows stay what they were."""
    c = moe_case(dev, 16, 6, 2, 512, inter, F16, kind)
    layer, clean = moe_check(c)
    hit = (layer.ids[:16] == 4).any(1)
    assert 0 < int(hit.sum()) < 16
    for bank in c["banks"]:
        bank.s[4] = float("inf")
    y = layer(c["x"])
    assert torch.equal(y[~hit], clean[~hit]) and not bool(y[hit].isfinite().any())


@pytest.mark.parametrize("kind", ["u4b8", "u4", "e4m3"])
@pytest.mark.parametrize("inter", [256, 384, 896])  # few launches, and more
def test_moe_activations_past_fp16(dev, kind, inter):
    """Activations beyond 65504 under a small routing scale: the layer's output is finite."""
    c = moe_case(dev, 5, 6, 2, 512, inter, F16, kind)
    c["x"] *= 1000 if kind == "e4m3" else 300
    layer, y = moe_check(c, scale=2.0 ** -8)
    e = int(layer.ids[0, 0])
    g, u = (np64(c["x"][0]) @ dequant(b, kind, c["group"])[e] for b in c["raw"][:2])
    assert (np.maximum(g, 0) * u).max() > 65504 and bool(y.isfinite().all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind,group", [("u4b8", 128), ("u4", 16), ("e4m3", 128)])
@pytest.mark.parametrize("tokens,inter", [(3, 256), (16, 256), (3, 1280), (16, 1280)])
def test_moe_rounds_its_output_only(dev, dtype, kind, group, tokens, inter):
    """The error of y (2-norm) is that of its one rounding: the activation's 16 bits add a part of
    2^-16 a term, against y's half step of 2^-11 or more; a tenth is left for fp32 sums and
    for the number of elements."""
    c = moe_case(dev, tokens, 6, 2, 512, inter, dtype, kind, group)
    _, y = moe_check(c)
    w = [dequant(b, kind, group) for b in c["raw"]]
    want = ref.moe_layer(np64(c["x"]), np64(c["router"]), *w, 2, True, 1.0, None, 2.0 ** -16)[0]
    rounded = np64(torch.from_numpy(want).to(dtype))
    assert np.linalg.norm(np64(y) - want) <= 1.1 * np.linalg.norm(rounded - want)


# ---- streams and graphs -----------------------------------------------------------------------

def test_a_decode_step_on_another_stream_and_in_a_graph(dev):
    """All four on a side stream, then captured and replayed on changed inputs: the replays
    give what eager calls give."""
    c = attn_case(dev, [100, 37], 4, 2, 128, 16, BF16, poison=False, max_len=400)
    m = moe_case(dev, 2, 4, 2, 512, 256, BF16)
    layer = decode.MoELayer(*m["banks"], m["router"], 2)
    plan = decode.PagedAttention(c["cache"], 2, 4, 400, dtype=BF16)
    norm_w = normal(m["g"], (512,), BF16)
    inv = torch.rand(64, device=dev)
    x, delta = normal(m["g"], (2, 512), BF16), normal(m["g"], (2, 512), BF16)
    q, k, v = (normal(m["g"], (2, h, 128), BF16) for h in (4, 2, 2))
    slots = c["table"][:, 6].long() * 16 + 4
    pos = torch.tensor([100, 100], dtype=torch.int32, device=dev)
    lens = torch.tensor([101, 101], dtype=torch.int32, device=dev)

    def step():
        y, s = decode.add_rms_norm(x, norm_w, delta=delta)
        qr = decode.rope_append(q, k, v, c["cache"], slots, positions=pos, inv_freq=inv)
        o = plan(qr, c["table"], lens)
        z = layer((y + o.flatten(1)), residual=s)
        return y, s, qr, o, z

    eager = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        x.copy_(normal(m["g"], (2, 512), BF16))
        q.copy_(normal(m["g"], (2, 4, 128), BF16))
        lens.fill_(101 + 40 * i)
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, held)), i


def test_the_example_layer_against_its_formula(dev):
    """examples/decode_layer.py, a small layer: eager and graph steps agree bit for bit, and the
    first step is what the formula gives, within 1.5% (2-norm): six 16-bit roundings in a row,
    each 2^-11 of its value, through products that keep their inputs' relative error."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.run(3, 5, 100, hidden=512, q_heads=8, kv_heads=2, head_dim=64, inter=256,
                    experts=4)
    assert torch.equal(r["eager"], r["graph"])
    layer, n = r["layer"], 3

    def weight(w):  # [k][n] in 64 bits
        out = torch.empty((w.k, w.n), dtype=torch.float16, device=dev)
        wq.wq_dequant(w.b, w.s, w.z, out, k=w.k, n=w.n)
        return np64(out)

    def expert(bank, e):
        out = torch.empty((bank.k, bank.n), dtype=torch.float16, device=dev)
        wq.wq_dequant(bank.b[e], bank.s[e], None, out, k=bank.k, n=bank.n)
        return np64(out)

    y, s = ref.add_rms_norm(np64(r["x"]), np64(r["delta"]), 1.0, 1e-6)
    qkv = y @ weight(layer.w_qkv)
    q = qkv[:, :512].reshape(n, 8, 64)
    pos = r["start"].cpu().numpy()[None]
    q, _ = ref.rotate(q, pos, layer.inv_freq.cpu().numpy(), [32], False)
    # the cache holds the prompts and the steps' keys and values
    o, _, _, _ = ref.paged_attention(q, np64(layer.cache.k), np64(layer.cache.v),
                                     layer.table.cpu().numpy(), pos[0] + 1, 1 / 8)
    o = o.reshape(n, -1) @ weight(layer.w_out)
    y, s = ref.add_rms_norm(s, o, 1.0, 1e-6)
    pairs = [expert(layer.moe.gate_up, e).reshape(512, -1, 2, 16) for e in range(4)]
    gate, up = (np.stack([p[:, :, i].reshape(512, -1) for p in pairs]) for i in range(2))
    down = np.stack([expert(layer.moe.down, e) for e in range(4)])
    want, _, _, _ = ref.moe_layer(y, np64(layer.moe.router), gate, up, down, 2, True, 1.0, s, 0.0)
    got = np64(r["eager"][0])
    assert np.linalg.norm(got - want) <= 0.015 * np.linalg.norm(want)
