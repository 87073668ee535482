"""The 4-bit cache's operators and the token's choice as they are used together: a step of them on
other streams and in graphs, the example's layer and its tokens; and the largest strides and batches."""

import importlib.util
import math
import os

import numpy as np
import pytest

from oracle import decode as ref

torch = pytest.importorskip("torch")
wq = pytest.importorskip("weight_only_quantized_gemm_amd")
from weight_only_quantized_gemm_amd import decode  # noqa: E402

from test_decode_gpu import BF16, F16, normal, np64, rng_of  # noqa: E402
from test_decode4_gpu import attn_case, attn_check, attn_run, paged4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


class Step:
    """Norms, rotary positions and the cache write, attention, a product to logits, and the choice,
    for two sequences, one of them long enough to be cut into ranges."""

    def __init__(self, dev, dtype, seed, order):
        g = self.g = rng_of(dev, seed)
        self.dtype, self.hq, self.hkv, self.d, self.vocab = dtype, 8, 2, 128, 4001
        pages, top = 700, 9000
        self.cache = paged4(dev, pages, 16, self.hkv, self.d, 64, dtype, order, g)
        self.table = torch.stack([torch.randperm(pages, generator=g, device=dev)[:563]
                                  for _ in range(2)]).to(torch.int32)
        self.plan = decode.PagedAttention(self.cache, 2, self.hq, top, dtype=dtype)
        assert self.plan.workspace.numel()
        self.sampler = decode.Sampler(2, self.vocab, dtype=dtype, device=dev)
        self.norms = [1 + normal(g, (self.d,), dtype, 0.1) for _ in range(2)]
        self.inv = torch.rand(self.d // 2, generator=g, device=dev)
        self.w = normal(g, (self.hq * self.d, self.vocab), dtype, 0.2)
        self.qkv = torch.empty((2, (self.hq + 2 * self.hkv) * self.d), dtype=dtype, device=dev)
        self.lens = torch.empty(2, dtype=torch.int32, device=dev)
        self.u = torch.empty(2, device=dev)
        self.settings = dict(temperature=torch.tensor([0.7, 1.2], device=dev),
                             top_k=torch.tensor([0, 50], dtype=torch.int32, device=dev),
                             top_p=torch.tensor([0.9, 0.95], device=dev))
        self.next()

    def next(self):
        self.qkv.copy_(normal(self.g, self.qkv.shape, self.dtype))
        self.lens.copy_(torch.tensor([int(torch.randint(1, 8900, (1,), generator=self.g,
                                                        device=self.g.device)), 150]))
        self.u.copy_(torch.rand(2, generator=self.g, device=self.g.device))

    def __call__(self):
        d = self.d
        q, k, v = (x.unflatten(1, (-1, d)) for x in
                   self.qkv.split([self.hq * d, self.hkv * d, self.hkv * d], dim=1))
        page = self.table.gather(1, (self.lens // 16).long()[:, None])[:, 0].long()
        slots = page * 16 + self.lens % 16
        q = decode.rope_append(q, k, v, self.cache, slots, positions=self.lens, inv_freq=self.inv,
                               q_norm=self.norms[0], k_norm=self.norms[1])
        o, lse = self.plan(q, self.table, self.lens + 1, lse=True)
        logits = o.flatten(1) @ self.w
        ids, logprob = self.sampler(logits, self.u, logprob=True, **self.settings)
        return (q, o, lse, logits, ids, logprob, *self.cache.read(slots))


@pytest.mark.parametrize("dtype,order", [(F16, "hnd"), (BF16, "nhd")])
def test_a_step_on_other_streams_and_in_graphs(dev, dtype, order):
    """Two steps of their own caches and plans: at once on two streams, then each captured and
    replayed on changed inputs with eager work between the replays."""
    steps = [Step(dev, dtype, 50 + i, order) for i in range(2)]
    eager = [[t.clone() for t in s()] for s in steps]
    for s, e in zip(steps, eager):  # the choice is the oracle's
        for r in range(2):
            kw = {n: float(x[r]) for n, x in s.settings.items()}
            kw["top_k"] = int(kw["top_k"])
            want, _, certain, _ = ref.sample(np64(e[3][r]), float(s.u[r]), **kw)
            assert not certain or int(e[4][r]) == want
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in steps]
    others = []
    for side, s in zip(sides, steps):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            others.append(s())
    torch.cuda.synchronize()
    for e, o in zip(eager, others):
        assert all(torch.equal(a, b) for a, b in zip(e, o))
    graphs, held = [], []
    for s in steps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(s())
    for i in range(4):
        for s in steps:
            s.next()
        eager = [[t.clone() for t in s()] for s in steps]
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for e, h in zip(eager, held):
            assert all(torch.equal(a, b) for a, b in zip(e, h)), i


def example_module():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


SHAPE = dict(hidden=512, q_heads=8, kv_heads=2, head_dim=64, inter=256, experts=4)


def test_the_example_layer_on_a_4_bit_cache(dev):
    """The layer with a 4-bit cache and normed heads: eager and graph steps agree bit for bit, and
    the first step is what the formula gives on the cache's own values, within 1.5% (2-norm): the
    16-bit roundings between its products, each 2^-11 of its value."""
    r = example_module().run(3, 5, 100, cache4=True, qk_norm=True, **SHAPE)
    assert torch.equal(r["eager"], r["graph"])
    layer, n = r["layer"], 3

    def weight(w):  # [k][n] in 64 bits
        out = torch.empty((w.k, w.n), dtype=F16, device=dev)
        wq.wq_dequant(w.b, w.s, w.z, out, k=w.k, n=w.n)
        return np64(out)

    def expert(bank, e):
        out = torch.empty((bank.k, bank.n), dtype=F16, device=dev)
        wq.wq_dequant(bank.b[e], bank.s[e], None, out, k=bank.k, n=bank.n)
        return np64(out)

    y, s = ref.add_rms_norm(np64(r["x"]), np64(r["delta"]), 1.0, 1e-6)
    q = (y @ weight(layer.w_qkv))[:, :512].reshape(n, 8, 64)
    q, _ = ref.head_norm(q, np64(layer.q_norm), 1e-6)
    pos = r["start"].cpu().numpy()[None]
    q, _ = ref.rotate(q, pos, layer.inv_freq.cpu().numpy(), [32], False)
    cache = layer.cache  # the prompts' keys and values, and the steps'
    kv = [ref.values4(x.cpu().numpy(), np64(p))
          for x, p in ((cache.k, cache.k_pairs), (cache.v, cache.v_pairs))]
    o, _, _, _ = ref.paged_attention(q, *kv, layer.table.cpu().numpy(), pos[0] + 1, 1 / 8)
    o = o.reshape(n, -1) @ weight(layer.w_out)
    y, s = ref.add_rms_norm(s, o, 1.0, 1e-6)
    pairs = [expert(layer.moe.gate_up, e).reshape(512, -1, 2, 16) for e in range(4)]
    gate, up = (np.stack([p[:, :, i].reshape(512, -1) for p in pairs]) for i in range(2))
    down = np.stack([expert(layer.moe.down, e) for e in range(4)])
    want, _, _, _ = ref.moe_layer(y, np64(layer.moe.router), gate, up, down, 2, True, 1.0, s, 0.0)
    got = np64(r["eager"][0])
    assert np.linalg.norm(got - want) <= 0.015 * np.linalg.norm(want)


@pytest.mark.parametrize("cache4", [True, False])
def test_the_example_generates_tokens(dev, cache4):
    """Tokens that feed the next step: those of the graph are those of the eager steps, and the last
    ones are the oracle's choice from the last logits."""
    r = example_module().generate(3, 6, 90, 1024, cache4=cache4, qk_norm=True, **SHAPE)
    (ids, logprob), (graph_ids, graph_logprob) = r["eager"], r["graph"]
    assert torch.equal(ids, graph_ids) and torch.equal(logprob, graph_logprob)
    layer = r["layer"]
    assert torch.equal(layer.ids, ids[-1]) and bool(((ids >= 0) & (ids < 1024)).all())
    for b in range(3):
        want, share, certain, off = ref.sample(
            np64(layer.logits[b]), float(r["u"][-1, b]), float(layer.temperature[b]), 40,
            float(layer.top_p[b]))
        if certain:
            assert int(ids[-1, b]) == want
            assert abs(float(logprob[-1, b]) - share) <= abs(share) * 2.0 ** -23 + 2 * off


def test_pages_far_apart(dev):
    """Strides of pages of more than 2^32 elements, for codes and pairs, and of a whole page's slots."""
    d, hkv, page, group = 64, 2, 16, 32
    g = rng_of(dev, 77)
    near = paged4(dev, 3, page, hkv, d, group, BF16, "nhd", g)
    far_page = (1 << 31) + 64  # bytes of codes
    pool = torch.empty(2 * (2 * far_page + page * hkv * d), dtype=torch.uint8, device=dev)
    order = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=dev)
    q, lens = normal(g, (1, 6, d), BF16), torch.tensor([43], dtype=torch.int32, device=dev)
    want = decode.PagedAttention(near, 1, 6, 48, dtype=BF16)(q, order, lens)
    for slot_bytes in (hkv * d // 2, far_page // page // 64 * 64):
        step = far_page if slot_bytes < 1024 else hkv * d // 2
        # far slots: a page's span is 2^31 bytes, and pages lie between each other's slots
        kv = [torch.as_strided(pool, (3, page, hkv, d // 2), (step, slot_bytes, d // 2, 1), at)
              for at in (0, 1 << 12)]
        for x, y in zip(kv, (near.k, near.v)):
            for i in range(3):
                x[i].copy_(y[i])
        far = decode.PagedCache4(*kv, near.k_pairs, near.v_pairs)
        got = decode.PagedAttention(far, 1, 6, 48, dtype=BF16)(q, order, lens)
        assert torch.equal(got, want), slot_bytes
        slots = torch.tensor([5, 47, 5, 20], device=dev)
        for a, b in zip(far.read(slots), near.read(slots)):
            assert torch.equal(a, b), slot_bytes


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,group,hq,hkv", [(64, 32, 4, 4), (80, 80, 6, 3), (128, 64, 8, 2),
                                            (128, 32, 32, 2), (256, 32, 5, 1)])
def test_query_heads_of_infinities_and_nan(dev, dtype, d, group, hq, hkv):
    """They give NaN, of a sequence with live positions, and leave all others as they are."""
    for cut in (False, True):
        c = attn_case(dev, [300, 64, 0, 1], hq, hkv, d, group, 16, dtype)
        clean, clean_lse = attn_run(c, cut)
        hit = torch.zeros((4, hq), dtype=torch.bool, device=dev)
        hit[0, 1] = hit[3, 2] = True
        for bad in (math.nan, math.inf, -math.inf):
            q = c["q"].clone()
            q[0, 1, 5] = q[3, 2, d - 1] = q[2, 0, 0] = bad
            out, lse = attn_run(dict(c, q=q), cut)
            assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all()), (cut, bad)
            assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,group", [(64, 32), (80, 80), (128, 128), (128, 64), (256, 32)])
def test_query_heads_with_a_large_element(dev, dtype, d, group):
    """A few large elements (some just below a power of two) beside small ones, which still count."""
    c = attn_case(dev, [300, 64, 1, 700], 6, 2, d, group, 16, dtype)
    q = c["q"] * 0.25
    for i, x in enumerate((40.0, 31.9, 63.75, 500.0, 128.0, 3.98)):
        q[:, i, (7 * i) % d] = x
        q[0, i, (11 * i + 20) % d] = -x
    c["q"] = q
    for cut in (False, True):
        attn_check(c, *attn_run(c, cut), f"cut {cut}")


def test_head_norms_below_normal_squares(dev):
    """Squares among fp32's smallest numbers count: with an eps of 0 a head is of size one."""
    k = torch.full((2, 1, 64), 2.0 ** -70, dtype=BF16, device=dev)
    k[1] = 2.0 ** -66
    cache = decode.PagedCache.empty(1, 16, 1, 64, BF16, dev)
    decode.rope_append(None, k, k, cache, torch.arange(2, device=dev), k_norm=torch.ones_like(k[0, 0]),
                       eps=0.0)
    assert bool((cache.k[0, :2] == 1).all())


def test_a_slot_read_twice(dev):
    cache = paged4(dev, 2, 16, 3, 128, 64, F16, "hnd")
    slots = torch.tensor([7, 7, 31, 7, -1], device=dev)
    k, v = cache.read(slots)
    for x in (k, v):
        assert torch.equal(x[0], x[1]) and torch.equal(x[0], x[3]) and bool((x[4] == 0).all())


def test_the_most_rows_of_a_choice(dev):
    """65535 rows: top_k of one is the largest logit's token, and so is a temperature of zero."""
    rows, vocab = 65535, 37
    g = rng_of(dev, 3)
    z = torch.randperm(rows * vocab, generator=g, device=dev).view(rows, vocab).float() * 1e-3
    u = torch.rand(rows, generator=g, device=dev)
    plan = decode.Sampler(rows, vocab, device=dev)
    one = torch.ones(rows, dtype=torch.int32, device=dev)
    best = z.argmax(1).int()
    assert torch.equal(plan(z, u, top_k=one), best)
    assert torch.equal(plan(z, u, temperature=torch.zeros(rows, device=dev)), best)
    ids, logprob = plan(z, u, top_p=torch.full((rows,), math.inf, device=dev), logprob=True)
    assert bool(((ids >= 0) & (ids < vocab)).all()) and bool((logprob <= 0).all())
