"""The choice of the next token on the GPU against its 64-bit form (oracle/decode.py).

A token has to be the formula's wherever the formula's own borders leave it certain.  logprob is the
log of a share, as far as that is certain, rounded to fp32."""

import math

import numpy as np
import pytest

from oracle import decode as ref

torch = pytest.importorskip("torch")
wq = pytest.importorskip("weight_only_quantized_gemm_amd")
from weight_only_quantized_gemm_amd import decode  # noqa: E402

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def run(logits, u, plan=None, **settings):
    dev = logits.device
    plan = plan or decode.Sampler(logits.shape[0], logits.shape[1], dtype=logits.dtype, device=dev)
    plan.workspace.fill_(0xFF)  # its contents need no initialization
    given = {n: torch.tensor(x, dtype=torch.int32 if n == "top_k" else F32, device=dev)
             for n, x in settings.items() if x is not None}
    return plan(logits, torch.tensor(u, dtype=F32, device=dev), logprob=True, **given)


def verify(logits, u, ids, logprob, label="", **settings):
    """How many rows are certain, all of them checked."""
    z, u = logits.double().cpu().numpy(), np.asarray(u, dtype=np.float32).astype(np.float64)
    ids, logprob = ids.cpu().numpy(), logprob.double().cpu().numpy()
    clear = 0
    for r in range(len(z)):
        kw = {n: (int(x[r]) if n == "top_k" else float(np.float32(x[r])))
              for n, x in settings.items() if x is not None}
        want, want_log, certain, off = ref.sample(z[r], u[r], **kw)
        if not certain:
            continue
        clear += 1
        assert ids[r] == want, (label, r, kw, u[r], int(ids[r]), want)
        if math.isnan(want_log):
            assert math.isnan(logprob[r]), (label, r)
        else:
            assert abs(logprob[r] - want_log) <= abs(want_log) * 2.0 ** -24 * 1.01 + 2 * off + 2.0 ** -40, (label, r)
    return clear


def sample_check(logits, u, label="", most=0, **settings):
    ids, logprob = run(logits, u, **settings)
    clear = verify(logits, u, ids, logprob, label, **settings)
    assert clear >= len(u) - most, (label, clear)
    return ids, logprob


def logits_of(g, rows, vocab, dtype, sd=2.5):
    """Rows of a wide middle and a few tokens that stand out."""
    z = g.normal(size=(rows, vocab)) * sd
    hot = g.integers(0, vocab, (rows, min(vocab, 40)))
    np.put_along_axis(z, hot, np.take_along_axis(z, hot, 1) + g.uniform(0, 14, hot.shape), 1)
    return torch.tensor(z, dtype=dtype, device="cuda:0")


SETTINGS = [
    dict(), dict(temperature=[0.7, 1.5, 0.0, 5.0]), dict(top_k=[1, 5, 50, 1000]),
    dict(top_k=[0, -3, 10 ** 6, 2]), dict(top_p=[0.1, 0.9, 0.99, 1.0]), dict(top_p=[0.0, 0.5, 2.0, 0.9999]),
    dict(min_p=[0.0, 0.05, 0.5, 1.0]), dict(top_k=[20, 20, 300, 3000], top_p=[0.5, 0.95, 0.9, 0.999]),
    dict(temperature=[0.8, 1.2, 1.0, 0.3], top_k=[0, 40, 7, 0], top_p=[0.9, 1.0, 0.8, 0.95],
         min_p=[0.02, 0.1, 0.0, 0.001]),
]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("vocab", [1, 2, 7, 63, 64, 65, 255, 257, 511, 512, 513, 1000, 4097, 8193, 50001, 128000])
def test_sample(dev, dtype, vocab):
    g = np.random.default_rng(vocab)
    for i, settings in enumerate(SETTINGS):
        z = logits_of(g, 4, vocab, dtype)
        sample_check(z, g.random(4).astype(np.float32), f"settings {i}", **settings)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,vocab", [(1, 200003), (2, 524288), (40, 32000), (300, 1001), (513, 300), (1500, 50)])
def test_sample_batches(dev, dtype, rows, vocab):
    g = np.random.default_rng(rows)
    z = logits_of(g, rows, vocab, dtype)
    pick = lambda *x: np.asarray(x)[g.integers(0, len(x), rows)]  # noqa: E731
    # (2^19 borders, each uncertain over 2^-21 of the sum)
    sample_check(z, g.random(rows).astype(np.float32), most=2 if vocab == 524288 else 1, temperature=pick(0.0, 0.5, 1.0, 2.0),
                 top_k=pick(0, 0, 1, 30, 900), top_p=pick(1.0, 0.3, 0.95), min_p=pick(0.0, 0.0, 0.03))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("sd", [0.0, 1e-3, 0.3])
def test_sample_flat_logits(dev, dtype, sd):
    """All equal, nearly equal, and close together: ties of thousands, cuts inside them."""
    g = np.random.default_rng(5)
    for settings in (dict(), dict(top_k=[1, 3, 20000, 49999]), dict(top_p=[1e-6, 0.1, 0.5, 0.99]),
                     dict(top_k=[7, 300, 30000, 50000], top_p=[0.4, 0.999, 0.5, 0.7]),
                     dict(min_p=[0.2, 0.9, 0.99, 1.0], temperature=[1.0, 3.0, 100.0, 0.01])):
        z = torch.tensor(g.normal(size=(4, 50001)) * sd, dtype=dtype, device=dev)
        # of 50001 equal tokens a border is at every multiple of 1 / n: 2^-24 may fall on one
        sample_check(z, g.random(4).astype(np.float32), str(settings), most=1, **settings)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_sample_ties_at_the_cut_go_by_number(dev, dtype):
    z = torch.zeros((6, 3000), dtype=dtype, device=dev)
    z[:, [17, 1000, 2999]] = 2.0
    z[:, 5::7] += 1.0  # (not among the three)
    z[:, [17, 1000, 2999]] = 2.0
    u = [0.0, 0.3, 0.5, 0.7, 0.95, 1 - 2.0 ** -24]
    ids, _ = sample_check(z, u, most=1, top_k=[2] * 6)  # (0.5 lies on the border, exactly)
    assert ids.tolist() == [17, 17, 1000, 1000, 1000, 1000]
    ids, _ = sample_check(z, u, top_k=[5] * 6)  # and the two lowest of the next value
    ones = [i for i in range(5, 3000, 7) if i not in (17, 1000, 2999)][:2]
    assert set(ids.tolist()) <= {17, 1000, 2999, *ones} and ids[0] == ones[0]
    ids, logprob = run(z, u, top_k=[1] * 6)
    assert ids.tolist() == [17] * 6 and logprob.tolist() == [0.0] * 6


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("vocab", [9, 700, 40000])
def test_sample_masked_and_infinite_logits(dev, dtype, vocab):
    """-inf and the type's lowest value are never chosen; +inf takes all; NaN and nothing at all."""
    low = torch.finfo(dtype).min
    z = torch.full((7, vocab), -math.inf, dtype=dtype, device=dev)
    z[0, 4] = -3.0
    z[1] = low
    z[1, [2, 7]] = 1.0
    z[2] = 0.5
    z[2, 3] = math.inf
    z[3] = 0.5
    z[3, [1, 8]] = math.inf
    z[4] = 0.5
    z[4, vocab - 1] = math.nan
    z[6, 1:] = -math.inf
    z[6, 0] = low
    u = [0.99, 0.6, 0.2, 0.7, 0.5, 0.5, 0.5]
    for settings in (dict(), dict(top_k=[3] * 7), dict(top_p=[0.9] * 7), dict(min_p=[0.3] * 7),
                     dict(top_k=[5] * 7, top_p=[0.8] * 7), dict(temperature=[0.0] * 7)):
        ids, logprob = sample_check(z, u, str(settings), **settings)
        hot = settings.get("temperature") is None
        assert ids.tolist() == [4, 7 if hot else 2, 3, 8 if hot else 1, -1, -1, 0]
        assert bool(logprob[4:6].isnan().all()) and logprob[[0, 2, 6]].tolist() == [0.0] * 3


def test_sample_temperatures_and_settings_out_of_range(dev):
    g = np.random.default_rng(8)
    z = logits_of(g, 8, 5000, F32)
    u = g.random(8).astype(np.float32)
    t = [0.0, -1.0, math.nan, 1e-30, 1e-44, 3e38, math.inf, 1e-3]
    ids, logprob = sample_check(z, u, temperature=[x if x == x else 0.0 for x in t])
    again, _ = run(z, u, temperature=t)
    assert torch.equal(ids, again)
    top = z.argmax(1)
    assert torch.equal(ids[:5].long(), top[:5]) and logprob[:5].tolist() == [0.0] * 5
    base = run(z, u)
    for settings in (dict(top_k=[0, -1, -2 ** 31, 5000, 5001, 2 ** 31 - 1, 0, 0]),
                     dict(top_p=[1.0, 1.5, math.nan, math.inf, 1.0, 1.0, 1.0, 1.0]),
                     dict(min_p=[0.0, -1.0, math.nan, -math.inf, 0.0, 0.0, 0.0, 0.0])):
        got = run(z, u, **settings)
        assert torch.equal(got[0], base[0]) and torch.equal(got[1], base[1])
    for settings in (dict(top_p=[0.0, -1.0, -math.inf, 1e-40] * 2), dict(min_p=[1.0, 1.5, math.inf, 3e38] * 2)):
        ids, logprob = run(z, u, **settings)
        assert torch.equal(ids.long(), top) and logprob.tolist() == [0.0] * 8


def test_sample_random_numbers_at_the_ends(dev):
    z = torch.full((7, 600), -math.inf, device=dev)
    z[:, [3, 300, 590]] = torch.tensor([0.0, 1.0, -1.0], device=dev)
    u = [0.0, -1.0, math.nan, 1 - 2.0 ** -24, 1.0, 5.0, math.inf]
    ids, _ = run(z, u)
    assert ids.tolist() == [3, 3, 3, 590, 590, 590, 590]


def test_sample_frequencies(dev):
    """Evenly spaced random numbers hit each token in proportion, within one."""
    p = np.array([0.5, 0.25, 0.125, 0.0625, 0.0625])
    z = torch.full((4000, 1000), -math.inf, device=dev)
    at = [0, 255, 256, 511, 999]
    z[:, at] = torch.tensor(np.log(p), dtype=F32, device=dev)
    ids, _ = run(z, (np.arange(4000) + 0.5) / 4000)
    for i, share in zip(at, p):
        assert abs(int((ids == i).sum()) - 4000 * share) <= 1


@pytest.mark.parametrize("dtype", [F16, F32])
def test_sample_strided_rows(dev, dtype):
    """Rows at every offset from 16 bytes; the elements around them are never used."""
    g = np.random.default_rng(11)
    wide = torch.full((5, 5013), math.nan, dtype=dtype, device=dev)
    z = logits_of(g, 5, 4999, dtype)
    u = g.random(5).astype(np.float32)
    settings = dict(top_k=[0, 50, 0, 9, 0], top_p=[0.9, 1.0, 1.0, 0.5, 1.0])
    want = sample_check(z, u, **settings)
    for start in range(1, 9):
        view = wide[:, start:start + 4999]
        view.copy_(z)
        got = run(view, u, **settings)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), start
        wide.fill_(math.nan)


def test_sample_fewer_rows_than_planned_and_given_outputs(dev):
    g = np.random.default_rng(12)
    z = logits_of(g, 9, 3001, BF16)
    u = g.random(9).astype(np.float32)
    plan = decode.Sampler(9, 3001, dtype=BF16, device=dev)
    want = run(z, u, plan, top_p=[0.9] * 9)
    one = run(z[4:5], u[4:5], plan, top_p=[0.9])
    assert torch.equal(one[0], want[0][4:5]) and torch.equal(one[1], want[1][4:5])
    ids = torch.full((9,), -7, dtype=torch.int32, device=dev)
    got = plan(z, torch.tensor(u, device=dev), top_p=torch.full((9,), 0.9, device=dev), ids=ids)
    assert got is ids and torch.equal(ids, want[0])


def test_sample_on_another_stream_and_in_a_graph(dev):
    """Replays on changed inputs give what eager calls give; two plans' graphs do not mix."""
    g = np.random.default_rng(13)
    z = [logits_of(g, 3, 30011, BF16) for _ in range(2)]
    u = torch.tensor(g.random(3), dtype=F32, device=dev)
    kw = dict(temperature=torch.tensor([1.0, 0.5, 0.0], device=dev),
              top_k=torch.tensor([0, 40, 0], dtype=torch.int32, device=dev),
              top_p=torch.tensor([0.9, 0.8, 1.0], device=dev))
    plans = [decode.Sampler(3, 30011, dtype=BF16, device=dev) for _ in range(2)]
    eager = [p(x, u, logprob=True, **kw) for p, x in zip(plans, z)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = plans[0](z[0], u, logprob=True, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager[0], other))
    graphs, held = [], []
    for p, x in zip(plans, z):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(p(x, u, logprob=True, **kw))
    for i in range(3):
        for x in z:
            x.copy_(logits_of(g, 3, 30011, BF16))
        u.copy_(torch.tensor(g.random(3), dtype=F32))
        eager = [[t.clone() for t in p(x, u, logprob=True, **kw)] for p, x in zip(plans, z)]
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, held):
            assert all(torch.equal(s, t) for s, t in zip(a, b)), i


@pytest.mark.parametrize("vocab", [700, 128000])
def test_sample_is_deterministic(dev, vocab):
    g = np.random.default_rng(14)
    z = logits_of(g, 5, vocab, F32, 0.5)
    u = g.random(5).astype(np.float32)
    kw = dict(top_p=[0.9, 0.99, 0.5, 0.95, 1.0], top_k=[0, 10000, 0, 500, 0])
    first = run(z, u, **kw)
    for _ in range(5):
        again = run(z, u, **kw)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
