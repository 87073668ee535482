"""How near the 4-bit attention comes to its formula, on the GPU: against the 64-bit form for the q
that its products take (oracle/decode.py: held4), so that only fp32 arithmetic and the output's
rounding are left to the bounds.  These are held against the outputs' own size: a bound that would
let a wrong output pass fails its test."""

import math

import numpy as np
import pytest

from oracle import decode as ref

torch = pytest.importorskip("torch")
wq = pytest.importorskip("weight_only_quantized_gemm_amd")

from test_decode_gpu import BF16, F16, check, half_step, np64  # noqa: E402
from test_decode4_gpu import attn_case, attn_run  # noqa: E402

pytestmark = pytest.mark.gpu

# d, group, q heads, KV heads, order: each head size with its groups, in one and two sets of columns
# and with two KV heads to a set
SHAPES = [
    (16, 16, 2, 1, "hnd"), (24, 24, 40, 2, "nhd"), (64, 32, 4, 4, "nhd"), (64, 64, 20, 1, "hnd"),
    (64, 32, 18, 2, "hnd"), (72, 72, 6, 2, "hnd"), (80, 80, 3, 3, "nhd"), (96, 32, 10, 2, "hnd"),
    (96, 96, 34, 2, "nhd"), (120, 120, 4, 2, "hnd"), (128, 32, 16, 2, "hnd"), (128, 32, 2, 2, "nhd"),
    (128, 64, 8, 2, "nhd"), (128, 64, 18, 2, "hnd"), (128, 128, 40, 2, "nhd"), (136, 136, 2, 1, "hnd"),
    (160, 32, 4, 2, "hnd"), (184, 184, 2, 1, "nhd"), (192, 32, 6, 2, "nhd"), (192, 64, 3, 3, "hnd"),
    (192, 192, 8, 2, "nhd"), (224, 32, 5, 1, "hnd"), (256, 32, 4, 4, "hnd"), (256, 32, 6, 2, "nhd"),
    (256, 64, 4, 4, "nhd"), (256, 128, 17, 1, "hnd"), (256, 256, 8, 2, "nhd")]


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def exact(c, **kw):
    cache = c["cache"]
    k, v = ((x.cpu().numpy(), np64(y))
            for x, y in ((cache.k, cache.k_pairs), (cache.v, cache.v_pairs)))
    return ref.paged_attention4(np64(c["q"]), k, v, c["table"].cpu().numpy(), c["lens"].cpu().numpy(),
                                c["scale"], c["window"], c["softcap"],
                                None if c["keep"] is None else c["keep"].cpu().numpy(), **kw)


def near(c):
    want, want_lse, err, lse_err = exact(c)
    long = (c["lens"] >= 300).cpu().numpy()
    size, room, n = (np.linalg.norm(want[long], axis=-1), np.linalg.norm(err[long], axis=-1),
                     c["lens"].cpu().numpy()[long][:, None])
    # (scores of 1 / sqrt(d) of q's and K's products; a bound grows with theirs)
    q = np64(c["q"])
    scores = max(1.0, abs(c["scale"]) * math.sqrt(np.square(q).mean() * q.shape[-1]))
    assert (room <= 0.15 * scores * size).all(), float((room / size).max())
    for cut in (False, True):
        out, lse = attn_run(c, cut)
        check(out, want, err, f"out, cut {cut}")
        check(lse, want_lse, lse_err, f"lse, cut {cut}")
        # the positions' errors have signs of their own: of n, the bound's 1 / sqrt(n), four times
        off = np.linalg.norm((np64(out) - want)[long], axis=-1)
        assert (off <= half_step(c["dtype"]) * size + 4 * room / np.sqrt(n)).all(), cut


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,group,hq,hkv,order", SHAPES)
def test_attention_comes_near_its_formula(dev, dtype, d, group, hq, hkv, order):
    c = attn_case(dev, [0, 1, 33, 64, 129, 300, 600], hq, hkv, d, group, 16, dtype, order)
    near(c)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kw", [dict(window=310), dict(softcap=5.0), dict(window=400, softcap=30.0)])
@pytest.mark.parametrize("d,group,hq,hkv", [(64, 32, 18, 2), (128, 64, 8, 2), (256, 32, 4, 2)])
def test_attention_of_windows_and_caps_comes_near_its_formula(dev, dtype, kw, d, group, hq, hkv):
    c = attn_case(dev, [700, 33, 1, 320], hq, hkv, d, group, 16, dtype, **kw)
    near(c)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,group,hq,hkv,order", SHAPES)
def test_what_lies_far_below_a_groups_largest_element_counts(dev, dtype, d, group, hq, hkv, order):
    """All elements of q but one of each group at 2^-16 of it: the last of three pieces holds them.  With
    two the log of the sum is another."""
    c = attn_case(dev, [600, 300, 64], hq, hkv, d, group, 16, dtype, order)
    c["q"].fill_(2.0 ** -16)
    c["q"][:, :, group // 3::group] = 1.0
    _, want_lse, _, lse_err = exact(c)
    _, lost_lse, _, _ = exact(c, pieces=2)
    for cut in (False, True):
        _, lse = attn_run(c, cut)
        check(lse, want_lse, lse_err, f"lse, cut {cut}")
        off = np.abs(np64(lse) - lost_lse)
        assert (off > 2 * (lse_err + np.abs(want_lse) * 2.0 ** -24)).all(), float(off.min())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("scale,softcap", [(-0.09, 0.0), (0.0, 0.0), (-0.2, 4.0), (2.0 ** -140, 0.0), (1e-3, 0.5)])
@pytest.mark.parametrize("d,group,hq,hkv", [(64, 32, 18, 2), (128, 64, 8, 2), (256, 32, 4, 2)])
def test_attention_of_scales_of_any_sign(dev, dtype, scale, softcap, d, group, hq, hkv):
    """A negative scale turns the order of the scores, one of 0 makes them alike."""
    c = attn_case(dev, [700, 33, 1, 320], hq, hkv, d, group, 16, dtype, softcap=softcap)
    c["scale"] = scale
    near(c)


@pytest.mark.parametrize("power", [-95, -60, 60, 110])
@pytest.mark.parametrize("d,group,hq,hkv", [(64, 32, 18, 2), (128, 64, 8, 2), (256, 32, 4, 2)])
def test_attention_of_queries_of_any_size(dev, power, d, group, hq, hkv):
    """Queries far from 1, which the scale takes back."""
    c = attn_case(dev, [700, 33, 1, 320], hq, hkv, d, group, 16, BF16)
    c["q"] *= 2.0 ** power
    c["scale"] *= 2.0 ** -power
    near(c)


@pytest.mark.parametrize("power", [-100, 100, 112])
@pytest.mark.parametrize("d,group,hq,hkv", [(64, 32, 18, 2), (128, 64, 8, 2), (256, 32, 4, 2)])
def test_attention_of_values_of_any_size(dev, power, d, group, hq, hkv):
    """V's pairs far from 1: scales of up to 2^111.4, 31 of which 700 positions add up below 2^126."""
    c = attn_case(dev, [700, 33, 1, 320], hq, hkv, d, group, 16, BF16, poison=False)
    c["cache"].v_pairs.mul_(2.0 ** power)
    near(c)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,group,hq,hkv,order", SHAPES)
def test_the_log_of_one_positions_sum_is_its_score(dev, dtype, d, group, hq, hkv, order):
    """Of a single position, to fp32's arithmetic (2-norm over all heads): a group's code part and its
    offset's part are each rounded to 2^-24 of themselves, the former with each of three pieces, the
    latter with its sum of q; four such steps are allowed.  Queries of two pieces miss it by far."""
    c = attn_case(dev, [1] * 40, hq, hkv, d, group, 16, dtype, order)
    codes, pairs = c["cache"].k.cpu().numpy(), np64(c["cache"].k_pairs)
    at = c["table"][:, 0].cpu().numpy(), np.zeros(40, dtype=int)
    q = np64(c["q"]).reshape(40, hq, d // group, group)
    code, pair = (np.repeat(x[at].reshape(40, hkv, d // group, -1), hq // hkv, axis=1)
                  for x in (ref.unpack4(codes), pairs))
    parts = np.abs(pair[..., 0] * (code * q).sum(-1)) + np.abs(pair[..., 1] * q.sum(-1))
    sizes = parts.sum(-1) * c["scale"]
    _, want, _, _ = exact(c)
    _, lost, _, _ = exact(c, pieces=2)
    most = 4 * 2.0 ** -24 * np.linalg.norm(sizes)
    for cut in (False, True):
        _, lse = attn_run(c, cut)
        assert np.linalg.norm(np64(lse) - want) <= most, cut
    if dtype is F16:
        assert np.linalg.norm(np64(lse) - lost) > most
