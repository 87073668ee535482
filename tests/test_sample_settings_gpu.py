"""Settings of the token choice at their ends, on the GPU against the 64-bit form."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
wq = pytest.importorskip("weight_only_quantized_gemm_amd")

from test_sample_gpu import BF16, F16, F32, logits_of, run, sample_check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("vocab", [9, 5000])
@pytest.mark.parametrize("cuts", [{}, dict(top_k=[5] * 8), dict(top_p=[0.999] * 8),
                                  dict(top_k=[3] * 8, top_p=[0.9] * 8)])
def test_min_p_past_one_leaves_the_first_token(dev, dtype, vocab, cuts):
    """Of several equal largest logits the lowest token, for certain; a min_p of 1 leaves them all."""
    z = torch.zeros((8, vocab), dtype=dtype, device=dev)
    z[:, [2, 5, vocab - 1]] = 3.0
    z[3, [1, 4]] = math.inf
    z[6, 7] = math.nan
    u = (np.arange(8) / 8 + 0.07).astype(np.float32)
    for min_p in (1 + 2.0 ** -23, 1.5, math.inf):
        ids, logprob = sample_check(z, u, min_p=[min_p] * 8, **cuts)
        assert ids.tolist() == [2, 2, 2, 1, 2, 2, -1, 2]
        assert logprob[6].isnan() and logprob[[0, 1, 2, 3, 4, 5, 7]].tolist() == [0.0] * 7
    again, shares = run(z, u, min_p=[1.0] * 8, top_k=[3] * 8)
    assert again.tolist() == [2, 2, 2, 1, 5, vocab - 1, -1, vocab - 1]
    assert math.isclose(float(shares[0]), -math.log(3), rel_tol=2.0 ** -23)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("cuts", [dict(top_k=[1, 3, 600, 50, 4990, 4999, 5, 2]), dict(top_p=[0.5, 0.9, 0.1, 0.999] * 2),
                                  dict(top_k=[700] * 8, top_p=[0.8] * 8, min_p=[0.0, 0.1] * 4)])
def test_cuts_at_temperatures_of_any_size(dev, dtype, cuts):
    """Exponents from none to past every bin: those of a tiny temperature pass 32 bits, and -inf over
    an infinite one is no number."""
    g = np.random.default_rng(21)
    z = logits_of(g, 8, 5000, dtype)
    z[:, 7::9] = -math.inf
    u = g.random(8).astype(np.float32)
    # (of some hundreds of tokens that are all alike, a border may be where u falls)
    sample_check(z, u, most=1, temperature=[1e-44, 1e-30, 1e-7, 1e-3, 1e4, 1e30, 3e38, math.inf], **cuts)
