"""4-bit attention of shapes whose instances few other shapes share, on the GPU against its 64-bit form."""

import numpy as np
import pytest

from oracle import decode as ref

torch = pytest.importorskip("torch")
wq = pytest.importorskip("weight_only_quantized_gemm_amd")

from test_decode_gpu import BF16, F16, half_step, np64  # noqa: E402
from test_decode4_gpu import attn_case, attn_check, attn_run  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,group,hq,hkv,order", [
    (256, 32, 2, 2, "hnd"), (256, 32, 4, 4, "nhd"), (256, 32, 3, 3, "hnd"), (224, 32, 4, 4, "hnd"),
    (224, 32, 3, 3, "nhd"), (192, 32, 4, 4, "nhd"), (192, 32, 5, 5, "hnd"), (160, 32, 4, 4, "hnd"),
    (160, 32, 3, 3, "nhd"), (256, 64, 6, 3, "hnd"), (96, 32, 6, 3, "nhd")])
def test_few_query_heads_to_several_kv_heads(dev, dtype, d, group, hq, hkv, order):
    """Five to eight groups with one query head to a KV head, three and four with two: two KV heads
    share an instance's columns where it is made for that.  The outputs' distance (2-norm) from the
    formula's is half a step of the type, and 2^-9 for the scores: elements of q within 2^-14.95 of
    the largest (4.5), codes within 7.5 of their mean, scales of 0.4 and 16 = sqrt(256) terms make
    2^-11 of p, four times which is allowed."""
    c = attn_case(dev, [0, 1, 33, 64, 65, 127, 300, 1500], hq, hkv, d, group, 16, dtype, order)
    cache = c["cache"]
    k, v = (ref.values4(x.cpu().numpy(), np64(y))
            for x, y in ((cache.k, cache.k_pairs), (cache.v, cache.v_pairs)))
    want, _, _, _ = ref.paged_attention(np64(c["q"]), k, v, c["table"].cpu().numpy(),
                                        c["lens"].cpu().numpy(), c["scale"])
    for cut in (False, True):
        out, lse = attn_run(c, cut)
        attn_check(c, out, lse, f"cut {cut}")
        off = np.linalg.norm(np64(out) - want, axis=-1)
        assert (off <= (half_step(dtype) + 2.0 ** -9) * np.linalg.norm(want, axis=-1)).all(), cut
