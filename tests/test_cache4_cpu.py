"""What PagedCache4.empty is asked for is what it makes, or it refuses."""

import pytest

torch = pytest.importorskip("torch")
wq = pytest.importorskip("weight_only_quantized_gemm_amd")
from weight_only_quantized_gemm_amd import decode  # noqa: E402


@pytest.mark.parametrize("head_dim", range(16, 257, 8))
def test_an_empty_cache_has_the_groups_asked_for(head_dim):
    for group in (None, 16, 32, 48, 64, 80, 128, head_dim, 256, 0, -32):
        if group is None or group == head_dim or (group in (32, 64, 128) and head_dim % group == 0):
            cache = decode.PagedCache4.empty(2, 8, 3, head_dim, torch.float16, "cpu", group)
            assert cache.head_dim == head_dim and cache.group == (
                group or (64 if head_dim % 64 == 0 else head_dim))
        else:
            with pytest.raises(ValueError):
                decode.PagedCache4.empty(2, 8, 3, head_dim, torch.float16, "cpu", group)


def test_an_empty_cache_refuses_heads_of_an_odd_size():
    with pytest.raises(ValueError):
        decode.PagedCache4.empty(2, 8, 3, 65, torch.float16, "cpu")
