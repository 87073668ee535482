"""Refusals of the calls on a 4-bit cache (fake device pointers, nothing is launched), the
binding's own checks, and pins of their 64-bit forms."""

import ctypes
import math

import numpy as np
import pytest

import weight_only_quantized_gemm_amd as wq
from oracle import decode as ref
from test_decode_cpu import ABI, ALIGN, BAD, CACHE_REFUSALS, FLAGS, NULL, OVER, P, SPACE, cache_args, refused

torch = pytest.importorskip("torch")
from weight_only_quantized_gemm_amd import decode  # noqa: E402

KV4, FP8 = wq.WQ_FLAG_KV4, wq.WQ_FLAG_FP8


def pairs_args(groups=2, **kw):
    return wq.wq_kv_pairs(k=20 * P, v=21 * P, page_stride=16 * 2 * groups, slot_stride=groups,
                          head_stride=16 * groups, group_size=32, **kw)


PAIR_REFUSALS = [
    ({"pairs.k": None}, NULL), ({"pairs.v": None}, NULL), ({"pairs.k": P + 2}, ALIGN),
    ({"pairs.group_size": 0}, BAD), ({"pairs.group_size": 16}, BAD), ({"pairs.group_size": 48}, BAD),
    ({"pairs.group_size": 128}, BAD), ({"pairs.group_size": -32}, BAD),
    ({"pairs.page_stride": -1}, BAD), ({"pairs.slot_stride": 1}, BAD),
    ({"pairs.head_stride": 0}, BAD), ({"pairs.page_stride": 1 << 61}, OVER),
    ({"pairs.reserved": 1}, ABI), ({"cache.k_scale": P}, FLAGS), ({"cache.v": P + 8}, ALIGN),
    ({"cache.slot_stride": 4}, BAD), ({"cache.head_dim": 60}, BAD),
]


def norm_rope_args(**kw):
    a = wq.versioned(wq.wq_norm_rope_args, cache=cache_args(), q=3 * P, k=4 * P, v=5 * P,
                     q_out=6 * P, q_norm=10 * P, k_norm=11 * P, slots=7 * P, positions=8 * P,
                     inv_freq=9 * P, tokens=3, q_heads=4, ldq=256, ldk=128, ldv=128, ldqo=256,
                     rot_dim=64, axes=2, eps=1e-6, **kw)
    a.sections[0], a.sections[1] = 20, 12
    return a


@pytest.mark.parametrize("changes,want", CACHE_REFUSALS + [
    (dict(tokens=0), BAD), (dict(tokens=1 << 24), BAD), (dict(q_heads=-1), BAD), (dict(ldq=248), BAD),
    (dict(ldk=120), BAD), (dict(ldv=132), BAD), (dict(ldqo=0), BAD), (dict(rot_dim=4), BAD),
    (dict(rot_dim=72), BAD), (dict(rot_dim=56), BAD), (dict(axes=0), BAD), (dict(axes=5), BAD),
    (dict(axes=1), BAD), (dict(interleaved=2), FLAGS), (dict(q=None), NULL), (dict(k=None), NULL),
    (dict(q_out=None), NULL), (dict(v=P + 8), ALIGN), (dict(slots=P + 4), ALIGN),
    (dict(positions=None), NULL), (dict(inv_freq=P + 2), ALIGN), (dict(q_norm=P + 8), ALIGN),
    (dict(k_norm=P + 2), ALIGN), (dict(eps=-1e-6), BAD), (dict(eps=math.nan), BAD),
    (dict(flags=FP8 | KV4), FLAGS), ({"pairs.k": P}, FLAGS), ({"pairs.group_size": 64}, FLAGS),
    (dict(abi_version=2), ABI),
])
def test_norm_rope_refusals(changes, want):
    refused(wq.wq_norm_rope_append, norm_rope_args(), changes, want)


@pytest.mark.parametrize("changes,want", PAIR_REFUSALS)
def test_norm_rope_refusals_of_a_4_bit_cache(changes, want):
    refused(wq.wq_norm_rope_append, norm_rope_args(pairs=pairs_args(), flags=KV4), changes, want)


def read_args():
    return wq.versioned(wq.wq_cache4_read_args, cache=cache_args(), pairs=pairs_args(), slots=3 * P,
                        k_out=4 * P, v_out=5 * P, tokens=7, ldk=128, ldv=128)


@pytest.mark.parametrize("changes,want", PAIR_REFUSALS + [
    (dict(tokens=0), BAD), (dict(tokens=1 << 24), BAD), (dict(ldk=120), BAD), (dict(ldv=132), BAD),
    (dict(slots=None), NULL), (dict(slots=P + 4), ALIGN), (dict(k_out=P + 8), ALIGN),
    (dict(v_out=P + 2), ALIGN), (dict(flags=KV4), FLAGS), (dict(flags=FP8), FLAGS),
    (dict(struct_size=0), ABI), (dict(reserved=1), ABI),
])
def test_read_refusals(changes, want):
    refused(wq.wq_cache4_read, read_args(), changes, want)


def attn4_args():
    return wq.versioned(wq.wq_attn4_args, cache=cache_args(), pairs=pairs_args(), q=3 * P, out=4 * P,
                        block_table=5 * P, lens=6 * P, workspace=7 * P, workspace_bytes=1 << 30,
                        batch=2, q_heads=4, max_len=40000, table_stride=2500, ldq=256, ldo=256,
                        scale=0.1)


@pytest.mark.parametrize("changes,want", PAIR_REFUSALS + [
    (dict(batch=0), BAD), (dict(batch=65536), BAD), (dict(q_heads=3), BAD), (dict(q_heads=0), BAD),
    (dict(max_len=0), BAD), (dict(max_len=(1 << 30) + 1), BAD), (dict(table_stride=2499), BAD),
    (dict(keep=P, keep_stride=39999), BAD), (dict(ldq=128), BAD), (dict(ldo=260), BAD),
    (dict(window=-1), BAD), (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD),
    (dict(softcap=-1.0), BAD), (dict(softcap=math.inf), BAD), (dict(q=None), NULL),
    (dict(out=P + 8), ALIGN), (dict(lse=P + 2), ALIGN), (dict(block_table=None), NULL),
    (dict(lens=P + 1), ALIGN), (dict(workspace=None), SPACE), (dict(workspace_bytes=64), SPACE),
    (dict(workspace=P + 8), ALIGN), (dict(flags=KV4), FLAGS), (dict(flags=FP8), FLAGS),
    (dict(abi_version=2), ABI), (dict(struct_size=8), ABI), (dict(reserved=1), ABI),
])
def test_attention4_refusals(changes, want):
    refused(wq.wq_paged_attention4, attn4_args(), changes, want)


def test_attention4_workspace():
    f = wq.wq_paged_attention4_workspace_bytes
    assert f(1, 8, 2, 64, 32, 1) == 0 == f(1, 8, 2, 64, 64, 256)  # no sequence is split
    assert f(3, 8, 2, 64, 32, 1 << 20) > 0 == f(1, 8, 2, 64, 32, 1 << 20, 600)
    with pytest.raises(wq.WQError) as e:
        f(65535, 512, 512, 64, 64, 128)                           # work-groups of one launch
    assert e.value.code == wq.WQ_ERR_OVERFLOW
    with pytest.raises(wq.WQError) as e:
        f(65535, 8, 2, 64, 64, 1 << 30)                           # steps of all sequences
    assert e.value.code == wq.WQ_ERR_OVERFLOW
    for bad in ((0, 8, 2, 64, 32, 1), (1, 7, 2, 64, 32, 1), (1, 8, 0, 64, 32, 1), (1, 8, 2, 20, 20, 1),
                (1, 8, 2, 64, 16, 1), (1, 8, 2, 80, 32, 1), (1, 8, 2, 64, 128, 1)):
        with pytest.raises(wq.WQError):
            f(*bad)


def sample_args():
    return wq.versioned(wq.wq_sample_args, logits=P, u=2 * P, temperature=3 * P, top_k=4 * P,
                        top_p=5 * P, min_p=6 * P, ids=7 * P, logprob=8 * P, workspace=9 * P,
                        workspace_bytes=1 << 40, rows=3, vocab=50001, ld=50001)


@pytest.mark.parametrize("changes,want", [
    (dict(rows=0), BAD), (dict(rows=65536), BAD), (dict(vocab=0), BAD),
    (dict(vocab=(1 << 19) + 1, ld=1 << 20), BAD), (dict(ld=50000), BAD), (dict(ld=-1), BAD),
    (dict(ld=1 << 60), OVER), (dict(logits=None), NULL), (dict(u=None), NULL), (dict(ids=None), NULL),
    (dict(logits=P + 1), ALIGN), (dict(logits=P + 2, flags=wq.WQ_FLAG_FP32), ALIGN),
    (dict(u=P + 2), ALIGN), (dict(temperature=P + 1), ALIGN), (dict(top_k=P + 2), ALIGN),
    (dict(top_p=P + 2), ALIGN), (dict(min_p=P + 1), ALIGN), (dict(ids=P + 2), ALIGN),
    (dict(logprob=P + 2), ALIGN), (dict(flags=FP8), FLAGS),
    (dict(flags=wq.WQ_FLAG_FP32 | wq.WQ_FLAG_BF16), FLAGS), (dict(abi_version=2), ABI),
    (dict(struct_size=8), ABI), (dict(reserved=1), ABI),
])
def test_sample_refusals(changes, want):
    refused(wq.wq_sample, sample_args(), changes, want)


def test_sampler_refuses_before_the_library():
    plan = decode.Sampler(4, 100, dtype=torch.float16, device="cpu")
    z, u = torch.zeros((4, 100), dtype=torch.float16), torch.zeros(4)
    with pytest.raises(TypeError):
        decode.Sampler(4, 100, dtype=torch.float64, device="cpu")
    with pytest.raises(wq.WQError):
        decode.Sampler(4, (1 << 19) + 1, device="cpu")
    for args, kw in (((z[:, :99], u), {}), ((torch.cat([z, z]), u), {}), ((z[:0], u[:0]), {}),
                     ((z, u[:3]), {}), ((z, u), dict(top_p=u[:2])),
                     ((torch.zeros((4, 200), dtype=torch.float16)[:, ::2], u), {})):
        with pytest.raises(ValueError):
            plan(*args, **kw)
    for args, kw in (((z.float(), u), {}), ((z, u.double()), {}), ((z, u), dict(top_k=u)),
                     ((z, u), dict(temperature=u.half())), ((z, u), dict(ids=u.long())),
                     ((z, u), dict(logprob=u.half()))):
        with pytest.raises(TypeError):
            plan(*args, **kw)


def test_null_structs_and_sizes():
    L = wq.lib()
    for name, cls in (("wq_norm_rope_append", wq.wq_norm_rope_args),
                      ("wq_cache4_read", wq.wq_cache4_read_args),
                      ("wq_paged_attention4", wq.wq_attn4_args),
                      ("wq_sample", wq.wq_sample_args)):
        assert getattr(L, name)(None) == (wq.WQ_STAGE_ARGS << 16) | wq.WQ_ERR_NULL
        with pytest.raises(wq.WQError) as e:  # the binding's size passes, later checks fail
            getattr(wq, name)(wq.versioned(cls))
        assert e.value.code != wq.WQ_ERR_ABI
    assert ctypes.sizeof(wq.wq_kv_pairs) == 48


def tensors4(pages=3, page=16, heads=2, d=64, groups=2, dtype=torch.float16):
    codes = [torch.zeros((pages, page, heads, d // 2), dtype=torch.uint8) for _ in range(2)]
    pairs = [torch.zeros((pages, page, heads, groups, 2), dtype=dtype) for _ in range(2)]
    return codes + pairs


def test_cache4_refuses_what_it_cannot_describe():
    k, v, kp, vp = tensors4()
    cache = decode.PagedCache4(k, v, kp, vp)
    assert (cache.group, cache.head_dim, cache.page_size) == (32, 64, 16)
    for bad in ((k, v[:2], kp, vp), (k, v, kp, vp[:, :, :, :1]), (k, v, kp[:2], vp[:2]),
                (k[..., ::2], v[..., ::2], kp, vp), (k, v, kp[..., :1], vp[..., :1]),
                (k, v, *(torch.zeros((3, 16, 2, 3, 2), dtype=torch.float16) for _ in range(2))),
                (k, v, *(torch.zeros((3, 16, 2, 2, 3), dtype=torch.float16)[..., :2]
                         for _ in range(2))),
                (k, v, *(torch.zeros(200, dtype=torch.float16)[1:193].view(3, 16, 2, 1, 2)
                         for _ in range(2)))):
        with pytest.raises(ValueError):
            decode.PagedCache4(*bad)
    for bad in ((k.char(), v.char(), kp, vp), (k, v, kp.float(), vp.float()), (k, v, kp, vp.bfloat16())):
        with pytest.raises(TypeError):
            decode.PagedCache4(*bad)
    assert decode.PagedCache4.empty(2, 8, 1, 192, torch.bfloat16, "cpu").group == 64
    assert decode.PagedCache4.empty(2, 8, 1, 80, torch.bfloat16, "cpu").group == 80


def test_binding_refuses_before_the_library():
    cache = decode.PagedCache4(*tensors4())
    f16 = torch.float16
    k, slots = torch.zeros((5, 2, 64), dtype=f16), torch.zeros(5, dtype=torch.int64)
    w = torch.ones(64, dtype=f16)
    with pytest.raises(TypeError):
        decode.rope_append(None, k.bfloat16(), k.bfloat16(), cache, slots)
    with pytest.raises(ValueError):
        decode.rope_append(None, k, k, cache, slots, q_norm=w)
    with pytest.raises(ValueError):
        decode.rope_append(None, k, k, cache, slots, k_norm=w[:32])
    with pytest.raises(TypeError):
        decode.rope_append(None, k, k, cache, slots, k_norm=w.float())
    with pytest.raises(TypeError):
        cache.read(slots.int())
    with pytest.raises(ValueError):
        cache.read(slots, k_out=k[:4])
    with pytest.raises(TypeError):
        cache.read(slots, v_out=k.float())
    plan = decode.PagedAttention(cache, 5, 4, 48, dtype=f16)
    with pytest.raises(TypeError):
        decode.PagedAttention(cache, 5, 4, 48, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        plan(torch.zeros((4, 4, 64), dtype=f16), torch.zeros((5, 3), dtype=torch.int32),
             torch.zeros(5, dtype=torch.int32))


# ---- pins of the 64-bit forms --------------------------------------------------------------------

def test_reference_head_norm_against_torch():
    g = np.random.default_rng(3)
    x, w = g.normal(size=(3, 2, 24)), g.normal(size=24)
    t = torch.nn.functional.rms_norm(torch.tensor(x), (24,), torch.tensor(w), 1e-3)
    assert np.allclose(ref.head_norm(x, w, 1e-3)[0], t.numpy())


def test_reference_codes_and_their_check():
    codes = np.array([[0x21, 0x43, 0xF0, 0x08]], dtype=np.uint8)
    pairs = np.array([[[0.5, -1.0], [2.0, 3.0]]])
    assert ref.unpack4(codes).tolist() == [[1, 2, 3, 4, 0, 15, 8, 0]]
    assert ref.values4(codes, pairs).tolist() == [[-0.5, 0, 0.5, 1, 3, 33, 19, 3]]
    x = np.array([[0.0, 1.0, 2.0, 15.0]])
    good, pair = np.array([[0x10, 0xF2]], dtype=np.uint8), np.array([[[1.0, 0.0]]])
    ref.check_quantized4(x, 0.0, good, pair, 2.0 ** -11, 0.0)
    for codes, pair in (([[0x10, 0xF3]], [[[1.0, 0.0]]]), ([[0x10, 0xF2]], [[[1.01, 0.0]]]),
                        ([[0x10, 0xF2]], [[[1.0, 0.1]]])):
        with pytest.raises(AssertionError):
            ref.check_quantized4(x, 0.0, np.array(codes, dtype=np.uint8), np.array(pair),
                                 2.0 ** -11, 0.0)


def test_reference_sampling_against_its_steps():
    g = np.random.default_rng(4)
    z = g.normal(size=40) * 2
    p = np.exp(z - z.max())
    order = np.argsort(-z)
    for u in g.random(20):
        full = np.cumsum(p / p.sum())
        assert ref.sample(z, u)[0] == int((full <= u).sum())
        top = np.sort(order[:5])
        share = np.cumsum(p[top] / p[top].sum())
        got, logp, _, _ = ref.sample(z, u, top_k=5)
        assert got == top[int((share <= u).sum())] and np.isclose(logp, np.log(p[got] / p[top].sum()))
    # the shortest run that holds half
    run = 1 + int((np.cumsum(p[order]) < 0.5 * p.sum()).sum())
    seen = {ref.sample(z, u, top_p=0.5)[0] for u in np.linspace(0, 0.9999, 4000)}
    assert seen == set(order[:run].tolist())
    seen = {ref.sample(z, u, min_p=0.2, temperature=2.0)[0] for u in np.linspace(0, 0.9999, 4000)}
    assert seen == set(np.flatnonzero(np.exp((z - z.max()) / 2) >= 0.2).tolist())
    assert ref.sample(z, 0.7, temperature=0.0)[:2] == (order[0], 0.0)
    assert ref.sample(np.array([0.0, np.nan]), 0.5)[0] == -1
    assert ref.sample(np.full(3, -np.inf), 0.5)[0] == -1
    assert ref.sample(np.array([1.0, np.inf, 2.0]), 0.99)[0] == 1
