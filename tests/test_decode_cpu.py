"""Refusals of the decode-step calls (fake device pointers, nothing is launched), the binding's
own checks, and pins of the 64-bit forms the GPU tests compare with."""

import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import weight_only_quantized_gemm_amd as wq
from oracle import decode as ref

ARGS, SHAPE = wq.WQ_STAGE_ARGS, wq.WQ_STAGE_SHAPE
ABI, NULL, ALIGN = (ARGS, wq.WQ_ERR_ABI), (ARGS, wq.WQ_ERR_NULL), (ARGS, wq.WQ_ERR_ALIGN)
BAD, FLAGS = (SHAPE, wq.WQ_ERR_SHAPE), (ARGS, wq.WQ_ERR_FLAGS)
SPACE, OVER = (ARGS, wq.WQ_ERR_WORKSPACE), (SHAPE, wq.WQ_ERR_OVERFLOW)
P = 0x10000


def set_path(args, path, value):
    *at, last = path.split(".")
    for name in at:
        args = getattr(args, name)
    setattr(args, last, value)


def refused(call, args, changes, want):
    for path, value in changes.items():
        set_path(args, path, value)
    with pytest.raises(wq.WQError) as e:
        call(args)
    assert (e.value.stage, e.value.code) == want, str(e.value)


def norm_args():
    return wq.versioned(wq.wq_norm_args, x=P, weight=2 * P, y=3 * P, delta=4 * P, sum_out=5 * P,
                        rows=2, n=64, ldx=64, ldd=64, lds=64, ldy=64, eps=1e-6)


@pytest.mark.parametrize("changes,want", [
    (dict(abi_version=2), ABI), (dict(struct_size=8), ABI), (dict(reserved=1), ABI),
    (dict(x=None), NULL), (dict(weight=None), NULL), (dict(y=None), NULL),
    (dict(x=P + 8), ALIGN), (dict(delta=P + 2), ALIGN), (dict(sum_out=P + 2), ALIGN),
    (dict(rows=0), BAD), (dict(rows=1 << 22), BAD), (dict(n=0), BAD), (dict(n=60), BAD),
    (dict(n=65544, ldx=65544), BAD),
    (dict(ldx=56), BAD), (dict(ldy=68), BAD), (dict(ldd=8), BAD), (dict(lds=60), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD), (dict(delta=None), FLAGS),
    (dict(sum_out=3 * P), FLAGS), (dict(flags=wq.WQ_FLAG_FP8), FLAGS),
])
def test_norm_refusals(changes, want):
    refused(wq.wq_add_rms_norm, norm_args(), changes, want)


def cache_args(d=64):
    return wq.wq_kv_cache(k=P, v=2 * P, page_stride=16 * 2 * d, slot_stride=d,
                          head_stride=16 * d, num_pages=5, page_size=16, kv_heads=2, head_dim=d)


CACHE_REFUSALS = [
    ({"cache.k": None}, NULL), ({"cache.v": P + 8}, ALIGN), ({"cache.num_pages": 0}, BAD),
    ({"cache.page_size": 0}, BAD), ({"cache.kv_heads": 0}, BAD), ({"cache.head_dim": 8}, BAD),
    ({"cache.head_dim": 264}, BAD), ({"cache.head_dim": 60}, BAD),
    ({"cache.page_stride": -8}, BAD), ({"cache.slot_stride": 4}, BAD),
    ({"cache.head_stride": 32}, BAD), ({"cache.page_stride": 1 << 60}, OVER),
    ({"cache.k_scale": P}, FLAGS), ({"flags": wq.WQ_FLAG_FP8, "cache.v_scale": P + 2}, ALIGN),
    ({"flags": wq.WQ_FLAG_FP8, "cache.k": P + 4}, ALIGN), ({"flags": wq.WQ_FLAG_HAS_ZP}, FLAGS),
    ({"abi_version": 4}, ABI), ({"struct_size": 0}, ABI), ({"reserved": 3}, ABI),
]


def rope_args():
    a = wq.versioned(wq.wq_rope_args, cache=cache_args(), q=3 * P, k=4 * P, v=5 * P, q_out=6 * P,
                     slots=7 * P, positions=8 * P, inv_freq=9 * P, tokens=3, q_heads=4, ldq=256,
                     ldk=128, ldv=128, ldqo=256, rot_dim=64, axes=2)
    a.sections[0], a.sections[1] = 20, 12
    return a


@pytest.mark.parametrize("changes,want", CACHE_REFUSALS + [
    (dict(tokens=0), BAD), (dict(tokens=1 << 24), BAD), (dict(q_heads=-1), BAD), (dict(ldq=248), BAD),
    (dict(ldk=120), BAD),
    (dict(ldv=132), BAD), (dict(ldqo=0), BAD), (dict(rot_dim=4), BAD), (dict(rot_dim=72), BAD),
    (dict(rot_dim=56), BAD), (dict(axes=0), BAD), (dict(axes=5), BAD), (dict(axes=1), BAD),
    (dict(interleaved=2), FLAGS), (dict(q=None), NULL), (dict(k=None), NULL),
    (dict(q_out=None), NULL), (dict(v=P + 8), ALIGN), (dict(slots=P + 4), ALIGN),
    (dict(positions=None), NULL), (dict(inv_freq=P + 2), ALIGN),
])
def test_rope_refusals(changes, want):
    refused(wq.wq_rope_append, rope_args(), changes, want)


def test_rope_negative_section():
    a = rope_args()
    a.sections[0], a.sections[1] = 40, -8
    refused(wq.wq_rope_append, a, {}, BAD)


def attn_args():
    return wq.versioned(wq.wq_attn_args, cache=cache_args(), q=3 * P, out=4 * P, block_table=5 * P,
                        lens=6 * P, workspace=7 * P, workspace_bytes=1 << 30, batch=2, q_heads=4,
                        max_len=4000, table_stride=250, ldq=256, ldo=256, scale=0.1)


@pytest.mark.parametrize("changes,want", CACHE_REFUSALS + [
    (dict(batch=0), BAD), (dict(batch=65536), BAD), (dict(q_heads=3), BAD), (dict(q_heads=0), BAD),
    (dict(max_len=0), BAD), (dict(max_len=(1 << 30) + 1), BAD), (dict(table_stride=249), BAD),
    (dict(keep=P, keep_stride=3999), BAD), (dict(ldq=128), BAD), (dict(ldo=260), BAD),
    (dict(window=-1), BAD), (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD),
    (dict(softcap=-1.0), BAD), (dict(softcap=math.inf), BAD), (dict(q=None), NULL),
    (dict(out=P + 8), ALIGN), (dict(lse=P + 2), ALIGN), (dict(block_table=None), NULL),
    (dict(lens=P + 1), ALIGN), (dict(workspace=None), SPACE), (dict(workspace_bytes=64), SPACE),
    (dict(workspace=P + 8), ALIGN),
])
def test_attention_refusals(changes, want):
    refused(wq.wq_paged_attention, attn_args(), changes, want)


def test_attention_workspace():
    f = wq.wq_paged_attention_workspace_bytes
    assert f(1, 8, 2, 64, 1) == 0 == f(65535, 8, 2, 64, 128)  # no sequence is split
    # two partials for each of 384 ranges, [2 KV heads][4 query heads] of head_dim + 2 floats,
    # 8 bytes a sequence
    assert f(3, 8, 2, 64, 769) == f(3, 8, 2, 64, 1 << 20) == 2 * 384 * 8 * 66 * 4 + 24
    # whole sequences up to a KiB of keys for each work-group, between 96 and 256
    assert f(3, 8, 2, 64, 768) == 0 == f(100, 8, 2, 64, 1600) < f(100, 8, 2, 64, 1601)
    assert f(4096, 8, 2, 64, 2048) == 0 < f(4096, 8, 2, 64, 2049)
    assert f(1, 8, 2, 64, 1 << 20, 700) == 0                  # a window that one work-group covers
    assert f(1, 8, 2, 128, 500, 0, wq.WQ_FLAG_FP8) == 0 < f(1, 8, 2, 128, 500)
    with pytest.raises(wq.WQError):
        f(1, 8, 2, 64, 1, 0, wq.WQ_FLAG_SWIGLU)
    with pytest.raises(wq.WQError) as e:
        f(65535, 512, 512, 64, 128)                           # work-groups of one launch
    assert e.value.code == wq.WQ_ERR_OVERFLOW
    assert f(65535, 8, 2, 64, 1 << 20) > 0 == f(65535, 8, 2, 64, 1 << 30, 100)
    with pytest.raises(wq.WQError) as e:
        f(65535, 8, 2, 64, 1 << 30)                           # steps of all sequences
    assert e.value.code == wq.WQ_ERR_OVERFLOW
    for bad in ((0, 8, 2, 64, 1), (1, 7, 2, 64, 1), (1, 8, 0, 64, 1), (1, 8, 2, 20, 1)):
        with pytest.raises(wq.WQError):
            f(*bad)


def test_attention_ranges_of_a_rounded_up_grid(tmp_path):
    """Every (row, unit) is one work-group's, those of the rounded-up grid past the last row have
    none, and a range's first granule is right (against 64 bits) up to 2^30 granules."""
    csrc = os.path.join(os.path.dirname(wq.__file__), "csrc")
    source, program = tmp_path / "ranges.cc", tmp_path / "ranges"
    source.write_text(r"""
        #include <cstdio>
        #include <vector>
        #include "wq_ranges.h"
        int main() {
          for (int near = 0; near < 2; ++near)
            for (int rows : {1, 2, 7, 8, 9, 64, 100})
              for (int units : {1, 3, 513}) {
                std::vector<int> hits(rows * units);
                const int grid = (near ? (rows + 7) / 8 * 8 : rows) * units;
                for (int block = 0, row, unit; block < grid; ++block) {
                  const bool in = wq::place_of_block(block, units, near, rows, row, unit);
                  if (in != (row < rows) || row < 0 || unit < 0 || unit >= units)
                    return std::printf("block %d of %d x %d: %d %d", block, rows, units, row, unit);
                  if (in) ++hits[row * units + unit];
                }
                for (int n : hits)
                  if (n != 1) return std::printf("%d x %d: %d hits", rows, units, n);
              }
          for (long long total : {0ll, 1ll, 129ll, 306783379ll, (1ll << 29) + 1, 1ll << 30})
            for (int ranges : {1, 2, 3, 42, 256, 768}) {
              long long length = (total + ranges - 1) / ranges, left = total;
              if (length < 1) length = 1;
              for (int row = 0; row < ranges; ++row) {
                const long long first = row * length, got = wq::range_first(row, total, ranges);
                if (got != (first < total ? first : -1))
                  return std::printf("range %d of %d, %lld: %lld", row, ranges, total, got);
                if (got >= 0) left -= total - first < length ? total - first : length;
              }
              if (left) return std::printf("%d ranges of %lld leave %lld", ranges, total, left);
            }
        }""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", csrc, str(source), "-o", str(program)],
                   check=True)
    done = subprocess.run([str(program)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0, done.stdout


def bank_args(k, n):
    return wq.wq_expert_bank(b=P, s=2 * P, b_stride_bytes=k * n // 2, s_stride_bytes=k // 128 * n * 2,
                             group_size=128)


def moe_args():
    return wq.versioned(wq.wq_moe_args, x=P, router=2 * P, gate_up=bank_args(512, 768),
                        down=bank_args(384, 512), y=3 * P, workspace=4 * P, workspace_bytes=1 << 30,
                        tokens=4, n_expert=8, top_k=2, hidden=512, inter=384, ldx=512, ldy=512,
                        routed_scale=1.0, renormalize=1)


@pytest.mark.parametrize("changes,want", [
    (dict(abi_version=1), ABI), (dict(struct_size=1), ABI), (dict(reserved=1), ABI),
    ({"down.reserved": 1}, ABI), (dict(tokens=0), BAD), (dict(tokens=17), BAD),
    (dict(n_expert=0), BAD), (dict(n_expert=257), BAD), (dict(top_k=0), BAD), (dict(top_k=9), BAD),
    (dict(n_expert=64, top_k=17), BAD), (dict(hidden=384), BAD), (dict(inter=200), BAD),
    (dict(hidden=1 << 20, inter=1 << 20), OVER), (dict(ldx=256), BAD), (dict(ldy=516), BAD),
    (dict(residual=P, ldr=504), BAD), (dict(residual=P + 2, ldr=512), ALIGN), (dict(x=None), NULL),
    (dict(router=P + 8), ALIGN), (dict(y=None), NULL), (dict(ids=P + 2), ALIGN),
    (dict(weights=P + 1), ALIGN), (dict(renormalize=2), FLAGS),
    (dict(flags=wq.WQ_FLAG_HAS_ZP), FLAGS), ({"down.zp": P}, FLAGS),
    (dict(flags=wq.WQ_FLAG_HAS_ZP | wq.WQ_FLAG_FP8), FLAGS), (dict(flags=wq.WQ_FLAG_SWIGLU), FLAGS),
    (dict(flags=wq.WQ_FLAG_FP8), BAD), ({"gate_up.group_size": 24}, BAD),
    ({"gate_up.group_size": 0}, BAD), ({"down.group_size": 256}, BAD),
    ({"gate_up.b_stride_bytes": 16}, BAD), ({"down.s_stride_bytes": 1544}, BAD),
    ({"gate_up.b": None}, NULL), ({"down.s": P + 4}, ALIGN), (dict(workspace=None), SPACE),
    (dict(workspace_bytes=100), SPACE), (dict(workspace=P + 8), ALIGN),
])
def test_moe_refusals(changes, want):
    refused(wq.wq_moe_layer, moe_args(), changes, want)


def test_null_structs():
    L = wq.lib()
    for name in ("wq_add_rms_norm", "wq_rope_append", "wq_paged_attention", "wq_moe_layer"):
        assert getattr(L, name)(None) == (ARGS << 16) | wq.WQ_ERR_NULL
    assert L.wq_moe_layer_workspace_bytes(1, 1, 1, 256, 128, None) == (ARGS << 16) | wq.WQ_ERR_NULL


# ---- the binding's own checks -------------------------------------------------------------------

torch = pytest.importorskip("torch")
from weight_only_quantized_gemm_amd import decode  # noqa: E402


def test_binding_refuses_before_the_library():
    f16 = torch.float16
    x, w = torch.zeros((2, 64), dtype=f16), torch.zeros(64, dtype=f16)
    with pytest.raises(TypeError):
        decode.add_rms_norm(x.float(), w)
    with pytest.raises(TypeError):
        decode.add_rms_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        decode.add_rms_norm(x, w[:32])
    with pytest.raises(ValueError):
        decode.add_rms_norm(x, w, sum_out=x)
    with pytest.raises(ValueError):
        decode.add_rms_norm(x, w, delta=x[:1])
    k = torch.zeros((3, 16, 2, 64), dtype=f16)
    with pytest.raises(ValueError):
        decode.PagedCache(k, k[:2])
    with pytest.raises(ValueError):
        decode.PagedCache(k, k, torch.ones(2))
    with pytest.raises(TypeError):
        decode.PagedCache(k.float(), k.float())
    cache = decode.PagedCache(k, k.clone())
    kn, slots = torch.zeros((5, 2, 64), dtype=f16), torch.zeros(5, dtype=torch.int64)
    with pytest.raises(TypeError):
        decode.rope_append(None, kn.bfloat16(), kn.bfloat16(), cache, slots)
    with pytest.raises(ValueError):
        decode.rope_append(None, kn, kn[:4], cache, slots)
    with pytest.raises(TypeError):
        decode.rope_append(None, kn, kn, cache, slots.int())
    inv, pos = torch.ones(32), torch.zeros((2, 5), dtype=torch.int32)
    for kw in (dict(), dict(positions=pos), dict(positions=pos, sections=(32,))):
        with pytest.raises(ValueError):
            decode.rope_append(None, kn, kn, cache, slots, inv_freq=inv, **kw)
    plan = decode.PagedAttention(cache, 5, 4, 48, dtype=f16)
    q, table = torch.zeros((5, 4, 64), dtype=f16), torch.zeros((5, 3), dtype=torch.int32)
    lens = torch.zeros(5, dtype=torch.int32)
    for args in ((q[:4], table, lens), (q, table[:4], lens), (q, table, lens[:1]),
                 (q.transpose(1, 2).contiguous().transpose(1, 2), table, lens)):
        with pytest.raises(ValueError):
            plan(*args)
    with pytest.raises(TypeError):
        plan(q, table.long(), lens)
    with pytest.raises(ValueError):
        plan(q, table, lens, keep=torch.ones((4, 48), dtype=torch.uint8))


# ---- pins of the 64-bit forms --------------------------------------------------------------------

def test_reference_attention_against_softmax():
    g = np.random.default_rng(0)
    q, k, v = g.normal(size=(2, 4, 16)), g.normal(size=(6, 4, 2, 16)), g.normal(size=(6, 4, 2, 16))
    table, lens = [[3, 1], [5, 0]], [7, 3]
    out, lse, _, _ = ref.paged_attention(q, k, v, table, lens, 0.25)
    for b in range(2):
        kk = np.concatenate([k[p] for p in table[b]])[: lens[b]]
        vv = np.concatenate([v[p] for p in table[b]])[: lens[b]]
        for h in range(4):
            s = torch.tensor(kk[:, h // 2] @ q[b, h] * 0.25)
            p = torch.softmax(s, 0).numpy()
            assert np.allclose(out[b, h], p @ vv[:, h // 2])
            assert np.isclose(lse[b, h], torch.logsumexp(s, 0).item())


def test_reference_rotation_is_a_complex_product():
    g = np.random.default_rng(1)
    x, pos, inv = g.normal(size=(3, 2, 12)), g.integers(0, 99, (1, 3)), g.uniform(size=4)
    for inter in (False, True):
        y, _ = ref.rotate(x, pos, inv, [4], inter)
        a, b = (np.s_[..., 0:8:2], np.s_[..., 1:8:2]) if inter else (np.s_[..., :4], np.s_[..., 4:8])
        z = (x[a] + 1j * x[b]) * np.exp(1j * pos[0][:, None, None] * inv)
        assert np.allclose(y[a] + 1j * y[b], z) and np.array_equal(y[..., 8:], x[..., 8:])


def test_reference_norm_and_moe_against_torch():
    g = np.random.default_rng(2)
    x, d, w = g.normal(size=(3, 24)), g.normal(size=(3, 24)), g.normal(size=24)
    y, s = ref.add_rms_norm(x, d, w, 1e-3)
    t = torch.nn.functional.rms_norm(torch.tensor(x + d), (24,), torch.tensor(w), 1e-3)
    assert np.allclose(y, t.numpy()) and np.array_equal(s, x + d)
    router, gate, up, down = (g.normal(size=sh) for sh in ((5, 24), (5, 24, 8), (5, 24, 8), (5, 8, 24)))
    got, ids, weights, _ = ref.moe_layer(x, router, gate, up, down, 2, True, 1.0, d, 0.0)
    for t in range(3):
        p = torch.softmax(torch.tensor(router @ x[t]), 0)
        top = torch.topk(p, 2)
        assert ids[t].tolist() == top.indices.tolist()
        assert np.allclose(weights[t], (top.values / top.values.sum()).numpy())
        want = d[t].copy()
        for i, wt in zip(ids[t], weights[t]):
            h = torch.nn.functional.silu(torch.tensor(x[t] @ gate[i])).numpy() * (x[t] @ up[i])
            want += wt * (h @ down[i])
        assert np.allclose(got[t], want)


def test_argument_structs_match_the_library():
    """A struct of the binding's size passes the version check (and fails a later one)."""
    for call, cls in ((wq.wq_add_rms_norm, wq.wq_norm_args), (wq.wq_rope_append, wq.wq_rope_args),
                      (wq.wq_paged_attention, wq.wq_attn_args), (wq.wq_moe_layer, wq.wq_moe_args)):
        with pytest.raises(wq.WQError) as e:
            call(wq.versioned(cls))
        assert e.value.code != wq.WQ_ERR_ABI
    assert ctypes.sizeof(wq.wq_kv_cache) == 72
