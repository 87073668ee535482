"""Pins of the 4-bit attention's 64-bit form, and that its bounds refuse wrong outputs."""

import numpy as np
import pytest

from oracle import decode as ref


def test_reference_numbers_of_four_bits():
    x = np.array([0.0, 0.125, 1.125, 2.125, 2.375, 17.0, 19.0, 21.0, 248.0, 247.875, -2.375, 2.0 ** -9])
    assert ref.e4m3(x).tolist() == [0.0, 0.125, 1.125, 2.0, 2.5, 16.0, 20.0, 20.0, 256.0, 240.0, -2.5,
                                    2.0 ** -9]


@pytest.mark.parametrize("pieces", [2, 3])
def test_reference_pieces_hold_a_query(pieces):
    """A piece of four bits leaves at most half of its step: of numbers below 2^8 2^3, which four bits
    down is below 2^7 or 2^7 itself, so that the next leaves 2^-1 at most, the third 2^-5, beside a
    largest element of 124 at least.  Of the types' own numbers less is left: bf16's eight bits past the
    first piece's four are the second's where its steps of 2^-3 / 16 reach, which leaves half of these,
    2^-8; fp16's eleven are three pieces', which leave 2^-12.  Whole numbers below 2^7 are held."""
    g = np.random.default_rng(pieces)
    q = g.normal(size=(50, 64)) * 2.0 ** g.integers(-40, 40, (50, 1))
    held = ref.held4(q, pieces)
    most = np.abs(q).max(axis=1, keepdims=True)
    assert (np.abs(held - q) <= most * 2.0 ** (7 - 4 * pieces) / 124).all()
    bits = 8 if pieces == 2 else 11
    step = 2.0 ** (np.floor(np.log2(np.abs(q))) - bits + 1)
    typed = np.rint(q / step) * step
    top = np.abs(typed).max(axis=1, keepdims=True)
    assert (np.abs(ref.held4(typed, pieces) - typed) <= top * 2.0 ** (-4 * pieces) / 124).all()
    whole = np.arange(-127.0, 128.0)[None]
    assert np.array_equal(ref.held4(whole, 3), whole) and not ref.held4(whole * 0, 2).any()


def cache(g, pages, page, heads, d, group):
    codes = g.integers(0, 256, (pages, page, heads, d // 2)).astype(np.uint8)
    scale = g.random((pages, page, heads, d // group)) * 0.2 + 0.2
    return codes, np.stack([scale, scale * -7.5 + 0.3 * g.normal(size=scale.shape)], axis=-1)


@pytest.mark.parametrize("kw", [{}, dict(window=200), dict(softcap=3.0), dict(keep=True)])
def test_reference_attention_of_codes(kw):
    """With pieces enough it is the attention over the codes' values, with two another; and its bounds are a small part of the output, so that zeros, another group's offsets, or codes in
    another order do not pass."""
    g = np.random.default_rng(5)
    k, v = cache(g, 30, 16, 2, 64, 32), cache(g, 30, 16, 2, 64, 32)
    q = g.normal(size=(3, 8, 64))
    table = np.stack([g.permutation(30)[:28] for _ in range(3)])
    table[1, 3] = -1
    lens = [448, 300, 0]
    kw = dict(kw, keep=g.integers(0, 4, (3, 448)) if kw.get("keep") else None)
    want, lse, _, _ = ref.paged_attention(q, ref.values4(*k), ref.values4(*v), table, lens, 0.125, **kw)
    same, same_lse, err, lse_err = ref.paged_attention4(q, k, v, table, lens, 0.125, pieces=9, **kw)
    assert np.allclose(same, want, atol=1e-9) and np.allclose(same_lse[:2], lse[:2], atol=1e-9)
    assert (same_lse[2] == -np.inf).all() and (same[2] == 0).all()
    two, _, _, _ = ref.paged_attention4(q, k, v, table, lens, 0.125, pieces=2, **kw)
    # an element of q off by 2^-1 / 124 of the largest, 64 of them with codes within 7.5 of their mean
    # and scales of 0.4, shifts a score by so much at most, and p by e to it
    shift = np.abs(q).max() / 248 * 64 * 7.5 * 0.4 * 0.125
    assert 0 < np.abs(two - want).max() <= np.expm1(2 * shift) * np.abs(ref.values4(*v)).max()
    rms = np.sqrt((want[:2] ** 2).mean())
    assert np.sqrt((err[:2] ** 2).mean()) <= 0.1 * rms
    assert (err <= (2 * lse_err.max() + 1e-3) * 40).all()
    wrong = [np.zeros_like(want)]
    for codes, pairs in ((v[0], v[1][..., ::-1, :]), (v[0] >> 4 | v[0] << 4, v[1])):
        wrong.append(ref.paged_attention4(q, k, (codes, pairs), table, lens, 0.125, pieces=2, **kw)[0])
    for x in wrong:
        passed = np.abs(x - want)[:2] <= err[:2] + np.abs(want[:2]) * 2.0 ** -8
        assert passed.mean() < 0.2
