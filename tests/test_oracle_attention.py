"""Pins of the attention and eviction oracle against values that follow from
the definitions alone: elementwise sums in plain Python, rows whose result is
known, ties, and compaction by hand."""

import math

import numpy as np
import pytest

from oracle import attention, formats


def _codes(rng, shape, fmt):
    """Random finite codes."""
    c = rng.integers(0, 256, shape, dtype=np.uint8)
    return np.where(np.isfinite(formats.decode(c, fmt)), c, 0).astype(np.uint8)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("kind", ["tensor", "head", "channel"])
def test_kv_attention_by_elementwise_sums(fmt, kind):
    rng = np.random.default_rng(3 + fmt)
    H, Hk, D, bs, slots = 4, 2, 6, 3, 24
    lens, news = [7, 4, 1], [2, 1, 1]
    table = rng.permutation(slots // bs)[:9 - 1].tolist() + [-1]
    table = np.array(table, np.int64).reshape(3, 3)
    starts = np.concatenate([[0], np.cumsum(news)])
    kc, vc = _codes(rng, (slots, Hk, D), fmt), _codes(rng, (slots, Hk, D), fmt)
    n = {"tensor": 1, "head": Hk, "channel": Hk * D}[kind]
    ks, vs = rng.uniform(1e-3, 2e-3, n), rng.uniform(0.5, 2, n)
    q = rng.standard_normal((sum(news), H, D))
    got = attention.kv_attention(q, kc, vc, table, bs, starts, lens, ks, vs, fmt, 0.4)

    def scale(s, h, d):
        return s[0] if kind == "tensor" else s[h] if kind == "head" else s[h * D + d]

    for b in range(3):
        received = np.zeros((Hk, lens[b]))
        for i in range(news[b]):
            for h in range(H):
                kh, terms = h // 2, []
                for j in range(lens[b] - news[b] + i + 1):
                    s = int(table[b, j // bs]) * bs + j % bs
                    dot = sum(q[starts[b] + i, h, d] * formats.decode_code(int(kc[s, kh, d]), fmt) * scale(ks, kh, d)
                              for d in range(D))
                    terms.append((0.4 * dot, s))
                top = max(x for x, _ in terms)
                l = sum(math.exp(x - top) for x, _ in terms)
                assert got[b]["lse"][i, h] == pytest.approx(top + math.log(l), rel=1e-12)
                for j, (x, _) in enumerate(terms):
                    received[kh, j] += math.exp(x - top) / l
                for d in range(D):
                    o = sum(math.exp(x - top) / l * formats.decode_code(int(vc[s, kh, d]), fmt) * scale(vs, kh, d)
                            for x, s in terms)
                    assert got[b]["out"][i, h, d] == pytest.approx(o, rel=1e-9, abs=1e-9)
        assert np.allclose(got[b]["weights"], received, rtol=1e-12, atol=1e-14)


def test_rows_that_see_one_position_or_none():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 2, 4)), rng.standard_normal((5, 1, 4)), rng.standard_normal((5, 1, 4))
    out, lse, p, _, _ = attention.attend(q, k, v, [0, 1, 5], 0.5)
    assert (out[0] == 0).all() and (lse[0] == -np.inf).all() and (p[0] == 0).all()
    assert np.allclose(out[1], v[0, 0]) and np.allclose(lse[1], (q[1] @ k[0, 0]) * 0.5)
    assert np.allclose(p[2].sum(-1), 1)
    # equal scores: the mean of the values
    out, lse, _, _, _ = attention.attend(np.zeros((1, 2, 4)), k, v, [5], 1.0)
    assert np.allclose(out[0], v[:, 0].mean(0)) and np.allclose(lse, math.log(5))


def test_pages_outside_the_pool_are_left_out():
    rng = np.random.default_rng(2)
    kc, vc = _codes(rng, (8, 1, 4), 0), _codes(rng, (8, 1, 4), 0)
    q = rng.standard_normal((2, 1, 4))
    args = ([0, 2], [6], [1.0], [1.0], 0, 0.01)
    holed = attention.kv_attention(q, kc, vc, np.array([[1, -1, 0]]), 2, *args)[0]
    whole = attention.kv_attention(q, kc, vc, np.array([[1, 0]]), 2, [0, 2], [4], *args[2:])[0]
    assert np.array_equal(holed["out"], whole["out"]) and np.array_equal(holed["lse"], whole["lse"])
    assert (holed["weights"][0, 2:4] == 0).all()


def test_evict_select_by_hand():
    w = np.zeros((3, 2, 8), np.float32)
    w[0] = [[1, 5, 2, 2, 2, 0, 0, 9], [0, 0, 1, 1, 1, 0, 8, 9]]     # scores 1 5 3 3 3 0 8 18
    w[1] = 1.0
    w[2, 0] = [np.nan, 2, np.inf, -1, 0, 1, 0, 0]
    kept, lens = attention.evict_select(w, [8, 3, 7], 4, 1, 1)
    assert kept.tolist() == [[0, 1, 6, 7], [0, 1, 2, -1], [0, 1, 2, 6]] and lens.tolist() == [4, 3, 4]
    kept, _ = attention.evict_select(w, [8, 8, 7], 4, 0, 0)
    assert kept.tolist() == [[1, 2, 6, 7], [0, 1, 2, 3], [1, 2, 4, 5]]


def test_compact_by_hand():
    cache = np.arange(12, dtype=np.uint8).reshape(6, 1, 2)
    table = np.array([[2, 0]])                                       # slots 4 5 0 1
    kept, lens = np.array([[1, 3, -1]]), np.array([2])
    out = attention.compact(cache, table, table, 2, kept, lens)
    assert out[4].tolist() == cache[5].tolist() and out[5].tolist() == cache[1].tolist()
    assert np.array_equal(out[:4], cache[:4])
    out = attention.compact(cache, table, np.array([[-1, 1]]), 2, kept, lens)
    assert np.array_equal(out, cache)                                 # positions 0 and 1 lie in the dropped page
