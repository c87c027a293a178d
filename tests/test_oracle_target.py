"""Pins of the oracle's verification-pass functions (oracle/target.py): closed
forms, hand-computed sets and invariants."""
import numpy as np
import pytest

import oracle as O


def test_e4m3_and_e2m1_values():
    v = O.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0**-9 and v[8] == 2.0**-6 and v[0x38] == 1.0 and v[0x7E] == 448.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and v[0xB8] == -1.0
    assert np.all(np.diff(v[:127]) > 0)
    assert O.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def test_quantise_ties_and_limits():
    """With a group maximum of 6 the scale is 1: midpoints go to the even code."""
    y = np.array([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, 0.2, 0.3, 4.9, 5.1, -6.0, 0.0]])
    codes, scale = O.quantise_fp4(y)
    assert scale.tolist() == [[0x38]]
    assert codes[0].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 0, 1, 6, 7, 15, 0]
    big, s = O.quantise_fp4(np.full((1, 16), 1e6))
    assert s.tolist() == [[0x7E]] and set(big[0]) == {7}  # clamped at 6 * 448
    tiny, s = O.quantise_fp4(np.full((1, 16), 6 * 2.0**-10))
    assert s.tolist() == [[0]] and set(tiny[0]) == {0}  # a tie with zero: even


def test_quantised_values_are_within_half_a_step():
    rng = np.random.default_rng(3)
    y = O.round_bf16(rng.standard_normal((50, 64)))
    v = O.fp4_values(*O.quantise_fp4(y))
    top = np.abs(y.reshape(50, 4, 16)).max(-1, keepdims=True)
    # the scale is at most 2^-4 off max / 6: an element in [4, 6] of the scale is at most 1 off, one beyond clamped
    assert np.all(np.abs(y - v).reshape(50, 4, 16) <= top / 6 * (1 + 2.0**-4))


def test_rotation_keeps_lengths_and_depends_on_distance():
    rng = np.random.default_rng(4)
    d = 32
    inv = 1e6 ** (-np.arange(0, d, 2) / d)
    cs = lambda p: (np.cos(p * inv), np.sin(p * inv))
    q, k = rng.standard_normal((2, d))
    dots = [float(O.rotate(q, *cs(p + 7)) @ O.rotate(k, *cs(p))) for p in (0, 5, 1000)]
    assert np.allclose(dots, dots[0], atol=32 * 2.0**-8)
    assert abs(np.linalg.norm(O.rotate(q, *cs(99))) - np.linalg.norm(q)) < 32 * 2.0**-8
    assert np.array_equal(O.rotate(q, *cs(0)), O.round_bf16(q))


def visible(C, n, j, mode, window, sinks, pos=None, tree=None):
    pos = pos if pos is not None else [C + i for i in range(n)]
    return [c for c in range(-1, C + n + 2) if O.sees(C, n, j, c, mode, window, sinks, pos, tree)]


def test_visible_slots_by_hand():
    assert visible(3, 2, 0, "causal", 0, 0) == [0, 1, 2, 3]
    assert visible(3, 2, 1, "causal", 0, 0) == [0, 1, 2, 3, 4]
    assert visible(3, 2, 0, "block", 0, 0) == [0, 1, 2, 3, 4]
    assert visible(8, 2, 1, "causal", 3, 0) == [7, 8, 9]
    assert visible(8, 2, 1, "causal", 3, 2) == [0, 1, 7, 8, 9]
    assert visible(8, 1, 0, "causal", 1, 0) == [8]
    assert visible(0, 1, 0, "causal", 0, 0) == [0]
    # a tree: node 2 is node 0's child at depth 1, like node 1
    tree = [[1, 0, 0], [1, 1, 0], [1, 0, 1]]
    assert visible(4, 3, 2, "tree", 0, 0, [4, 5, 5], tree) == [0, 1, 2, 3, 4, 6]
    assert visible(4, 3, 2, "tree", 2, 1, [4, 5, 5], tree) == [0, 4, 6]
    assert visible(4, 3, 1, "tree", 1, 0, [4, 5, 5], [[0] * 3] * 3) == []  # nothing left


@pytest.mark.parametrize("mode", ["causal", "block"])
def test_attention_closed_forms(mode):
    rng = np.random.default_rng(5)
    C, n, d = 5, 2, 8
    k, v, q = rng.standard_normal((C + n, 1, d)), rng.standard_normal((C + n, 1, d)), rng.standard_normal((n, 3, d))
    pos = [C, C + 1]
    # a window of one leaves a row its own value, whatever the scores
    out, mass, _ = O.paged_attention(q, k, v, C, "causal", 1, 0, pos)
    assert np.allclose(out, v[C:, [0, 0, 0]]) and np.allclose(mass, np.abs(out))
    # equal keys: the mean of the visible values
    out, _, _ = O.paged_attention(q, np.ones_like(k), v, C, mode, 0, 0, pos)
    assert np.allclose(out[0, 0], v[: C + (1 if mode == "causal" else n), 0].mean(0))
    # no slot: zeros
    out, _, _ = O.paged_attention(q, k, v, C, "tree", 1, 0, pos, [[0] * n] * n)
    assert not out.any()


def test_counts_and_rules_by_hand():
    c = np.zeros(8, dtype=np.uint16)
    O.count_tokens(c, [1, 2, 2, -1, 8], prompt=False)
    O.count_tokens(c, [2, 3], prompt=True)
    assert c.tolist() == [0, 1, 0x8002, 0x8000, 0, 0, 0, 0]
    c[5] = 32767
    O.count_tokens(c, [5], prompt=False)
    assert c[5] == 32767
    x = np.array([1.0, 2.0, -2.0, 4.0, 1.0, 0.0, 3.0, 3.0])
    c[5] = 0
    got = O.logit_rules(x, c, [6, 2], 2.0, 0.5, 0.25, [(7, 1.0), (7, 2.0), (9, 5.0)], np.arange(8) != 4)
    assert got.tolist() == [1.0, 1.0 - 0.75, -4.0 - 1.75, 2.0, -np.inf, 0.0, 1.5 - 0.75, 6.0]
