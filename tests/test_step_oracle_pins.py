"""Pins of the oracles of oracle/step.py: closed forms and invariants."""
import math

import numpy as np
import pytest

from oracle import step


def test_plan_two_requests_by_hand():
    table = np.array([[5, -1, -1], [7, 9, -1]])
    r = step.page_plan([127, 256], [2, 3], [20, 21, 22], table, S1=3, T=6, num_blocks=30)
    assert r["block_table"].tolist() == [[5, 20, -1], [7, 9, 21]]
    assert r["act_seqs"].tolist() == [129, 259] and r["num_taken"] == 2 and r["status"] == 0
    assert r["cache_index"].tolist() == [5 * 128 + 127, 20 * 128, -1, 21 * 128, 21 * 128 + 1, 21 * 128 + 2]
    assert r["positions"].tolist() == [127, 128, 0, 256, 257, 258]
    assert r["seq_ids"].tolist() == [0, 0, -1, 1, 1, 1] and r["cu_seqs"].tolist() == [0, 2, 5]
    assert r["tree_mask"] == [1, 3, 0, 1, 3, 7]


def test_plan_tree_by_hand():
    #       0        root of the draft
    #      / \
    #     1   2
    #     |   |\
    #     3   4 5
    r = step.page_plan([10], None, [], np.array([[0]]), S1=6, T=6, num_blocks=1, parents=[[-1, 0, 0, 1, 2, 2]])
    assert r["positions"].tolist() == [10, 11, 11, 12, 12, 12]
    assert r["tree_mask"] == [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b100101]


def test_plan_without_pages():
    r = step.page_plan([0, 0], None, [3], np.array([[-1], [-1]]), S1=2, T=4, num_blocks=4)
    assert r["cache_index"].tolist() == [384, 385, -1, -1] and r["status"] == step.NO_PAGE and r["num_taken"] == 1


def test_rope_frequencies_closed_forms():
    f = step.rope_freqs(64)
    assert f[0] == 1 and abs(f[16] - 0.01) < 1e-17
    np.testing.assert_allclose(step.rope_freqs(64, scaling="linear", factor=8.0) * 8, f, rtol=1e-15)
    # the slowest pair of the ntk form is stretched by exactly the factor, the fastest not at all
    g = step.rope_freqs(64, scaling="ntk", factor=8.0)
    assert g[0] == 1 and abs(g[-1] * 8 / f[-1] - 1) < 1e-12
    y = step.rope_freqs(64, scaling="yarn", factor=40.0)
    assert y[0] == f[0] and abs(y[-1] * 40 / f[-1] - 1) < 1e-12 and (np.diff(y) < 0).all()
    # f (1 - r) + f / 1 r is f up to four roundings (1 - r, two products, the sum) of half a step, 2^-53 each
    np.testing.assert_allclose(step.rope_freqs(64, scaling="yarn", factor=1.0), f, rtol=4 * 2.0 ** -53, atol=0)


@pytest.mark.parametrize("half", [False, True])
def test_rope_turns_scores_by_relative_position(half):
    """q . k after the rotation depends on the distance of their positions alone, and the inverse undoes it."""
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 40))
    f = step.rope_freqs(32)

    def dot(a, b):
        return float((step.rope_apply(q, [a], f, rot_off=8, half=half)
                      * step.rope_apply(k, [b], f, rot_off=8, half=half)).sum())
    assert math.isclose(dot(3, 10), dot(1003, 1010), rel_tol=1e-10)
    y = step.rope_apply(q, [77], f, rot_off=8, half=half)
    np.testing.assert_allclose(step.rope_apply(y, [77], f, rot_off=8, half=half, inverse=True), q, atol=1e-14)
    np.testing.assert_array_equal(y[..., :8], q[..., :8])
