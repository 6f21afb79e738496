"""Pins of the oracle of the operators around a GDN layer (oracle/layers.py):
hand-worked cases and identities."""
import numpy as np

from oracle import layers


def test_attention_hand_worked():
    # Two tokens on one page, scores 0 and ln 3 -> weights 1/4 and 3/4.
    k = np.zeros((1, 1, 2, 1))
    k[0, 0, 1, 0] = np.log(3.0)
    v = np.array([[[[4.0], [8.0]]]])
    o, lse, drawn, _ = layers.paged_attention(np.ones((1, 1, 1, 1)), k, v, np.zeros((1, 1), int), [2], scale=1.0)
    assert abs(o.item() - 7.0) < 1e-14 and abs(lse.item() - np.log(4.0)) < 1e-14
    np.testing.assert_allclose(drawn[0, 0], [0.25, 0.75], atol=1e-15)


def test_attention_pages_and_split_do_not_matter():
    rng = np.random.default_rng(0)
    k, v = rng.normal(size=(2, 5, 2, 4, 8))
    q = rng.normal(size=(1, 2, 4, 8))
    table = np.array([[3, 0, 4]])
    whole, _, drawn, _ = layers.paged_attention(q, k, v, table, [11])
    # The same tokens as a prompt of 4 and beams' tables of 7 more.
    beam = (k, v, np.broadcast_to(table[:, None, 1:], (1, 2, 2)), np.full((1, 2), 7))
    split, _, _, _ = layers.paged_attention(q, k, v, table, [4], beam=beam)
    np.testing.assert_allclose(whole, split, atol=1e-14)
    assert abs(drawn.sum() - 2 * 4) < 1e-12


def test_empty_row_is_zero():
    o, lse, _, _ = layers.paged_attention(np.ones((1, 1, 1, 2)), np.ones((1, 1, 2, 2)), np.ones((1, 1, 2, 2)),
                                          np.zeros((1, 1), int), [0])
    assert (o == 0).all() and np.isneginf(lse).all()


def test_kept_positions():
    w = np.array([5.0, np.nan, 7.0, 5.0, -0.0, 0.0, 1.0])
    assert layers.kept_positions(w, 7, 4, 1) == [0, 2, 3, 6]
    assert layers.kept_positions(w, 7, 3, 1) == [0, 2, 6]     # the tie goes to the smaller position
    assert layers.kept_positions(w, 7, 6, 1) == [0, 2, 3, 4, 5, 6]
    assert layers.kept_positions(w, 7, 5, 1) == [0, 2, 3, 4, 6]
    assert layers.kept_positions(w, 2, 5, 3) == [0, 1]
    assert layers.kept_positions(w, 7, 3, 3) == [4, 5, 6]


def test_block_norm_hand_worked():
    x, n = layers.block_norm(y=[[3.0, 4.0]], x=[[1.0, 1.0]], w_post=[2.0, 1.0], alpha=0.5, w_pre=[1.0, 1.0], eps=0.0)
    r = np.sqrt(12.5)
    np.testing.assert_allclose(x, [[1 + 3 / r, 1 + 2 / r]], atol=1e-14)
    np.testing.assert_allclose((n ** 2).mean(), 1.0, atol=1e-14)
    g, _ = layers.block_norm(y=[[1.0, 2.0]], gate=[[0.0, np.log(3.0)]], act="sigmoid")
    np.testing.assert_allclose(g, [[0.5, 1.5]], atol=1e-14)
