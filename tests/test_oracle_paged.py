"""The paged operators' oracle against closed forms (CPU)."""
import numpy as np

from oracle import batch as ob
from oracle import paged as op
from oracle import rope as orope


def test_rotation_by_quarter_turns():
    x = np.random.default_rng(1).standard_normal((3, 2, 128))
    for halves in (False, True):
        i, j = op.partners(64, halves)
        y, _ = op.norm_rope(x, None, 0.0, np.full((3, 64), np.pi / 2), halves)
        np.testing.assert_allclose(y[..., i], -x[..., j], atol=1e-15)
        np.testing.assert_allclose(y[..., j], x[..., i], atol=1e-15)


def test_products_depend_on_the_distance():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((1, 1, 128)), rng.standard_normal((1, 1, 128))
    f = op.frequencies((64, 32), 1e4)
    for halves in (False, True):
        dot = [(op.norm_rope(q, None, 0, op.angles([[p + 7, p - 3]], f, (32, 16)), halves)[0]
                * op.norm_rope(k, None, 0, op.angles([[p, p]], f, (32, 16)), halves)[0]).sum() for p in (0, 5, 100000)]
        np.testing.assert_allclose(dot, dot[0], rtol=1e-9)


def test_norm_and_untouched_dims():
    x = np.random.default_rng(3).standard_normal((4, 2, 128)) * 5
    w = np.linspace(0.5, 1.5, 128)
    y, _ = op.norm_rope(x, w, 1e-6, np.zeros((4, 10)), False)
    np.testing.assert_allclose(y, x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6) * w)
    np.testing.assert_allclose(((y / w) ** 2).mean(-1), 1, rtol=1e-5)


def test_three_axes_agree_with_the_models_tables():
    """The frequencies and the order of the axes are those of the DiT's own tables (which round angles to fp32)."""
    tc, ts, ic, is_ = orope.token_tables(9, 4, 6)
    h, w = 4, 6
    pos = orope.image_positions(9, h, w)
    a = op.angles(pos, op.frequencies((16, 56, 56), 1e4), (8, 28, 28))
    np.testing.assert_allclose(np.cos(a), ic, atol=9 * 2.0 ** -22)
    np.testing.assert_allclose(np.sin(a), is_, atol=9 * 2.0 ** -22)


def test_pages_are_the_rows_they_hold():
    rng = np.random.default_rng(4)
    pages = rng.standard_normal((7, 16, 2, 128))
    got = op.rows_of(pages, [3, -1, 0, 99], 50)
    np.testing.assert_array_equal(got, np.concatenate([pages[3], np.zeros((16, 2, 128)), pages[0], np.zeros((2, 2, 128))]))


def test_attention_is_that_of_the_same_rows_in_a_row():
    rng = np.random.default_rng(5)
    k, v = rng.standard_normal((2, 9, 16, 2, 128))
    q = rng.standard_normal((2, 3, 4, 128))
    table = np.array([[1, 5, 2], [8, 0, 3]])
    for causal in (False, True):
        o, A, *_ = op.paged_attention(q, k, v, table, [40, 2], None, causal, 0.1, 48)
        rows = [np.stack([op.rows_of(x, t, 48) for t in table]) for x in (k, v)]
        z = np.zeros((0, 2, 128))
        ref, RA = ob.prefix_attention(q, *rows, z, z, [40, 2], causal, 0.1)
        np.testing.assert_allclose(o, ref, atol=1e-14)
        np.testing.assert_allclose(A, RA, atol=1e-14)


def test_rows_past_a_chunk_and_empty_rows():
    rng = np.random.default_rng(6)
    k, v = rng.standard_normal((2, 3, 16, 1, 128))
    q = rng.standard_normal((3, 4, 1, 128))
    o, _, _, _, live = op.paged_attention(q, k, v, np.array([[0], [1], [2]]), [2, 16, 0], [4, 2, 1], True, 1.0, 16)
    assert live.tolist() == [[True] * 4, [True, True, False, False], [True, False, False, False]]
    assert not o[0, :2].any() and o[0, 2:].any() and not o[2].any()   # rows before the first key; no keys at all
    np.testing.assert_allclose(o[0, 2, 0], v[0, 0, 0])
