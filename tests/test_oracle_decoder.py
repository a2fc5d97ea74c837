"""Pins of the decoder oracle (norms, rotation, cache codes, attention) by
identities and hand-worked values -- no GPU."""
import numpy as np
import pytest

from oracle import decoder as od


def test_norm_of_constant_rows_is_the_weight():
    w = np.array([1.0, -2.0, 0.5, 3.0])
    r, y = od.norm_residual(None, np.full((2, 4), 7.0), None, None, 1.0, w, 0.0)
    np.testing.assert_allclose(r, 7.0)
    np.testing.assert_allclose(y, np.broadcast_to(w, (2, 4)))


def test_norm_parts():
    x, res = np.array([[3.0, -4.0]]), np.array([[1.0, 1.0]])
    r, y = od.norm_residual(x, res, [1.0, 2.0], [10.0, 100.0], 0.5, None, 0.0)
    rms = np.sqrt(12.5)
    np.testing.assert_allclose(r, [[1 + 0.5 * 10 * 3 / rms, 1 + 0.5 * 100 * 2 * -4 / rms]])
    np.testing.assert_allclose(np.mean(y ** 2), 1.0)


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_keeps_norms_and_composes(pairs):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 16)).astype(np.float32)
    a = rng.uniform(0, 6, 4)
    y = od.rotate(x, np.cos(a), np.sin(a), pairs)
    np.testing.assert_allclose((y ** 2).sum(1), (x ** 2).sum(1), rtol=1e-6)
    assert np.array_equal(y[:, 8:], x[:, 8:])
    back = od.rotate(y, np.cos(-a), np.sin(-a), pairs)
    np.testing.assert_allclose(back, x, atol=1e-6)
    quarter = od.rotate(np.eye(8, dtype=np.float32)[:1], np.zeros(4), np.ones(4), pairs)
    assert quarter[0, 1 if pairs else 4] == 1.0


@pytest.mark.parametrize("amax,E", [(0.0, 87), (127.0, 127), (127.5, 128), (126.9, 127), (63.5, 126),
                                    (127.0 * 2.0 ** 40, 167), (128.0 * 2.0 ** 40, 255),
                                    (float("inf"), 255), (float("nan"), 255), (1e-30, 87)])
def test_scale_byte(amax, E):
    assert od.scale_byte(amax) == E


def empty(n_pages=4, heads=1, page=32, dim=16):
    z = np.zeros((n_pages, heads, page, dim), np.int8)
    e = np.full((n_pages, heads, page // 32), 200, np.uint8)   # whatever was there
    return od.Cache(z, z, e, e)


def test_append_grows_the_unit_and_rerounds_held_codes():
    c = empty()
    table = np.array([[2]])
    small, big = np.zeros((1, 1, 16), np.float32), np.zeros((1, 1, 16), np.float32)
    small[0, 0, :4] = [127, 3, -5, 1]
    big[0, 0, 0] = 508                                          # needs 4 times the unit
    c.append(table, [0], [0, 1], small, small)
    assert c.scales[0][2, 0, 0] == 127 and list(c.codes[0][2, 0, 0, :4]) == [127, 3, -5, 1]
    c.append(table, [1], [0, 1], big, small)
    assert c.scales[0][2, 0, 0] == 129 and c.scales[1][2, 0, 0] == 127
    assert list(c.codes[0][2, 0, 0, :4]) == [32, 1, -1, 0]      # 31.75, 0.75, -1.25, 0.25
    assert c.codes[0][2, 0, 1, 0] == 127
    np.testing.assert_array_equal(c.values([2], 1, 0)[0, :1], [508.0])


def test_append_marks_and_restarts_a_block():
    c = empty()
    x = np.ones((1, 1, 16), np.float32)
    bad = x.copy()
    bad[0, 0, 3] = np.inf
    c.append(np.array([[1]]), [4], [0, 1], bad, x)
    assert c.scales[0][1, 0, 0] == 255 and np.isnan(c.values([1], 0, 0)).all()
    c.append(np.array([[1]]), [5], [0, 1], x, x)
    assert c.scales[0][1, 0, 0] == 255
    c.append(np.array([[1]]), [0], [0, 1], x, x)                # a first token starts afresh
    assert c.scales[0][1, 0, 0] == 121


def test_append_skips_tokens_without_a_page():
    c = empty()
    before = c.codes[0].copy()
    x = np.ones((3, 1, 16), np.float32)
    c.append(np.array([[9], [1], [-1]]), [0, 32, 0], [0, 1, 2, 3], x, x)
    assert np.array_equal(c.codes[0], before)


def test_attention_identities():
    rng = np.random.default_rng(2)
    c = empty(n_pages=3, heads=2, page=64, dim=16)
    for s in c.scales:
        s[:] = 120
    for k in c.codes:
        k[:] = rng.integers(-127, 128, k.shape)
    table = np.array([[2, 0]])
    q = rng.standard_normal((1, 4, 16))
    # one visible position: its value, whatever the scores
    out, _, _ = od.attention(c, table, [70], [0, 1], 1, q, 0.3, window=1)
    for h in range(4):
        np.testing.assert_allclose(out[0, h], c.values(table[0], 70, 1)[h // 2])
    # equal scores: the mean
    out, _, _ = od.attention(c, table, [9], [0, 1], 1, 0 * q, 0.3)
    np.testing.assert_allclose(out[0, 0], np.mean([c.values(table[0], j, 1)[0] for j in range(10)], axis=0))
    # a sink equal to the (zero) scores counts as one more position of value 0
    sunk, _, _ = od.attention(c, table, [9], [0, 1], 1, 0 * q, 0.3, sinks=np.zeros(4))
    np.testing.assert_allclose(sunk, out * 10 / 11)
    # nothing visible: 0
    out, _, _ = od.attention(c, np.array([[7, 7]]), [9], [0, 1], 1, q, 0.3)
    assert not out.any()


def test_bound_is_tight_enough_to_see_a_mistake():
    """A lost position, a shifted window or a swapped head is outside the bound."""
    rng = np.random.default_rng(3)
    c = empty(n_pages=3, heads=2, page=64, dim=64)
    for s in c.scales:
        s[:] = 122
    for k in c.codes:
        k[:] = np.clip(np.rint(30 * rng.standard_normal(k.shape)), -127, 127)
    table = np.array([[2, 0]])
    q = rng.standard_normal((1, 4, 64))
    good, mag, xmag = od.attention(c, table, [100], [0, 1], 1, q, 0.125)
    for dtype in ("float32", "float16", "bfloat16"):
        bound = od.attention_bound(dtype, 64, 101, good, mag, xmag)
        for other in (od.attention(c, table, [99], [0, 1], 1, q, 0.125)[0],
                      od.attention(c, table, [100], [0, 1], 1, q, 0.125, window=100)[0],
                      good[:, ::-1]):
            assert (np.abs(other - good) > bound).any()
