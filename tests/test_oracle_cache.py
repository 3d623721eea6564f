"""Pins of the 4-bit cache, attention-weight and eviction oracle (CPU)."""

import numpy as np
import pytest

import oracle as O
from oracle import cache_oracle as C


def test_grids_hold_the_formats_values():
    assert C.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert len(C.E4M3) == 127 and C.E4M3[-1] == 448 and C.E4M3[1] == 2.0 ** -9 and C.E4M3[0x38] == 1.0


@pytest.mark.parametrize("v,code", [(0.25, 0), (0.26, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6),
                                    (5.01, 7), (1e30, 7)])
def test_ties_go_to_the_even_code_and_large_values_saturate(v, code):
    assert C.nearest_code(np.array([v]), C.E2M1)[0] == code


def test_representable_rows_come_back_unchanged():
    rng = np.random.default_rng(0)
    s = C.E4M3[rng.integers(8, 100, size=(5, 3))]
    y = C.E2M1[rng.integers(0, 7, size=(5, 3, 16))] * rng.choice([-1, 1], size=(5, 3, 16))
    y[..., 3] = 6.0  # the block's largest magnitude fixes the scale
    y = (y * s[..., None]).reshape(5, 48)
    for ls in (1.0, 2.0 ** -7):
        c4, s8 = C.fp4_quantise(y * ls, ls)
        assert np.array_equal(O.fp4_values(c4, s8, ls), y * ls)


def test_first_feature_is_the_low_half():
    y = np.zeros((1, 16))
    y[0, 0], y[0, 1] = 6.0, -3.0
    c4, s8 = O.fp4_quantise(y)
    assert c4[0, 0] == 0x7 | (0xD << 4) and s8[0, 0] == 0x38


def test_error_is_bounded_by_half_a_step():
    y = np.random.default_rng(1).standard_normal((64, 512))
    v = O.fp4_values(*O.fp4_quantise(y))
    s = np.repeat(np.abs(y).reshape(64, 32, 16).max(-1) / 6.0, 16, -1).reshape(y.shape)
    # the widest step is 2 scales; a scale is at most 2^-4 below amax / 6, so 6 scales may fall short by 2^-4
    assert (np.abs(v - y) <= s * (1 + 2.0 ** -4) * 1.0).all()


def test_nan_block_reads_as_nan_and_zero_block_as_zero():
    y = np.zeros((1, 48))
    y[0, 20], y[0, 40] = np.nan, 1.0
    v = O.fp4_values(*O.fp4_quantise(y))[0]
    assert (v[:16] == 0).all() and np.isnan(v[16:32]).all() and v[40] == pytest.approx(1.0, rel=2.0 ** -4)


def test_weights_are_the_softmax_summed_over_heads():
    rng = np.random.default_rng(2)
    T, n_h, L = 3, 2, 7
    q, qp = rng.standard_normal((T, n_h, 32)), rng.standard_normal((T, n_h, 4))
    c, k = rng.standard_normal((L, 32)), rng.standard_normal((L, 4))
    lse = np.empty((T, n_h))
    for s in range(T):
        n = L - T + s + 1
        _, lse[s], _ = O.latent_attention(q[s], qp[s], c[:n], k[:n], 0.3)
    w = O.token_weights(q, qp, c, k, 0.3, lse)
    assert w.sum() == pytest.approx(T * n_h, rel=1e-12)  # each head of each token hands out weight 1
    lse[1] = -np.inf
    assert O.token_weights(q, qp, c, k, 0.3, lse).sum() == pytest.approx((T - 1) * n_h, rel=1e-12)
    assert w[-1] < n_h  # the last row is seen by the last token alone


def test_evict_map_on_a_worked_case():
    acc = [9, 1, 5, 1, 7, 3, 1, 8]
    # sink row 0, recent row 7; of rows 1..6 the heaviest two are 4 and 2; rows kept: 0 2 4 7
    assert O.evict_map(acc, 8, 4, 1, 1) == [0, 4, 2, 7]
    assert O.evict_map(acc, 4, 4, 1, 1) == [0, 1, 2, 3]
    assert O.evict_map([1] * 6, 6, 3, 0, 0) == [0, 1, 2]           # ties: the lower rows
    assert O.evict_map([np.nan, 0, -1, 0], 4, 2, 0, 0) == [3, 1]   # a NaN is the least
    assert O.evict_map(acc, 8, 2, 1, 1) == [0, 7]


@pytest.mark.parametrize("mistake", ["ceil_scale", "block32", "nibbles", "ties_up"])
def test_planted_mistakes_change_the_values(mistake):
    rng = np.random.default_rng(3)
    y = rng.standard_normal((8, 64))
    y[:, 0::16] = 6.0      # scale exactly 1
    y[:, 1::16] = 2.5      # a tie
    y[:, 2::16] = rng.uniform(-6, 6, (8, 4))
    good = O.fp4_values(*O.fp4_quantise(y))
    if mistake == "nibbles":
        c4, s8 = O.fp4_quantise(y)
        bad = O.fp4_values(((c4 >> 4) | (c4 << 4)).astype(np.uint8), s8)
    elif mistake == "block32":
        c4, s8 = O.fp4_quantise(y)
        bad = O.fp4_values(c4, np.repeat(s8[:, ::2], 2, -1))
        y2 = y.copy()
        y2[:, 16:32] *= 4
        c4, s8 = O.fp4_quantise(y2)
        good, bad = O.fp4_values(c4, s8), O.fp4_values(c4, np.repeat(s8[:, ::2], 2, -1))
    elif mistake == "ceil_scale":
        y3 = y * 1.07
        c4, s8 = O.fp4_quantise(y3)
        good, bad = O.fp4_values(c4, s8), O.fp4_values(c4, s8 + 1)
    else:
        bad = good.copy()
        bad[np.abs(y) == 2.5] = 3.0
    assert not np.array_equal(good, bad)
