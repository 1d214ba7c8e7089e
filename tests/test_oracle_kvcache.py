"""Pins of the paged-cache oracle: its attention against the one-token oracle
and against a two-position softmax by hand, its quantiser against the
activation quantiser's oracle, and its places against a table by hand."""
import math

import numpy as np

import oracle.kvcache as OK
from kv_util import bf16_values, bits


def test_places_by_hand():
    # three sequences: 2 new rows of 5 positions, none, 2 new rows of 1 position (the first has no place)
    got = list(OK.places([0, 2, 2, 4], [5, 3, 1], [[7, 4], [9, 9], [2, 0]], 4))
    assert got == [(0, 0, 3, 7, 3), (1, 0, 4, 4, 0), (3, 2, 0, 2, 0)]


def test_quantise_is_the_activation_quantiser(O):
    x = bf16_values(np.random.default_rng(1), (40, 128), 3.0)
    x[3] = 0
    x[4] = 1e-7
    code, step = OK.quantise(x)
    q, s_x, _ = O.quantize_input(bits(x))
    assert np.array_equal(code, q)
    assert np.array_equal(step, (np.float32(1) / s_x).astype(np.float32))


def test_quantise_marks_rows_without_a_scale():
    x = np.ones((3, 64), np.float32)
    x[0, 5], x[2, 63] = np.inf, np.nan
    code, step = OK.quantise(x)
    assert (code[[0, 2]] == 0).all() and np.isnan(step[[0, 2]]).all()
    assert (code[1] == 127).all() and np.isfinite(step[1])


def test_attention_two_positions_by_hand():
    d = 64
    q = np.zeros((2, 1, d))
    q[:, 0, 0] = 2.0
    k = np.zeros((2, 1, d))
    k[1, 0, 0] = 1.5
    v = np.stack([np.full((1, d), 1.0), np.full((1, d), 5.0)])
    out, _, mag, seen = OK.attention(q, [k], [v], [0, 2], [2], 0.5, True, np.zeros((2, 1, d)))
    w = math.exp(1.5) / (1 + math.exp(1.5))
    assert np.allclose(out[0], 1.0) and np.allclose(out[1], 1.0 + 4.0 * w, rtol=1e-14)
    assert seen.tolist() == [[1], [2]] and mag[1, 0] == 1.5


def test_attention_of_one_row_is_the_decode_oracle(O):
    import oracle.attention as OA
    rng = np.random.default_rng(2)
    k, v, q = rng.standard_normal((33, 2, 64)), rng.standard_normal((33, 2, 64)), rng.standard_normal((1, 8, 64))
    out, _, _, _ = OK.attention(q, [k], [v], [0, 1], [33], 0.125, True, np.zeros((1, 8, 64)))
    assert np.allclose(out.reshape(-1), OA.attn_decode(q.reshape(-1), k, v, 33, 8, 2, 64, 0.125), rtol=1e-13)


def test_attention_row_that_sees_nothing_is_zeros():
    out, _, _, seen = OK.attention(np.ones((3, 1, 64)), [np.ones((1, 1, 64))], [np.ones((1, 1, 64))], [0, 2], [1],
                                   1.0, True, np.full((3, 1, 64), 7.0))
    assert (out[0] == 0).all() and (out[1] == 1).all() and (out[2] == 7).all() and seen[0, 0] == 0
