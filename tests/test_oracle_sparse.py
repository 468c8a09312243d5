"""The oracle of the rotated append and of block-sparse decode, pinned to closed forms."""

import numpy as np
import pytest

from oracle import attention as OA
from oracle import sparse as OS


def test_rotation_is_complex_multiplication():
    rng = np.random.default_rng(0)
    R, P = 16, 50
    angles = np.arange(P)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
    table = np.concatenate([np.cos(angles), np.sin(angles)], axis=1)
    x, pos = rng.standard_normal((7, 3, 24)), rng.integers(0, P, 7)
    for interleaved in (False, True):
        y = OS.rotate(x, table, pos, interleaved=interleaved)
        pick = (lambda z: z[..., 0:R:2] + 1j * z[..., 1:R:2]) if interleaved else \
            (lambda z: z[..., :R // 2] + 1j * z[..., R // 2:R])
        assert np.allclose(pick(y), pick(x) * np.exp(1j * angles[pos])[:, None], atol=1e-14)
        assert np.array_equal(y[..., R:], x[..., R:])


def test_rotated_logits_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    R = 32
    angles = np.arange(200)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
    table = np.concatenate([np.cos(angles), np.sin(angles)], axis=1)
    q, k = rng.standard_normal((1, 1, R)), rng.standard_normal((1, 1, R))
    dots = [float((OS.rotate(q, table, [p + 17]) * OS.rotate(k, table, [p])).sum()) for p in (0, 3, 150)]
    assert np.ptp(dots) < 1e-12


def test_axes_take_their_own_positions():
    rng = np.random.default_rng(2)
    angles = np.arange(40)[:, None] * np.array([1.0, 0.1, 0.01, 0.5])
    table = np.concatenate([np.cos(angles), np.sin(angles)], axis=1)
    x = rng.standard_normal((5, 2, 8))
    pos = rng.integers(0, 40, (2, 5))
    both = OS.rotate(x, table, pos, pair_axis=[0, 1, 1, 0])
    one = [OS.rotate(x, table, pos[a]) for a in (0, 1)]
    for j, a in enumerate((0, 1, 1, 0)):
        for d in (j, j + 4):
            assert np.array_equal(both[..., d], one[a][..., d])


def test_scores_bound_every_logit_and_are_reached_by_single_rows():
    rng = np.random.default_rng(3)
    kc = rng.standard_normal((9, 2, 4, 16))
    tables, lens = np.array([[3, 1, 8], [0, 5, -1]]), [10, 5]
    lo, hi = np.zeros((9, 2, 16)), np.zeros((9, 2, 16))
    OS.block_bounds(kc, tables, lens, lo, hi)
    q = rng.standard_normal((2, 6, 16))
    scores, _ = OS.block_scores(q, lo, hi, tables, lens, 0.25, 4)
    for i, h, b in np.ndindex(2, 2, 3):
        rows = min(4, lens[i] - 4 * b)
        if rows <= 0:
            assert scores[i, h, b] == -np.inf
            continue
        logits = 0.25 * q[i, 3 * h:3 * h + 3] @ kc[tables[i, b], h, :rows].T
        assert scores[i, h, b] >= logits.max() - 1e-12
        if rows == 1:
            assert np.isclose(scores[i, h, b], logits.max())


def test_select_keeps_the_ends_and_the_best():
    nan = float("nan")
    s = np.array([[[0., 5., 1., 5., nan, -np.inf, 5., 9.]]])
    pick = lambda **k: OS.block_select(s, [8], 1, **k)[0, 0].tolist()
    assert pick(num_selected=3) == [1, 4, 7]
    assert pick(num_selected=4) == [1, 3, 4, 7]
    assert pick(num_selected=3, sink=1, recent=1) == [0, 4, 7]
    assert pick(num_selected=2, sink=1, recent=1) == [0, 7]
    assert pick(num_selected=9) == list(range(8)) + [-1]
    assert OS.block_select(s, [0], 1, 2)[0, 0].tolist() == [-1, -1]


@pytest.mark.parametrize("group", [1, 3])
def test_all_blocks_selected_is_dense_attention(group):
    rng = np.random.default_rng(4)
    H, D, bs, lens = 2, 8, 4, [11, 4, 0]
    kc, vc = rng.standard_normal((12, H, bs, D)), rng.standard_normal((12, H, bs, D))
    tables = np.array([[7, 2, 9], [4, 0, 0], [1, 1, 1]])
    q = rng.standard_normal((3, H * group, D))
    every = np.broadcast_to(np.array([2, 0, 1, -1]), (3, H, 4))
    out, _, _ = OS.sparse_attention(q, kc, vc, tables, lens, every, 0.3)
    dense = OA.paged_decode_attention(q, kc.repeat(group, axis=1), vc.repeat(group, axis=1), tables,
                                      lens, 0.3, bs, "f64")
    assert np.allclose(out, dense, atol=1e-13)
