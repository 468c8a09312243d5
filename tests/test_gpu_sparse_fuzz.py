"""Seeded random configurations of the rotary append and the block-sparse decode, each against the
oracle with the checks and tolerances of test_gpu_append_rope and test_gpu_sparse."""

import numpy as np
import pytest
import torch

import test_gpu_append_rope as A
import test_gpu_sparse as S
from oracle import sparse as OS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def _lengths(rng, most):
    hi = int(rng.choice(most))
    lens = rng.integers(0, hi + 1, int(rng.integers(1, 9)))
    lens[0] = hi
    return lens


@pytest.mark.parametrize("seed", range(60))
def test_sparse_decode_random_configuration(B, seed):
    rng = np.random.default_rng(7000 + seed)
    D, H, bs = int(rng.choice([64, 128, 256])), int(rng.integers(1, 6)), int(rng.choice([8, 16, 32, 48, 80]))
    group = int(rng.choice([1, 2, 3, 5, 7, 8, 9, 12, 16, 17, 33]))
    lens, keep = _lengths(rng, [3, 40, 300, 1500, 4000]), int(rng.choice([1, 2, 3, 7, 20, 64, 300, 700]))
    dtype = [torch.float16, torch.bfloat16][int(rng.integers(2))]
    out_dtype = [torch.float32, torch.float16, torch.bfloat16][int(rng.integers(3))]
    b = S.make(seed, lens, H * group, H, D, bs, dtype, wide=int(rng.integers(0, 4)))
    rec = B.new_error_record()
    s = S.scores_of(B, b, error_record=rec)
    S.check_scores(s, b)
    sink = int(rng.integers(0, min(3, keep) + 1))
    recent = int(rng.integers(0, min(4, keep - sink) + 1))
    sel = B.paged_block_select(s, S.dev(lens), bs, keep, sink, recent, error_record=rec).cpu().numpy()
    assert np.array_equal(sel, OS.block_select(s.cpu().numpy(), lens, bs, keep, sink, recent))
    for listed in (sel, S.lists(rng, b, keep)):
        S.check_attention(S.attend(B, b, listed, out_dtype=out_dtype, error_record=rec), b, listed)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]


@pytest.mark.parametrize("seed", range(40))
def test_select_random_configuration(B, seed):
    rng = np.random.default_rng(8000 + seed)
    rows, width = int(rng.choice([5, 300, 700])), int(rng.choice([3, 100, 900, 1100, 3000, 9000, 20000]))
    keep = int(rng.integers(1, min(width, 400) + 1))
    sink = int(rng.integers(0, keep + 1))
    recent = int(rng.integers(0, keep - sink + 1))
    s = rng.standard_normal((rows, 1, width)).astype(np.float32)
    kind = int(rng.integers(4))
    if kind == 1:
        s = np.round(s * 4)
    elif kind == 2:
        s = (s * np.float32(10.0) ** rng.integers(-44, 38, s.shape)).astype(np.float32)
    elif kind == 3:
        s = np.round(s)
        for v in (np.nan, np.inf, -np.inf):
            s[rng.random(s.shape) < 0.02] = v
    lens = rng.integers(0, width + 1, rows)
    rec = B.new_error_record()
    got = B.paged_block_select(torch.from_numpy(s).cuda(), S.dev(lens), 1, keep, sink, recent,
                               error_record=rec).cpu().numpy()
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    some = rng.choice(rows, min(rows, 40), replace=False)
    assert np.array_equal(got[some], OS.block_select(s[some], lens[some], 1, keep, sink, recent))


@pytest.mark.parametrize("seed", range(60))
def test_append_random_configuration(B, seed):
    rng = np.random.default_rng(9000 + seed)
    D = int(rng.choice([16, 32, 48, 64, 96, 128, 192, 256]))
    R = int(rng.integers(0, D // 16 + 1)) * 16
    bs, H = int(rng.choice([1, 3, 8, 16, 32, 100, 700])), int(rng.integers(1, 6))
    group = int(rng.choice([1, 2, 3, 5, 8, 17]))
    lens = _lengths(rng, [3, 40, 300, 1500])
    news = np.minimum(lens, rng.integers(0, int(rng.choice([2, 2, 4, 5, 6, 30, 400])), len(lens)))
    news[0] = max(1, news[0])
    st = A.make(seed, lens, news, H * group, H, D, R, bs, [torch.float16, torch.bfloat16][int(rng.integers(2))],
                int(rng.integers(1, 5)) if R else 1, bool(rng.integers(2)), pad=int(rng.integers(0, 3)))
    before, rec = A.snapshot(st), B.new_error_record()
    out = A.call(B, st, error_record=rec)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    A.check(B, st, out, before)
