"""Seeded random configurations of the grouped chunk attention, the attention weights and the eviction: head
layouts, block sizes, lengths from nothing to thousands, windows, lists; checked as in test_gpu_evict, whose
tolerances hold here too."""

import numpy as np
import pytest
import torch

import test_gpu_evict as E
import test_gpu_sparse as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def layout(rng, most_group):
    H = int(rng.choice([1, 1, 2, 3, 5]))
    group = int(rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 31, 64, 128) if g <= most_group // H]))
    return H * group, H, int(rng.choice([64, 128, 256])), int(rng.choice([8, 16, 32, 48, 64])), (
        torch.bfloat16 if rng.random() < 0.5 else torch.float16)


def lengths(rng, budget):
    """Lengths whose sum is about the budget, some of them nothing."""
    n = int(rng.choice([1, 1, 2, 3, 7, 20]))
    lens = rng.integers(0, max(2, 2 * budget // n), n)
    lens[rng.random(n) < 0.1] = 0
    return lens.astype(np.int32)


@pytest.mark.parametrize("seed", range(40))
def test_chunks_and_their_weights(B, seed):
    rng = np.random.default_rng(500 + seed)
    Hq, H, D, bs, dtype = layout(rng, 128)
    lens = lengths(rng, 6000 if Hq <= 8 else 1500)
    most = int(rng.choice([1, 3, 20, 200 if Hq <= 16 else 20]))
    news = np.minimum(lens, rng.integers(0, most + 1, len(lens)))
    b = E.chunk_batch(600 + seed, lens, news, Hq, H, D, bs, dtype, wide=int(rng.integers(0, 3)))
    out, lse, rec = E.run_chunk(B, b, out_dtype=dtype if rng.random() < 0.5 else torch.float32)
    assert rec == [0, 0, 0, 0]
    E.check_chunk(b, out, lse)
    window = int(rng.choice([0, 1, 2, 7, 32]))
    lse = E.given_lse(b)
    before, got, rec = E.run_weights(B, b, lse, window)
    assert rec == [0, 0, 0, 0]
    E.check_chunk_weights(b, lse, before, got, window)


@pytest.mark.parametrize("seed", range(40))
def test_decode(B, seed):
    rng = np.random.default_rng(700 + seed)
    Hq, H, D, bs, dtype = layout(rng, 300)
    b = S.make(800 + seed, lengths(rng, 20000 if Hq <= 32 else 4000), Hq, H, D, bs, dtype, wide=int(rng.integers(0, 3)))
    before, got, out, rec = E.run_decode(B, b, out_dtype=dtype if rng.random() < 0.5 else torch.float32)
    assert rec == [0, 0, 0, 0]
    E.check_decode(b, before, got, out)


@pytest.mark.parametrize("seed", range(40))
def test_evictions(B, seed):
    rng = np.random.default_rng(900 + seed)
    H, D, bs = int(rng.choice([1, 2, 5, 40])), int(rng.choice([8, 64, 96, 128, 256])), int(rng.choice([1, 8, 16, 48]))
    lens = lengths(rng, 2000)
    K = int(rng.choice([1, 5, 64, 129, 1000, 3000]))
    b = S.make(1000 + seed, lens, H, H, D, bs, torch.float16, wide=int(rng.integers(0, 3)))
    kept = E.pick(rng, lens, H, K)
    new = None
    if rng.random() < 0.5:             # into blocks of their own, but for some places that stay
        own = -(-min(K, int(lens.max())) // bs) + 1
        total = len(b["kc"])
        fresh = rng.permutation(len(lens) * own).reshape(len(lens), own).astype(np.int32) + total
        for k in ("kc", "vc"):
            b[k] = torch.cat([b[k], torch.zeros((len(lens) * own, *b[k].shape[1:]), dtype=b[k].dtype, device="cuda")])
        stay = rng.random(fresh.shape) < 0.3
        width = min(own, b["tables"].shape[1])
        stay[:, width:] = False
        new = fresh.copy()
        held = b["tables"][:, :width]
        new[:, :width] = np.where(stay[:, :width] & (held >= 0), held, fresh[:, :width])
    E.check_evict(B, b, kept, new_tables=new, weights=bool(rng.random() < 0.8))
