"""The dense calls know one number of heads: caches with fewer key heads than query heads, which
kv_cache_append_rope and the block-sparse calls take, are refused before anything is enqueued."""

import pytest
import torch


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def calls(B, q, k, v, kc, vc):
    tables, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    start = torch.arange(3, dtype=torch.int32)
    return {"decode": lambda: B.paged_attn_decode(q, kc, vc, tables, lens, 0.1),
            "decode_append": lambda: B.paged_attn_decode_append(q, k, v, kc, vc, tables, lens, 0.1),
            "prefill": lambda: B.paged_attn_prefill(q, start, 1, kc, vc, tables, lens, 0.1),
            "noalloc": lambda: B.paged_attn_decode_noalloc(q, kc, vc, tables, lens, 0.1, torch.zeros(q.shape)),
            "append": lambda: B.kv_cache_append(k, v, torch.zeros(2, dtype=torch.int64), kc, vc)}


def half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


@pytest.mark.parametrize("name", ["decode", "decode_append", "prefill", "noalloc", "append"])
@pytest.mark.parametrize("cache,other", [((9, 2, 16, 64), (9, 2, 16, 64)),     # grouped
                                         ((9, 8, 16, 32), (9, 8, 16, 32)),     # fewer channels
                                         ((9, 8, 16, 64), (9, 2, 16, 64)),     # the values alone
                                         ((9, 8, 16, 64), (5, 8, 16, 64)),     # fewer blocks of values
                                         ((9, 8, 16, 64), (9, 8, 8, 64))])     # shorter ones
def test_caches_of_other_heads_are_refused(B, name, cache, other):
    q = half(2, 8, 64)
    with pytest.raises(ValueError, match="the caches must be"):
        calls(B, q, q, q, half(*cache), half(*other))[name]()


@pytest.mark.parametrize("name", ["decode_append", "append"])
def test_new_rows_of_other_heads_are_refused(B, name):
    q, few, cache = half(2, 8, 64), half(2, 2, 64), half(9, 8, 16, 64)
    for k, v in ((q, few), (few, q), (q, half(1, 8, 64))):
        with pytest.raises(ValueError, match="rows of new keys" if k is q or name == "decode_append"
                           else "the caches must be"):
            calls(B, q, k, v, cache, cache)[name]()


@pytest.mark.parametrize("name", ["decode", "decode_append", "prefill", "noalloc", "append"])
def test_caches_of_these_heads_are_not(B, name):
    q, cache = half(2, 8, 64), half(9, 8, 16, 64)
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):     # the next check: all on the host
        calls(B, q, q, q, cache, cache.clone())[name]()


def test_block_copy_refuses_caches_that_are_not_alike(B):
    """One call copies blocks of one size: key bounds beside their caches would be addressed as caches."""
    kc, lo, pairs = half(9, 2, 16, 64), half(9, 2, 64), torch.zeros(1, 2, dtype=torch.int64)
    bound = lo[:, :, None]
    for k, v in (([kc, bound], [kc, bound]), ([kc], [bound]), ([kc], [kc.float()]),
                 ([kc, kc], [kc, half(5, 2, 16, 64)])):
        with pytest.raises(ValueError, match="must be alike"):
            B.block_copy(k, v, pairs)
    with pytest.raises(ValueError, match="2 key caches and 1 value"):
        B.block_copy([kc, kc], [kc], pairs)
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        B.block_copy([kc], [kc.to(torch.bfloat16)], pairs)     # the bytes are copied as they are
