"""Corners of the grouped chunk attention and the attention weights."""

import numpy as np
import pytest
import torch

import test_gpu_evict as E
from gpu_util import assert_matches_oracle

pytestmark = pytest.mark.gpu

BAD_SEQ_LEN = 6
INF = float("inf")
BF, FH = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


@pytest.mark.parametrize("lens,news", [([150, 40], [100, 3]), ([9000, 700], [3, 2])])   # one part, several
@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("D", [64, 256])
def test_rows_of_minus_infinity_alone(B, lens, news, dtype, D):
    """softmax over logits that are all -infinity is 0 / 0: the outputs are NaN, the logarithm of the sum
    -infinity, the weights NaN.  Rows with one number among them are as ever."""
    b = E.chunk_batch(31, lens, news, 4, 2, D, 16, dtype)
    b["q"].abs_()
    where = [(int(b["tables"][0, t // 16]), t % 16) for t in range(lens[0])]
    at, row = (torch.tensor(x, device="cuda") for x in zip(*where))
    b["kc"][at, 1, row] = -INF                          # sequence 0, key head 1: query heads 2 and 3
    first = lens[0] - news[0]
    for out_dtype in (torch.float32, dtype):
        out, lse, rec = E.run_chunk(B, b, out_dtype=out_dtype)
        assert rec == [0, 0, 0, 0]
        n = news[0]
        assert bool(torch.isnan(out[:n, 2:]).all()) and bool((lse[:n, 2:] == -INF).all())
        assert bool(torch.isfinite(out[:n, :2]).all()) and bool(torch.isfinite(lse[:n, :2]).all())
        assert bool(torch.isfinite(out[n:]).all()) and bool(torch.isfinite(lse[n:]).all())
        w = torch.zeros((2, 2, b["tables"].shape[1] * 16), device="cuda")
        B.paged_chunk_weights(b["q"], lse, E.dev(b["start"]), b["most"], b["kc"], E.dev(b["tables"]), E.dev(b["lens"]),
                              b["scale"], w)
        assert bool(torch.isnan(w[0, 1, :lens[0]]).all()) and bool(torch.isfinite(w[0, 0]).all())
        assert bool(torch.isfinite(w[1]).all()) and not bool(w[0, 1, lens[0]:].any())
    # decode of the last rows: the same
    last = torch.stack([b["q"][news[0] - 1], b["q"][sum(news) - 1]])
    w = torch.zeros((2, 2, b["tables"].shape[1] * 16), device="cuda")
    out = B.paged_attn_decode_weights(last, b["kc"], b["vc"], E.dev(b["tables"]), E.dev(b["lens"]), b["scale"], w)
    assert bool(torch.isnan(out[0, 2:]).all()) and bool(torch.isfinite(out[0, :2]).all())
    # One number, at the last token before the chunk: the row is that token's.  Its probability p is near 1, as
    # the reference is its logit rounded; the two halves of p are within 2^-16 (bf16) or 2^-21 (fp16) of it, the sum
    # is p, their products, sum, quotient and product add 8 u.
    t = first - 1
    b["kc"][at[t], 1, row[t]] = 0.5
    out, lse, _ = E.run_chunk(B, b)
    v = b["vc"][at[t], 1, row[t]].float()
    tol = (2.0 ** (-16 if dtype is BF else -21) + 8 * E.U) * v.abs()
    assert bool(((out[:news[0], 2:] - v).abs() <= tol).all())
    assert bool(torch.isfinite(lse[:news[0], 2:]).all())
    # infinity among them: NaN, as inf - inf is
    b["kc"][at[t], 1, row[t]] = INF
    out, lse, _ = E.run_chunk(B, b)
    assert bool(torch.isnan(out[:news[0], 2:]).all()) and bool(torch.isfinite(out[:news[0], :2]).all())


@pytest.mark.parametrize("lens,news,most", [([50, 60, 40, 70], [5, 8, 3, 7], 7), ([9000, 40], [3, 2], 2)])
def test_more_queries_than_the_call_allows(B, lens, news, most):
    """One query over max_query_len, though a tile would hold it: left out by both calls."""
    b = E.chunk_batch(7, lens, news, 6, 2, 64, 16, FH)
    b["most"] = most
    skip = int(np.argmax(news))
    out, lse, rec = E.run_chunk(B, b)
    assert rec == [BAD_SEQ_LEN, 1, skip, lens[skip]]
    E.check_chunk(b, out, lse, skip=(skip,))
    lse = E.given_lse(b)
    before, got, rec = E.run_weights(B, b, lse, 0)
    assert rec == [BAD_SEQ_LEN, 1, skip, lens[skip]]
    E.check_chunk_weights(b, lse, before, got, 0, skip=(skip,))


def test_any_bound_on_queries_for_a_batch(B):
    """max_query_len is a bound: 64 sequences, 8 key heads and 2^31 - 1 are no more work than 70."""
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 300, 64)
    news = np.minimum(lens, rng.integers(0, 70, 64))
    b = E.chunk_batch(33, lens, news, 24, 8, 64, 16, BF)
    want, wlse, rec = E.run_chunk(B, b)
    out, lse, wide = E.run_chunk(B, {**b, "most": 2 ** 31 - 1})
    assert rec == wide == [0, 0, 0, 0]
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    E.check_chunk(b, out, lse)


@pytest.mark.parametrize("N,lens,wide,shared", [(50, 700, 100, True), (80, 700, 100, False), (80, 700, 600, True),
                                                (120, 700, 100, False), (152, 1300, 600, False), (77, 2600, 300, True)])
def test_parts_of_wide_heads(B, N, lens, wide, shared):
    """256 channels, one thread block an SM: 50 items are shared out, 80 and more where tables are long, 152 and
    one a place are not."""
    rng = np.random.default_rng(N)
    lens = rng.integers(500, lens, N)
    b = E.chunk_batch(35, lens, [2] * N, 4, 1, 256, 16, BF, wide=wide)
    need = B.paged_attn_chunk_workspace_needed(N, 4, 1, 256, 16, b["tables"].shape[1], 2)
    assert (need > 0) == shared
    for out_dtype in (torch.float32, BF):
        out, lse, rec = E.run_chunk(B, b, out_dtype=out_dtype)
        assert rec == [0, 0, 0, 0]
        E.check_chunk(b, out, lse)


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("lens,news,Hq,H,D", [([300, 200], [300, 200], 8, 8, 128), ([300, 200], [300, 200], 8, 2, 128),
                                              ([2000], [64], 8, 2, 128), ([400], [400], 4, 4, 64),
                                              ([300], [300], 4, 1, 256), ([9000, 5000], [3, 4], 4, 1, 128)])
def test_half_precision_outputs_keep_the_librarys_bound(B, lens, news, Hq, H, D, dtype):
    """2e-3 and half a step of the output's type at the oracle's value, as everywhere; and with a head of its own
    each, a bf16 cache and keys that are not shared out, the bits of the dense prefill."""
    b = E.chunk_batch(3, lens, news, Hq, H, D, 16, dtype)
    q, kc = E.f64(b["q"]), E.f64(b["kc"])
    out, _, rec = E.run_chunk(B, b, out_dtype=dtype)
    assert rec == [0, 0, 0, 0]
    for i, length in enumerate(lens):
        a, e = int(b["start"][i]), int(b["start"][i + 1])
        places = length - (e - a) + np.arange(e - a)
        w, _, _ = E.OE.softmax_rows(q[a:e], kc, b["tables"][i], length, places, b["scale"])
        want, _, _ = E.OE.weighted(w, E.f64(b["vc"]), b["tables"][i], length)
        assert_matches_oracle(out[a:e], want, f"sequence {i}")
    if Hq == H and dtype is BF:
        dense = torch.full_like(out, 7)
        B.paged_attn_prefill(b["q"], E.dev(b["start"]), b["most"], b["kc"], b["vc"], E.dev(b["tables"]),
                             E.dev(b["lens"]), b["scale"], out=dense)
        assert torch.equal(out, dense)
