"""Both numbers of a probability, and fp16's smallest: many small weights beside a large one, outputs to the
bound that the kernels' larger probabilities give.

An fp16 number is off by half a step of 2^-24 at the smallest, 2^-25.  The chunk's probabilities are kept 2^7
larger against a running reference that never exceeds the row's largest logit, the decode's 2^12 larger against
that largest logit: a weight is off by 2^-32 or 2^-37 of the largest besides its relative error (two numbers
2^-22 at most, one 2^-11).  The other terms are those of test_gpu_evict.
"""

import numpy as np
import pytest
import torch

import test_gpu_evict as E
import test_gpu_sparse as S
from gpu_util import half_ulp

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
BF, FH = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def bound(b, q, table, length, places, small, half, out_dtype):
    """What rows q of a sequence are to give, and by how much they may be off."""
    w, _, reach = E.OE.softmax_rows(q, E.f64(b["kc"]), table, length, places, b["scale"])
    want, spread, size = E.OE.weighted(w, E.f64(b["vc"]), table, length)
    n = (np.asarray(places) + 1)[:, None]
    tol = (4 * ((b["D"] + 8) * U * reach + (n + 16) * U) + half)[..., None] * spread + small * size
    if out_dtype is not torch.float32:
        tol = tol + half_ulp(np.abs(want) + tol, out_dtype)
    return want, tol


@pytest.mark.parametrize("out_dtype", [torch.float32, FH])
@pytest.mark.parametrize("lens,news,Hq,H,D", [([2000], [5], 8, 2, 128), ([500, 400], [60, 400], 4, 4, 64),
                                              ([1500], [9], 3, 1, 256), ([9000], [2], 4, 1, 64)])
def test_chunk_to_the_bound_of_its_lift(B, lens, news, Hq, H, D, out_dtype):
    b = E.chunk_batch(41, lens, news, Hq, H, D, 16, FH)
    out, _, rec = E.run_chunk(B, b, out_dtype=out_dtype)
    assert rec == [0, 0, 0, 0]
    half = 2.0 ** -21 if out_dtype is torch.float32 else 2.0 ** -11
    for i, length in enumerate(lens):
        a, e = int(b["start"][i]), int(b["start"][i + 1])
        want, tol = bound(b, E.f64(b["q"])[a:e], b["tables"][i], length, length - (e - a) + np.arange(e - a),
                          2.0 ** -32, half, out_dtype)
        E.close(out[a:e], want, tol, f"sequence {i}")


@pytest.mark.parametrize("out_dtype", [torch.float32, FH])
@pytest.mark.parametrize("lens,Hq,H,D", [([2000], 8, 2, 128), ([1000] * 3, 4, 4, 64), ([900, 20], 20, 1, 256),
                                         ([9000], 4, 1, 64)])
def test_decode_to_the_bound_of_its_lift(B, lens, Hq, H, D, out_dtype):
    b = S.make(43, lens, Hq, H, D, 16, FH)
    _, _, out, rec = E.run_decode(B, b, out_dtype=out_dtype)
    assert rec == [0, 0, 0, 0]
    for i, length in enumerate(lens):
        want, tol = bound(b, E.f64(b["q"])[i:i + 1], b["tables"][i], length, [length - 1], 2.0 ** -37, 2.0 ** -21,
                          out_dtype)
        E.close(out[i:i + 1], want, tol, f"sequence {i}")


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("n,N,inside", [(1000, 2, True), (6000, 1, False)])
def test_decode_of_many_small_weights_next_to_a_large_one(B, dtype, n, N, inside):
    """A first key that has nearly all of the weight, and the others 2^-25 of it each, whose values are all
    there is to see; with the logits inside a thread block, and with rows in parts."""
    D = 64
    b = S.make(47, [n] * N, 4, 1, D, 16, dtype)
    assert (B.paged_attn_decode_weights_workspace_needed(N, 4, 1, D, 16, b["tables"].shape[1]) == 0) == inside
    b["q"][:] = 1.0
    b["kc"][:], b["vc"][:] = 0.0, 1.0
    for first in b["tables"][:, 0]:
        b["kc"][int(first), 0, 0, 0], b["vc"][int(first), 0, 0] = 140.0, 0.0     # a logit of 17.5
    small = (n - 1) * np.exp(-17.5)
    want = small / (1 + small)
    d = (D + 8) * U * 17.5 + (n + 16) * U
    for out_dtype in (torch.float32, dtype):
        before, w, out, rec = E.run_decode(B, b, out_dtype=out_dtype)
        assert rec == [0, 0, 0, 0]
        tol = (4 * d + 2.0 ** -16) * want + 2.0 ** -37 * n
        if out_dtype is not torch.float32:
            tol += float(half_ulp(np.array(want + tol), dtype))
        assert float((out.double() - want).abs().max()) <= tol
        each = np.exp(-17.5) / (1 + small)
        got = (w.double() - before.double())[:, 0, 1:n]
        assert float((got - 4 * each).abs().max()) <= (2 * d + 8 * U) * 4 * each + U * 2


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_both_halves_of_a_probability_count(B, dtype, D):
    """Few tokens of nearly equal weight: small logits and short sums leave a bound below what one half-precision
    number of each probability would be off by (2^-9 or 2^-12 of each, of about 20)."""
    lens = [9, 17, 24, 23]
    half, small = (2.0 ** -16, 0) if dtype is BF else (2.0 ** -21, 2.0 ** -32)
    b = E.chunk_batch(51, lens, [1, 3, 2, 7], 8, 2, D, 16, dtype)
    b["scale"] = float(np.float32(D ** -0.5 / 64))
    out, _, rec = E.run_chunk(B, b)
    assert rec == [0, 0, 0, 0]
    for i, length in enumerate(lens):
        a, e = int(b["start"][i]), int(b["start"][i + 1])
        want, tol = bound(b, E.f64(b["q"])[a:e], b["tables"][i], length, length - (e - a) + np.arange(e - a), small, half,
                          torch.float32)
        E.close(out[a:e], want, tol, f"chunk of sequence {i}")
    b["q"] = b["q"][:4].contiguous()
    _, _, out, rec = E.run_decode(B, b)
    assert rec == [0, 0, 0, 0]
    for i, length in enumerate(lens):
        want, tol = bound(b, E.f64(b["q"])[i:i + 1], b["tables"][i], length, [length - 1], small * 2.0 ** -5, half,
                          torch.float32)
        E.close(out[i:i + 1], want, tol, f"decode of sequence {i}")
