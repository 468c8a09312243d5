"""paged_attn_chunk, paged_chunk_weights, paged_attn_decode_weights and kv_cache_evict on the GPU against
the fp64 oracle, each by itself and as they are used together.

Tolerances (derived, u = 2^-23: a sum on the tensor cores may drop a unit in the last place at each
addition).  A logit is off by at most d = (D + 8) u * max_t scale sum_d |q_d k_td|: D products, their sum,
the scaling to base 2 and the subtraction of a maximum.  Over n tokens:
* lse: d, the sum's (n + 16) u, the logarithm's and its product's 2 u |lse|.
* a softmax weight: numerator and denominator within e^(+-d), the exponentials' and the sum's (n + 16) u:
  2 (d + (n + 16) u) of it in all; its sum over rows and heads and with what was there adds u of that for
  each.
* a weight from a given lse: d, 2 u |lse| for lse in base 2, 4 u for the exponential, the sum's.
* outputs: twice the weights' bound and 2^-16 (bf16) or 2^-21 (fp16), the two half-precision numbers of a
  probability, of sum_t w_t |v_t|; fp16 numbers have steps of 2^-24 at least, so that each token may be off
  by 2^-25 of a largest weight of at least 1; a half-precision output is rounded by half a step on top.
  Chunks with half-precision outputs have probabilities in one number: 2^-8 (bf16) or 2^-11 (fp16), the half
  step of its rounding, in place of 2^-16 and 2^-21.
"""

import numpy as np
import pytest
import torch

import test_gpu_sparse as S
from gpu_util import bits, half_ulp
from oracle import evict as OE
from oracle import sparse as OS

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
NAN = float("nan")
BAD_BLOCK, BAD_SEQ_LEN, BAD_POSITION = 4, 6, 12
f64, dev = S.f64, S.dev
BF, FH = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def place(b, weights=None, seed=1):
    """Weights that tokens have had, NaN at places without one."""
    N, MB = b["tables"].shape
    rng = np.random.default_rng(seed)
    w = rng.random((N, b["H"], MB * b["bs"] + 3)).astype(np.float32)
    past = np.arange(w.shape[2]) >= np.asarray(b["lens"])[:, None, None]
    w[np.broadcast_to(past, w.shape)] = NAN
    return torch.from_numpy(w).cuda()


def close(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= tol)
    bad &= ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3])


def out_bound(b, w, reach, n, table, length, dtype, out_dtype, one=False):
    want, spread, size = OE.weighted(w, f64(b["vc"]), table, length)
    d = (b["D"] + 8) * U * reach
    half = 2.0 ** -16 if dtype is BF else 2.0 ** -21
    if one and out_dtype is not torch.float32:
        half = 2.0 ** -8 if dtype is BF else 2.0 ** -11
    tol = (4 * (d + (n + 16) * U) + half)[..., None] * spread + (2.0 ** -25 * size if dtype is FH else 0)
    if out_dtype is not torch.float32:
        tol = tol + half_ulp(np.abs(want) + tol, out_dtype)
    return want, tol


# ------------------------------------------------------------------------ chunks
def chunk_batch(seed, lens, news, Hq, H, D, bs, dtype, wide=0):
    b = S.make(seed, lens, Hq, H, D, bs, dtype, wide)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1000)
    b["start"] = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    b["q"] = torch.randn((int(b["start"][-1]) + 2, Hq, D), generator=gen, device="cuda").to(dtype)
    b["most"] = max(1, int(np.max(news)))
    return b


def run_chunk(B, b, out_dtype=torch.float32, **kw):
    out = torch.full((*b["q"].shape,), 7, dtype=out_dtype, device="cuda")
    lse = torch.full(b["q"].shape[:2], 7.0, device="cuda")
    rec = B.new_error_record()
    got = B.paged_attn_chunk(b["q"], dev(b["start"]), b["most"], b["kc"], b["vc"], dev(b["tables"]),
                             dev(b["lens"]), b["scale"], out=out, lse=lse, error_record=rec, **kw)
    assert got is out
    return out, lse, B.pa_error_read(rec)


def check_chunk(b, out, lse, skip=()):
    q, kc = f64(b["q"]), f64(b["kc"])
    for i, length in enumerate(b["lens"]):
        a, e = int(b["start"][i]), int(b["start"][i + 1])
        if i in skip:
            assert bool((out[a:e] == 7).all() and (lse[a:e] == 7).all())
            continue
        if a == e:
            continue
        places = int(length) - (e - a) + np.arange(e - a)
        w, want_lse, reach = OE.softmax_rows(q[a:e], kc, b["tables"][i], int(length), places, b["scale"])
        n = (places + 1)[:, None]
        want, tol = out_bound(b, w, reach, n, b["tables"][i], int(length), b["q"].dtype, out.dtype,
                              one=True)
        close(out[a:e], want, tol, f"out of sequence {i}")
        close(lse[a:e], want_lse, (b["D"] + 8) * U * reach + (n + 16) * U + 2 * U * np.abs(want_lse),
              f"lse of sequence {i}")
    end = int(b["start"][-1])
    assert bool((out[end:] == 7).all()) and bool((lse[end:] == 7).all())   # rows behind the last sequence


SHAPES = [(8, 8, 64, 8, FH), (8, 2, 128, 16, BF), (7, 1, 256, 32, FH), (33, 1, 64, 16, BF),
          (128, 1, 64, 16, FH), (15, 3, 128, 64, FH), (10, 2, 256, 8, BF), (40, 8, 128, 16, BF)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lens,news", [([1, 2, 9, 200], [1, 2, 5, 3]), ([70, 0, 333, 64], [70, 0, 31, 1]),
                                       ([150], [150])])
def test_chunk_matches_the_oracle(B, shape, lens, news):
    Hq, H, D, bs, dtype = shape
    b = chunk_batch(3, lens, news, Hq, H, D, bs, dtype, wide=2)
    out, lse, rec = run_chunk(B, b)
    assert rec == [0, 0, 0, 0]
    check_chunk(b, out, lse)
    out, lse, _ = run_chunk(B, b, out_dtype=dtype)
    check_chunk(b, out, lse)


@pytest.mark.parametrize("lens", [[300, 40, 777], [300, 40, 512]])
def test_chunk_with_a_head_of_its_own_each_agrees_with_the_prefill(B, lens):
    """Where tables hold at most 512 tokens, so that no item's keys are shared out, bit for bit."""
    b = chunk_batch(5, lens, [129, 7, 500], 4, 4, 128, 16, BF)
    out, lse, _ = run_chunk(B, b)
    want = torch.full_like(out, 7)
    B.paged_attn_prefill(b["q"], dev(b["start"]), b["most"], b["kc"], b["vc"], dev(b["tables"]), dev(b["lens"]),
                         b["scale"], out=want)
    check_chunk(b, out, lse)
    check_chunk(b, want, lse)
    if max(lens) <= 512:
        assert torch.equal(out, want)
    # in another dispatch order, and without lse, the same bits
    again, _, _ = run_chunk(B, b, seq_order=dev([2, 0, 1]))
    assert torch.equal(out, again)
    bare = B.paged_attn_chunk(b["q"], dev(b["start"]), b["most"], b["kc"], b["vc"], dev(b["tables"]),
                              dev(b["lens"]), b["scale"])
    assert torch.equal(bare[:int(b["start"][-1])], out[:int(b["start"][-1])])


def test_few_rows_over_a_long_context(B):
    """Drafted tokens of one and of three sequences over contexts that are shared out over thread blocks."""
    for lens, news in (([20011], [3]), ([9000, 17, 12345], [1, 5, 2]), ([30000], [40])):
        b = chunk_batch(11, lens, news, 8, 1, 64, 16, BF)
        out, lse, rec = run_chunk(B, b)
        assert rec == [0, 0, 0, 0]
        check_chunk(b, out, lse)
        out, lse, _ = run_chunk(B, b, out_dtype=BF)
        check_chunk(b, out, lse)
        need = B.paged_attn_chunk_workspace_needed(len(lens), 8, 1, 64, 16, b["tables"].shape[1], b["most"])
        assert need == B.paged_attn_chunk_workspace_size(len(lens), 8, 1, 64, 16, b["tables"].shape[1], b["most"]) > 0
        given = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        again, _, _ = run_chunk(B, b, out_dtype=BF, workspace=given)
        assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", [BF, FH])
def test_many_small_weights_next_to_a_large_one(B, dtype):
    """A first key that has nearly all of the weight, and thousands of 2^-25 of it each, whose values are
    all there is to see: none of them may be lost.  The bound is that of the outputs above, with 2^-32 of
    the largest weight for each token, as fp16 numbers are kept 2^7 larger."""
    n, D = 6000, 64
    b = chunk_batch(14, [n], [3], 4, 1, D, 16, dtype)
    b["q"][:] = 1.0
    b["kc"][:], b["vc"][:] = 0.0, 1.0
    first = int(b["tables"][0, 0])
    b["kc"][first, 0, 0, 0], b["vc"][first, 0, 0] = 140.0, 0.0   # a logit of 17.5
    for out_dtype in (torch.float32, dtype):
        out, lse, rec = run_chunk(B, b, out_dtype=out_dtype)
        assert rec == [0, 0, 0, 0]
        for j in range(3):
            small = (n - 3 + j) * np.exp(-17.5)
            want = small / (1 + small)
            one = out_dtype is not torch.float32
            half = (2.0 ** -8 if dtype is BF else 2.0 ** -11) if one else 2.0 ** -16
            tol = (4 * ((D + 8) * U * 17.5 + (n + 16) * U) + half) * want + 2.0 ** -32 * n
            if one:
                tol += float(half_ulp(np.array(want + tol), dtype))
            assert float((out[j].double() - want).abs().max()) <= tol
            assert float((lse[j].double() - (17.5 + np.log1p(small))).abs().max()) <= (
                (D + 8) * U * 17.5 + (n + 16) * U + 2 * U * 17.5)


@pytest.mark.parametrize("shape", SHAPES)
def test_chunks_shared_out_over_parts(B, shape):
    """Lengths around the ends of parts, one sequence without queries, with an order."""
    Hq, H, D, bs, dtype = shape
    lens, news = [2049, 511, 512, 513, 1000, 3000], [2, 3, 5, 1, 0, 4]
    b = chunk_batch(12, lens, news, Hq, H, D, bs, dtype)
    for kw in ({}, dict(seq_order=dev([5, 4, 3, 2, 1, 0]))):
        out, lse, rec = run_chunk(B, b, **kw)
        assert rec == [0, 0, 0, 0]
        check_chunk(b, out, lse)


@pytest.mark.parametrize("dtype", [BF, FH])
def test_a_nan_far_from_the_large_weights_is_seen(B, dtype):
    """Over parts, a NaN counts in every row that sees it, though its part's weight is 0 in fp32."""
    b = chunk_batch(15, [5000], [4], 4, 2, 64, 16, dtype)
    b["q"][:] = 1.0
    b["kc"][:] = 0.0
    b["kc"][int(b["tables"][0, 0]), :, 0] = 40.0      # a logit of 320, the others' 0
    at = int(b["tables"][0, 4000 // 16]), 0, 4000 % 16
    for which, channel in (("kc", slice(None)), ("vc", 9), ("q", slice(None))):
        c = {k: b[k].clone() for k in ("q", "kc", "vc")}
        if which == "q":
            c["q"][1, 2] = NAN
        else:
            c[which][(*at, channel)] = NAN
        out, lse, rec = run_chunk(B, {**b, **c})
        assert rec == [0, 0, 0, 0]
        want = torch.zeros(b["q"].shape, dtype=torch.bool)
        if which == "q":
            want[1, 2] = True
        else:
            want[:4, :2, channel] = True
        assert torch.equal(torch.isnan(out).cpu(), want), which
        assert torch.equal(torch.isnan(lse).cpu(), want.all(2)), which
        if which != "q":
            w = torch.zeros(1, 2, b["tables"].shape[1] * 16, device="cuda")
            out = B.paged_attn_decode_weights(b["q"][:1], c["kc"], c["vc"], dev(b["tables"]), dev(b["lens"]),
                                              b["scale"], w)
            assert torch.equal(torch.isnan(out).cpu(), want[:1]), which
            assert bool(torch.isnan(w[0, 0, :5000]).all()) == (which == "kc") and not bool(torch.isnan(w[0, 1]).any())


def test_more_queries_allowed_than_there_can_be(B):
    """max_query_len is a bound, however large."""
    b = chunk_batch(16, [3000, 70], [3, 70], 6, 2, 64, 16, BF)
    out, lse, rec = run_chunk(B, b)
    wide = {**b, "most": 2 ** 31 - 1}
    again, wlse, wrec = run_chunk(B, wide)
    assert rec == wrec == [0, 0, 0, 0]
    check_chunk(wide, again, wlse)
    w = [torch.zeros(2, 2, b["tables"].shape[1] * 16, device="cuda") for _ in range(2)]
    for most, to in ((b["most"], w[0]), (2 ** 31 - 1, w[1])):
        B.paged_chunk_weights(b["q"], lse, dev(b["start"]), most, b["kc"], dev(b["tables"]), dev(b["lens"]), b["scale"],
                              to, window=4)
    assert torch.equal(w[0], w[1])


@pytest.mark.parametrize("n,Hq,H,D,most", [(60, 16, 8, 64, 200), (6, 16, 8, 256, 3000), (300, 4, 2, 64, 90)])
def test_the_order_of_sequences_changes_nothing(B, n, Hq, H, D, most):
    """More items than thread blocks, as they are dealt out by themselves and in given orders."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, most + 1, n)
    lens[1] = most
    news = np.minimum(lens, rng.integers(0, 5, n))
    b = chunk_batch(21, lens, news, Hq, H, D, 16, BF)
    b["lens"] = b["lens"].copy()
    skip = int(np.flatnonzero(news > 1)[0])
    b["lens"][skip] = news[skip] - 1
    want, wlse, rec = run_chunk(B, b)
    assert rec == [BAD_SEQ_LEN, 1, skip, news[skip] - 1]
    check_chunk(b, want, wlse, skip=(skip,))
    for order in (np.arange(n), rng.permutation(n)):
        out, lse, _ = run_chunk(B, b, seq_order=dev(order.astype(np.int32)))
        assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("lens,news,Hq,H,cap", [
    ([7003], [640], 32, 2, 7200),                                   # 160 items: a part and half a part each
    ([5000, 17, 4096, 4097, 3, 2900, 1] + [600] * 25, [3] * 32, 8, 2, 5000),   # 64: four and half a part
    ([9000] + [40] * 39, [3] * 40, 16, 4, 9000),                    # 160, of which only four have a second part
])
@pytest.mark.parametrize("out_dtype", [torch.float32, FH])
def test_parts_of_two_sizes(B, lens, news, Hq, H, cap, out_dtype):
    news = [min(n, length) for n, length in zip(news, lens)]
    b = chunk_batch(22, lens, news, Hq, H, 64, 16, FH, wide=max(0, cap // 16 - (max(lens) + 15) // 16))
    out, lse, rec = run_chunk(B, b, out_dtype=out_dtype)
    assert rec == [0, 0, 0, 0]
    check_chunk(b, out, lse)
    again, wlse, _ = run_chunk(B, b, out_dtype=out_dtype)
    assert torch.equal(again, out) and torch.equal(wlse, lse)


def test_chunk_leaves_out_inconsistent_sequences(B):
    b = chunk_batch(7, [50, 30, 60, 40], [5, 4, 8, 3], 6, 2, 64, 16, FH)
    b["lens"] = b["lens"].copy()
    b["lens"][1] = 3                                   # fewer tokens than queries
    out, lse, rec = run_chunk(B, b)
    assert rec == [BAD_SEQ_LEN, 1, 1, 3]
    check_chunk(b, out, lse, skip=(1,))
    b = chunk_batch(7, [50, 30, 60, 40], [5, 4, 64, 3], 6, 2, 64, 16, FH, wide=1)
    b["most"] = 7                                      # more queries than promised
    b["lens"] = np.array([50, 30, 64, 40], np.int32)
    out, lse, rec = run_chunk(B, b)
    assert rec == [BAD_SEQ_LEN, 1, 2, 64]
    check_chunk(b, out, lse, skip=(2,))


def test_chunk_records_a_bad_block(B):
    b = chunk_batch(8, [50, 200], [5, 40], 6, 2, 64, 16, FH)
    want, wlse, _ = run_chunk(B, b)
    b["tables"][1, 4] = 10 ** 6
    out, lse, rec = run_chunk(B, b)
    assert rec[0] == BAD_BLOCK and rec[2:] == [1, 10 ** 6] and rec[1] >= 1
    assert torch.equal(out[:5], want[:5]) and torch.equal(lse[:5], wlse[:5])


# --------------------------------------------------------------- weights of a chunk
def check_chunk_weights(b, lse, before, got, window, skip=()):
    q, kc = f64(b["q"]), f64(b["kc"])
    want, tol = f64(before).copy(), np.zeros(got.shape)
    for i, length in enumerate(b["lens"]):
        a, e = int(b["start"][i]), int(b["start"][i + 1])
        if window:
            a = max(a, e - window)
        if i in skip or a == e:
            continue
        n = int(length)
        places = n - (e - a) + np.arange(e - a)
        w, own, reach = OE.softmax_rows(q[a:e], kc, b["tables"][i], n, places, b["scale"])
        given = f64(lse)[a:e]
        w = w * np.exp(own - given)[..., None]
        rows = (e - a) * q.shape[1] // b["H"]
        bound = (b["D"] + 8) * U * reach + 2 * U * np.abs(given) + (rows + 20) * U
        want[i, :, :n] += OE.by_key_head(w, b["H"])
        tol[i, :, :n] = OE.by_key_head(w * bound[..., None], b["H"]) + U * np.abs(want[i, :, :n]) + 1e-37
    close(got, want, tol, "weights")


def given_lse(b):
    """lse of every row, in fp32 of the oracle's; rows outside every sequence NaN."""
    lse = np.full(b["q"].shape[:2], NAN, np.float32)
    q, kc = f64(b["q"]), f64(b["kc"])
    for i, length in enumerate(b["lens"]):
        a, e = int(b["start"][i]), int(b["start"][i + 1])
        places = int(length) - (e - a) + np.arange(e - a)
        lse[a:e] = OE.softmax_rows(q[a:e], kc, b["tables"][i], int(length), places, b["scale"])[1]
    return torch.from_numpy(lse).cuda()


def run_weights(B, b, lse, window, weights=None):
    before = place(b) if weights is None else weights
    w, rec = before.clone(), B.new_error_record()
    B.paged_chunk_weights(b["q"], lse, dev(b["start"]), b["most"], b["kc"], dev(b["tables"]), dev(b["lens"]),
                          b["scale"], w, window=window, error_record=rec)
    return before, w, B.pa_error_read(rec)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 6, 40])
@pytest.mark.parametrize("lens,news", [([1, 2, 9, 300], [1, 2, 5, 3]), ([70, 0, 533, 257], [70, 0, 41, 9])])
def test_chunk_weights_match_the_oracle(B, shape, window, lens, news):
    Hq, H, D, bs, dtype = shape
    b = chunk_batch(13, lens, news, Hq, H, D, bs, dtype, wide=1)
    b["q"][int(b["start"][-1]):] = NAN                  # rows behind the last sequence
    lse = given_lse(b)
    before, got, rec = run_weights(B, b, lse, window)
    assert rec == [0, 0, 0, 0]
    check_chunk_weights(b, lse, before, got, window)


@pytest.mark.parametrize("news,window,group", [([400, 700], 0, 3), ([400, 700], 0, 16), ([33, 500, 64], 64, 4)])
def test_weights_of_whole_prompts(B, news, window, group):
    """Many tiles of rows, causal triangles; and windows of one, two and three tiles side by side."""
    b = chunk_batch(17, [max(500, n) for n in news], news, 2 * group, 2, 64, 8, BF)
    lse = given_lse(b)
    before, got, rec = run_weights(B, b, lse, window)
    assert rec == [0, 0, 0, 0]
    check_chunk_weights(b, lse, before, got, window)


def test_weights_of_prompts_of_all_lengths(B):
    """Enough of them that some thread blocks have several, dealt out longest first; two without rows."""
    news = [37 * i % 331 for i in range(50)]
    news[7], news[31] = 0, 700
    b = chunk_batch(18, [max(n, 1) + (i % 3) * 64 for i, n in enumerate(news)], news, 40, 2, 64, 8, FH)
    lse = given_lse(b)
    before, got, rec = run_weights(B, b, lse, 0)
    assert rec == [0, 0, 0, 0]
    check_chunk_weights(b, lse, before, got, 0)


def test_weights_of_many_sequences(B):
    """More sequences than are counted together at a time, some with nothing to do."""
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 60, 700)
    news = np.minimum(lens, rng.integers(0, 4, 700))
    lens[5], news[5] = 1500, 2
    b = chunk_batch(19, lens, news, 4, 2, 64, 16, FH)
    lse = given_lse(b)
    before, got, rec = run_weights(B, b, lse, 2)
    assert rec == [0, 0, 0, 0]
    check_chunk_weights(b, lse, before, got, 2)


def test_chunk_weights_leave_out_inconsistent_sequences(B):
    b = chunk_batch(7, [50, 30, 60, 40], [5, 4, 8, 3], 6, 2, 64, 16, FH)
    lse = given_lse(b)
    b["lens"] = b["lens"].copy()
    b["lens"][1] = 3
    b["most"] = 7
    before, got, rec = run_weights(B, b, lse, 0)
    assert rec[:2] == [BAD_SEQ_LEN, 2] and rec[2] in (1, 2)
    check_chunk_weights(b, lse, before, got, 0, skip=(1, 2))


def test_chunk_weights_record_a_bad_block(B):
    b = chunk_batch(8, [50, 400], [5, 40], 6, 2, 64, 16, FH)
    lse = given_lse(b)
    before, want, _ = run_weights(B, b, lse, 0)
    b["tables"][1, 20] = -5
    _, got, rec = run_weights(B, b, lse, 0)
    assert rec == [BAD_BLOCK, 1, 1, -5]
    same = np.ones(400, bool)
    same[320:336] = False
    assert torch.equal(got[0].nan_to_num(9), want[0].nan_to_num(9))
    assert np.array_equal(f64(got[1])[:, :400][:, same], f64(want[1])[:, :400][:, same])


def test_a_nan_key_makes_its_own_weight_nan(B):
    b = chunk_batch(9, [300], [4], 4, 2, 64, 16, BF)
    lse = given_lse(b)
    at = 123
    b["kc"][int(b["tables"][0, at // 16]), 1, at % 16, 5] = NAN
    _, got, _ = run_weights(B, b, lse, 0)
    bad = torch.isnan(got[0, :, :300])
    assert bad.nonzero().tolist() == [[1, at]]


# ------------------------------------------------------------------------- decode
def run_decode(B, b, **kw):
    before = place(b)
    w, rec = before.clone(), B.new_error_record()
    out = B.paged_attn_decode_weights(b["q"], b["kc"], b["vc"], dev(b["tables"]), dev(b["lens"]), b["scale"], w,
                                      error_record=rec, **kw)
    return before, w, out, B.pa_error_read(rec)


def check_decode(b, before, got, out, lens=None):
    q, kc = f64(b["q"]), f64(b["kc"])
    want, tol = f64(before).copy(), np.zeros(got.shape)
    for i, length in enumerate(b["lens"] if lens is None else lens):
        n = int(length)
        if n == 0:
            assert not bool(out[i].any())
            continue
        w, _, reach = OE.softmax_rows(q[i:i + 1], kc, b["tables"][i], n, [n - 1], b["scale"])
        d = 2 * ((b["D"] + 8) * U * reach + (n + 16) * U) + (q.shape[1] // b["H"] + 4) * U
        want[i, :, :n] += OE.by_key_head(w, b["H"])
        tol[i, :, :n] = OE.by_key_head(w * d[..., None], b["H"]) + U * np.abs(want[i, :, :n]) + 1e-37
        o, otol = out_bound(b, w, reach, n, b["tables"][i], n, b["q"].dtype, out.dtype)
        close(out[i:i + 1], o, otol, f"out of sequence {i}")
    close(got, want, tol, "weights")


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lens", [[1, 0, 17, 300], [9, 8, 7], [1023], [5000, 1, 64]])
def test_decode_matches_the_oracle(B, shape, lens):
    Hq, H, D, bs, dtype = shape
    b = S.make(23, lens, Hq, H, D, bs, dtype, wide=1)
    before, got, out, rec = run_decode(B, b)
    assert rec == [0, 0, 0, 0]
    check_decode(b, before, got, out)
    _, _, half, _ = run_decode(B, b, out_dtype=dtype)
    check_decode(b, before, got, half)


@pytest.mark.parametrize("N,H,G,most", [(60, 4, 1, 900), (200, 2, 3, 700), (3, 1, 4, 20000), (40, 8, 8, 1500)])
def test_decode_of_batches(B, N, H, G, most):
    """Launches of every kind: logits inside a thread block, rows shared out over several."""
    lens = np.random.default_rng(N).integers(0, most, N)
    b = S.make(29, lens, H * G, H, 64, 16, BF)
    before, got, out, rec = run_decode(B, b)
    assert rec == [0, 0, 0, 0]
    check_decode(b, before, got, out)


def test_decode_agrees_with_attention_over_all_blocks(B):
    b = S.make(31, [700, 33, 1200], 12, 4, 128, 16, BF)
    _, _, out, _ = run_decode(B, b)
    every = np.tile(np.arange(b["tables"].shape[1], dtype=np.int32), (3, 4, 1))
    other = S.attend(B, b, every)
    assert float((out - other).abs().max()) < 1e-4


def test_the_weights_of_a_row_sum_to_its_heads(B):
    b = S.make(37, [3000, 50], 20, 4, 64, 16, FH)
    zero = torch.zeros((2, 4, b["tables"].shape[1] * 16), device="cuda")
    B.paged_attn_decode_weights(b["q"], b["kc"], b["vc"], dev(b["tables"]), dev(b["lens"]), b["scale"], zero)
    assert float((zero.double().sum(-1) - 5).abs().max()) < 5 * 3100 * U
    assert not bool(zero[1, :, 50:].any())


def test_decode_records_bad_entries(B):
    b = S.make(41, [100, 90], 4, 2, 64, 16, BF, wide=1)
    _, want, out0, _ = run_decode(B, b)
    bad = dict(b, tables=b["tables"].copy())
    bad["tables"][0, 2] = 10 ** 7
    _, got, out, rec = run_decode(B, bad)
    assert rec == [BAD_BLOCK, 1, 0, 10 ** 7]
    assert torch.equal(out[1], out0[1]) and torch.equal(got[1].nan_to_num(9), want[1].nan_to_num(9))
    for length, clamped in ((-4, 0), (10 ** 6, b["tables"].shape[1] * 16)):
        c = dict(b, lens=np.array([100, length], np.int32), tables=b["tables"].copy())
        c["tables"][1] = c["tables"][0]
        c["kc"], c["vc"] = c["kc"].nan_to_num(0.5), c["vc"].nan_to_num(0.5)
        c["tables"][:, -1] = 0
        before = torch.zeros_like(want)
        w, rec = before.clone(), B.new_error_record()
        out = B.paged_attn_decode_weights(c["q"], c["kc"], c["vc"], dev(c["tables"]), dev(c["lens"]), c["scale"], w,
                                          error_record=rec)
        assert B.pa_error_read(rec) == [BAD_SEQ_LEN, 1, 1, length]
        check_decode(c, before, w, out, lens=[100, clamped])


def test_infinite_keys_and_values(B):
    """One key of +infinity: its row is NaN, as softmax has it, and no other row is."""
    b = S.make(43, [100, 90], 4, 2, 64, 16, BF)
    b["kc"][int(b["tables"][0, 1]), 0, 3] = float("inf")
    _, got, out, _ = run_decode(B, b)
    assert bool(torch.isnan(out[0, :2]).all()) and not bool(torch.isnan(out[0, 2:]).any())
    assert not bool(torch.isnan(out[1]).any())
    assert bool(torch.isnan(got[0, 0, :100]).all()) and not bool(torch.isnan(got[0, 1, :100]).any())


# ----------------------------------------------------------------------- eviction
def pick(rng, lens, H, K, step=1):
    """Ascending random places, then -1."""
    kept = np.full((len(lens), H, K), -1, np.int32)
    for i, n in enumerate(lens):
        for h in range(H):
            m = min(int(n), K)
            kept[i, h, :m] = np.sort(rng.permutation(int(n))[:m])
    return kept


def check_evict(B, b, kept, new_tables=None, total=None, weights=True, expect=(0, 0, 0, 0), skip=None):
    w = place(b) if weights else None
    k, v = bits(b["kc"]).copy(), bits(b["vc"]).copy()
    want_w = None if w is None else w.cpu().numpy().copy()
    allowed = kept.copy()
    if skip is not None:
        for i, h, j in skip:
            allowed[i, h, j] = -1
    OE.evict(k, v, b["tables"], b["lens"], allowed, want_w, new_tables)
    if skip is not None and w is not None:
        for i, h, j in skip:
            want_w[i, h, j] = w[i, h, j].item()
    rec = B.new_error_record()
    B.kv_cache_evict(b["kc"], b["vc"], dev(b["tables"]), dev(b["lens"]), dev(kept), weights=w,
                     new_tables=None if new_tables is None else dev(new_tables), error_record=rec)
    assert B.pa_error_read(rec) == list(expect)
    assert np.array_equal(bits(b["kc"]), k) and np.array_equal(bits(b["vc"]), v)
    if w is not None:
        assert np.array_equal(w.cpu().numpy().view(np.int32), want_w.view(np.int32))


@pytest.mark.parametrize("H,D,bs,dtype", [(1, 64, 8, FH), (3, 128, 16, BF), (2, 256, 64, BF), (2, 40, 5, FH),
                                          (1, 8, 1, BF), (1, 1024, 16, FH)])
@pytest.mark.parametrize("lens,K", [([1, 2, 50, 300], 7), ([700, 0, 40], 100), ([64, 64, 3], 64), ([900], 640)])
def test_evict_moves_what_the_oracle_moves(B, H, D, bs, dtype, lens, K):
    b = S.make(47, lens, H, H, D, bs, dtype, wide=1)
    check_evict(B, b, pick(np.random.default_rng(5), lens, H, K))
    b = S.make(47, lens, H, H, D, bs, dtype)
    check_evict(B, b, pick(np.random.default_rng(6), lens, H, K), weights=False)


@pytest.mark.parametrize("N,H,L,K", [(1, 1, 20000, 9000), (1, 8, 9000, 4096), (100, 4, 500, 300), (2, 2, 5000, 4999)])
def test_evict_of_long_lists(B, N, H, L, K):
    """Many rounds, alone and over clusters; a list that moves nearly every row by one place."""
    lens = np.full(N, L)
    b = S.make(53, lens, H, H, 64, 16, BF)
    check_evict(B, b, pick(np.random.default_rng(N), lens, H, K))


def test_lists_that_are_no_ascending_ones(B):
    """Any place at or past the new one may be taken, twice too; -1 leaves a place, wherever it is."""
    b = S.make(59, [200, 200], 2, 2, 64, 16, BF)
    rng = np.random.default_rng(1)
    kept = rng.integers(np.arange(150), 200, (2, 2, 150)).astype(np.int32)
    kept[rng.random(kept.shape) < 0.2] = -1
    check_evict(B, b, kept)


def test_evict_records_bad_entries(B):
    b = S.make(61, [100, 90], 2, 2, 64, 16, BF)
    kept = pick(np.random.default_rng(3), [100, 90], 2, 40)
    kept[1, 0, 20] = 19                                # before its new place
    check_evict(B, b, kept, expect=(BAD_POSITION, 1, 2, 19), skip=[(1, 0, 20)])
    kept = pick(np.random.default_rng(3), [100, 90], 2, 40)
    kept[0, 1, 7] = 100                                # past the last token
    check_evict(B, S.make(61, [100, 90], 2, 2, 64, 16, BF), kept, expect=(BAD_POSITION, 1, 1, 100),
                skip=[(0, 1, 7)])
    kept = pick(np.random.default_rng(3), [100, 90], 2, 40)
    kept[0, 1, 8] = -2
    check_evict(B, S.make(61, [100, 90], 2, 2, 64, 16, BF), kept, expect=(BAD_POSITION, 1, 1, -2),
                skip=[(0, 1, 8)])


def test_evict_leaves_out_rows_of_bad_blocks(B):
    b = S.make(67, [64], 1, 1, 64, 16, BF)
    kept = np.arange(32, 64, dtype=np.int32)[None, None]
    before = bits(b["kc"]).copy()
    tables = b["tables"].copy()
    tables[0, 2] = 10 ** 6
    rec = B.new_error_record()
    B.kv_cache_evict(b["kc"], b["vc"], dev(tables), dev([64]), dev(kept), error_record=rec)
    code, count, index, value = B.pa_error_read(rec)
    assert (code, count, index, value) == (BAD_BLOCK, 16, 0, 10 ** 6)
    after, t = bits(b["kc"]), b["tables"][0]
    assert np.array_equal(after[t[0]], before[t[0]]) and np.array_equal(after[t[1]], before[t[3]])
    # a length out of range is clamped
    rec = B.new_error_record()
    B.kv_cache_evict(b["kc"], b["vc"], dev(b["tables"]), dev([-3]), dev(kept), error_record=rec)
    assert B.pa_error_read(rec) == [BAD_SEQ_LEN, 1, 0, -3] and np.array_equal(bits(b["kc"]), after)


def test_forks_are_evicted_into_fresh_blocks(B):
    """Samples of one prompt, each with lists of its own; one keeps all it has."""
    bs, H, D = 16, 2, 64
    alloc = B.BlockAllocator(64, bs, np.random.default_rng(0).permutation(64))
    alloc.add(0, 100)
    alloc.fork(0, 1)
    alloc.add(2, 50)
    alloc.fork(0, 3)
    slots, pairs = alloc.batch_append([1])             # sequence 1 has a last block of its own
    gen = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn((64, H, bs, D), generator=gen, device="cuda").to(FH) for _ in range(2))
    B.block_copy([kc], [vc], torch.from_numpy(pairs).cuda())
    seqs = [0, 1, 2, 3]
    tables, lens = alloc.batch_block_tables(seqs, 8)
    alloc.batch_evict(seqs[:3], 60)
    alloc.check()
    new, after = alloc.batch_block_tables(seqs, 8)
    assert after.tolist() == [60, 60, 50, 100] and np.array_equal(new[2:], tables[2:])
    assert not set(new[0][new[0] >= 0]) & set(tables[3][tables[3] >= 0])
    b = dict(kc=kc, vc=vc, tables=tables[:3], lens=lens[:3], bs=bs, H=H)
    check_evict(B, b, pick(np.random.default_rng(4), lens[:3], H, 60), new_tables=new[:3])


# -------------------------------------------------------------- together, and around
def rounds(B, dtype, Hq, H, D, bs, keep=48, steps=40):
    """Prompts of grouped heads, their attention and its last rows' weights, eviction, decode steps with
    evictions whenever a sequence has 24 tokens too many."""
    lens = [150, 30, 97]
    alloc = B.BlockAllocator(80, bs, np.random.default_rng(1).permutation(80))
    for i, n in enumerate(lens):
        alloc.add(i, n)
    alloc.fork(0, 3)
    seqs, MB = [0, 1, 2, 3], -(-160 // bs)
    gen = torch.Generator(device="cuda").manual_seed(7)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
    kc, vc = (torch.zeros((80, H, bs, D), dtype=dtype, device="cuda") for _ in range(2))
    weights = torch.zeros((4, H, MB * bs), device="cuda")
    scale, rec = D ** -0.5, B.new_error_record()
    table = B.rope_cos_sin(512, D)
    at = np.array(lens + lens[:1])                     # the positions of the next tokens
    kw = dict(error_record=rec)

    def on_gpu(which=seqs):
        t, n = alloc.batch_block_tables(which, MB)
        return dev(t), dev(n)

    def evict():
        t, n = on_gpu()
        kept = B.paged_block_select(weights, n, 1, keep, sink_blocks=2, recent_blocks=16, **kw)
        old = f64(kc), f64(vc), t.cpu().numpy(), n.cpu().numpy()
        alloc.batch_evict(seqs, keep)
        alloc.check()
        new, _ = on_gpu()
        before = weights.cpu().numpy().copy()
        B.kv_cache_evict(kc, vc, t, n, kept, weights=weights, new_tables=new, **kw)
        k, v = old[0].copy(), old[1].copy()
        chosen = OS.block_select(before, old[3], 1, keep, 2, 16)
        assert np.array_equal(kept.cpu().numpy(), chosen)
        OE.evict(k, v, old[2], old[3], chosen, before, new.cpu().numpy())
        live = np.unique(new.cpu().numpy()[new.cpu().numpy() >= 0])
        assert np.array_equal(f64(kc)[live], k[live]) and np.array_equal(f64(vc)[live], v[live])
        assert np.array_equal(weights.cpu().numpy(), before)

    t, n = on_gpu([0, 1, 2])
    start = np.concatenate([[0], np.cumsum(lens)])
    T = int(start[-1])
    q = B.kv_cache_append_rope(randn(T, Hq, D), randn(T, H, D), randn(T, H, D), dev(start), 150, kc, vc, t, n, table,
                               **kw)
    lse = torch.empty((T, Hq), device="cuda")
    out = B.paged_attn_chunk(q, dev(start), 150, kc, vc, t, n, scale, lse=lse, **kw)
    b = dict(q=q, kc=kc, vc=vc, tables=t.cpu().numpy(), lens=n.cpu().numpy(), start=start, scale=scale, D=D, H=H,
             bs=bs)
    check_chunk(b, out, lse)
    before = weights[:3].clone()
    B.paged_chunk_weights(q, lse, dev(start), 150, kc, t, n, scale, weights[:3], window=8, **kw)
    check_chunk_weights(b, lse, before, weights[:3], 8)
    weights[3] = weights[0]
    evict()
    for step in range(steps):
        slots, pairs = alloc.batch_append(seqs)
        if len(pairs):
            B.block_copy([kc], [vc], torch.from_numpy(pairs).cuda())
        t, n = on_gpu()
        q = B.kv_cache_append_rope(randn(4, Hq, D), randn(4, H, D), randn(4, H, D), dev(np.arange(5)), 1, kc, vc, t, n,
                                   table, positions=dev(at + step), **kw)
        before = weights.clone()
        out = B.paged_attn_decode_weights(q, kc, vc, t, n, scale, weights, **kw)
        if step % 13 == 0:
            check_decode(dict(q=q, kc=kc, vc=vc, tables=t.cpu().numpy(), lens=n.cpu().numpy(), scale=scale, D=D, H=H,
                              bs=bs), before, weights, out)
        if int(n.max()) >= keep + 24:
            evict()
    assert B.pa_error_read(rec) == [0, 0, 0, 0]


@pytest.mark.parametrize("dtype,Hq,H,D,bs", [(BF, 8, 2, 128, 16), (FH, 6, 6, 64, 8), (BF, 12, 1, 256, 32)])
def test_prompts_weights_eviction_and_decode_together(B, dtype, Hq, H, D, bs):
    rounds(B, dtype, Hq, H, D, bs)


def test_two_captured_steps_replay_side_by_side(B):
    """Two graphs of a decode step and an eviction, each with its own buffers, replayed on two streams;
    and the bits are those of eager calls."""
    def batch(seed):
        b = S.make(seed, [5000, 700], 8, 2, 64, 16, BF)
        b["dt"], b["dl"] = dev(b["tables"]), dev(b["lens"])
        b["w0"] = place(b, seed=seed).nan_to_num(0.0)
        b["k0"], b["v0"] = b["kc"].clone(), b["vc"].clone()
        b["w"], b["out"] = b["w0"].clone(), torch.empty((2, 8, 64), device="cuda")
        b["start"], b["lse"] = dev([0, 1, 2]), torch.empty((2, 8), device="cuda")
        return b

    def step(b):
        B.paged_attn_decode_weights(b["q"], b["kc"], b["vc"], b["dt"], b["dl"], b["scale"], b["w"], out=b["out"])
        B.paged_attn_chunk(b["q"], b["start"], 1, b["kc"], b["vc"], b["dt"], b["dl"], b["scale"], lse=b["lse"])
        B.paged_chunk_weights(b["q"], b["lse"], b["start"], 1, b["kc"], b["dt"], b["dl"], b["scale"], b["w"])
        kept = B.paged_block_select(b["w"], b["dl"], 1, 300, 4, 30)
        B.kv_cache_evict(b["kc"], b["vc"], b["dt"], b["dl"], kept, weights=b["w"])

    def reset(b):
        b["kc"].copy_(b["k0"])
        b["vc"].copy_(b["v0"])
        b["w"].copy_(b["w0"])

    def state(b):
        return [x.clone() for x in (b["w"], b["out"], b["kc"].nan_to_num(3), b["vc"].nan_to_num(3))]

    two = [batch(71), batch(72)]
    want = []
    for b in two:
        step(b)
        want.append(state(b))
    graphs = []
    for b in two:
        reset(b)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(b)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for b in two:
            reset(b)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for b, w in zip(two, want):
            assert all(torch.equal(x, y) for x, y in zip(state(b), w))


@pytest.mark.parametrize("lens,news,Hq,H", [([9000, 17], [3, 2], 8, 1), ([7003], [640], 32, 2)])
def test_captured_chunks_in_parts(B, lens, news, Hq, H):
    """Replayed with other queries and lengths, two calls behind each other through one workspace."""
    b = chunk_batch(24, lens, news, Hq, H, 64, 16, BF)
    start, tables, lengths = dev(b["start"]), dev(b["tables"]), dev(b["lens"])
    need = B.paged_attn_chunk_workspace_needed(len(lens), Hq, H, 64, 16, b["tables"].shape[1], b["most"])
    assert need > 0
    space = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.full_like(b["q"], 7) for _ in range(2)]

    def step():
        for out, v in zip(outs, (b["vc"], b["kc"])):
            B.paged_attn_chunk(b["q"], start, b["most"], b["kc"], v, tables, lengths, b["scale"], out=out,
                               workspace=space)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for shorter in (0, 1500):
        b["q"].copy_(torch.randn(b["q"].shape, device="cuda"))
        lengths.copy_(dev(b["lens"]) - torch.tensor([shorter] + [0] * (len(lens) - 1), device="cuda", dtype=torch.int32))
        graph.replay()
        got = [out.clone() for out in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, outs))
        lse = torch.full(b["q"].shape[:2], 7.0, device="cuda")
        B.paged_attn_chunk(b["q"], start, b["most"], b["kc"], b["vc"], tables, lengths, b["scale"], out=outs[0], lse=lse)
        assert torch.equal(outs[0], got[0])
        check_chunk({**b, "lens": lengths.cpu().numpy()}, got[0], lse)


def test_captured_weights_of_whole_prompts(B):
    """The launch in clusters, captured and replayed."""
    b = chunk_batch(75, [600, 500], [600, 400], 14, 2, 64, 8, BF)
    lse = given_lse(b)
    before, want, _ = run_weights(B, b, lse, 0)
    start, tables, lens = dev(b["start"]), dev(b["tables"]), dev(b["lens"])
    w = before.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.paged_chunk_weights(b["q"], lse, start, b["most"], b["kc"], tables, lens, b["scale"], w)
    for _ in range(3):
        w.copy_(before)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(w.nan_to_num(9), want.nan_to_num(9))


def test_the_same_call_gives_the_same_bits(B):
    lens = np.random.default_rng(0).integers(50, 3000, 20)
    b = chunk_batch(73, lens, np.minimum(lens, 50), 16, 2, 128, 16, BF)
    d = S.make(73, lens, 16, 2, 128, 16, BF)
    first = None
    for _ in range(5):
        out, lse, _ = run_chunk(B, b)
        _, w, _ = run_weights(B, b, lse, 32)
        _, dw, dout, _ = run_decode(B, d)
        now = [x.nan_to_num(9) for x in (out, lse, w, dw, dout)]
        assert first is None or all(torch.equal(x, y) for x, y in zip(first, now))
        first = now


def test_a_given_stream_and_offsets_past_32_bits(B):
    """A cache of over 2^32 elements: blocks at its far end, on another stream."""
    H, D, bs, nb = 2, 128, 16, (1 << 20) + 64
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    kc = torch.zeros((nb, H, bs, D), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    gen = torch.Generator(device="cuda").manual_seed(9)
    tables = np.array([[nb - 1, nb - 40, 3]], np.int32)
    for t in tables[0]:
        for c in (kc, vc):
            c[int(t)] = torch.randn((H, bs, D), generator=gen, device="cuda").to(BF)
    where = [int(t) for t in tables[0]]
    q = torch.randn((1, 4, D), generator=gen, device="cuda").to(BF)
    small = dict(tables=np.array([[0, 1, 2]], np.int32), lens=np.array([41], np.int32), kc=kc[where], vc=vc[where], q=q,
                 start=np.array([0, 1]), bs=bs, scale=float(np.float32(0.1)), D=D, H=H)
    td, ld, start = dev(tables), dev([41]), dev([0, 1])
    w = torch.zeros((1, H, 48), device="cuda")
    lse = torch.empty((1, 4), device="cuda")
    kept = dev(pick(np.random.default_rng(1), [41], H, 20))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = B.paged_attn_chunk(q, start, 1, kc, vc, td, ld, 0.1, lse=lse, stream=side)
    B.paged_chunk_weights(q, lse, start, 1, kc, td, ld, 0.1, w, stream=side)
    side.synchronize()
    check_chunk(small, out, lse)
    check_chunk_weights(small, lse, torch.zeros_like(w), w, 0)
    before = w.clone()
    side.wait_stream(torch.cuda.current_stream())
    out = B.paged_attn_decode_weights(q, kc, vc, td, ld, 0.1, w, stream=side)
    side.synchronize()
    check_decode(small, before, w, out)
    k, v = bits(small["kc"]).copy(), bits(small["vc"]).copy()
    OE.evict(k, v, small["tables"], [41], kept.cpu().numpy())
    side.wait_stream(torch.cuda.current_stream())
    B.kv_cache_evict(kc, vc, td, ld, kept, stream=side)
    side.synchronize()
    assert np.array_equal(bits(kc[where]), k) and np.array_equal(bits(vc[where]), v)


def test_the_largest_batch(B):
    """65535 sequences, the most a call takes, two tokens each in a block of its own; one more is
    refused."""
    N, D, bs = 65535, 64, 8
    gen = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(FH)
    kc, vc = randn(N + 1, 1, bs, D), randn(N + 1, 1, bs, D)
    tables = torch.arange(N + 1, dtype=torch.int32, device="cuda").flip(0)[:, None].contiguous()
    lens = torch.full((N + 1,), 2, dtype=torch.int32, device="cuda")
    start = torch.arange(N + 2, dtype=torch.int32, device="cuda")
    q, rec = randn(N + 1, 2, D), B.new_error_record()
    w = torch.zeros((N + 1, 1, bs), device="cuda")
    lse = torch.empty((N + 1, 2), device="cuda")
    n = N
    out = B.paged_attn_chunk(q[:n], start[:n + 1], 1, kc, vc, tables[:n], lens[:n], 0.125, lse=lse[:n], error_record=rec)
    B.paged_chunk_weights(q[:n], lse[:n], start[:n + 1], 1, kc, tables[:n], lens[:n], 0.125, w[:n], error_record=rec)
    at = [0, 1, 30000, N - 1]
    blocks = [N - i for i in at]
    b = dict(tables=np.arange(4)[:, None], lens=np.full(4, 2), kc=kc[blocks], vc=vc[blocks], q=q[at], start=np.arange(5),
             bs=bs, scale=0.125, D=D, H=1)
    check_chunk(b, out[at], lse[at])
    check_chunk_weights(b, lse[at], torch.zeros_like(w[at]), w[at], 0)
    before = w[at].clone()
    out = B.paged_attn_decode_weights(q[:n], kc, vc, tables[:n], lens[:n], 0.125, w[:n], error_record=rec)
    check_decode(b, before, w[at], out[at])
    kept = torch.ones((n, 1, 1), dtype=torch.int32, device="cuda")
    second = kc[blocks, 0, 1].clone()
    B.kv_cache_evict(kc, vc, tables[:n], lens[:n], kept, weights=w[:n], error_record=rec)
    assert torch.equal(kc[blocks, 0, 0], second) and B.pa_error_read(rec) == [0, 0, 0, 0]
    kept = torch.ones((N + 1, 1, 1), dtype=torch.int32, device="cuda")
    for call in (lambda: B.paged_chunk_weights(q, lse, start, 1, kc, tables, lens, 0.125, w),
                 lambda: B.paged_attn_decode_weights(q, kc, vc, tables, lens, 0.125, w),
                 lambda: B.kv_cache_evict(kc, vc, tables, lens, kept)):
        with pytest.raises(B.PagedKVError, match="INVALID_ARG"):
            call()


def test_the_example_runs(B):
    """paged_kv_cache_317_gb300/examples/bounded_step.py: its last step is the oracle's for the cache it has."""
    import os
    import runpy
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = runpy.run_path(os.path.join(root, "paged_kv_cache_317_gb300", "examples", "bounded_step.py"))
    lens = env["lengths"].cpu().numpy()
    assert lens.tolist() == [512 + 100 % 64, 300 + 100] and env["alloc"].num_free() == 1024 - 35 - 25
    b = dict(lens=lens, tables=env["tables"].cpu().numpy(), kc=env["kc"], vc=env["vc"], q=env["q"], bs=16,
             scale=128 ** -0.5, D=128, H=8)
    w = torch.zeros_like(env["weights"])
    out = B.paged_attn_decode_weights(env["q"], env["kc"], env["vc"], env["tables"], env["lengths"], b["scale"], w)
    assert torch.equal(out, env["out"])
    check_decode(b, torch.zeros_like(w), w, out)
    assert bool(torch.isfinite(env["weights"]).all()) and not bool(env["weights"][0, :, 548:].any())
