"""paged_block_scores, paged_block_select and paged_attn_sparse on the GPU against the fp64
oracle, each by itself and as the decode step that they form.

Tolerances (derived, u = 2^-23: a sum on the tensor cores may drop a unit in the last place
at each addition):
* scores: 2 D products, exact in fp32, and their sum: (2 D + 4) u times the sum of the terms'
  magnitudes.
* attention: a logit is off by at most d = (D + 4) u * max_t scale sum_d |q_d k_td|, so a
  weight by a factor within e^(+-d); the probabilities enter the product as two half-precision
  numbers, off by 2^-17 (bf16) of the weight at most; exponentials, n products and sums add
  (n + 16) u.  Numerator and denominator both, so the result is within twice that of the sum of
  w_t |v_t|; a half-precision output is rounded by half a step on top.  fp16 has steps of 2^-24 at
  least and holds 2^12 times the weight: 2^-37 (of a largest weight of 1) per token and |v| besides.
"""

import numpy as np
import pytest
import torch

from gpu_util import bits, half_ulp
from oracle import sparse as OS

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def f64(t):
    return t.detach().cpu().double().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def make(seed, lens, Hq, H, D, bs, dtype, wide=0):
    """Caches with NaN in every row without a token, tables (wider than needed by `wide`)."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
    lens = np.asarray(lens, np.int32)
    N, nb = len(lens), -(-lens // bs)
    MB, total = max(1, int(nb.max())) + wide, int(nb.sum()) + 3
    tables = np.full((N, MB), -1, np.int32)
    tables[np.arange(MB)[None, :] < nb[:, None]] = rng.permutation(total)[:int(nb.sum())]
    live = np.zeros((total, bs), bool)
    for i in range(N):
        for t in range(int(lens[i])):
            live[tables[i, t // bs], t % bs] = True
    dead = torch.from_numpy(~live).cuda()[:, None, :, None]
    kc, vc = (randn(total, H, bs, D).masked_fill(dead, NAN) for _ in range(2))
    lo, hi = (torch.full((total, H, D), NAN, dtype=dtype, device="cuda") for _ in range(2))
    wlo, whi = f64(lo).copy(), f64(hi).copy()
    OS.block_bounds(f64(kc), tables, lens, wlo, whi)
    lo, hi = torch.from_numpy(wlo).cuda().to(dtype), torch.from_numpy(whi).cuda().to(dtype)
    return dict(lens=lens, tables=tables, kc=kc, vc=vc, lo=lo, hi=hi, q=randn(N, Hq, D), bs=bs,
                scale=float(np.float32(D ** -0.5)), D=D, H=H)


def scores_of(B, b, **kw):
    return B.paged_block_scores(b["q"], b["lo"], b["hi"], dev(b["tables"]), dev(b["lens"]), b["scale"],
                                b["bs"], **kw)


def attend(B, b, selected, **kw):
    return B.paged_attn_sparse(b["q"], b["kc"], b["vc"], dev(b["tables"]), dev(b["lens"]),
                               dev(selected), b["scale"], **kw)


def check_scores(got, b, dtype=None):
    want, size = OS.block_scores(f64(b["q"]), f64(b["lo"]), f64(b["hi"]), b["tables"], b["lens"],
                                 b["scale"], b["bs"])
    got = f64(got)
    past = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), past)
    err = np.abs(got[~past] - want[~past])
    assert (err <= (2 * b["D"] + 4) * U * size[~past] + 1e-30).all(), err.max()


def check_attention(out, b, selected, kc=None, vc=None):
    """NaN rows are cut by the oracle; a NaN in the result is an error here."""
    ref, spread, reach = OS.sparse_attention(f64(b["q"]), f64(b["kc"] if kc is None else kc),
                                             f64(b["vc"] if vc is None else vc), b["tables"],
                                             b["lens"], selected, b["scale"])
    n = selected.shape[-1] * b["bs"]
    d = (b["D"] + 4) * U * reach[..., None]
    split = 2.0 ** -17
    bound = 2 * (np.expm1(2 * d) + split + (n + 16) * U) * spread
    if b["q"].dtype == torch.float16:
        bound = bound + n * 2.0 ** -37 * float(torch.nan_to_num(b["vc"].float()).abs().max())
    if out.dtype != torch.float32:
        bound = bound + half_ulp(np.abs(ref) + bound, out.dtype)
    err = np.abs(f64(out) - ref)
    assert (err <= bound).all(), (np.nanmax(err), bound.max(), np.isnan(err).sum())


def lists(rng, b, keep, spoil=True):
    """Distinct blocks in any order with -1 (and blocks past the end) between them."""
    N, H, MB = len(b["lens"]), b["H"], b["tables"].shape[1]
    out = np.full((N, H, keep), -1, np.int32)
    for i in range(N):
        held = -(-int(b["lens"][i]) // b["bs"])
        for h in range(H):
            n = min(held, rng.integers(0, keep + 1)) if spoil else min(held, keep)
            at = rng.choice(keep, n, replace=False)
            out[i, h, at] = rng.choice(held, n, replace=False) if n else 0
            if spoil and held < MB and n < keep:
                out[i, h, np.flatnonzero(out[i, h] == -1)[0]] = rng.integers(held, MB)
    return out


SHAPES = [
    # lens, Hq, H, D, bs
    ([1], 1, 1, 64, 16),
    ([17, 0, 33, 16, 200], 8, 8, 128, 16),
    ([40, 7, 1, 100, 31], 8, 2, 128, 8),
    ([333, 64], 16, 1, 64, 32),
    ([65, 129, 2], 15, 3, 256, 16),
    ([130], 32, 1, 128, 48),
    ([1000, 3], 14, 2, 128, 64),
    ([50, 90], 80, 2, 256, 8),
    ([90, 47], 34, 2, 64, 16),
]
IDS = ["x".join(map(str, s[1:])) for s in SHAPES]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_scores_match_the_oracle(B, shape, dtype):
    b = make(1, *shape, dtype, wide=2)
    rec = B.new_error_record()
    check_scores(scores_of(B, b, error_record=rec), b)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("keep", [1, 3, 40])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_attention_matches_the_oracle(B, shape, keep, dtype):
    b = make(2, *shape, dtype, wide=2)
    sel = lists(np.random.default_rng(keep), b, keep)
    rec = B.new_error_record()
    for out_dtype in (torch.float32, dtype):
        check_attention(attend(B, b, sel, out_dtype=out_dtype, error_record=rec), b, sel)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]


@pytest.mark.parametrize("seqs,keep,H,G", [(1, 300, 1, 4), (2, 600, 2, 1), (1, 1500, 1, 8), (70, 33, 2, 2)])
def test_long_lists(B, seqs, keep, H, G):
    rng = np.random.default_rng(keep)
    lens = rng.integers(keep * 16, keep * 18, seqs)
    b = make(3, lens, H * G, H, 128, 16, torch.bfloat16)
    sel = lists(rng, b, keep, spoil=False)
    check_attention(attend(B, b, sel), b, sel)


@pytest.mark.parametrize("dtype,D,Hq,H,keep,bs", [(torch.bfloat16, 128, 1, 1, 700, 64),
                                                  (torch.float16, 256, 9, 1, 600, 32),
                                                  (torch.bfloat16, 64, 34, 2, 4000, 8)])
def test_few_rows_with_long_lists(B, dtype, D, Hq, H, keep, bs):
    """A row's list spread over several clusters, whose sums a second kernel joins; without a
    workspace over one; rows without tokens, and with less than one chunk a cluster, among them."""
    rng = np.random.default_rng(D)
    for lens in ([keep * bs - 3], [bs * keep // 3, 0, 5]):
        b = make(12, lens, Hq, H, D, bs, dtype, wide=keep - (-(-max(lens) // bs)))
        sel = lists(rng, b, keep, spoil=len(lens) > 1)
        need = B.paged_attn_sparse_workspace_size(len(lens), Hq, H, D, bs, b["tables"].shape[1], keep)
        assert need > 0
        ws, rec = torch.full((need,), 255, dtype=torch.uint8, device="cuda"), B.new_error_record()
        for od in (torch.float32, dtype):
            out = attend(B, b, sel, out_dtype=od, workspace=ws, error_record=rec)
            check_attention(out, b, sel)
            assert torch.equal(out, attend(B, b, sel, out_dtype=od))
        assert B.pa_error_read(rec) == [0, 0, 0, 0]
        lib, one = B.load_library(), torch.empty_like(b["q"])
        tables, lens_d, sel_d = dev(b["tables"]), dev(b["lens"]), dev(sel)
        assert lib.paged_attn_sparse(b["q"].data_ptr(), b["kc"].data_ptr(), b["vc"].data_ptr(),
                                     tables.data_ptr(), lens_d.data_ptr(),
                                     sel_d.data_ptr(), keep, len(lens), Hq, H, D, bs,
                                     b["tables"].shape[1], len(b["kc"]), b["scale"], B._DTYPE[dtype],
                                     one.data_ptr(), B._DTYPE[dtype], None, 0, None,
                                     torch.cuda.current_stream().cuda_stream) == 0
        check_attention(one, b, sel)
        with pytest.raises(B.PagedKVError, match="INVALID_ARG"):
            attend(B, b, sel, workspace=ws[:-1])
    # every logit -infinity in all parts: no softmax; in all but one: that one's alone
    b["kc"].fill_(-INF), b["q"].abs_(), b["q"].add_(1)
    sel = lists(rng, b, keep, spoil=False)
    assert torch.isnan(attend(B, b, sel)[0]).all()
    b["kc"][int(b["tables"][0, 1])] = 0.5
    only = np.full_like(sel, -1)
    only[0, :, 0] = 1
    only[2] = -1
    out = attend(B, b, np.where(np.arange(3)[:, None, None] == 2, -1, sel).astype(np.int32))
    check_attention(out, b, only)


def test_short_lists_spread_over_clusters(B):
    """Few rows, one query head in the last tile of a group: the clusters' blocks have next to
    nothing to do after they have read one another's sums, and must still wait for one another
    before they leave."""
    b = make(11, [3, 0, 1, 1, 2], 66, 2, 128, 48, torch.float16, wide=3)
    sel = lists(np.random.default_rng(0), b, 7)
    tables, lens, sel_d = dev(b["tables"]), dev(b["lens"]), dev(sel)
    first = attend(B, b, sel)
    check_attention(first, b, sel)
    for _ in range(3000):
        out = B.paged_attn_sparse(b["q"], b["kc"], b["vc"], tables, lens, sel_d, b["scale"])
    assert torch.equal(out, first)


def test_all_blocks_listed_equals_the_dense_decode(B):
    b = make(4, [130, 16, 77, 1], 4, 4, 128, 16, torch.bfloat16)
    every = np.broadcast_to(np.arange(9, dtype=np.int32), (4, 4, 9))
    dense = B.paged_attn_decode(b["q"], b["kc"], b["vc"], dev(b["tables"]), dev(b["lens"]), b["scale"])
    out = attend(B, b, every)
    check_attention(out, b, every)
    assert float((out - dense).abs().max()) < 2e-3


def test_rows_without_tokens_are_zero(B):
    b = make(5, [0, 20, 40], 4, 2, 64, 16, torch.float16, wide=3)
    sel = np.array([[[0, 1]] * 2, [[-1, -1], [4, 2]], [[1, -1], [-1, -1]]], np.int32)
    rec = B.new_error_record()
    out = attend(B, b, sel, error_record=rec)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    assert (out[:2] == 0).all() and (out[2, 2:] == 0).all() and (out[2, :2] != 0).any()
    none = np.zeros((3, 2, 0), np.int32)
    assert (attend(B, b, none) == 0).all()


def test_a_block_listed_twice_counts_twice(B):
    b = make(6, [40], 2, 1, 64, 16, torch.float16)
    sel = np.array([[[1, 2, 1]]], np.int32)
    check_attention(attend(B, b, sel), b, sel)


def test_infinite_keys_in_listed_blocks(B):
    b = make(7, [40], 1, 1, 64, 16, torch.bfloat16)
    b["q"].abs_()
    sel = np.array([[[0, 1, 2]]], np.int32)
    b["kc"][int(b["tables"][0, 0])] = -INF          # a whole block of logits -inf: weight 0
    ref = np.array([[[1, 2, -1]]], np.int32)
    check_attention(attend(B, b, sel), b, ref)
    b["kc"][:] = -INF                               # every logit -inf: no softmax
    assert torch.isnan(attend(B, b, sel)).all()
    assert (scores_of(B, make(7, [0], 1, 1, 64, 16, torch.bfloat16)) == -INF).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_small_weights_next_to_a_large_one(B, dtype):
    """8000 weights of 2^-25.5 of the largest, whose value is 0: they are all of the result."""
    b = make(10, [8001], 1, 1, 64, 16, dtype)
    b["kc"].fill_(0), b["vc"].fill_(1), b["q"].fill_(0)
    b["q"][..., 0] = 1
    first = int(b["tables"][0, 0])
    b["kc"][first, 0, 0, 0], b["vc"][first, 0, 0] = 17.625, 0     # 25.43 / log2(e)
    b["scale"] = 1.0
    sel = np.arange(501, dtype=np.int32)[None, None]
    out = attend(B, b, sel)
    check_attention(out, b, sel)
    assert float(out.min()) > 1e-4


def test_nan_bounds_make_nan_scores_that_are_kept(B):
    b = make(8, [100], 4, 2, 128, 16, torch.float16)
    b["lo"][int(b["tables"][0, 3]), 1, 5] = NAN
    s = scores_of(B, b)
    assert torch.isnan(s[0, 1, 3]) and int(torch.isnan(s).sum()) == 1
    assert 3 in B.paged_block_select(s, dev(b["lens"]), 16, 1)[0, 1].tolist()


def test_bad_entries_are_recorded(B):
    b = make(9, [40, 70], 4, 2, 64, 16, torch.float16)
    rec = B.new_error_record()
    sel = np.array([[[0, 5], [0, 1]], [[-2, 1], [0, 1]]], np.int32)
    out = attend(B, b, sel, error_record=rec)
    got = B.pa_error_read(rec)
    assert got[0] == 4 and got[1] == 2 and (got[2], got[3]) in ((0, 5), (2, -2))
    check_attention(out, b, np.array([[[0, -1], [0, 1]], [[-1, 1], [0, 1]]]))
    B.pa_error_clear(rec)
    good = b["tables"].copy()
    b["tables"][1, 0] = len(b["kc"])
    b["tables"][0, 0] = 0                            # block 0 read in place of a bad one
    sel = np.zeros((2, 2, 1), np.int32)
    clean = torch.where(torch.isnan(b["kc"]), 0, b["kc"]), torch.where(torch.isnan(b["vc"]), 0, b["vc"])
    bad = dict(b, kc=clean[0], vc=clean[1])
    out = attend(B, bad, sel, error_record=rec)
    assert B.pa_error_read(rec) == [4, 2, 1, len(b["kc"])]     # by both key heads' lists
    bad["tables"] = np.where(b["tables"] == len(b["kc"]), 0, b["tables"])
    check_attention(out, bad, sel)
    B.pa_error_clear(rec)
    lo, hi = torch.nan_to_num(b["lo"]), torch.nan_to_num(b["hi"])
    s = scores_of(B, dict(b, lo=lo, hi=hi), error_record=rec)
    assert B.pa_error_read(rec) == [4, 1, 1, len(b["kc"])]
    check_scores(s, dict(bad, lo=lo, hi=hi))
    # lengths out of range are clamped
    b["tables"], b["lens"] = good, np.array([-1, 81], np.int32)
    for call in (lambda: scores_of(B, b, error_record=rec), lambda: attend(B, b, sel, error_record=rec),
                 lambda: B.paged_block_select(torch.zeros(2, 2, 5, device="cuda"), dev(b["lens"]), 16, 2,
                                              error_record=rec)):
        B.pa_error_clear(rec)
        call()
        got = B.pa_error_read(rec)
        assert got[0] == 6 and got[1] == 2 and (got[2], got[3]) in ((0, -1), (1, 81))


# ------------------------------------------------------------------------------ select
@pytest.mark.parametrize("width,lens,keep,sink,recent", [
    (1, [1, 0], 1, 0, 0), (7, [7, 3, 5], 3, 1, 1), (40, [40, 33, 2], 4, 2, 2),
    (300, [300, 257, 256, 1], 50, 0, 3), (1031, [1031, 800], 64, 4, 8),
    (2100, [2100, 2049], 1000, 1, 1), (5000, [4999], 1, 0, 1), (9001, [9001, 4097], 300, 0, 0),
    (20000, [20000, 19999, 7], 2000, 1, 4), (70001, [70001, 69000], 500, 3, 5),
    (131072, [131072, 5], 20000, 1, 9)])
@pytest.mark.parametrize("kind", ["normal", "ties", "odd", "wide"])
def test_select_matches_the_oracle(B, width, lens, keep, sink, recent, kind):
    rng = np.random.default_rng(width)
    s = rng.standard_normal((len(lens), 3, width)).astype(np.float32)
    if kind == "ties":
        s = np.round(s)                              # also -0 and 0
    elif kind == "odd":
        s = np.round(s * 4)
        for v in (NAN, -NAN, INF, -INF, 1e-42, -1e-42, -0.0):
            s[rng.random(s.shape) < 0.05] = v
        s[0, 0] = 2.5
    elif kind == "wide":                             # finite, of every size
        s = (s * np.float32(10.0) ** rng.integers(-44, 38, s.shape)).astype(np.float32)
        s[-1] = 1 + rng.integers(0, 9, s[-1].shape) * np.float32(2.0 ** -23)
        s[0, 1] = np.float32(3e38) * rng.choice([-1, 1], width)
    rec = B.new_error_record()
    got = B.paged_block_select(torch.from_numpy(s).cuda(), dev(lens), 1, keep, sink, recent,
                               error_record=rec)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    assert np.array_equal(got.cpu().numpy(), OS.block_select(s, lens, 1, keep, sink, recent))


@pytest.mark.parametrize("kind", ["normal", "ties", "odd", "wide"])
@pytest.mark.parametrize("rows,width,keep", [(700, 40, 7), (650, 256, 256), (700, 300, 17), (620, 1024, 100),
                                             (640, 1500, 64), (610, 2048, 1), (20, 2049, 9), (3, 33000, 200)])
def test_select_of_many_rows(B, rows, width, keep, kind):
    """A warp a row, a thread block a row and a cluster a row: by the width and how many rows."""
    rng = np.random.default_rng(rows + width)
    s = rng.standard_normal((rows, 1, width)).astype(np.float32)
    if kind == "ties":
        s = np.round(s)
    elif kind == "odd":
        s = np.round(s * 4)
        for v in (NAN, -NAN, INF, -INF, 1e-42, -1e-42, -0.0):
            s[rng.random(s.shape) < 0.03] = v
        s[1] = -1.5
    elif kind == "wide":
        s = (s * np.float32(10.0) ** rng.integers(-44, 38, s.shape)).astype(np.float32)
    lens = rng.integers(0, width + 1, rows)
    lens[0] = width
    sink, recent = (1, 2) if keep > 4 else (0, 0)
    rec = B.new_error_record()
    got = B.paged_block_select(torch.from_numpy(s).cuda(), dev(lens), 1, keep, sink, recent, error_record=rec)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    assert np.array_equal(got.cpu().numpy(), OS.block_select(s, lens, 1, keep, sink, recent))


@pytest.mark.parametrize("width", [9, 300, 3000, 40000])
def test_select_of_the_ends_alone(B, width):
    """Nothing competes for a place: the first and last blocks, whatever the scores."""
    s = torch.full((609, 1, width), NAN, device="cuda")
    got = B.paged_block_select(s, dev([width] * 609), 1, 5, 2, 3)[:, 0].cpu().numpy()
    assert (got == [0, 1, width - 3, width - 2, width - 1]).all()


def test_select_reads_nothing_past_a_sequence(B):
    s = torch.full((1, 1, 50), NAN, device="cuda")
    s[..., :30] = torch.arange(30, device="cuda").flip(0).float()
    assert B.paged_block_select(s, dev([30 * 8 - 7]), 8, 4)[0, 0].tolist() == [0, 1, 2, 3]


# ---------------------------------------------------------------------------- the step
def _step(B, b, st, keep, q, k, v, start, most, rec, out=None):
    """Append with rotation, score, select, attend."""
    turned = B.kv_cache_append_rope(q, k, v, start, most, b["kc"], b["vc"], st["tables"], st["lens"],
                                    st["cos_sin"], k_min=b["lo"], k_max=b["hi"], q_out=st.get("q_out"),
                                    error_record=rec)
    s = B.paged_block_scores(turned, b["lo"], b["hi"], st["tables"], st["lens"], b["scale"], b["bs"],
                             out=st.get("scores"), error_record=rec)
    sel = B.paged_block_select(s, st["lens"], b["bs"], keep, 1, 2, out=st.get("sel"), error_record=rec)
    return turned, s, sel, B.paged_attn_sparse(turned, b["kc"], b["vc"], st["tables"], st["lens"], sel,
                                               b["scale"], out=out, out_dtype=q.dtype, error_record=rec)


@pytest.mark.parametrize("dtype,Hq,H,D,bs", [(torch.bfloat16, 8, 2, 128, 16), (torch.float16, 4, 4, 64, 8)])
def test_prompts_then_decode_steps(B, dtype, Hq, H, D, bs):
    """Prompts through the rotated append and the dense prefill; then decode steps whose lists
    agree with the scores and whose outputs agree with the oracle; the dense decode over the
    same caches where every block fits the list."""
    prompts, steps, keep = [150, 33, 7], 20, 5
    N, T = len(prompts), sum(prompts)
    final = np.array(prompts, np.int32) + steps
    b = make(20, final, Hq, H, D, bs, dtype)
    b["kc"].fill_(NAN), b["vc"].fill_(NAN), b["lo"].fill_(NAN), b["hi"].fill_(NAN)
    gen = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
    st = {"tables": dev(b["tables"]), "lens": dev(prompts), "cos_sin": B.rope_cos_sin(400, D)}
    start = np.concatenate([[0], np.cumsum(prompts)])
    rec = B.new_error_record()
    q, k, v = randn(T, Hq, D), randn(T, H, D), randn(T, H, D)
    turned = B.kv_cache_append_rope(q, k, v, dev(start), max(prompts), b["kc"], b["vc"], st["tables"],
                                    st["lens"], st["cos_sin"], k_min=b["lo"], k_max=b["hi"],
                                    error_record=rec)
    if Hq == H:
        pre = B.paged_attn_prefill(turned, dev(start), max(prompts), b["kc"], b["vc"], st["tables"],
                                   st["lens"], b["scale"], error_record=rec)
        assert torch.isfinite(pre).all()
    lens = np.array(prompts, np.int32)
    for step in range(steps):
        lens = lens + 1
        st["lens"] = dev(lens)
        turned, s, sel, out = _step(B, b, st, keep, randn(N, Hq, D), randn(N, H, D), randn(N, H, D),
                                    dev(np.arange(N + 1)), 1, rec)
        now = dict(b, lens=lens, q=turned)
        if step % 6 == 0 or step == steps - 1:
            check_scores(s, now)
            sel_h = sel.cpu().numpy()
            assert np.array_equal(sel_h, OS.block_select(s.cpu().numpy(), lens, bs, keep, 1, 2))
            check_attention(out, now, sel_h)
            lo, hi = torch.empty_like(b["lo"]), torch.empty_like(b["hi"])
            B.kv_block_bounds(b["kc"], st["tables"], st["lens"], lo, hi, error_record=rec)
            held = sorted({int(x) for i in range(N) for x in b["tables"][i, :-(-int(lens[i]) // bs)]})
            assert torch.equal(lo[held], b["lo"][held]) and torch.equal(hi[held], b["hi"][held])
    assert B.pa_error_read(rec) == [0, 0, 0, 0]


def test_two_captured_steps_replay_side_by_side(B):
    """Two steps captured into graphs of their own share no scratch: replayed on two streams at
    once, each gives what it gives alone, with lengths and inputs written into its buffers."""
    graphs = []
    for seed in (30, 31):
        b = make(seed, [200, 90, 33], 8, 2, 128, 16, torch.bfloat16)
        st = {"tables": dev(b["tables"]), "lens": dev(b["lens"]), "cos_sin": B.rope_cos_sin(256, 128)}
        gen = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
        q, k, v = randn(3, 8, 128), randn(3, 2, 128), randn(3, 2, 128)
        start, rec = dev(np.arange(4)), B.new_error_record()
        want = _step(B, b, st, 4, q, k, v, start, 1, rec)
        st["q_out"], st["scores"], st["sel"] = (torch.empty_like(x) for x in want[:3])
        out = torch.empty_like(want[3])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _step(B, b, st, 4, q, k, v, start, 1, rec, out=out)
        graphs.append((g, want, out, st, rec, b, q, k, v, start))   # a graph keeps no tensor alive
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for g, want, out, st, rec, *_ in graphs:
        assert torch.equal(out, want[3]) and torch.equal(st["sel"], want[2])
        assert torch.equal(st["scores"], want[1]) and B.pa_error_read(rec) == [0, 0, 0, 0]


def test_the_same_call_gives_the_same_bits(B):
    b = make(40, np.random.default_rng(0).integers(1, 3000, 20), 16, 2, 128, 16, torch.bfloat16)
    first = None
    for _ in range(5):
        s = scores_of(B, b)
        sel = B.paged_block_select(s, dev(b["lens"]), 16, 64, 1, 2)
        out = B.paged_attn_sparse(b["q"], b["kc"], b["vc"], dev(b["tables"]), dev(b["lens"]), sel, b["scale"])
        now = (bits(s.to(torch.bfloat16)), sel.cpu().numpy(), out.cpu().numpy())
        if first is not None:
            assert all(np.array_equal(x, y) for x, y in zip(first, now))
        first = now


def test_a_given_stream_and_offsets_past_32_bits(B):
    """A cache of over 2^32 elements: blocks at its far end, on another stream."""
    H, D, bs, nb = 2, 128, 16, (1 << 20) + 64
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    kc = torch.zeros((nb, H, bs, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    lo, hi = (torch.zeros((nb, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(9)
    tables = np.array([[nb - 1, nb - 40, 3]], np.int32)
    for t in tables[0]:
        for c in (kc, vc):
            c[int(t)] = torch.randn((H, bs, D), generator=gen, device="cuda").to(torch.bfloat16)
    q = torch.randn((1, 4, D), generator=gen, device="cuda").to(torch.bfloat16)
    lens = np.array([41], np.int32)
    k = torch.randn((1, H, D), generator=gen, device="cuda").to(torch.bfloat16)
    lens_d, tables_d, start = dev(lens), dev(tables), dev([0, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.kv_block_bounds(kc, tables_d, lens_d, lo, hi, stream=side)
    B.kv_cache_append_rope(None, k, k, start, 1, kc, vc, tables_d, lens_d, None, k_min=lo, k_max=hi,
                           stream=side)
    s = B.paged_block_scores(q, lo, hi, tables_d, lens_d, 0.1, bs, stream=side)
    sel = B.paged_block_select(s, lens_d, bs, 3, stream=side)
    out = B.paged_attn_sparse(q, kc, vc, tables_d, lens_d, sel, 0.1, stream=side)
    side.synchronize()
    pick = [int(t) for t in tables[0]]
    small = dict(tables=np.array([[0, 1, 2]]), lens=lens, kc=kc[pick], vc=vc[pick], lo=lo[pick], hi=hi[pick],
                 q=q, bs=bs, scale=float(np.float32(0.1)), D=D, H=H)
    assert sel.tolist() == [[[0, 1, 2], [0, 1, 2]]]
    assert torch.equal(small["kc"][2, :, 8], k[0])
    check_scores(s, small)
    check_attention(out, small, sel.cpu().numpy())


def test_the_example_runs(B):
    """paged_kv_cache_317_gb300/examples/sparse_step.py: its output is the oracle's for its lists."""
    import os
    import runpy
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = runpy.run_path(os.path.join(root, "paged_kv_cache_317_gb300", "examples", "sparse_step.py"))
    lens, sel = env["lengths"].cpu().numpy(), env["blocks"].cpu().numpy()
    assert lens.tolist() == [5001, 301] and (sel[1, :, 19:] == -1).all() and (sel[0] >= 0).all()
    b = dict(lens=lens, tables=env["tables"].cpu().numpy(), kc=env["kc"], vc=env["vc"], q=env["q"], bs=16,
             scale=128 ** -0.5, D=128)
    check_attention(env["out"], b, sel)


def test_a_million_tokens(B):
    b = make(50, [(1 << 20) - 7], 4, 1, 64, 16, torch.bfloat16)
    rec = B.new_error_record()
    s = scores_of(B, b, error_record=rec)
    check_scores(s, b)
    sel = B.paged_block_select(s, dev(b["lens"]), 16, 4096, 1, 4, error_record=rec)
    assert np.array_equal(sel.cpu().numpy(), OS.block_select(s.cpu().numpy(), b["lens"], 16, 4096, 1, 4))
    check_attention(attend(B, b, sel.cpu().numpy(), error_record=rec), b, sel.cpu().numpy())
    assert B.pa_error_read(rec) == [0, 0, 0, 0]


def test_the_largest_batch(B):
    """65535 sequences, the most a call takes, two tokens each in a block of its own; one more is
    refused."""
    N, D, bs = 65535, 64, 8
    gen = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.float16)
    kc, vc = randn(N + 1, 1, bs, D), randn(N + 1, 1, bs, D)
    lo, hi = torch.empty_like(kc[:, :, 0]), torch.empty_like(kc[:, :, 0])
    tables = torch.arange(N + 1, dtype=torch.int32, device="cuda").flip(0)[:, None].contiguous()
    lens = torch.full((N + 1,), 2, dtype=torch.int32, device="cuda")
    start = torch.arange(N + 2, dtype=torch.int32, device="cuda")
    q, k, v = randn(N + 1, 2, D), randn(N + 1, 1, D), randn(N + 1, 1, D)
    table, rec = B.rope_cos_sin(8, D), B.new_error_record()

    def step(n):
        B.kv_block_bounds(kc, tables[:n], lens[:n] - 1, lo, hi, error_record=rec)
        turned = B.kv_cache_append_rope(q[:n], k[:n], v[:n], start[:n + 1], 1, kc, vc, tables[:n], lens[:n],
                                        table, k_min=lo, k_max=hi, error_record=rec)
        s = B.paged_block_scores(turned, lo, hi, tables[:n], lens[:n], 0.125, bs, error_record=rec)
        sel = B.paged_block_select(s, lens[:n], bs, 1, error_record=rec)
        return turned, s, B.paged_attn_sparse(turned, kc, vc, tables[:n], lens[:n], sel, 0.125,
                                              error_record=rec)

    turned, s, out = step(N)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    pick = np.array([0, 1, 30000, N - 1])
    blocks = [N - int(i) for i in pick]
    small = dict(tables=np.arange(4)[:, None], lens=np.full(4, 2), kc=kc[blocks], vc=vc[blocks], lo=lo[blocks],
                 hi=hi[blocks], q=turned[pick], bs=bs, scale=0.125, D=D, H=1)
    check_scores(s[pick], small)
    check_attention(out[pick], small, np.zeros((4, 1, 1), np.int32))
    # prompts: two tokens of each
    starts = 2 * start[:N + 1]
    two = randn(2 * N, 1, D)
    B.kv_cache_append_rope(None, two, two, starts, 2, kc, vc, tables[:N], lens[:N], None, k_min=lo, k_max=hi,
                           error_record=rec)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    at = torch.from_numpy(pick).cuda()
    assert torch.equal(kc[blocks, 0, 1], two[2 * at + 1, 0]) and torch.equal(vc[blocks, 0, 0], two[2 * at, 0])
    assert torch.equal(lo[blocks, 0], torch.minimum(two[2 * at, 0], two[2 * at + 1, 0]))
    with pytest.raises(B.PagedKVError, match="INVALID_ARG"):
        step(N + 1)
