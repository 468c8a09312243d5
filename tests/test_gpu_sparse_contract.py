"""What the documentation of the rotary append and of the block-sparse decode promises besides values:
bad entries in each of the append's kernels, rows that share a block table, equal bits on every run.

The append runs one of three kernels by max_query_len: 1, 2 to 4, more.  The tolerances are those of
test_gpu_sparse, whose checks are used.
"""

import numpy as np
import pytest
import torch

import test_gpu_append_rope as A
import test_gpu_sparse as S
from gpu_util import bits
from oracle import sparse as OS

pytestmark = pytest.mark.gpu

BAD_BLOCK, BAD_SEQ_LEN = 4, 6
NAMES = ("kc", "vc", "k_min", "k_max")


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def _batch(most, Hq=40, H=3):
    """Three sequences in blocks of 8; the middle one's new tokens lie in several blocks, if they are
    several."""
    news = {1: [1, 1, 1], 3: [3, 2, 1], 30: [30, 25, 3]}[most]
    return A.make(most, [40, 41, 33], news, Hq, H, 64, 64, 8, torch.float16)


def _run(B, st, most, **kw):
    out = torch.full_like(st["q"], 7)
    rec = B.new_error_record()
    args = dict(k_min=st["k_min"], k_max=st["k_max"], q_out=out, error_record=rec)
    args.update(kw)
    B.kv_cache_append_rope(st["q"], st["k"], st["v"], A.dev(st["start"]), most, st["kc"], st["vc"],
                           A.dev(st["tables"]), A.dev(st["lens"]), st["cos_sin"], **args)
    return out, B.pa_error_read(rec)


@pytest.mark.parametrize("value", [10 ** 6, -7])
@pytest.mark.parametrize("most,entry", [(1, 5), (3, 4), (3, 5), (30, 2), (30, 4), (30, 5)])
def test_a_bad_block_number_leaves_out_its_tile_alone(B, most, entry, value):
    st, ref = _batch(most), _batch(most)
    want, clean = _run(B, ref, most)
    assert clean == [0, 0, 0, 0]
    before = {k: bits(st[k]).copy() for k in NAMES}
    block = int(st["tables"][1, entry])
    st["tables"][1, entry] = value
    out, rec = _run(B, st, most)
    assert rec == [BAD_BLOCK, 1, 1, value]                    # once for the tile
    assert np.array_equal(bits(out), bits(want))              # queries need no block
    others = np.arange(len(st["kc"])) != block
    for k in NAMES:
        got = bits(st[k])
        assert np.array_equal(got[others], bits(ref[k])[others]), k
        assert np.array_equal(got[block], before[k][block]), k


@pytest.mark.parametrize("most", [1, 3, 30])
@pytest.mark.parametrize("length", [-3, 0, 6 * 8 + 1])
def test_a_bad_length_leaves_out_its_sequence_alone(B, most, length):
    st, ref = _batch(most), _batch(most)
    want, _ = _run(B, ref, most)
    before = {k: bits(st[k]).copy() for k in NAMES}
    st["lens"][1] = length
    out, rec = _run(B, st, most)
    assert rec == [BAD_SEQ_LEN, 1, 1, length]
    mine = slice(int(st["start"][1]), int(st["start"][2]))
    assert bool((out[mine] == 7).all())
    rest = np.ones(len(out), bool)
    rest[mine] = False
    assert np.array_equal(bits(out)[rest], bits(want)[rest])
    blocks = np.zeros(len(st["kc"]), bool)
    blocks[st["tables"][1][st["tables"][1] >= 0]] = True
    for k in NAMES:
        got = bits(st[k])
        assert np.array_equal(got[~blocks], bits(ref[k])[~blocks]), k
        assert np.array_equal(got[blocks], before[k][blocks]), k


@pytest.mark.parametrize("most", [1, 3, 30])
def test_bad_ranges_are_recorded_once_each(B, most):
    """More new tokens than promised, than the sequence has, and a range behind the last token; over
    200 sequences, so that more than one thread block checks them."""
    N = 300
    news = np.full(N, 1)
    news[5], lens = most + 1, np.full(N, 64)
    lens[200] = 0
    st = A.make(3, np.full(N, 64), news, 2, 1, 16, 16, 16, torch.bfloat16)
    st["lens"] = lens.astype(np.int32)
    st["start"][N] += 1                                       # the last one: beyond the tokens
    before = {k: bits(st[k]).copy() for k in NAMES}
    out, rec = _run(B, st, most)
    assert rec[0] == BAD_SEQ_LEN and rec[1] == 3 and rec[2] in (5, 200, N - 1)
    bad = [5, 200, N - 1]
    for i in bad:
        assert bool((out[int(st["start"][i]):int(st["start"][i + 1])] == 7).all())
        for k in NAMES:
            at = st["tables"][i]
            assert np.array_equal(bits(st[k])[at], before[k][at])
    good = [i for i in range(N) if i not in bad]
    at = st["tables"][good, 3]
    assert torch.equal(st["vc"][at, :, 15], st["v"][st["start"][good]])
    assert not bool((out[st["start"][good]] == 7).all(2).any())


# ------------------------------------------------------------- rows that share a table
@pytest.mark.parametrize("dtype,Hq,H,D,bs", [(torch.bfloat16, 8, 2, 128, 16), (torch.float16, 9, 9, 64, 8),
                                             (torch.bfloat16, 20, 1, 256, 32)])
def test_query_tokens_of_one_sequence_as_rows(B, dtype, Hq, H, D, bs):
    """Drafted tokens: each a row with the sequence's table and a length of its own, beside another
    sequence's; and each gives what it gives alone."""
    b = S.make(1, [203, 90], Hq, H, D, bs, dtype, wide=1)
    rows, lens = [0, 0, 0, 0, 1, 1, 0], np.array([200, 201, 202, 203, 90, 89, 1], np.int32)
    b["tables"], b["lens"] = b["tables"][rows], lens
    gen = torch.Generator(device="cuda").manual_seed(2)
    b["q"] = torch.randn((len(rows), Hq, D), generator=gen, device="cuda").to(dtype)
    rec = B.new_error_record()
    s = S.scores_of(B, b, error_record=rec)
    S.check_scores(s, b)
    sel = B.paged_block_select(s, S.dev(lens), bs, 4, 1, 1, error_record=rec)
    assert np.array_equal(sel.cpu().numpy(), OS.block_select(s.cpu().numpy(), lens, bs, 4, 1, 1))
    out = S.attend(B, b, sel.cpu().numpy(), error_record=rec)
    S.check_attention(out, b, sel.cpu().numpy())
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    for i in range(len(rows)):
        one = dict(b, tables=b["tables"][i:i + 1], lens=lens[i:i + 1], q=b["q"][i:i + 1])
        assert torch.equal(S.scores_of(B, one), s[i:i + 1])
        S.check_attention(S.attend(B, one, sel[i:i + 1].cpu().numpy()), one, sel[i:i + 1].cpu().numpy())


def test_forks_of_one_prefix(B):
    """Sequences whose tables begin with the same blocks and end in blocks of their own."""
    bs, lens = 16, np.array([100, 100, 97], np.int32)
    b = S.make(5, lens, 8, 2, 128, bs, torch.bfloat16)
    b["tables"][1:, :6] = b["tables"][0, :6]
    s = S.scores_of(B, b)
    S.check_scores(s, b)
    assert torch.equal(S.scores_of(B, dict(b, q=b["q"][:1].expand(3, -1, -1).contiguous()))[..., :6],
                       s[:1, :, :6].expand(3, -1, -1))
    sel = S.lists(np.random.default_rng(0), b, 5)
    S.check_attention(S.attend(B, b, sel), b, sel)


# ------------------------------------------------------------------ the same bits
@pytest.mark.parametrize("N,lens,Hq,H,keep", [(70, 3000, 16, 2, 64),      # a thread block a row
                                              (2, 3000, 16, 2, 64),       # a cluster a row
                                              (1, 9000, 8, 1, 500)])      # several clusters a row
def test_the_same_bits_on_every_run(B, N, lens, Hq, H, keep):
    D, bs = 128, 16
    rng = np.random.default_rng(N)
    b = S.make(40, np.maximum(rng.integers(lens // 2, lens, N), 1), Hq, H, D, bs, torch.bfloat16)
    width, n = b["tables"].shape[1], S.dev(b["lens"])
    assert (B.paged_attn_sparse_workspace_needed(N, Hq, H, D, bs, width, keep) > 0) == (keep == 500)
    first = None
    for _ in range(20):
        s = S.scores_of(B, b)
        sel = B.paged_block_select(s, n, bs, keep, 1, 2)
        out = S.attend(B, b, sel.cpu().numpy())
        lo, hi = torch.zeros_like(b["lo"]), torch.zeros_like(b["hi"])
        B.kv_block_bounds(b["kc"], S.dev(b["tables"]), n, lo, hi)
        now = [s.view(torch.int32), sel, out.view(torch.int32), lo.view(torch.int16), hi.view(torch.int16)]
        if first is not None:
            assert all(torch.equal(x, y) for x, y in zip(first, now))
        first = now


@pytest.mark.parametrize("most", [1, 3, 30])
def test_the_append_gives_the_same_bits_on_every_run(B, most):
    first = None
    for _ in range(20):
        st = _batch(most, 7, 7)
        out, rec = _run(B, st, most)
        now = [out] + [st[k] for k in NAMES]
        if first is not None:
            assert all(np.array_equal(bits(x), bits(y)) for x, y in zip(first, now))
        first = now
