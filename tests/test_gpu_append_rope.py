"""kv_cache_append_rope and kv_block_bounds on the GPU against the fp64 oracle.

Tolerance of a rotated value x' = x c - y s in the storage type: half a step of the type
at the result (one rounding at the end), plus the fp32 roundings of two products and one
difference, each at most 2^-24 of |x c| + |y s|, plus half the smallest step of the type.
Values, unrotated dims, untouched rows and key bounds (of the rows as stored) are exact.
"""

import numpy as np
import pytest
import torch

from gpu_util import bits
from oracle import sparse as OS

pytestmark = pytest.mark.gpu

CODE = {"PA_ERR_BAD_BLOCK": 4, "PA_ERR_BAD_SEQ_LEN": 6, "PA_ERR_BAD_POSITION": 12}


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def f64(t):
    return t.detach().cpu().double().numpy()


def make(seed, lens, news, Hq, H, D, R, bs, dtype, axes=1, interleaved=False, pad=0, reach=None):
    """A batch on the GPU with NaN in every row that holds no token yet."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
    lens, news = np.asarray(lens, np.int32), np.asarray(news, np.int32)
    N, nb = len(lens), -(-lens // bs)
    MB, total = max(1, int(nb.max())), int(nb.sum()) + 3
    order = rng.permutation(total)
    tables = np.full((N, MB), -1, np.int32)
    tables[np.arange(MB)[None, :] < nb[:, None]] = order[:int(nb.sum())]
    st = {"lens": lens, "news": news, "tables": tables, "bs": bs, "Hq": Hq, "H": H, "D": D, "R": R,
          "interleaved": interleaved, "dtype": dtype, "start": np.concatenate([[0], np.cumsum(news)])}
    T = int(news.sum()) + pad
    st["q"], st["k"], st["v"] = randn(T, Hq, D), randn(T, H, D), randn(T, H, D)
    live = np.zeros((total, bs), bool)
    for i in range(N):
        for t in range(int(lens[i] - news[i])):
            live[tables[i, t // bs], t % bs] = True
    dead = torch.from_numpy(~live).cuda()[:, None, :, None]
    st["kc"] = randn(total, H, bs, D).masked_fill(dead, float("nan"))
    st["vc"] = randn(total, H, bs, D).masked_fill(dead, float("nan"))
    held = torch.from_numpy(live).cuda()[:, None, :, None]
    inf = float("inf")
    st["k_min"] = st["kc"].float().masked_fill(~held, inf).amin(2).to(dtype)
    st["k_max"] = st["kc"].float().masked_fill(~held, -inf).amax(2).to(dtype)
    reach = reach or max(64, int(lens.max()))
    st["cos_sin"] = None
    if R:
        angles = np.arange(reach)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
        st["cos_sin"] = torch.from_numpy(np.concatenate([np.cos(angles), np.sin(angles)], 1)
                                         .astype(np.float32)).cuda()
    st["positions"] = st["pair_axis"] = None
    if axes > 1:
        st["positions"] = torch.from_numpy(rng.integers(0, reach, (axes, T)).astype(np.int32)).cuda()
        st["pair_axis"] = [int(x) for x in rng.integers(0, axes, R // 2)]
    return st


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def call(B, st, q=True, bounds=True, **kw):
    a = dict(interleaved=st["interleaved"], positions=st["positions"], pair_axis=st["pair_axis"])
    if bounds:
        a.update(k_min=st["k_min"], k_max=st["k_max"])
    a.update(kw)
    return B.kv_cache_append_rope(st["q"] if q is True else q, st["k"], st["v"], dev(st["start"]),
                                  int(st["news"].max(initial=0)), st["kc"], st["vc"],
                                  dev(st["tables"]), dev(st["lens"]), st["cos_sin"], **a)


def near(got, x, ref, st, place_pos, what):
    """got within the stated tolerance of ref = rotate(x)."""
    if not st["R"]:
        assert np.array_equal(got, ref), what
        return
    table = np.abs(f64(st["cos_sin"]))
    size = np.zeros_like(ref)
    half = st["R"] // 2
    pos = np.atleast_2d(place_pos)
    for j in range(half):
        at = pos[0 if st["pair_axis"] is None else st["pair_axis"][j]]
        c, s = table[at, j][:, None], table[at, half + j][:, None]
        d0, d1 = (2 * j, 2 * j + 1) if st["interleaved"] else (j, j + half)
        a, b = np.abs(x[..., d0]), np.abs(x[..., d1])
        size[..., d0], size[..., d1] = a * c + b * s, b * c + a * s
    eps = torch.finfo(st["dtype"]).eps
    tiny = 2.0 ** -25 if st["dtype"] == torch.float16 else 0.0
    bound = (eps / 2) * (np.abs(ref) + 2.0 ** -22 * size) + 2.0 ** -22 * size + tiny
    bad = ~(np.abs(got - ref) <= bound)
    bad &= size > 0
    assert not bad.any(), (what, np.abs(got - ref).max())
    same = size == 0
    assert np.array_equal(got[same], ref[same]), what


def check(B, st, q_out, before):
    """q_out, caches and bounds of st after a call against the oracle."""
    places = OS.new_places(st["start"], st["lens"])
    rows = np.array([t for t, _, _ in places], int)
    place = np.array([p for _, _, p in places], int)
    pos = place if st["positions"] is None else st["positions"].cpu().numpy()[..., rows]
    turn = lambda x: OS.rotate(x, f64(st["cos_sin"]), pos, st["pair_axis"], st["interleaved"]) \
        if st["R"] else x
    if q_out is not None:
        x = f64(st["q"])[rows]
        near(f64(q_out)[rows], x, turn(x), st, pos, "q")
    kc, vc = f64(st["kc"]), f64(st["vc"])
    blk = np.array([st["tables"][i, p // st["bs"]] for _, i, p in places], int)
    row = place % st["bs"]
    x = f64(st["k"])[rows]
    near(kc[blk, :, row], x, turn(x), st, pos, "k")
    assert np.array_equal(vc[blk, :, row], f64(st["v"])[rows])
    kept = np.ones(kc.shape[0:1] + kc.shape[2:3], bool)
    kept[blk, row] = False
    for name in ("kc", "vc"):
        assert np.array_equal(np.moveaxis(bits(st[name]), 2, 1)[kept],
                              np.moveaxis(before[name], 2, 1)[kept]), name
    # bounds: exact over the rows as stored
    lo, hi = before["k_min"].astype(np.float64), before["k_max"].astype(np.float64)
    OS.block_bounds(kc, st["tables"], st["lens"], lo, hi, st["lens"] - st["news"])
    for i in np.flatnonzero(st["news"] == 0):   # nothing new: nothing touched
        for b in st["tables"][i][:-(-int(st["lens"][i]) // st["bs"])]:
            lo[b], hi[b] = before["k_min"][b], before["k_max"][b]
    assert np.array_equal(f64(st["k_min"]), lo, equal_nan=True)
    assert np.array_equal(f64(st["k_max"]), hi, equal_nan=True)


def snapshot(st):
    return {"kc": bits(st["kc"]).copy(), "vc": bits(st["vc"]).copy(),
            "k_min": f64(st["k_min"]).copy(), "k_max": f64(st["k_max"]).copy()}


CASES = [
    # lens, news, Hq, H, D, R, bs, axes, interleaved
    ([1], [1], 4, 1, 64, 64, 16, 1, False),
    ([17, 1, 33, 16, 200], [1, 1, 1, 1, 1], 8, 8, 128, 128, 16, 1, False),
    ([40, 7, 100, 5, 31], [40, 3, 37, 0, 1], 8, 2, 128, 64, 16, 1, True),
    ([40, 7, 100, 5, 31], [39, 3, 100, 0, 30], 6, 3, 64, 32, 8, 3, False),
    ([65, 130], [65, 2], 5, 1, 256, 256, 32, 2, True),
    ([9, 50, 3], [9, 20, 3], 3, 3, 48, 16, 5, 1, False),
    ([300], [299], 4, 2, 128, 128, 64, 4, False),
    ([20, 21], [4, 21], 2, 2, 16, 16, 1, 1, False),
    ([17, 4, 33, 64, 200], [2, 4, 0, 3, 1], 6, 2, 128, 64, 16, 3, False),   # a few tokens each
    ([9, 5, 3], [3, 3, 2], 40, 5, 64, 64, 2, 1, True),
    ([700, 130], [600, 130], 3, 2, 64, 32, 500, 1, False),                  # long blocks
    ([2500], [2400], 1, 1, 32, 32, 2100, 1, True),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[2:7])))
def test_matches_the_oracle(B, case, dtype):
    lens, news, Hq, H, D, R, bs, axes, inter = case
    st = make(len(lens) + D, lens, news, Hq, H, D, R, bs, dtype, axes, inter)
    before, rec = snapshot(st), B.new_error_record()
    out = call(B, st, error_record=rec)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    check(B, st, out, before)


def test_many_sequences_of_mixed_lengths(B):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 90, 300)
    news = np.minimum(lens, rng.integers(0, 40, 300))
    st = make(6, lens, news, 4, 2, 64, 64, 16, torch.bfloat16)
    before, rec = snapshot(st), B.new_error_record()
    out = call(B, st, error_record=rec)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    check(B, st, out, before)


@pytest.mark.parametrize("Hq,H,D,bs", [(12, 10, 16, 8), (40, 3, 32, 16), (33, 33, 16, 4)])
def test_large_batches_of_prompts(B, Hq, H, D, bs):
    """Enough tiles that a thread block takes all of its 32 heads."""
    rng = np.random.default_rng(Hq)
    lens = rng.integers(1, 900, 40)
    news = np.maximum(lens - rng.integers(0, 30, 40), 0)
    st = make(Hq, lens, news, Hq, H, D, 16, bs, torch.float16, axes=2)
    before, rec = snapshot(st), B.new_error_record()
    out = call(B, st, error_record=rec)
    assert B.pa_error_read(rec) == [0, 0, 0, 0]
    check(B, st, out, before)


@pytest.mark.parametrize("news", [[1, 1, 1], [1, 30, 7]])
def test_without_rotation_it_is_the_plain_append(B, news):
    st = make(7, [33, 64, 7], news, 4, 4, 64, 0, 16, torch.float16)
    kc, vc = st["kc"].clone(), st["vc"].clone()
    slots = np.array([st["tables"][i, p // 16] * 16 + p % 16
                      for _, i, p in OS.new_places(st["start"], st["lens"])], np.int64)
    B.kv_cache_append(st["k"], st["v"], torch.from_numpy(slots).cuda(), kc, vc)
    out = call(B, st)
    assert np.array_equal(bits(st["kc"]), bits(kc)) and np.array_equal(bits(st["vc"]), bits(vc))
    assert np.array_equal(bits(out), bits(st["q"]))


def test_slices_of_one_projection_and_a_given_output(B):
    st = make(8, [70, 20, 1], [50, 1, 1], 4, 2, 64, 64, 16, torch.bfloat16)
    ref = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in st.items()}
    want = call(B, ref)
    fused = torch.cat([st["q"].flatten(1), st["k"].flatten(1), st["v"].flatten(1),
                       st["q"].flatten(1)], 1)
    sl = fused.split([4 * 64, 2 * 64, 2 * 64, 4 * 64], 1)
    st["q"], st["k"], st["v"] = (x.unflatten(1, (-1, 64)) for x in sl[:3])
    out = torch.empty_like(want)
    assert call(B, st, q_out=out) is out
    for a, b in ((out, want), (st["kc"], ref["kc"]), (st["vc"], ref["vc"]),
                 (st["k_min"], ref["k_min"]), (st["k_max"], ref["k_max"])):
        assert np.array_equal(bits(a), bits(b))


def test_in_place_and_without_queries(B):
    st = make(9, [70, 20, 1], [50, 1, 1], 4, 2, 64, 32, 16, torch.float16)
    ref = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in st.items()}
    want = call(B, ref)
    assert call(B, st, q_out=st["q"]) is st["q"]
    assert np.array_equal(bits(st["q"]), bits(want))
    st["kc"].fill_(0)
    assert call(B, st, q=None, bounds=False) is None
    rows = [(st["tables"][i, p // 16], p % 16) for _, i, p in OS.new_places(st["start"], st["lens"])]
    for b, r in rows:
        assert np.array_equal(bits(st["kc"][b, :, r]), bits(ref["kc"][b, :, r]))


def test_rows_outside_every_sequence_stay(B):
    st = make(10, [40, 20], [6, 20], 4, 2, 64, 64, 16, torch.float16, pad=9)
    st["start"] = st["start"] + 4               # four rows before, five behind
    out = torch.full_like(st["q"], 7)
    call(B, st, q_out=out)
    assert (out[:4] == 7).all() and (out[30:] == 7).all() and not (out[4:30] == 7).all(2).any()
    before = {k: bits(st[k]).copy() for k in ("kc", "vc", "k_min", "k_max")}
    st["news"] = np.zeros(2, np.int32)          # no new token at all
    st["start"] = np.array([0, 0, 0])
    call(B, st, q_out=out)
    assert all(np.array_equal(bits(st[k]), before[k]) for k in before)


def test_bounds_are_combined_within_a_block_and_begin_anew_at_its_first_row(B):
    H, D, bs = 2, 64, 16
    st = make(11, [20], [1], 2, H, D, 0, bs, torch.bfloat16)
    b = int(st["tables"][0, 1])
    st["k_min"][b], st["k_max"][b] = -100, 100
    st["k"].fill_(3)
    call(B, st)
    assert (st["k_min"][b] == -100).all() and (st["k_max"][b] == 100).all()
    st["lens"] = np.array([17], np.int32)       # row 0 of the block
    call(B, st)
    assert (st["k_min"][b] == 3).all() and (st["k_max"][b] == 3).all()
    st["lens"] = np.array([18], np.int32)
    st["k"][0, 0, 5] = float("nan")
    call(B, st)
    assert torch.isnan(st["k_min"][b, 0, 5]) and torch.isnan(st["k_max"][b, 0, 5])
    assert int(torch.isnan(st["k_min"][b].float()).sum()) == 1


def test_bad_indices_are_recorded_and_skipped(B):
    st = make(12, [40, 20, 33], [1, 1, 1], 4, 2, 64, 64, 16, torch.float16)
    st["tables"][1, 1] = 10 ** 6
    before, rec = snapshot(st), B.new_error_record()
    call(B, st, error_record=rec)
    assert B.pa_error_read(rec) == [CODE["PA_ERR_BAD_BLOCK"], 1, 1, 10 ** 6]
    good = [0, 2]
    for i in good:
        b, r = st["tables"][i, (st["lens"][i] - 1) // 16], (st["lens"][i] - 1) % 16
        assert np.array_equal(f64(st["vc"])[b, :, r], f64(st["v"])[i])
    same = np.ones(len(before["vc"]), bool)
    same[[st["tables"][i, (st["lens"][i] - 1) // 16] for i in good]] = False
    assert np.array_equal(bits(st["vc"])[same], before["vc"][same])


@pytest.mark.parametrize("most", [1, 30])
def test_bad_lengths_are_recorded_and_skipped(B, most):
    st = make(13, [40, 20, 33], [1, 1, 1], 4, 2, 64, 64, 16, torch.float16)
    before, rec = snapshot(st), B.new_error_record()
    st["lens"] = np.array([-3, 0, 49], np.int32)   # negative; fewer than the new; over the table
    args = (st["q"], st["k"], st["v"], dev(st["start"]), most, st["kc"], st["vc"],
            dev(st["tables"]), dev(st["lens"]), st["cos_sin"])
    out = torch.full_like(st["q"], 7)
    B.kv_cache_append_rope(*args, k_min=st["k_min"], k_max=st["k_max"], q_out=out, error_record=rec)
    got = B.pa_error_read(rec)
    assert got[0] == CODE["PA_ERR_BAD_SEQ_LEN"] and got[1] == 3
    assert all(np.array_equal(bits(st[k]), before[k]) for k in ("kc", "vc"))
    assert (out == 7).all()
    # more new tokens than promised, and ranges that leave the tokens or decrease
    for start in ([0, 2, 3, 3], [0, 1, 2, 4], [0, -1, 2, 3]):
        B.pa_error_clear(rec)
        st2 = make(13, [40, 20, 33], [1, 1, 1], 4, 2, 64, 64, 16, torch.float16)
        B.kv_cache_append_rope(st2["q"], st2["k"], st2["v"], dev(start), 1, st2["kc"], st2["vc"],
                               dev(st2["tables"]), dev(st2["lens"]), st2["cos_sin"], error_record=rec)
        assert B.pa_error_read(rec)[0] == CODE["PA_ERR_BAD_SEQ_LEN"]


def test_positions_out_of_range_are_recorded_and_kept_in_range(B):
    st = make(14, [40, 20, 33], [1, 2, 3], 4, 2, 64, 64, 16, torch.float16, reach=64)
    st["positions"] = dev([5, 63, 0, 64, -1, 7])
    rec = B.new_error_record()
    out = call(B, st, error_record=rec)
    code, count, index, value = B.pa_error_read(rec)
    assert code == CODE["PA_ERR_BAD_POSITION"] and count == 2 and (index, value) in ((3, 64), (4, -1))
    st["positions"] = dev([5, 63, 0, 63, 0, 7])
    assert np.array_equal(bits(out), bits(call(B, st)))


def test_far_positions_keep_their_angles(B):
    table = B.rope_cos_sin(1 << 17, 64)
    far = (1 << 17) - 1
    angles = far * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    want = np.concatenate([np.cos(angles), np.sin(angles)])
    # the angle itself carries 2^-53 of 131071 radians in 64 bits, the entry half a step of fp32
    assert np.abs(f64(table[far]) - want).max() <= 2.0 ** -25 + 2.0 ** -33


def test_replays_from_a_graph_and_runs_on_another_stream(B):
    st = make(15, [40, 20, 33], [1, 1, 1], 4, 2, 64, 64, 16, torch.bfloat16)
    ref = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in st.items()}
    want = call(B, ref)
    side = torch.cuda.Stream()
    lens, start, tables = dev(st["lens"]), dev(st["start"]), dev(st["tables"])
    out = torch.empty_like(st["q"])
    torch.cuda.synchronize()
    run = lambda **k: B.kv_cache_append_rope(st["q"], st["k"], st["v"], start, 1, st["kc"], st["vc"],
                                             tables, lens, st["cos_sin"], k_min=st["k_min"],
                                             k_max=st["k_max"], **k)
    got = run(stream=side)
    side.synchronize()
    assert np.array_equal(bits(got), bits(want)) and np.array_equal(bits(st["kc"]), bits(ref["kc"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(q_out=out)
    st["q"].copy_(st["q"].flip(0))
    lens.copy_(dev([39, 19, 32]))
    graph.replay()
    ref["q"], ref["lens"] = st["q"], np.array([39, 19, 32], np.int32)
    assert np.array_equal(bits(out), bits(call(B, ref)))
    for k in ("kc", "vc", "k_min", "k_max"):
        assert np.array_equal(bits(st[k]), bits(ref[k]))


def test_copy_on_write_takes_the_bounds_along(B):
    st = make(16, [40], [1], 4, 2, 64, 64, 16, torch.bfloat16)
    pairs = torch.tensor([[int(st["tables"][0, 1]), int(st["tables"][0, 0])], [-1, -1]], device="cuda")
    B.block_copy([st["k_min"][:, :, None]], [st["k_max"][:, :, None]], pairs)
    for x in (st["k_min"], st["k_max"]):
        assert torch.equal(x[int(pairs[0, 0])], x[int(pairs[0, 1])])


# ------------------------------------------------------------------- kv_block_bounds
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,H,D,bs", [([1], 1, 8, 16), ([0, 5, 16, 17, 131], 3, 64, 16),
                                         ([64, 100], 2, 256, 64), ([33, 8], 8, 128, 8),
                                         ([10, 3], 5, 40, 3), ([1000], 1, 128, 1000)])
def test_bounds_match_the_oracle(B, lens, H, D, bs, dtype):
    st = make(sum(lens), lens, [0] * len(lens), 1, H, D, 0, bs, dtype)
    first = np.array([max(0, n - 20) if i % 2 else -1 for i, n in enumerate(lens)], np.int32)
    for f in (None, first):
        lo = torch.full_like(st["k_min"], 9)
        hi = torch.full_like(st["k_max"], 9)
        wlo, whi = f64(lo).copy(), f64(hi).copy()
        rec = B.new_error_record()
        B.kv_block_bounds(st["kc"], dev(st["tables"]), dev(lens), lo, hi,
                          first_token=None if f is None else dev(f), error_record=rec)
        assert B.pa_error_read(rec) == [0, 0, 0, 0]
        OS.block_bounds(f64(st["kc"]), st["tables"], lens, wlo, whi, f)
        assert np.array_equal(f64(lo), wlo) and np.array_equal(f64(hi), whi)


def test_bounds_after_a_rollback_and_of_bad_tables(B):
    st = make(17, [40, 30], [0, 0], 1, 2, 64, 0, 16, torch.float16)
    st["kc"][int(st["tables"][0, 1]), 1, 3, 7] = float("nan")
    st["tables"][1, 0] = -5
    rec = B.new_error_record()
    lo, hi = torch.full_like(st["k_min"], 9), torch.full_like(st["k_max"], 9)
    B.kv_block_bounds(st["kc"], dev(st["tables"]), dev(st["lens"]), lo, hi, error_record=rec)
    assert B.pa_error_read(rec) == [CODE["PA_ERR_BAD_BLOCK"], 1, 1, -5 & 0xffffffff] or \
        B.pa_error_read(rec) == [CODE["PA_ERR_BAD_BLOCK"], 1, 1, -5]
    b = int(st["tables"][0, 1])
    assert torch.isnan(lo[b, 1, 7]) and torch.isnan(hi[b, 1, 7])
    B.pa_error_clear(rec)
    B.kv_block_bounds(st["kc"], dev(st["tables"]), dev([19, 49]), lo, hi, error_record=rec)
    assert B.pa_error_read(rec) == [CODE["PA_ERR_BAD_SEQ_LEN"], 1, 1, 49]
    assert torch.equal(lo[b], st["kc"][b, :, :3].amin(1))   # rows 0 .. 2 alone
