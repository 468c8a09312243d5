"""kv_cache_evict where lists have places without an entry, entries that are refused and rows that are left
out, over blocks that forks hold too: bit for bit what oracle.evict moves."""

import numpy as np
import pytest
import torch

import test_gpu_evict as E
import test_gpu_sparse as S

pytestmark = pytest.mark.gpu

BAD_BLOCK, BAD_POSITION = 4, 12


@pytest.fixture(scope="module")
def B(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def forked(B, keep, bs=16, H=2, D=64, blocks=80):
    """Sequences 0, 1 (a fork that has grown) and 2 of which the first two are cut to `keep` tokens; 3 and 4
    are forks of 0 and 2 that are not listed.  Every block holds something."""
    alloc = B.BlockAllocator(blocks, bs, np.random.default_rng(0).permutation(blocks))
    alloc.add(0, 100)
    alloc.fork(0, 1)
    alloc.add(2, 50)
    alloc.fork(0, 3)
    alloc.fork(2, 4)
    slots, pairs = alloc.batch_append([1])
    gen = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn((blocks, H, bs, D), generator=gen, device="cuda").half() for _ in range(2))
    B.block_copy([kc], [vc], torch.from_numpy(pairs).cuda())
    tables, lens = alloc.batch_block_tables([0, 1, 2], 110 // bs + 1)
    alloc.batch_evict([0, 1, 2], keep)
    new, _ = alloc.batch_block_tables([0, 1, 2], 110 // bs + 1)
    assert np.array_equal(new[2], tables[2])            # of at most `keep` tokens: as it was, its fork's too
    return dict(kc=kc, vc=vc, tables=tables, lens=lens, bs=bs, H=H), new


@pytest.mark.parametrize("bs", [1, 8, 16])
@pytest.mark.parametrize("holes", [0.2, 1.0])
def test_places_without_an_entry_keep_their_rows_in_fresh_blocks(B, bs, holes):
    b, new = forked(B, 60, bs=bs, blocks=80 * 16 // bs)
    rng = np.random.default_rng(bs)
    kept = E.pick(rng, b["lens"], 2, 60)
    kept[rng.random(kept.shape) < holes] = -1
    E.check_evict(B, b, kept, new_tables=new)


def test_a_refused_entry_keeps_its_row_in_a_fresh_block(B):
    b, new = forked(B, 60)
    kept = E.pick(np.random.default_rng(4), b["lens"], 2, 60)
    kept[0, 1, 7] = 200                                 # past the last token
    E.check_evict(B, b, kept, new_tables=new, expect=(BAD_POSITION, 1, 1, 200), skip=[(0, 1, 7)])


def test_rows_that_a_fork_reads_are_not_moved(B):
    """Sequence 2 keeps its table, which sequence 4 holds too: a list that would move rows in it is refused."""
    b, new = forked(B, 60)
    kept = E.pick(np.random.default_rng(5), b["lens"], 2, 60)
    assert np.array_equal(kept[2, 1, :50], np.arange(50))
    kept[2, 1, 20] = 21
    E.check_evict(B, b, kept, new_tables=new, expect=(BAD_POSITION, 1, 5, 21), skip=[(2, 1, 20)])
    # in place, where the caller holds the blocks alone, the same list moves the row
    b, _ = forked(B, 60)
    own = {k: (v[2:] if k in ("tables", "lens") else v) for k, v in b.items()}
    E.check_evict(B, own, kept[2:])


@pytest.mark.parametrize("seed", range(12))
def test_random_lists_into_blocks_of_their_own(B, seed):
    """Lists with holes, one sequence shorter than the list, into tables of which some blocks stay."""
    rng = np.random.default_rng(1200 + seed)
    H, D, bs = int(rng.choice([1, 3, 40])), int(rng.choice([8, 64, 128])), int(rng.choice([1, 8, 16, 48]))
    lens = rng.integers(1, 900, 4).astype(np.int32)
    K = int(rng.choice([5, 129, 400, 1000]))
    b = S.make(1300 + seed, lens, H, H, D, bs, torch.bfloat16, wide=int(rng.integers(0, 3)))
    kept = E.pick(rng, lens, H, K)
    kept[rng.random(kept.shape) < 0.3] = -1
    own, total = -(-min(K, int(lens.max())) // bs), len(b["kc"])
    fresh = rng.permutation(len(lens) * own).reshape(len(lens), own).astype(np.int32) + total
    for k in ("kc", "vc"):
        more = torch.full((len(lens) * own, *b[k].shape[1:]), 9, dtype=b[k].dtype, device="cuda")
        b[k] = torch.cat([b[k], more])
    held = b["tables"][:, :own]
    new = np.where((rng.random(fresh.shape) < 0.3) & (held >= 0), held, fresh)
    E.check_evict(B, b, kept, new_tables=new, weights=bool(seed % 4))


@pytest.mark.parametrize("bs", [1, 8, 16])
def test_sequences_cut_to_lengths_of_their_own(B, bs):
    """Lists of one width, padded with -1: the places behind a sequence's new end have no block, and no need of
    one, though the sequence had fewer tokens than the list has room for."""
    blocks = 800 // bs
    alloc = B.BlockAllocator(blocks, bs, np.random.default_rng(0).permutation(blocks))
    lens, keeps = [100, 50, 70, 90], [64, 20, 70, 33]
    for i, n in enumerate(lens[:3]):
        alloc.add(i, n)
    alloc.fork(0, 3)
    alloc.free(3)
    alloc.add(3, lens[3])
    alloc.fork(2, 4)                                    # of which 2 keeps all it has
    alloc.fork(1, 5)
    gen = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn((blocks, 2, bs, 64), generator=gen, device="cuda").half() for _ in range(2))
    width = 110 // bs + 1
    tables, held = alloc.batch_block_tables(range(4), width)
    for i, keep in enumerate(keeps):
        alloc.batch_evict([i], keep)
    new, after = alloc.batch_block_tables(range(4), width)
    assert held.tolist() == lens and after.tolist() == keeps and np.array_equal(new[2], tables[2])
    rng = np.random.default_rng(bs)
    kept = np.full((4, 2, 80), -1, np.int32)
    for i, keep in enumerate(keeps):
        kept[i, :, :keep] = E.pick(rng, lens[i:i + 1], 2, keep)[0]
    E.check_evict(B, dict(kc=kc, vc=vc, tables=tables, lens=held, bs=bs, H=2), kept, new_tables=new)


def left_out(B, tables, kept, new=None, bad=10 ** 6):
    """A call with a block out of range, and what is to come of it: rows and weights that it leaves out are
    as they were."""
    b = S.make(67, [64], 1, 1, 64, 16, torch.float16)
    k, w = E.bits(b["kc"]).copy(), E.place(b)
    before = w.cpu().numpy().copy()
    t = b["tables"].copy()
    t[0, tables] = bad
    if new is not None:
        new = np.array([[b["tables"][0, n] if n is not None else bad for n in new]], np.int32)
    rec = B.new_error_record()
    B.kv_cache_evict(b["kc"], b["vc"], E.dev(t), E.dev([64]), E.dev(kept[None, None]), weights=w, error_record=rec,
                     new_tables=None if new is None else E.dev(new))
    return B.pa_error_read(rec), k, E.bits(b["kc"]), before[0, 0], w.cpu().numpy()[0, 0], b["tables"][0]


def test_a_weight_stays_where_its_row_is_left_out(B):
    # places 32 to 47, which 0 to 15 are to take, sit in the bad block
    rec, k, after, before, w, t = left_out(B, [2], np.arange(32, 64))
    assert rec == [BAD_BLOCK, 16, 0, 10 ** 6]
    assert np.array_equal(after[t[0]], k[t[0]]) and np.array_equal(after[t[1]], k[t[3]])
    assert np.array_equal(w[:16], before[:16]) and np.array_equal(w[16:32], before[48:64])
    assert not w[32:64].any()
    # the new places 16 to 31 have no block
    rec, k, after, before, w, t = left_out(B, [], np.arange(32, 64), new=[0, None])
    assert rec == [BAD_BLOCK, 16, 0, 10 ** 6]
    assert np.array_equal(after[t[0]], k[t[2]]) and np.array_equal(after[t[1:]], k[t[1:]])
    assert np.array_equal(w[:16], before[32:48]) and np.array_equal(w[16:32], before[16:32])
    assert not w[32:64].any()
