"""Refusals of the grouped chunk attention, the attention weights and the eviction on the host, and the
allocator's part of an eviction (no GPU needed)."""

import numpy as np
import pytest
import torch

from oracle.allocator_model import AllocatorError, BlockAllocatorModel

P = 1 << 20                       # never dereferenced: every call below fails its checks first
INV, UNS, OK = 1, 2, 0


@pytest.fixture(scope="module")
def binding(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def test_chunk_refuses(lib):
    def call(**kw):
        a = dict(q=P, start=P, T=64, most=8, kc=P, vc=P, bt=P, sl=P, N=4, Hq=8, H=2, D=64, bs=16, MB=4, B=64,
                 scale=0.125, dt=0, out=P, odt=2, lse=P, order=None, ws=None, wsb=0, err=None, stream=None)
        a.update(kw)
        return lib.paged_attn_chunk(*a.values())

    assert call(N=0) == call(T=0) == call(most=0) == OK
    for kw in (dict(N=-1), dict(T=-1), dict(most=-1), dict(Hq=0), dict(H=0), dict(Hq=7), dict(bs=0), dict(MB=0),
               dict(B=0), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(MB=1 << 28),
               dict(B=1 << 27), dict(N=1 << 20, most=1 << 16), dict(q=None), dict(start=None), dict(kc=None),
               dict(vc=None), dict(bt=None), dict(sl=None), dict(out=None), dict(q=P + 8), dict(kc=P + 8),
               dict(vc=P + 8), dict(out=P + 8), dict(ws=P + 8, wsb=1 << 30)):
        assert call(**kw) == INV, kw
    for kw in (dict(D=96), dict(dt=2), dict(odt=3), dict(bs=24), dict(bs=4), dict(Hq=258)):
        assert call(**kw) == UNS, kw
    # few sequences with long tables: no workspace, and one that is a byte short
    long = dict(N=1, MB=4096, B=8192)
    size, needed = lib.paged_attn_chunk_workspace_size, lib.paged_attn_chunk_workspace_needed
    need = needed(1, 8, 2, 64, 16, 4096, 8)
    assert need == size(1, 8, 2, 64, 16, 4096, 8) == size(500, 8, 2, 64, 16, 4096, 800) > 0
    assert call(**long) == INV and call(ws=P, wsb=need - 1, **long) == INV
    assert needed(500, 8, 2, 64, 16, 4096, 800) == needed(1, 8, 2, 64, 16, 32, 8) == size(1, 8, 2, 64, 16, 32, 8) == 0
    assert size(0, 8, 2, 64, 16, 4096, 8) == size(1, 7, 2, 64, 16, 4096, 8) == size(1, 8, 2, 96, 16, 4096, 8) == 0


def test_chunk_weights_refuse(lib):
    def call(**kw):
        a = dict(q=P, lse=P, start=P, T=64, most=8, kc=P, bt=P, sl=P, N=4, Hq=8, H=2, D=64, bs=16, MB=4, B=64,
                 scale=0.125, dt=0, window=0, w=P, room=64, err=None, stream=None)
        a.update(kw)
        return lib.paged_chunk_weights(*a.values())

    assert call(N=0) == call(T=0) == call(most=0) == OK
    for kw in (dict(N=-1), dict(T=-1), dict(most=-1), dict(window=-1), dict(Hq=0), dict(H=0), dict(Hq=7), dict(bs=0),
               dict(MB=0), dict(B=0), dict(scale=float("nan")), dict(MB=1 << 28), dict(room=63), dict(N=65536),
               dict(B=1 << 27), dict(N=60000, MB=1 << 18, room=1 << 22), dict(q=None), dict(lse=None),
               dict(start=None), dict(kc=None), dict(bt=None), dict(sl=None), dict(w=None), dict(q=P + 8),
               dict(kc=P + 8)):
        assert call(**kw) == INV, kw
    for kw in (dict(D=96), dict(dt=2), dict(bs=24), dict(bs=4), dict(Hq=258)):
        assert call(**kw) == UNS, kw


def test_decode_refuses(lib):
    def call(**kw):
        a = dict(q=P, kc=P, vc=P, bt=P, sl=P, N=4, Hq=8, H=2, D=64, bs=16, MB=4, B=64, scale=0.125, dt=0, out=P,
                 odt=2, w=P, room=64, ws=None, wsb=0, err=None, stream=None)
        a.update(kw)
        return lib.paged_attn_decode_weights(*a.values())

    assert call(N=0) == OK
    for kw in (dict(N=-1), dict(Hq=0), dict(H=0), dict(Hq=7), dict(bs=0), dict(MB=0), dict(B=0), dict(room=63),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(N=65536), dict(MB=1 << 28), dict(B=1 << 27),
               dict(q=None), dict(kc=None), dict(vc=None), dict(bt=None), dict(sl=None), dict(out=None), dict(w=None),
               dict(q=P + 8), dict(kc=P + 8), dict(vc=P + 8), dict(out=P + 8), dict(ws=P + 8, wsb=1 << 30)):
        assert call(**kw) == INV, kw
    for kw in (dict(D=96), dict(dt=2), dict(odt=3), dict(bs=24), dict(bs=4)):
        assert call(**kw) == UNS, kw
    long = dict(N=1, MB=4096, B=8192, room=65536)
    need = lib.paged_attn_decode_weights_workspace_needed(1, 8, 2, 64, 16, 4096)
    assert need == lib.paged_attn_decode_weights_workspace_size(1, 8, 2, 64, 16, 4096) > 0
    assert call(**long) == INV and call(ws=P, wsb=need - 1, **long) == INV


def test_evict_refuses(lib):
    def call(**kw):
        a = dict(kc=P, vc=P, bt=P, nt=None, sl=P, kept=P, K=8, w=P, room=64, N=4, H=2, D=64, bs=16, MB=4, NB=0, B=64,
                 dt=0, err=None, stream=None)
        a.update(kw)
        return lib.kv_cache_evict(*a.values())

    assert call(N=0) == OK
    for kw in (dict(N=-1), dict(H=0), dict(D=0), dict(bs=0), dict(MB=0), dict(B=0), dict(K=0), dict(K=-1),
               dict(nt=P, NB=0), dict(N=65536), dict(MB=1 << 28), dict(room=63), dict(kc=None), dict(vc=None),
               dict(bt=None), dict(sl=None), dict(kept=None), dict(kc=P + 8), dict(vc=P + 8)):
        assert call(**kw) == INV, kw
    for kw in (dict(D=60), dict(D=1032), dict(dt=2)):
        assert call(**kw) == UNS, kw


def test_workspace_sizes_never_fall(lib):
    size = lib.paged_attn_decode_weights_workspace_size
    needed = lib.paged_attn_decode_weights_workspace_needed
    for heads, kv, dim in ((8, 8, 64), (32, 8, 128), (64, 2, 256), (16, 1, 128)):
        for bs in (8, 16, 64):
            last = 0
            for n in (1, 2, 3, 5, 9, 30, 64, 65, 200, 1000):
                assert size(n, heads, kv, dim, bs, 500) >= last
                last = size(n, heads, kv, dim, bs, 500)
                assert needed(n, heads, kv, dim, bs, 500) in (0, last)
                assert size(n, heads, kv, dim, bs, 499) <= last <= size(n, heads, kv, dim, 2 * bs, 500)
    assert size(0, 8, 2, 64, 16, 64) == size(1, 7, 2, 64, 16, 64) == size(1, 8, 2, 96, 16, 64) == 0


def test_sizes_that_never_need_a_workspace(lib):
    """What the binding relies on where it does not ask."""
    for n in (1, 2, 7, 100, 1000, 65535):
        for kv in (1, 2, 8, 40):
            for dim in (64, 128, 256):
                for bs, mb in ((8, 128), (16, 64), (64, 16), (16, 1)):
                    for group in (1, 3, 8):
                        assert lib.paged_attn_decode_weights_workspace_needed(n, kv * group, kv, dim, bs, mb) == 0
                    assert lib.paged_attn_chunk_workspace_needed(n, kv, kv, dim, bs, mb // 2 or 1, 5) == 0


def test_the_binding_refuses_tensors_that_are_not_on_the_gpu(binding, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    h = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    i = torch.zeros(4, 4, dtype=torch.int32)
    w = torch.zeros(4, 2, 64)
    for call in (lambda: binding.paged_attn_chunk(h[:, :, 0], i[0], 1, h, h, i, i[0], 1.0),
                 lambda: binding.paged_chunk_weights(h[:, :, 0], w[:, :, 0], i[0], 1, h, i, i[0], 1.0, w),
                 lambda: binding.paged_attn_decode_weights(h[:, :, 0], h, h, i, i[0], 1.0, w),
                 lambda: binding.kv_cache_evict(h, h, i, i[0], i[None])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_the_binding_refuses_weights_that_are_too_short(binding):
    with pytest.raises(ValueError, match="at least 64"):
        binding._weights(torch.zeros(4, 2, 63), 0, (4, 2), 64)
    with pytest.raises(ValueError, match="at least 64"):
        binding._weights(torch.zeros(4, 64), 0, (4, 2), 64)


# --------------------------------------------------------------------- the allocator
def evict(model, seqs, keep):
    """The model's part: blocks that others hold when the call begins are replaced, fresh ones first."""
    if len(set(seqs)) < len(seqs) or any(s not in model.tables for s in seqs):
        raise AllocatorError("missing or twice")
    bs = model.block_size
    count = list(model.refcount)
    nb = -(-keep // bs)
    cut = [s for s in seqs if model.lens[s] > keep]
    swaps = [(s, j) for s in cut for j in range(nb) if count[model.tables[s][j]] > 1]
    if len(swaps) > len(model.free):
        raise AllocatorError("out of blocks")
    old = []
    for s, j in swaps:
        old.append(model.tables[s][j])
        model.tables[s][j] = model._take()
    for b in old:
        model._release(b)
    for s in cut:
        while len(model.tables[s]) > nb:
            model._release(model.tables[s].pop())
        model.lens[s] = keep


@pytest.mark.parametrize("seed", range(4))
def test_batch_evict_matches_the_model(lib, binding, seed):
    rng = np.random.default_rng(seed)
    nb, bs = 150, int(rng.choice([1, 4, 16]))
    order = rng.permutation(nb)
    cpp, model = binding.BlockAllocator(nb, bs, order), BlockAllocatorModel(nb, bs, order)
    fresh, refused = 0, 0
    for step in range(200):
        live = list(model.tables)
        op = int(rng.integers(0, 4))
        if op == 0 or not live:
            n = int(rng.integers(0, 12 * bs))
            if -(-n // bs) <= len(model.free):
                cpp.add(fresh, n)
                model.add(fresh, n)
                fresh += 1
        elif op == 1:
            p = int(rng.choice(live))
            cpp.fork(p, fresh)
            model.fork(p, fresh)
            fresh += 1
        elif op == 2 and len(live) > 6:
            s = int(rng.choice(live))
            cpp.free(s)
            model.free_seq(s)
        else:
            seqs = [int(x) for x in rng.permutation(live)[:int(rng.integers(0, 5))]]
            keep = int(rng.integers(1, 8 * bs))
            before = {s: list(model.tables[s]) for s in model.tables}
            try:
                evict(model, seqs, keep)
            except AllocatorError:
                refused += 1
                with pytest.raises(binding.PagedKVError, match="OOM"):
                    cpp.batch_evict(seqs, keep)
            else:
                cpp.batch_evict(seqs, keep)
                held = {b for s in before for b in before[s]}
                for s in seqs:              # a new place's block: its own of that place, or nobody's
                    for j, b in enumerate(model.tables[s]):
                        assert b == before[s][j] or b not in held
        cpp.check()
        model.check()
        for s in model.tables:
            assert cpp.block_table(s) == model.tables[s] and cpp.length(s) == model.lens[s]
        assert cpp.num_free() == len(model.free)


def test_batch_evict_is_all_or_nothing(binding):
    a = binding.BlockAllocator(10, 4)
    a.add(0, 16)
    a.fork(0, 1)
    a.add(2, 20)                            # one block left; evicting 0 and 1 needs two
    before = [a.block_table(s) for s in range(3)]
    for seqs, keep, code in (([0, 1], 4, "OOM"), ([0, 9], 4, "NO_SEQ"), ([2, 2], 4, "NO_SEQ"),
                             ([2], 0, "INVALID_ARG"), ([2], -1, "INVALID_ARG")):
        with pytest.raises(binding.PagedKVError, match=code):
            a.batch_evict(seqs, keep)
        assert [a.block_table(s) for s in range(3)] == before and a.num_free() == 1
    a.batch_evict([0], 4)                   # takes the free block, gives none back: 1 holds them
    assert a.num_free() == 0 and a.block_table(1) == before[1] and a.length(0) == 4
    a.batch_evict([], 4)
    a.batch_evict([0, 1, 2], 20)            # nothing is longer
    a.batch_evict([1, 2], 3)
    assert a.num_free() == 7 and a.length(1) == a.length(2) == 3
    a.check()


def test_the_example_is_the_one_shown():
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = open(os.path.join(root, "paged_kv_cache_317_gb300", "examples", "bounded_step.py")).read()
    body = code.split('"""', 2)[2].strip()
    assert body in open(os.path.join(root, "README.md")).read()
