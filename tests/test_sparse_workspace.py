"""The workspace of paged_attn_sparse: a buffer sized for the largest call serves every smaller one."""

import itertools

import numpy as np
import pytest
import torch

P = 1 << 20     # never dereferenced: the calls below fail their checks first
SHAPES = [(8, 1, 128), (16, 1, 64), (17, 1, 256), (32, 8, 128), (8, 2, 64)]


@pytest.fixture(scope="module")
def binding(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


@pytest.mark.parametrize("heads,kv,dim", SHAPES)
@pytest.mark.parametrize("keep", [129, 160, 192, 256, 512, 1000, 8192, 1 << 17])
def test_the_size_never_falls_as_sequences_are_added(binding, heads, kv, dim, keep):
    sizes = [binding.paged_attn_sparse_workspace_size(n, heads, kv, dim, 16, 8192, keep)
             for n in (*range(1, 70), 100, 257, 1000, 65535)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("heads,kv,dim", SHAPES)
def test_the_size_never_falls_with_longer_lists_or_wider_tables(binding, heads, kv, dim):
    for n in (1, 5, 9, 12, 40, 300):
        of = lambda keep, width, bs=16: binding.paged_attn_sparse_workspace_size(n, heads, kv, dim, bs,
                                                                                 width, keep)
        lengths = [1, 100, 128, *range(129, 600, 13), 1000, 4000, 1 << 17]
        for sizes in ([of(k, 1 << 17) for k in lengths], [of(1 << 17, w) for w in lengths],
                      [of(300, 1 << 17, bs) for bs in (8, 16, 32, 48, 64, 256)]):
            assert all(a <= b for a, b in zip(sizes, sizes[1:])), (n, sizes)


@pytest.mark.parametrize("heads,kv,dim", SHAPES)
def test_what_a_call_needs_is_the_size_or_nothing(binding, heads, kv, dim):
    spread = 0
    for n, keep, bs in itertools.product((1, 2, 3, 5, 7, 9, 11, 12, 17, 39, 153, 400, 2000),
                                         (1, 128, 129, 256, 1024, 5000, 1 << 15), (8, 16, 64)):
        a = (n, heads, kv, dim, bs, 1 << 16, keep)
        need, size = binding.paged_attn_sparse_workspace_needed(*a), binding.paged_attn_sparse_workspace_size(*a)
        cols = 8 if heads // kv <= 8 else 16
        rows = n * kv * -(-(heads // kv) // cols)
        assert need in (0, size) and size <= min(64 * rows, 1024) * cols * (dim * 4 + 8)
        if keep * bs <= 2048:
            assert size == 0
        spread += need > 0
    assert spread > 20


def test_sizes_that_no_call_has(binding):
    for a in ((0, 8, 2, 64, 16, 4096, 4096), (1, 7, 2, 64, 16, 4096, 4096), (1, 8, 2, 96, 16, 4096, 4096),
              (1, 8, 2, 64, 16, 4096, 0), (1, 8, 2, 64, 0, 4096, 9), (1, 8, 2, 64, 16, -1, 9)):
        assert binding.paged_attn_sparse_workspace_needed(*a) == 0
        assert binding.paged_attn_sparse_workspace_size(*a) == 0


def test_a_buffer_below_the_size_is_refused_where_a_list_is_spread(lib, binding):
    for n in range(1, 18):
        a = (n, 8, 1, 128, 16, 8192, 512)
        size = binding.paged_attn_sparse_workspace_size(*a)
        if binding.paged_attn_sparse_workspace_needed(*a):
            assert lib.paged_attn_sparse(P, P, P, P, P, P, 512, n, 8, 1, 128, 16, 8192, 1 << 18, 0.1, 1, P, 1,
                                         P, size - 1, None, None) == 1
    assert binding.paged_attn_sparse_workspace_needed(1, 8, 1, 128, 16, 8192, 512) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H,D", [(8, 1, 128), (16, 1, 64), (17, 1, 256), (6, 2, 64)])
def test_one_buffer_serves_a_batch_that_shrinks(binding, Hq, H, D):
    """12 sequences use less at a time than 11, and long lists less than short ones; a buffer made for
    all of them takes each, and what lies behind it stays."""
    B, bs, keep, width = binding, 16, 512, 600
    gen = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    kc, vc, q = randn(3000, H, bs, D), randn(3000, H, bs, D), randn(12, Hq, D)
    rng = np.random.default_rng(0)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    tables, lens = dev(rng.integers(0, 3000, (12, width))), dev(rng.integers(bs * keep, bs * width + 1, 12))
    sel = dev(rng.permuted(np.tile(np.arange(keep + 80), (12, H, 1)), axis=2)[:, :, :keep])
    need = B.paged_attn_sparse_workspace_size(12, Hq, H, D, bs, width, keep)
    whole = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    used = []
    for n in range(12, 0, -1):
        for s in (keep, 300, 129):
            part = sel[:n, :, :s].contiguous()
            args = (q[:n], kc, vc, tables[:n], lens[:n], part, 0.1)
            whole[:need] = 255
            got = B.paged_attn_sparse(*args, workspace=whole[:need])
            used.append(int((whole[:need] != 255).sum()))
            assert torch.equal(got, B.paged_attn_sparse(*args)) and bool(torch.isfinite(got).all())
            assert (used[-1] > 0) == (B.paged_attn_sparse_workspace_needed(n, Hq, H, D, bs, width, s) > 0)
    assert max(used[3:]) > used[0] and bool((whole[need:] == 77).all())
