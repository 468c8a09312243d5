"""Refusals of the rotated append and the block-sparse decode on the host: malformed arguments
are turned down before anything is enqueued (no GPU needed)."""

import ctypes

import pytest
import torch

P = 1 << 20                       # never dereferenced: every call below fails its checks first
INV, UNS, OK = 1, 2, 0


def _rope(binding, **kw):
    a = dict(cos_sin=P, max_position=64, rotary_dim=64, interleaved=0, num_axes=1, positions=None,
             pair_axis=None)
    a.update(kw)
    return binding.pa_rope(*a.values())


@pytest.fixture(scope="module")
def binding(lib):
    from paged_kv_cache_317_gb300 import binding
    return binding


def test_append_rope_refuses(lib, binding):
    def call(rope=None, **kw):
        a = dict(q=P, qs=8 * 64, k=P, ks=2 * 64, v=P, vs=2 * 64, start=P, T=0, most=4, kc=P, vc=P,
                 lo=P, hi=P, bt=P, sl=P, N=4, Hq=8, H=2, D=64, bs=16, MB=4, B=64, rope=rope, dt=0,
                 out=P, err=None, stream=None)
        a.update(kw)
        return lib.kv_cache_append_rope(*a.values())

    # sizes are checked even where there is nothing to do (T = 0)
    assert call() == OK and call(rope=_rope(binding)) == OK and call(T=5, N=0) == OK
    for kw in (dict(N=-1), dict(T=-1), dict(most=-1), dict(H=0), dict(bs=0), dict(MB=0), dict(B=0),
               dict(D=0), dict(N=65536), dict(MB=1 << 28)):
        assert call(**kw) == INV, kw
    for kw in (dict(dt=2), dict(D=72), dict(D=272)):
        assert call(**kw) == UNS, kw
    # pointers, alignment and strides, before any launch
    for kw in (dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(start=None), dict(bt=None),
               dict(sl=None), dict(out=None), dict(lo=None), dict(hi=None), dict(q=None), dict(k=P + 8),
               dict(q=P + 8), dict(kc=P + 2), dict(lo=P + 8), dict(out=P + 8), dict(qs=8 * 64 - 8),
               dict(ks=64), dict(vs=2 * 64 + 4), dict(qs=8 * 64 + 8, out=P), dict(Hq=0)):
        assert call(T=5, **kw) == INV, kw
    for kw, want in ((dict(rotary_dim=0), INV), (dict(rotary_dim=24), UNS), (dict(rotary_dim=80), UNS),
                     (dict(max_position=0), INV), (dict(num_axes=0), INV), (dict(num_axes=5), INV),
                     (dict(cos_sin=None), INV), (dict(cos_sin=P + 4), INV), (dict(num_axes=2), INV),
                     (dict(num_axes=2, positions=P), INV), (dict(pair_axis=bytes([1] * 32)), INV),
                     (dict(num_axes=2, positions=P, pair_axis=bytes([0] * 31 + [2])), INV)):
        assert call(rope=_rope(binding, **kw)) == want, kw


def test_bounds_refuses(lib):
    def call(**kw):
        a = dict(kc=P, bt=P, sl=P, first=None, N=4, H=2, D=64, bs=16, MB=4, B=64, dt=0, lo=P, hi=P,
                 err=None, stream=None)
        a.update(kw)
        return lib.kv_block_bounds(*a.values())

    assert call(N=0) == OK
    for kw in (dict(N=-1), dict(H=0), dict(D=0), dict(bs=0), dict(MB=0), dict(B=0), dict(N=65536),
               dict(MB=1 << 28), dict(kc=None), dict(bt=None), dict(sl=None), dict(lo=None), dict(hi=None),
               dict(kc=P + 8), dict(lo=P + 8), dict(hi=P + 8)):
        assert call(**kw) == INV, kw
    assert call(D=60) == UNS and call(dt=2) == UNS


def test_scores_refuses(lib):
    def call(**kw):
        a = dict(q=P, lo=P, hi=P, bt=P, sl=P, N=4, Hq=8, H=2, D=64, bs=16, MB=4, B=64, scale=0.125,
                 dt=0, s=P, err=None, stream=None)
        a.update(kw)
        return lib.paged_block_scores(*a.values())

    assert call(N=0) == OK
    for kw in (dict(N=-1), dict(Hq=0), dict(H=0), dict(Hq=7), dict(bs=0), dict(MB=0), dict(B=0),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(N=65536), dict(MB=1 << 28), dict(q=None), dict(lo=None), dict(hi=None), dict(bt=None),
               dict(sl=None), dict(s=None), dict(q=P + 8), dict(lo=P + 8), dict(hi=P + 8)):
        assert call(**kw) == INV, kw
    assert call(D=96) == UNS and call(dt=2) == UNS


def test_select_refuses(lib):
    def call(**kw):
        a = dict(s=P, sl=P, N=4, H=2, bs=16, MB=4, keep=4, sink=1, recent=1, out=P, err=None, stream=None)
        a.update(kw)
        return lib.paged_block_select(*a.values())

    assert call(N=0) == OK
    for kw in (dict(N=-1), dict(H=0), dict(bs=0), dict(MB=0), dict(keep=0), dict(sink=-1), dict(recent=-1),
               dict(sink=3, recent=2), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(N=65536),
               dict(MB=1 << 28), dict(s=None), dict(sl=None), dict(out=None)):
        assert call(**kw) == INV, kw
    assert call(MB=131073, bs=1) == UNS            # more blocks than a row may have


def test_attention_refuses(lib):
    def call(**kw):
        a = dict(q=P, kc=P, vc=P, bt=P, sl=P, sel=P, S=4, N=4, Hq=8, H=2, D=64, bs=16, MB=4, B=64,
                 scale=0.125, dt=0, out=P, odt=2, ws=None, wsb=0, err=None, stream=None)
        a.update(kw)
        return lib.paged_attn_sparse(*a.values())

    assert call(N=0) == OK
    for kw in (dict(N=-1), dict(Hq=0), dict(H=0), dict(Hq=7), dict(bs=0), dict(MB=0), dict(B=0),
               dict(S=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(N=65536),
               dict(MB=1 << 28), dict(B=1 << 27), dict(q=None), dict(kc=None), dict(vc=None),
               dict(bt=None), dict(sl=None), dict(sel=None), dict(out=None), dict(q=P + 8), dict(kc=P + 8),
               dict(vc=P + 8), dict(out=P + 8), dict(ws=P + 8, wsb=1 << 30)):
        assert call(**kw) == INV, kw
    # few rows with long lists: the workspace given is a byte short
    long = dict(N=1, S=4096, MB=4096, B=8192)
    need = lib.paged_attn_sparse_workspace_size(1, 8, 2, 64, 16, 4096, 4096)
    assert need > 0 and call(ws=P, wsb=need - 1, **long) == INV
    for kw in (dict(D=96), dict(dt=2), dict(odt=3), dict(bs=24), dict(bs=4)):
        assert call(**kw) == UNS, kw


def test_the_binding_refuses_tensors_that_are_not_on_the_gpu(binding, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    h = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    i = torch.zeros(4, 4, dtype=torch.int32)
    for call in (lambda: binding.kv_cache_append_rope(None, h[0], h[0], i, 1, h, h, i, i[0], None),
                 lambda: binding.kv_block_bounds(h, i, i[0], h[:, :, 0], h[:, :, 0]),
                 lambda: binding.paged_block_scores(h[:, :, 0], h[:, :, 0], h[:, :, 0], i, i[0], 1.0, 16),
                 lambda: binding.paged_block_select(torch.zeros(4, 2, 4), i[0], 16, 2),
                 lambda: binding.paged_attn_sparse(h[:, :, 0], h, h, i, i[0], torch.zeros(4, 2, 3), 1.0)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_rope_table_shape_and_values(binding):
    t = binding.rope_cos_sin(5, 8, base=100.0, device="cpu")
    assert t.shape == (5, 8) and t.dtype == torch.float32
    assert torch.equal(t[0], torch.tensor([1.0] * 4 + [0.0] * 4))
    assert abs(float(t[3, 1]) - float(torch.cos(torch.tensor(3 * 100.0 ** -0.25)))) < 1e-6


def test_the_example_is_the_one_shown():
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = open(os.path.join(root, "paged_kv_cache_317_gb300", "examples", "sparse_step.py")).read()
    body = code.split('"""', 2)[2].strip()
    assert body in open(os.path.join(root, "README.md")).read()


def test_attention_workspace_sizes(lib):
    size = lib.paged_attn_sparse_workspace_size
    assert size(1, 32, 8, 128, 16, 4096, 64) == 0          # short lists: one cluster a row
    assert size(64, 64, 8, 128, 16, 4096, 128) == 0        # many rows
    # rows x parts partials of 8 (16) columns: O in fp32, m and l
    for heads, cols in ((8, 8), (16, 16), (17, 16)):
        n = size(1, heads, 1, 128, 64, 512, 512)
        rows = -(-heads // cols)
        assert n > 0 and n % (rows * cols * (128 * 4 + 8)) == 0
        assert n // (rows * cols * (128 * 4 + 8)) <= 64
    for n in (1, 2, 7, 40, 300):                  # lists of up to 1024 tokens never need one
        for heads, kv in ((1, 1), (8, 1), (32, 8), (64, 2)):
            for dim in (64, 128, 256):
                assert size(n, heads, kv, dim, 8, 4096, 128) == size(n, heads, kv, dim, 64, 4096, 16) == 0
    assert size(0, 8, 2, 64, 16, 4096, 4096) == size(1, 7, 2, 64, 16, 4096, 4096) == 0
    assert size(1, 8, 2, 96, 16, 4096, 4096) == size(1, 8, 2, 64, 16, 4096, 0) == 0
