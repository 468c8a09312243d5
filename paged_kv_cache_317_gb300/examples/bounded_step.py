"""A bounded cache: prompts, the weight of their last rows, eviction, decode steps."""
import numpy as np
import torch
from paged_kv_cache_317_gb300 import binding as pa

# 8 key heads that 32 query heads share, one layer; at most 576 tokens a sequence, cut to 512
Hq, H, D, bs, nblk, MB, keep = 32, 8, 128, 16, 1024, 64, 512
kc = torch.zeros(nblk, H, bs, D, dtype=torch.bfloat16, device="cuda")
vc = torch.zeros_like(kc)
table = pa.rope_cos_sin(8192, D)               # cosines and sines of every position

alloc = pa.BlockAllocator(nblk, bs)
lens = [900, 300]
for i, n in enumerate(lens):
    alloc.add(i, n)
seqs, position = [0, 1], torch.tensor(lens, dtype=torch.int32, device="cuda")
weights = torch.zeros(2, H, MB * bs, device="cuda")   # the weight that each token has had


def on_gpu():
    tables, lengths = alloc.batch_block_tables(seqs, MB)
    return torch.from_numpy(tables).cuda(), torch.from_numpy(lengths).cuda()


def append(new, tables, lengths, positions=None):
    qkv = torch.randn(sum(new), (Hq + 2 * H) * D, dtype=torch.bfloat16, device="cuda")
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, H * D, H * D], dim=1))
    start = torch.tensor([0, *np.cumsum(new)], dtype=torch.int32, device="cuda")
    return start, pa.kv_cache_append_rope(q, k, v, start, max(new), kc, vc, tables, lengths, table,
                                          positions=positions)


def evict(tables, lengths):
    kept = pa.paged_block_select(weights, lengths, 1, keep, sink_blocks=4, recent_blocks=128)
    alloc.batch_evict(seqs, keep)              # shared blocks become fresh ones, the rest go back
    new_tables, _ = on_gpu()
    pa.kv_cache_evict(kc, vc, tables, lengths, kept, weights=weights, new_tables=new_tables)


# the prompts: attention, and what their last 32 rows attend to
tables, lengths = on_gpu()
start, q = append(lens, tables, lengths)
lse = torch.empty(sum(lens), Hq, device="cuda")
out = pa.paged_attn_chunk(q, start, max(lens), kc, vc, tables, lengths, D ** -0.5,
                          out_dtype=torch.bfloat16, lse=lse)
pa.paged_chunk_weights(q, lse, start, max(lens), kc, tables, lengths, D ** -0.5, weights, window=32)
evict(tables, lengths)
for step in range(100):                        # decode; evict when a sequence has 64 too many
    alloc.batch_append(seqs)
    tables, lengths = on_gpu()
    _, q = append([1, 1], tables, lengths, position + step)
    out = pa.paged_attn_decode_weights(q, kc, vc, tables, lengths, D ** -0.5, weights)
    if max(alloc.length(i) for i in seqs) >= keep + 64:
        evict(tables, lengths)
