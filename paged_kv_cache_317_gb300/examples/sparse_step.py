"""One block-sparse decode step: rotary append, scores, selection, attention."""
import torch
from paged_kv_cache_317_gb300 import binding as pa

# 8 key heads that 32 query heads share, one layer; bounds [num_blocks, key heads, head_dim]
Hq, H, D, bs, nblk, N = 32, 8, 128, 16, 4096, 2
kc = torch.zeros(nblk, H, bs, D, dtype=torch.bfloat16, device="cuda")
vc = torch.zeros_like(kc)
k_min = torch.zeros(nblk, H, D, dtype=torch.bfloat16, device="cuda")
k_max = torch.zeros_like(k_min)
table = pa.rope_cos_sin(8192, D)               # cosines and sines of every position

alloc = pa.BlockAllocator(nblk, bs)
lens = [5000, 300]
for i, n in enumerate(lens):
    alloc.add(i, n)


def append(new, max_new, tables, lens):        # q, k and v: slices of one projection
    qkv = torch.randn(sum(new), (Hq + 2 * H) * D, dtype=torch.bfloat16, device="cuda")
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, H * D, H * D], dim=1))
    start = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
    return pa.kv_cache_append_rope(q, k, v, start, max_new, kc, vc, tables, lens, table,
                                   k_min=k_min, k_max=k_max)


def on_gpu():
    tables, lengths = alloc.batch_block_tables([0, 1], max_blocks=512)
    return torch.from_numpy(tables).cuda(), torch.from_numpy(lengths).cuda()


append(lens, max(lens), *on_gpu())             # the prompts
alloc.batch_append([0, 1])                     # one decode step
tables, lengths = on_gpu()
q = append([1, 1], 1, tables, lengths)
scores = pa.paged_block_scores(q, k_min, k_max, tables, lengths, D ** -0.5, bs)
blocks = pa.paged_block_select(scores, lengths, bs, num_selected=64, sink_blocks=1,
                               recent_blocks=4)
out = pa.paged_attn_sparse(q, kc, vc, tables, lengths, blocks, D ** -0.5)
