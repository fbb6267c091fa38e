"""The operators on a batch of sequences one behind the other on a stream, without a wait between them: each kernel is on
the machine before the one ahead of it has ended, and must not take what that one writes too early.  Small integers
lie side by side in one buffer, so that a line of it is read by one call and written by the next.  The same calls
with a synchronisation after each give the same bytes."""

import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests.batch_reference import Batch

DEV = "cuda:0"


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("seqs,h,budget", [([(200, 1), (64, 1), (500, 1)], 8, 64), ([(900, 1)] * 20, 16, 130), ([(3000, 1), (70, 1)], 128, 256)])
def test_gpu_calls_behind_each_other(fmt, seqs, h, budget):
    B = len(seqs)
    new_blocks = -(-(budget + 3) // 64)
    batch = Batch(seqs, h, 51, fmt, spare=B * 3 * new_blocks, tree="chain")
    if fmt == "bf16":
        batch.cache = torch.nan_to_num(batch.cache, 0.25)
    else:
        batch.cache[batch.cache[:, 512] == 0xFF] = batch.cache[int(batch.slots(0)[0])].clone()
    used = {int(p) for p in batch.tables.flatten() if p >= 0}
    free = torch.tensor([p for p in range(batch.cache.shape[0] // 64) if p not in used], dtype=torch.int32)
    first, second = (free[i * B * new_blocks:(i + 1) * B * new_blocks].reshape(B, new_blocks) for i in range(2))
    cos_sin = torch.cat([torch.ones(4096, 32), torch.zeros(4096, 32)], dim=1).to(DEV)
    kv = torch.randn(B, 576, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    lists = torch.zeros(B, 1, dtype=torch.int32, device=DEV)

    def steps(wait):
        """Append, attend, gather, evict; the same over the new tables; evict those again."""
        results = []

        def note(*x):
            if wait:
                torch.cuda.synchronize()
            results.extend(x)

        ints = {"tables": batch.tables, "lengths": batch.lengths, "new_lengths": torch.full((B,), 7, dtype=torch.int32),
                "kept": torch.full((B, budget), 5, dtype=torch.int32), "first": first, "starts": batch.starts,
                "kept2": torch.full((B, budget), 9, dtype=torch.int32), "new_lengths2": torch.full((B,), 3, dtype=torch.int32), "second": second}
        buffer = torch.cat([v.flatten() for v in ints.values()]).to(DEV)
        at, v = 0, {}
        for k, x in ints.items():
            v[k] = buffer[at:at + x.numel()].view(x.shape)
            at += x.numel()
        cache, q = batch.cache.to(DEV), batch.q.to(DEV)
        slots = [torch.tensor([int(t[b, n // 64]) * 64 + n % 64 for b, n in enumerate(ns)], dtype=torch.int32, device=DEV)
                 for t, ns in ((batch.tables, [n for n, _ in seqs]), (first, [min(n, budget) for n, _ in seqs]))]
        positions = torch.zeros(B, dtype=torch.int32, device=DEV)
        blocks = batch.blocks
        wide = [torch.full((B, n * 64), 0.5, device=DEV) for n in (blocks, new_blocks, new_blocks)]
        o, l = torch.zeros(B, h, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(B, h, device=DEV)
        o2, l2 = torch.zeros_like(o), torch.zeros_like(l)
        torch.cuda.synchronize()
        mask = smla.sparse_mla_scatter_mask(lists, 1)
        smla.sparse_mla_append(kv, positions, slots[0], cache, cos_sin, kv_format=fmt)
        smla.sparse_mla_tree(q, cache, v["tables"], v["lengths"], v["starts"], mask=mask, out=o, lse=l, kv_format=fmt)
        note(o, l)
        smla.sparse_mla_weights(q, cache, v["tables"], v["lengths"], v["starts"], l, mask=mask, weights=wide[0], decay=0.5, out=wide[0], kv_format=fmt)
        note(wide[0])
        smla.sparse_mla_evict(cache, v["tables"], v["lengths"], wide[0], v["first"], budget, sinks=2, recent=5, kept=v["kept"],
                              new_lengths=v["new_lengths"], new_weights=wide[1], kv_format=fmt)
        note(v["kept"], v["new_lengths"])
        smla.sparse_mla_append(kv, positions, slots[1], cache, cos_sin, kv_format=fmt)
        smla.sparse_mla_tree(q, cache, v["first"], v["new_lengths"], v["starts"], mask=mask, out=o2, lse=l2, kv_format=fmt)
        note(o2, l2)
        smla.sparse_mla_weights(q, cache, v["first"], v["new_lengths"], v["starts"], l2, mask=mask, weights=wide[1], decay=0.5, out=wide[1],
                                kv_format=fmt)
        note(wide[1])
        smla.sparse_mla_evict(cache, v["first"], v["new_lengths"], wide[1], v["second"], budget // 2, sinks=1, recent=3,
                              kept=v["kept2"].view(-1)[:B * (budget // 2)].view(B, -1), new_lengths=v["new_lengths2"], new_weights=wide[2], kv_format=fmt)
        note(v["kept2"], v["new_lengths2"], wide[2], cache, buffer)
        smla.sync_status()
        return results

    want = steps(True)
    assert want[-5].ne(9).any() and want[-4].tolist() == [min(n, budget, budget // 2) for n, _ in seqs]
    for _ in range(10):
        for got, w in zip(steps(False), want):
            assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))
