"""Speculative decoding over caches kept to a budget, as the README has it, several rounds of it: the drafted tokens' rows
appended, attention over cached rows and trees, a path of each tree accepted and its rows appended behind the cached
ones, the weights gathered from the accepted tokens alone (a chain, with the lse that they had in the tree), the
lengths moved on, the caches cut into fresh pages.  Every stage is held to 64 bits over what the stages before it left;
tolerances are those of the operators' own tests."""

import copy

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import batch_reference as br
from tests import step_reference as ref
from tests.batch_reference import Batch
from tests.test_evict import _kept

DEV = "cuda:0"


def _within(got, want, tol):
    assert np.all(np.abs(ref.to64(got) - want) <= tol), float((np.abs(ref.to64(got) - want) - tol).max())


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("h,budget", [(16, 150), (8, 70)])
def test_gpu_rounds_of_verify_accept_gather_and_evict(fmt, h, budget):
    drafted, rounds, sinks, recent = [7, 12, 1, 5], 3, 4, 20
    B, T = len(drafted), sum(drafted)
    blocks = -(-(400 + 12) // 64)  # of every table
    batch = Batch([(200, 7), (63, 12), (400, 1), (20, 5)], h, budget, fmt, spare=(1 + rounds) * B * blocks)
    pages = batch.cache.shape[0] // 64
    used = {int(p) for p in batch.tables.flatten() if p >= 0}
    free = [p for p in range(pages) if p not in used]
    for b in range(B):  # whole tables: the caches grow
        for i in range(blocks):
            if batch.tables[b, i] < 0:
                batch.tables[b, i] = free.pop()
    g = torch.Generator().manual_seed(budget)
    table = ref.cos_sin_table(1000).to(DEV)
    cache, tables = batch.cache.to(DEV), batch.tables.to(DEV)
    lengths, w, text = batch.lengths.to(DEV), None, [n for n, _ in batch.seqs]  # text: tokens so far, a row's rotation
    for r in range(rounds):
        host_n, host_tables = lengths.tolist(), tables.cpu().long()

        def slot(b, at):
            return int(host_tables[b, at // 64]) * 64 + at % 64

        step = copy.copy(batch)
        trees = Batch([(0, d) for d in drafted], h, 60 + r, fmt)
        step.seqs, step.sees, step.mask, step.words = list(zip(host_n, drafted)), trees.sees, trees.mask, trees.words
        step.tables, step.lengths, step.starts = tables.cpu(), lengths.cpu(), trees.starts
        step.q = (torch.randn(T, h, 576, generator=g)).to(torch.bfloat16)
        kv = torch.randn(T, 576, generator=g).to(torch.bfloat16).to(DEV)
        positions, slots = [], []
        for b, d in enumerate(drafted):
            for j in range(d):
                positions.append(text[b] + int(step.sees[b][j].sum()) - 1)
                slots.append(slot(b, host_n[b] + j))
        positions = _ints(positions)
        smla.sparse_mla_append(kv, positions, _ints(slots), cache, table, kv_format=fmt)
        q, starts = step.q.to(DEV), step.starts.to(DEV)
        out, lse = smla.sparse_mla_tree(q, cache, tables, lengths, starts, mask=step.mask.to(DEV), kv_format=fmt)
        smla.sync_status()
        step.cache = cache.cpu()
        want_o, want_l, tol_o, tol_l = br.tree(step)
        _within(out, want_o, tol_o)
        _within(lse, want_l, tol_l)

        # a path of each tree is accepted
        paths = [np.nonzero(step.sees[b][d - 1])[0][:3 + r] for b, d in enumerate(drafted)]
        a = torch.tensor([int(step.starts[b]) + int(j) for b, path in enumerate(paths) for j in path], device=DEV)
        a_starts = _ints(np.cumsum([0] + [len(p) for p in paths]).tolist())
        a_slots = _ints([slot(b, host_n[b] + i) for b, path in enumerate(paths) for i in range(len(path))])
        smla.sparse_mla_append(kv[a], positions[a], a_slots, cache, table, kv_format=fmt)
        before = None if w is None else w.clone()
        w = smla.sparse_mla_weights(q[a], cache, tables, lengths, a_starts, lse[a], weights=w, decay=0.75, kv_format=fmt)
        lengths = lengths + a_starts.diff()
        smla.sync_status()
        chain = copy.copy(step)
        chain.seqs = [(n, len(p)) for n, p in zip(host_n, paths)]
        chain.sees, chain.mask = [np.tri(len(p), dtype=bool) for p in paths], None
        chain.starts, chain.q, chain.cache, chain.T = a_starts.cpu(), step.q[a.cpu()], cache.cpu(), a.numel()
        _within(w, *br.weights(chain, lse[a].cpu(), before, 0.75))
        # the accepted tokens see what they saw in the tree, so that each head's probabilities add up to one
        gained = w.double().sum(dim=1).cpu() - (0 if before is None else 0.75 * torch.stack([before[b, :n].double().sum() for b, n in enumerate(host_n)]).cpu())
        assert torch.allclose(gained, torch.tensor([float(len(p) * h) for p in paths], dtype=torch.float64), rtol=1e-4)
        text = [t + len(p) for t, p in zip(text, paths)]

        # cut to the budget, into pages that nobody uses
        fresh = torch.tensor([free.pop() for _ in range(B * blocks)], dtype=torch.int32, device=DEV).view(B, blocks)
        rows = cache.cpu()
        kept, new_lengths, new_w = smla.sparse_mla_evict(cache, tables, lengths, w, fresh, budget, sinks=sinks, recent=recent, kv_format=fmt)
        smla.sync_status()
        now, where = cache.cpu(), fresh.cpu().long()
        for b, n in enumerate(lengths.tolist()):
            mine = _kept(w[b].cpu().numpy(), n, budget, sinks, recent)
            assert kept[b].tolist() == mine + [-1] * (budget - len(mine)) and int(new_lengths[b]) == len(mine)
            assert torch.equal(new_w[b, :len(mine)], w[b, mine]) and new_w[b, len(mine):].eq(0).all()
            for i, p in enumerate(mine):
                assert torch.equal(now[int(where[b, i // 64]) * 64 + i % 64].view(torch.uint8), rows[slot(b, p)].view(torch.uint8))
        lengths, w, tables = new_lengths, new_w, fresh
