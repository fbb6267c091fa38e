"""sparse_mla_evict with its integers side by side in one buffer: the rows are copied while the selection may still
write what is kept, next to lengths and tables that the copy has already read.  Exact, as all of evict."""

import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests.test_evict import Case

DEV = "cuda:0"


def _packed(c, order, kept_before):
    """The case's integers in one buffer in this order, what a call leaves there filled with `kept_before`."""
    B = len(c.lengths)
    parts = dict(lengths=torch.tensor(c.lengths, dtype=torch.int32), block_tables=c.tables, new_tables=c.new_tables,
                 kept=torch.full((B, c.budget), kept_before, dtype=torch.int32), new_lengths=torch.full((B,), kept_before, dtype=torch.int32))
    buffer = torch.cat([parts[k].flatten() for k in order]).to(DEV)
    views, at = {}, 0
    for k in order:
        views[k] = buffer[at:at + parts[k].numel()].view(parts[k].shape)
        at += parts[k].numel()
    return views


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("order", [("lengths", "kept", "block_tables", "new_tables", "new_lengths"),
                                   ("block_tables", "new_lengths", "kept", "lengths", "new_tables")])
@pytest.mark.parametrize("lengths,budget,sinks,recent", [([900, 257, 4000], 256, 3, 40), ([700] * 30, 65, 0, 0), ([5000, 64, 0], 130, 1, 9),
                                                         ([300, 500], 3, 1, 1)])
def test_gpu_integers_side_by_side(fmt, order, lengths, budget, sinks, recent):
    for seed in range(4):  # other weights, over what the last call kept
        c = Case(lengths, budget, sinks, recent, 30 + seed, fmt)
        cache = c.cache.to(DEV)
        view = cache.view(torch.bfloat16) if fmt == "bf16" else cache
        v = _packed(c, order, kept_before=seed)
        weights = c.weights.to(DEV)
        for _ in range(3):
            kept, new_lengths, new_weights = smla.sparse_mla_evict(view, weights=weights, budget=budget, sinks=sinks, recent=recent, kv_format=fmt, **{
                "block_tables": v["block_tables"], "lengths": v["lengths"], "new_tables": v["new_tables"], "kept": v["kept"],
                "new_lengths": v["new_lengths"]})
        smla.sync_status()
        assert v["lengths"].tolist() == lengths and torch.equal(v["block_tables"].cpu(), c.tables) and torch.equal(v["new_tables"].cpu(), c.new_tables)
        c.check(kept.cpu(), new_lengths.cpu(), new_weights.cpu(), cache.cpu())
