"""The operators on a batch of sequences over caches of a few rows, over batches whose sequences differ in
everything that chooses how they are worked (few rows (token, head) and many, no cached rows and thousands,
tokens and none), and over block tables of the largest width.  Tolerances are those of each operator's own tests."""

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import test_tree, test_weights
from tests.batch_reference import Batch
from tests.test_evict import _kept

DEV = "cuda:0"


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("rows", [1, 3, 16, 63, 65])
@pytest.mark.parametrize("h", [1, 8, 64])
def test_gpu_caches_of_a_few_rows(fmt, rows, h):
    """Two sequences in one page of a cache that has `rows` rows: what lies past its end is masked."""
    batch = Batch([(rows // 2, rows - rows // 2), (1, 2)], h, rows, fmt, spare=0)
    batch.tables[batch.tables >= 0] = 0
    if rows > 64:
        batch.tables[0, 1] = 1
    full = Batch([(rows, 0)], 1, 5, fmt, spare=0)
    pages = full.tables[0].long()
    batch.cache = full.cache.reshape(-1, 64, full.cache.shape[1])[pages].reshape(-1, full.cache.shape[1])[:rows].contiguous()
    test_tree._check(batch, *test_tree._run(batch))
    lse, prev = test_weights._inputs(batch)
    test_weights._check(batch, test_weights._run(batch, lse, prev, 0.5), lse, prev, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("most", [8, 16, 40])
def test_gpu_sequences_of_all_kinds_in_one_batch(fmt, most):
    """Up to 128, 256 and 640 rows (token, head) a sequence, two to three sequences of each for every pair of CTAs: what
    a pair keeps between sequences of unlike kinds."""
    rng = np.random.default_rng(most)
    seqs = [(int(n), int(d)) for n, d in zip(rng.integers(0, 400, 200), rng.integers(0, most + 1, 200))]
    seqs[::9] = [(n, most) for n, _ in seqs[::9]]
    seqs[4::31] = [(0, d) for _, d in seqs[4::31]]
    batch = Batch(seqs, 16, 50 + most, fmt)
    test_tree._check(batch, *test_tree._run(batch))
    lse, prev = test_weights._inputs(batch)
    first = test_weights._run(batch, lse, prev, 0.5)
    test_weights._check(batch, first, lse, prev, 0.5)
    for _ in range(5):
        assert torch.equal(test_weights._run(batch, lse, prev, 0.5), first)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_eviction_in_a_cache_that_ends_inside_the_new_page(fmt):
    """A cache of 70 rows: page 0 is cut to 9 rows of page 1, which has 6; a sequence whose new page is outside keeps
    its list, length and weights.  Both are reported."""
    row = 576 if fmt == "bf16" else 656
    bits = torch.randint(0, 120, (70, row * (2 if fmt == "bf16" else 1)), dtype=torch.uint8, generator=torch.Generator().manual_seed(3))
    cache = bits.to(DEV)
    view = cache.view(torch.bfloat16) if fmt == "bf16" else cache
    w = torch.rand(2, 64, generator=torch.Generator().manual_seed(4))
    kept, lengths, weights = smla.sparse_mla_evict(
        view, torch.tensor([[0], [0]], dtype=torch.int32, device=DEV), torch.tensor([64, 20], dtype=torch.int32, device=DEV), w.to(DEV),
        torch.tensor([[1], [-1]], dtype=torch.int32, device=DEV), 9, sinks=1, recent=2, kv_format=fmt)
    with pytest.raises(smla.SparseMLAError, match="evict"):
        smla.sync_status()
    want = bits.clone()
    for b, n in enumerate((64, 20)):
        mine = _kept(w[b].numpy(), n, 9, 1, 2)
        assert kept[b].tolist() == mine and int(lengths[b]) == 9 and torch.equal(weights[b, :9].cpu(), w[b, mine])
        if b == 0:
            want[64:70] = bits[mine[:6]]
    assert torch.equal(cache.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("in_place", [True, False])
def test_gpu_many_sequences_without_tokens(fmt, in_place):
    """Some with more positions than a warp takes at once, their weights decayed beside the others' sums."""
    rng = np.random.default_rng(6)
    seqs = [(int(n), 0) for n in rng.integers(0, 9000, 40)]
    seqs[3], seqs[11], seqs[25], seqs[39] = (8500, 3), (0, 2), (4097, 1), (9100, 0)
    batch = Batch(seqs, 8, 61, fmt, extra_blocks=3)
    lse, prev = test_weights._inputs(batch)
    test_weights._check(batch, test_weights._run(batch, lse, prev, 0.75, in_place=in_place), lse, prev, 0.75)
    test_weights._check(batch, test_weights._run(batch, lse, None, 0.75), lse, None, 0.75)


@pytest.mark.gpu
def test_gpu_block_tables_of_the_largest_width():
    """2^31 - 16384 positions: every index is within 31 bits, loops' steps past the end included."""
    widest = 2 ** 25 - 256
    batch = Batch([(100, 2)], 8, 62)
    d = batch.to(DEV)
    want_o, want_l = smla.sparse_mla_tree(**d)
    want_w = smla.sparse_mla_weights(**d, lse=want_l)
    d["block_tables"] = torch.zeros(1, widest, dtype=torch.int32, device=DEV)
    d["block_tables"][0, :batch.blocks] = batch.tables[0].to(DEV)
    out, lse = smla.sparse_mla_tree(**d)
    assert torch.equal(out, want_o) and torch.equal(lse, want_l)
    w = torch.full((1, widest * 64), float("nan"), device=DEV)
    smla.sparse_mla_weights(**d, lse=lse, out=w)
    assert torch.equal(w[:, :want_w.shape[1]], want_w)
    assert not w[:, want_w.shape[1]:].count_nonzero()  # (NaN counts)
    used = set(batch.tables[0].tolist())
    free = [p for p in range(batch.cache.shape[0] // 64) if p not in used]
    new_tables = torch.zeros_like(d["block_tables"])
    new_tables[0, :2] = torch.tensor(free[:2], dtype=torch.int32, device=DEV)
    kept, lengths, weights = smla.sparse_mla_evict(d["kv_cache"], d["block_tables"], torch.tensor([100], dtype=torch.int32, device=DEV), w,
                                                   new_tables, 100)
    smla.sync_status()
    assert kept.tolist() == [list(range(100))] and lengths.tolist() == [100]
    assert torch.equal(weights[:, :100], w[:, :100]) and not weights[:, 100:].count_nonzero()
    with pytest.raises(smla.SparseMLAError, match="blocks"):
        smla.sparse_mla_tree(d["q"], d["kv_cache"], torch.zeros(1, widest + 1, dtype=torch.int32, device=DEV), d["lengths"], d["starts"])
