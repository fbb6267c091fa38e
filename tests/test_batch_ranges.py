"""Lengths and starts that leave their range, and drafted rows past the end of a table: sparse_mla_tree and
sparse_mla_weights bring the numbers into range on the device and compute what is then there.  Held to the 64-bit
definition over a batch with those numbers, by the tolerances of the operators' own tests."""

import copy

import numpy as np
import pytest
import torch

from tests import batch_reference as br
from tests import test_tree, test_weights
from tests.batch_reference import Batch


def _in_range(batch):
    """The batch that the numbers of this one stand for: lengths in [0, blocks * 64], starts in [0, T], the masks'
    bits of the tokens as they then lie."""
    c = copy.copy(batch)
    width = batch.blocks * 64
    lengths = [min(max(int(n), 0), width) for n in batch.lengths]
    first = [min(max(int(s), 0), batch.T) for s in batch.starts]
    c.seqs, c.sees, starts = [], [], []
    for b in range(len(lengths)):
        t0, t1 = first[b], first[b + 1]
        d = t1 - t0
        c.seqs.append((lengths[b], d))
        if batch.mask is None:
            c.sees.append(np.tri(d, dtype=bool))
        else:
            words = batch.mask[t0:t1].numpy().view(np.uint32).astype(np.uint64)
            bits = ((words[:, :, None] >> np.arange(32, dtype=np.uint64)) & np.uint64(1)).reshape(d, -1).astype(bool)
            c.sees.append(np.pad(bits, ((0, 0), (0, max(0, d - bits.shape[1]))))[:, :d])
        starts.append(t0)
    c.starts = torch.tensor(starts + [first[-1]], dtype=torch.int32)
    c.lengths = torch.tensor(lengths, dtype=torch.int32)
    return c


def _batch(name, fmt, tree):
    """A sequence's (cached rows, drafted tokens) here say only which pages the tables name; every row is finite."""
    if name == "lengths":
        batch = Batch([(100, 20), (40, 8), (300, 3)], 16, 11, fmt, extra_blocks=1, tree=tree)
        batch.lengths[:] = torch.tensor([10 ** 9, -5, -2 ** 31], dtype=torch.int32)
    elif name == "starts":
        batch = Batch([(100, 20), (40, 8)], 16, 12, fmt, extra_blocks=1, lead=1, pad=1, tree=tree)
        batch.starts[0], batch.starts[2] = -3, 10 ** 6
    elif name == "both":
        batch = Batch([(100, 20), (40, 8)], 16, 11, fmt, extra_blocks=1, lead=1, pad=1, tree=tree)
        batch.lengths[0], batch.lengths[1] = 10 ** 9, -5
        batch.starts[0], batch.starts[2] = -3, 10 ** 6
    elif name == "past the table":  # 180 cached rows and 30 drafted ones in three pages; 64 and one in one
        batch = Batch([(180, 30), (64, 1), (0, 200)], 8, 14, fmt, tree=tree)
        batch.blocks = 3
        batch.tables = batch.tables[:, :3].contiguous()
    batch.tables[batch.tables < 0] = 0
    if fmt == "bf16":
        batch.cache = torch.nan_to_num(batch.cache, 0.25)
    else:
        dead = batch.cache[:, 512] == 0xFF
        batch.cache[dead] = batch.cache[int(torch.nonzero(~dead)[0, 0])].clone()
    return batch


CASES = [(n, t) for n in ("lengths", "starts", "both", "past the table") for t in ("random", "chain")]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("name,tree", CASES)
def test_gpu_tree(name, tree, fmt):
    batch = _batch(name, fmt, tree)
    test_tree._check(_in_range(batch), *test_tree._run(batch))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("name,tree", CASES)
def test_gpu_weights(name, tree, fmt):
    batch = _batch(name, fmt, tree)
    meant = _in_range(batch)
    lse, prev = test_weights._inputs(meant)
    for in_place in (False, True):
        out = test_weights._run(batch, lse, prev, 0.75, in_place=in_place)
        test_weights._check(meant, out, lse, prev, 0.75)


def test_the_numbers_brought_into_range():
    """The reference of this file, by hand for one batch."""
    meant = _in_range(_batch("both", "bf16", "random"))
    assert meant.seqs == [(192, 21), (0, 9)] and meant.starts.tolist() == [0, 21, 30]
    assert [s.shape for s in meant.sees] == [(21, 21), (9, 9)]
    out, lse, _, _ = br.tree(meant)
    assert np.isfinite(out[:21]).all() and np.isfinite(lse).sum() >= 21 * 16


@pytest.mark.parametrize("seqs", [2 ** 31 - 1, 2 ** 31 - 600, 2 ** 31 - 1024])
def test_more_sequences_than_the_threads_can_share_are_refused(seqs):
    """The shares of a CTA's threads are rounded up and have to stay within 31 bits."""
    import token_sparse_mla_gb300 as smla

    lib, p = smla.library(), 0x1000
    assert lib.sparse_mla_tree(p, p, p, p, p, p, 4, 8, seqs, 3, 1, 256, 0, 0.04, p, p, p, 1 << 62, None) == 1
    assert "seqs" in lib.sparse_mla_last_error().decode()
    assert lib.sparse_mla_weights(p, p, p, p, p, p, p, p, 0.5, 4, 8, seqs, 3, 1, 256, 0, 0.04, p, None) == 1
    assert "seqs" in lib.sparse_mla_last_error().decode()
