"""NaN and infinite LSEs in the operators on a batch of sequences, where the batch is large enough that its cut
tiles are joined by the kernel for many of them (more than 57 groups of 32 rows on 152 SMs).  What a sequence's
tokens get must not depend on who else is in the batch, so NaN has to come out where the definition has it, and
everything else has to keep its bytes: no tolerance is needed."""

import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests.batch_reference import Batch

DEV = "cuda:0"


def _tree(batch):
    out, lse = smla.sparse_mla_tree(**batch.to(DEV), kv_format=batch.fmt)
    smla.sync_status()
    return out.cpu(), lse.cpu()


def _alone(batch, b):
    """Sequence b of the batch, as a batch of its own."""
    d = batch.to(DEV)
    t0, t1 = int(batch.starts[b]), int(batch.starts[b + 1])
    d.update(q=d["q"][t0:t1].contiguous(), block_tables=d["block_tables"][b:b + 1].contiguous(), lengths=d["lengths"][b:b + 1],
             starts=torch.tensor([0, t1 - t0], dtype=torch.int32, device=DEV), mask=None if d["mask"] is None else d["mask"][t0:t1].contiguous())
    out, lse = smla.sparse_mla_tree(**d, kv_format=batch.fmt)
    smla.sync_status()
    return out.cpu(), lse.cpu()


def _spoil(batch, slot):
    """NaN in the row, whatever its format."""
    if batch.fmt == "bf16":
        batch.cache[slot] = float("nan")
    else:
        batch.cache[slot, :512] = 0x7F
        batch.cache[slot, 528:] = 0xFF


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("seqs,h", [([(1500, 16)] * 16, 8), ([(128, 1)] * 8, 128), ([(700, 3), (0, 40), (300, 9)] * 10, 24)])
def test_gpu_a_query_with_nan_has_nan_in_every_batch(fmt, seqs, h):
    batch = Batch(seqs, h, 41, fmt)
    want_o, want_l = _tree(batch)
    hurt = torch.zeros(batch.T, h, dtype=torch.bool)
    for b in (0, len(seqs) // 2, len(seqs) - 1):
        hurt[int(batch.starts[b + 1]) - 1, (5 * b + 3) % h] = True
    batch.q[..., 70] = torch.where(hurt, torch.tensor(float("nan"), dtype=torch.bfloat16), batch.q[..., 70])
    out, lse = _tree(batch)
    assert torch.isnan(out[hurt]).all() and torch.isnan(lse[hurt]).all()
    assert torch.equal(out[~hurt], want_o[~hurt]) and torch.equal(lse[~hurt], want_l[~hurt])
    for b in (0, 1):
        mine = slice(int(batch.starts[b]), int(batch.starts[b + 1]))
        o, l = _alone(batch, b)
        assert torch.equal(torch.isnan(o), torch.isnan(out[mine])) and torch.equal(torch.isnan(l), torch.isnan(lse[mine]))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("n", [128, 256, 130])
def test_gpu_a_drafted_row_of_nan_alone_in_its_piece_is_not_lost(fmt, n):
    """Eight sequences of a few blocks of 128 keys: every block is a piece of its own, and behind 128 or 256 cached rows
    the last one holds the token's own row and nothing else."""
    batch = Batch([(n, 1)] * 8, 128, 42, fmt, tree="chain")
    want_o, want_l = _tree(batch)
    hurt = torch.zeros(8, dtype=torch.bool)
    for b in (0, 3, 7):
        _spoil(batch, int(batch.slots(b)[n]))
        hurt[b] = True
    out, lse = _tree(batch)
    assert torch.isnan(out[hurt]).all() and torch.isnan(lse[hurt]).all()
    assert torch.equal(out[~hurt], want_o[~hurt]) and torch.equal(lse[~hurt], want_l[~hurt])
    for b in (0, 1):
        o, l = _alone(batch, b)
        assert torch.equal(torch.isnan(o), torch.isnan(out[b:b + 1])) and torch.equal(torch.isnan(l), torch.isnan(lse[b:b + 1]))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("seqs,h", [([(300, 5), (64, 0), (129, 1), (0, 7)], 8), ([(900, 3), (40, 30)], 8), ([(300, 9), (64, 40), (700, 2)], 32)])
def test_gpu_rows_of_lse_minus_infinity_add_nothing(fmt, seqs, h):
    """Whatever their logits are: NaN or infinite queries (a padded batch's, or tokens that were not accepted) give the same
    bytes as any others.  Up to 128 rows a sequence, up to 256, and more."""
    batch = Batch(seqs, h, 43, fmt)
    _, lse = _tree(batch)
    g = torch.Generator().manual_seed(5)
    gone = torch.rand(batch.T, h, generator=g) < 0.3
    gone[int(batch.starts[1]) - 1] = True  # a token with all its heads
    lse[gone] = float("-inf")
    prev = torch.rand(len(seqs), batch.blocks * 64, generator=g)

    def run():
        out = smla.sparse_mla_weights(**batch.to(DEV), lse=lse.to(DEV), weights=prev.to(DEV), decay=0.5, kv_format=fmt)
        smla.sync_status()
        return out.cpu()

    want = run()
    assert torch.isfinite(want).all()
    for value in (float("nan"), float("inf"), float("-inf"), 3e38):
        batch.q[gone] = value
        assert torch.equal(run(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_nan_in_a_row_that_counts_is_not_lost(fmt):
    """Beside rows that add nothing: a NaN query with a finite lse, and an lse of NaN, reach every position that they see;
    an lse of +infinity makes finite logits nothing and NaN ones NaN."""
    for many in (3, 40):
        batch = Batch([(200, many), (70, many)], 8, 44, fmt)
        _, lse = _tree(batch)
        lse[many - 1, 2] = float("-inf")
        lse[0, 1] = float("inf")

        def run():
            out = smla.sparse_mla_weights(**batch.to(DEV), lse=lse.to(DEV), kv_format=fmt)
            smla.sync_status()
            return out.cpu()

        clean = run()
        assert torch.isfinite(clean).all()
        keep = batch.q.clone()
        for hurt in ("query", "query at +inf", "lse"):
            batch.q = keep.clone()
            at = lse[0, 3].item()
            if hurt == "query":
                batch.q[0, 3, 9] = float("nan")
            elif hurt == "query at +inf":
                batch.q[0, 1, 9] = float("nan")
            else:
                lse[0, 3] = float("nan")
            out = run()
            lse[0, 3] = at
            assert torch.isnan(out[0, :200]).all() and torch.equal(out[1], clean[1])
