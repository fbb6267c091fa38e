"""sparse_mla_evict: caches cut to a budget of rows by gathered attention weight.  Nothing is computed, so
everything is held to the definition exactly."""

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests.step_reference import CUDA0, STREAM, _d, base_fake, fake  # noqa: F401

DEV = "cuda:0"


def _kept(weights, n, budget, sinks, recent):
    """Positions kept of n, from their weights (numpy fp32)."""
    if n <= budget:
        return list(range(n))
    always = [i for i in range(n) if i < sinks or i >= n - recent]
    held = set(always)
    rank = [float("-inf") if np.isnan(x) else float(x) for x in weights[:n]]
    below = [bool(np.isnan(x)) for x in weights[:n]]  # NaN under -infinity
    rest = sorted((i for i in range(n) if i not in held), key=lambda i: (below[i], -rank[i], i))
    return sorted(always + rest[:budget - len(always)])


class Case:
    def __init__(self, lengths, budget, sinks, recent, seed, fmt="bf16", weights="exponential", new_blocks=None, extra_blocks=0):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.budget, self.sinks, self.recent, self.fmt = list(lengths), budget, sinks, recent, fmt
        B = len(lengths)
        self.blocks = max([1] + [-(-n // 64) for n in lengths]) + extra_blocks
        self.new_blocks = new_blocks or -(-budget // 64)
        old, new = [-(-n // 64) for n in lengths], [min(self.new_blocks, -(-min(n, budget) // 64)) for n in lengths]
        pages = sum(old) + sum(new) + 3
        perm = torch.randperm(pages, generator=g).int()
        self.tables = torch.full((B, self.blocks), -3, dtype=torch.int32)
        self.new_tables = torch.full((B, self.new_blocks), -3, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.tables[b, :old[b]] = perm[at:at + old[b]]
            at += old[b]
            self.new_tables[b, :new[b]] = perm[at:at + new[b]]
            at += new[b]
        row = 576 * 2 if fmt == "bf16" else 656
        self.cache = torch.randint(0, 256, (pages * 64, row), generator=g, dtype=torch.uint8)
        w = torch.empty(B, self.blocks * 64).exponential_(1.0, generator=g)
        if weights == "ties":
            w = (w * 2).floor()
        elif weights == "equal":
            w[:] = 0.25
        elif weights == "odd":
            w = torch.randn(w.shape, generator=g)
            w[:, ::7], w[:, 1::11], w[:, 2::13], w[:, 3::17], w[:, 4::5] = float("nan"), float("inf"), float("-inf"), -0.0, 0.0
        elif weights == "close":
            w = 1.0 + torch.randint(0, 40, w.shape, generator=g).float() * 2.0 ** -23
        self.weights = w

    def run(self, **kw):
        cache = self.cache.to(DEV)
        view = cache.view(torch.bfloat16) if self.fmt == "bf16" else cache
        B = len(self.lengths)
        guard = torch.full((B + 2, self.budget), 77, dtype=torch.int32, device=DEV)
        kept, lengths, weights = smla.sparse_mla_evict(
            view, self.tables.to(DEV), torch.tensor(self.lengths, dtype=torch.int32, device=DEV), self.weights.to(DEV),
            self.new_tables.to(DEV), self.budget, sinks=self.sinks, recent=self.recent, kv_format=self.fmt, kept=guard[1:B + 1], **kw)
        assert guard[0].eq(77).all() and guard[-1].eq(77).all()
        return kept.cpu(), lengths.cpu(), weights.cpu(), cache.cpu()

    def check(self, kept, lengths, weights, cache):
        want = self.cache.clone()
        for b, n in enumerate(self.lengths):
            mine = _kept(self.weights[b].numpy(), n, self.budget, self.sinks, self.recent)
            assert int(lengths[b]) == len(mine)
            assert kept[b].tolist() == mine + [-1] * (self.budget - len(mine))
            assert torch.equal(weights[b, :len(mine)].view(torch.int32), self.weights[b, mine].view(torch.int32))
            assert weights[b, len(mine):].eq(0).all()
            at, pos = torch.arange(len(mine)), torch.tensor(mine, dtype=torch.int64)
            want[self.new_tables[b].long()[at // 64] * 64 + at % 64] = self.cache[self.tables[b].long()[pos // 64] * 64 + pos % 64]
        assert torch.equal(cache, want)


SIZES = [([1], 1, 0, 0), ([2], 1, 0, 0), ([2], 1, 1, 0), ([2], 1, 0, 1), ([100], 100, 4, 10), ([101], 100, 4, 10), ([0, 5, 64, 65], 64, 0, 0),
         ([1000], 500, 4, 64), ([300, 7, 0, 1000, 64], 65, 3, 5), ([8191, 5000], 2001, 0, 128), ([777], 50, 20, 30),
         ([20000, 3], 4097, 4, 500), ([200] * 40, 64, 1, 1), ([70000], 1000, 0, 0), ([140000, 66000], 66001, 64, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_gpu_sizes(i, fmt):
    c = Case(*SIZES[i], seed=i, fmt=fmt, extra_blocks=i % 3)
    c.check(*c.run())
    smla.sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("weights", ["ties", "equal", "odd", "close"])
@pytest.mark.parametrize("lengths,budget,sinks,recent", [([900, 257, 4000], 256, 3, 40), ([9000], 4500, 0, 0), ([70001], 30000, 5, 9)])
def test_gpu_ties_and_odd_weights(weights, lengths, budget, sinks, recent):
    c = Case(lengths, budget, sinks, recent, 5, "fp8", weights)
    c.check(*c.run())
    smla.sync_status()


@pytest.mark.gpu
def test_gpu_wider_new_tables_and_lengths_out_of_range():
    c = Case([300, 64], 100, 0, 0, 6, new_blocks=5)
    c.check(*c.run())
    c.lengths = [10 ** 9, -4]
    c.tables[0, :] = torch.arange(5)  # the whole table: 320 positions
    c.new_tables[0, :2] = torch.tensor([6, 7])
    kept, lengths, weights, _ = c.run()
    assert lengths.tolist() == [100, 0]
    assert kept[0].tolist() == _kept(c.weights[0].numpy(), 320, 100, 0, 0) and kept[1].eq(-1).all()
    smla.sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_rows_outside_the_cache_are_reported_and_not_copied(fmt):
    for which in ("tables", "new_tables"):
        for page in (-1, 2 ** 31 - 1, None):
            c = Case([200], 150, 0, 0, 7, fmt)
            table = getattr(c, which)
            table[0, 1] = c.cache.shape[0] // 64 if page is None else page
            kept, lengths, _, cache = c.run()
            with pytest.raises(smla.SparseMLAError, match="INDEX_RANGE"):
                smla.sync_status()
            mine = _kept(c.weights[0].numpy(), 200, 150, 0, 0)
            assert kept[0].tolist() == mine and int(lengths) == 150
            want = c.cache.clone()
            for i, pos in enumerate(mine):
                if (pos if which == "tables" else i) // 64 != 1:
                    want[int(c.new_tables[0, i // 64]) * 64 + i % 64] = c.cache[int(c.tables[0, pos // 64]) * 64 + pos % 64]
            assert torch.equal(cache, want)
    smla.sync_status()


@pytest.mark.gpu
def test_gpu_streams_and_a_graph():
    cases = [Case([5000, 300], 700, 4, 20, 8 + i) for i in range(2)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    dev = [dict(kv_cache=c.cache.to(DEV).view(torch.bfloat16), block_tables=c.tables.to(DEV),
                lengths=torch.tensor(c.lengths, dtype=torch.int32, device=DEV), weights=c.weights.to(DEV),
                new_tables=c.new_tables.to(DEV)) for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [smla.sparse_mla_evict(**d, budget=700, sinks=4, recent=20, stream=s) for d, s in zip(dev, streams)]
    for s in streams:
        s.synchronize()
    for g, w, d in zip(got, want, dev):
        assert all(torch.equal(a.cpu(), b) for a, b in zip(g, w)) and torch.equal(d["kv_cache"].view(torch.uint8).cpu(), w[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = smla.sparse_mla_evict(**dev[0], budget=700, sinks=4, recent=20)
    for i in (1, 0):
        for k, v in dev[i].items():
            dev[0][k].copy_(cases[0].cache.to(DEV).view(torch.bfloat16) if k == "kv_cache" and i == 0 else v)
        if i == 0:
            dev[0]["weights"].copy_(cases[0].weights)
            dev[0]["block_tables"].copy_(cases[0].tables)
            dev[0]["new_tables"].copy_(cases[0].new_tables)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.cpu(), b) for a, b in zip(out, want[i]))
    smla.sync_status()


# ----------------------------------------------------------------------------- refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    return smla.library()


def _c(lib, **kw):
    a = dict(kv=0x1000, tables=0x1000, lengths=0x1000, weights=0x1000, new_tables=0x1000, seqs=2, blocks=3, new_blocks=2, budget=100, sinks=4,
             recent=8, num_slots=256, fmt=0, kept=0x1000, new_lengths=0x1000, new_weights=0x1000)
    a.update(kw)
    return lib.sparse_mla_evict(a["kv"], a["tables"], a["lengths"], a["weights"], a["new_tables"], a["seqs"], a["blocks"], a["new_blocks"],
                                a["budget"], a["sinks"], a["recent"], a["num_slots"], a["fmt"], a["kept"], a["new_lengths"],
                                a["new_weights"], None)


@pytest.mark.parametrize("kw", [
    dict(kv=0), dict(tables=0), dict(lengths=0), dict(weights=0), dict(new_tables=0), dict(kept=0), dict(new_lengths=0), dict(new_weights=0),
    dict(seqs=-1), dict(seqs=1 << 30), dict(blocks=0), dict(blocks=1 << 25), dict(new_blocks=0), dict(new_blocks=1 << 25), dict(budget=0),
    dict(budget=129), dict(sinks=-1), dict(recent=-1), dict(sinks=60, recent=41), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1),
    dict(num_slots=0), dict(num_slots=1 << 31), dict(fmt=2), dict(kv=0x1008), dict(tables=0x1002), dict(lengths=0x1002),
    dict(weights=0x1002), dict(new_tables=0x1002), dict(kept=0x1002), dict(new_lengths=0x1002), dict(new_weights=0x1002)])
def test_the_library_refuses(lib, kw):
    assert _c(lib, **kw) == 1
    assert lib.sparse_mla_last_error().decode()


def test_no_sequences_is_a_noop(lib):
    assert _c(lib, seqs=0, kv=0, tables=0, lengths=0, weights=0, new_tables=0, kept=0, new_lengths=0, new_weights=0) == 0


def _args():
    return dict(kv_cache=_d((640, 576), torch.bfloat16), block_tables=_d((2, 4), torch.int32), lengths=_d((2,), torch.int32),
                weights=_d((2, 256), torch.float32), new_tables=_d((2, 2), torch.int32), budget=100, kept=_d((2, 100), torch.int32),
                new_lengths=_d((2,), torch.int32), new_weights=_d((2, 128), torch.float32))


def test_marshalling(fake):
    a = _args()
    assert smla.sparse_mla_evict(**a, sinks=4, recent=9) == (a["kept"], a["new_lengths"], a["new_weights"])
    p = {k: v.data_ptr() for k, v in a.items() if k != "budget"}
    assert fake.lib.calls == [("sparse_mla_evict", (
        p["kv_cache"], p["block_tables"], p["lengths"], p["weights"], p["new_tables"], 2, 4, 2, 100, 4, 9, 640, 0, p["kept"],
        p["new_lengths"], p["new_weights"], STREAM))]
    assert fake.entered == [CUDA0]
    a["kv_cache"] = _d((640, 656), torch.uint8)
    smla.sparse_mla_evict(**a, kv_format="fp8")
    assert fake.lib.calls[-1][1][9:13] == (0, 0, 640, 1)


@pytest.mark.parametrize("kw", [
    dict(kv_cache=_d((640, 656), torch.uint8)), dict(kv_cache=torch.zeros(640, 576, dtype=torch.bfloat16)),
    dict(block_tables=_d((2, 0), torch.int32)), dict(block_tables=_d((2, 4), torch.int32, 1)), dict(lengths=_d((3,), torch.int32)),
    dict(weights=_d((2, 255), torch.float32)), dict(weights=_d((2, 256), torch.float32, 1)), dict(new_tables=_d((3, 2), torch.int32)),
    dict(new_tables=_d((2, 2), torch.int64)), dict(new_tables=_d((2, 2), torch.int32, 1)), dict(budget=0), dict(budget=129),
    dict(sinks=-1), dict(recent=-1), dict(sinks=50, recent=51), dict(kept=_d((2, 99), torch.int32)), dict(kept=_d((2, 100), torch.int64)),
    dict(new_lengths=_d((2,), torch.int32, 1)), dict(new_weights=_d((2, 100), torch.float32)), dict(kv_format="int8")])
def test_the_wrapper_refuses(fake, kw):
    a = dict(_args())
    a.update(kw)
    with pytest.raises(ValueError):
        smla.sparse_mla_evict(**a)
    assert fake.lib.calls == []
