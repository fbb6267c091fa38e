"""sparse_mla_tree: attention of a batch of sequences, each over its own cached rows and a tree of drafted tokens.

Tolerances, against the definition in 64 bits over the rows that the kernel multiplies (fp8 rows are
dequantised to bf16, as the forward does):
* a logit is an fp32 sum of 576 exact products: off by at most 576 * 2^-23 of their absolute sum A
  (the tensor cores' accumulation), so a probability by that factor e, and the LSE by e plus the
  fp32 rounding of its own value (2^-22) and of ex2 and log2 (2^-21 each);
* O is a sum of probabilities rounded to bf16 (2^-8 each) times values: off by (2^-8 + 2 e) of
  sum p |v|, plus its own rounding to bf16 (2^-8 of |O|).
"""

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import batch_reference as br
from tests import step_reference as ref
from tests.batch_reference import SCALE, Batch
from tests.step_reference import CUDA0, STREAM, _d, base_fake, fake  # noqa: F401
from token_sparse_mla_gb300 import _binding

DEV = "cuda:0"


def _run(batch, scale=SCALE, **kw):
    T, h = batch.T, batch.h
    guard_o = torch.full((T + 2, h, 512), 2.5, dtype=torch.bfloat16, device=DEV)
    guard_l = torch.full((T + 2, h), 2.5, dtype=torch.float32, device=DEV)
    need = smla.tree_workspace_bytes(T, h, len(batch.seqs))
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN where nothing is written
    out, lse = smla.sparse_mla_tree(**batch.to(DEV), scale=scale, out=guard_o[1:T + 1], lse=guard_l[1:T + 1], kv_format=batch.fmt,
                                    workspace=ws, **kw)
    smla.sync_status()
    assert guard_o[0].eq(2.5).all() and guard_o[T + 1].eq(2.5).all()
    assert guard_l[0].eq(2.5).all() and guard_l[T + 1].eq(2.5).all()
    assert ws[need:].eq(0xFF).all()
    return out.cpu(), lse.cpu()


def _check(batch, out, lse, scale=SCALE):
    want_o, want_l, tol_o, tol_l = br.tree(batch, scale)
    out, lse = ref.to64(out), ref.to64(lse)
    mine = ~np.isnan(want_l[:, 0])
    assert np.all(out[~mine] == 2.5) and np.all(lse[~mine] == 2.5)  # places of no sequence, as they were
    empty = np.isneginf(want_l) & mine[:, None]
    assert np.all(out[empty] == 0) and np.all(np.isneginf(lse[empty]))
    at = mine[:, None] & ~empty
    assert np.all(np.abs(lse[at] - want_l[at]) <= tol_l[at]), float((np.abs(lse[at] - want_l[at]) - tol_l[at]).max())
    assert np.all(np.abs(out[at] - want_o[at]) <= tol_o[at]), float((np.abs(out[at] - want_o[at]) - tol_o[at]).max())


BATCHES = [
    ([(0, 1)], 1), ([(1, 1)], 16), ([(63, 1)], 16), ([(64, 1)], 8), ([(127, 1)], 8), ([(128, 1)], 8), ([(1000, 8)], 8),
    ([(60, 8)], 16), ([(0, 70)], 8), ([(37, 100)], 3), ([(300, 64)], 64), ([(5, 130)], 1),
    ([(100, 3), (0, 0), (700, 1), (64, 64), (0, 5), (191, 33), (3, 0)], 16),
    ([(130 * i % 517, i % 7) for i in range(90)], 8),       # more tiles than pairs of CTAs
    ([(2000, 2), (10, 40), (5000, 1)], 13), ([(9000, 1)], 128), ([(700, 40), (700, 40)], 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_gpu_matches_the_definition(i, fmt):
    seqs, h = BATCHES[i]
    batch = Batch(seqs, h, 100 + i, fmt, pad=i % 3, lead=i % 2, extra_blocks=i % 4)
    _check(batch, *_run(batch))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("tree", ["chain", "any", "none"])
def test_gpu_masks(tree, fmt):
    """Chains without a mask; masks that are no trees; masks that leave a token nothing but the cached rows, or nothing."""
    batch = Batch([(0, 40), (70, 40), (63, 9), (500, 17), (0, 1)], 16, 7, fmt, tree=tree)
    _check(batch, *_run(batch))


@pytest.mark.gpu
def test_gpu_mask_of_fewer_words_than_drafted_tokens():
    batch = Batch([(30, 70), (64, 33), (10, 2)], 8, 8, words=1)
    _check(batch, *_run(batch))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_what_is_not_seen_may_hold_anything(fmt):
    """Drafted rows of infinities and NaN that some or all tokens do not see; a token that does see one has NaN."""
    for value in (float("nan"), float("inf"), float("-inf")):
        batch = Batch([(100, 20), (62, 5), (0, 33)], 16, 9, fmt)
        hurt = [(0, 3), (0, 19), (1, 1), (2, 0)]  # (sequence, drafted token)
        clean = Batch([(100, 20), (62, 5), (0, 33)], 16, 9, fmt)
        seen = np.zeros(batch.T, dtype=bool)
        for b, j in hurt:
            slot = int(batch.slots(b)[batch.seqs[b][0] + j])
            if fmt == "bf16":
                batch.cache[slot] = value
            else:
                batch.cache[slot, :512] = 0x7F if value != value else 0x38  # NaN codes, or ones by an infinite scale
                batch.cache[slot, 512:528] = torch.tensor([value] * 4).view(torch.uint8)
                batch.cache[slot, 528:] = torch.full((64,), value, dtype=torch.bfloat16).view(torch.uint8)
            for i in range(batch.seqs[b][1]):
                seen[int(batch.starts[b]) + i] |= bool(batch.sees[b][i, j])
        out, lse = _run(batch)
        want_o, want_l = _run(clean)
        assert torch.equal(out[~seen], want_o[~seen]) and torch.equal(lse[~seen], want_l[~seen])
        assert seen.any() and (~seen).any()
        if value != value:
            assert torch.isnan(out[seen]).all() and torch.isnan(lse[seen]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_pages_outside_the_cache_are_masked(fmt):
    batch = Batch([(700, 7), (64, 3)], 16, 5, fmt)
    pages = batch.cache.shape[0] // 64
    for i, page in ((0, -1), (3, pages), (4, 2 ** 31 - 1), (10, -2 ** 31)):
        batch.tables[0, i] = page
    _check(batch, *_run(batch))
    batch.tables[:] = -1
    out, lse = _run(batch)
    assert out.eq(0).all() and torch.isneginf(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("short", [1, 30, 33, 63])
def test_gpu_cache_that_ends_inside_a_page(fmt, short):
    batch = Batch([(500, 12)], 24, 6, fmt, spare=0)
    batch.cache = batch.cache[:batch.cache.shape[0] - short].contiguous()
    _check(batch, *_run(batch))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_numbers_out_of_range_are_brought_into_it(fmt):
    """Lengths past the table, negative ones, starts past the batch: what exists is computed, nothing else touched."""
    batch = Batch([(100, 20), (40, 8)], 16, 11, fmt, extra_blocks=1, lead=1, pad=1)
    batch.tables[batch.tables < 0] = 0
    batch.lengths[0], batch.lengths[1] = 10 ** 9, -5
    batch.starts[0], batch.starts[2] = -3, 10 ** 6
    out, lse = _run(batch)
    assert torch.isfinite(lse[22:]).all() and not out.eq(2.5).all(dim=2).any()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("order", ["up", "down"])
def test_gpu_running_max(order, fmt):
    """Keys sorted so that every row's max grows again and again, or never after the first block."""
    batch = Batch([(1500, 9)], 16, 77, fmt, q_sd=4.0)
    batch.q[:] = batch.q[:1, :1] * torch.linspace(0.5, 1.5, batch.T * 16).reshape(batch.T, 16, 1)
    slots = torch.from_numpy(batch.slots(0)[:1500])
    by = torch.argsort(torch.from_numpy(batch.rows())[slots] @ batch.q[0, 0].double(), descending=order == "down")
    batch.cache[slots] = batch.cache[slots[by]]
    _check(batch, *_run(batch))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_gpu_other_scales(scale):
    batch = Batch([(333, 3), (64, 20)], 16, 12)
    _check(batch, *_run(batch, scale), scale)


@pytest.mark.gpu
def test_gpu_nan_stays_in_its_row():
    batch = Batch([(900, 4), (50, 3)], 50, 13)
    want_o, want_l = _run(batch)
    batch.q[1, 3, 5] = float("nan")
    out, lse = _run(batch)
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
    same = torch.ones(batch.T, 50, dtype=torch.bool)
    same[1, 3] = False
    assert torch.equal(out[same], want_o[same]) and torch.equal(lse[same], want_l[same])


@pytest.mark.gpu
def test_gpu_no_tokens_and_no_sequences():
    batch = Batch([(100, 0), (0, 0)], 8, 14, pad=2)
    out, lse = _run(batch)
    assert out.eq(2.5).all() and lse.eq(2.5).all()
    d = batch.to(DEV)
    o, l = smla.sparse_mla_tree(d["q"][:0].contiguous(), d["kv_cache"], d["block_tables"], d["lengths"], d["starts"])
    assert o.shape == (0, 8, 512) and l.shape == (0, 8)
    smla.sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_repeated_calls_give_the_same_bytes(fmt):
    batch = Batch([(3000, 8), (100, 3), (777, 12), (2000, 1)], 16, 15, fmt)
    d = batch.to(DEV)
    first = smla.sparse_mla_tree(**d, kv_format=fmt)
    for _ in range(20):
        o, l = smla.sparse_mla_tree(**d, kv_format=fmt)
        assert torch.equal(o, first[0]) and torch.equal(l, first[1])
    smla.sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_streams_and_a_graph_whose_batch_grows(fmt):
    """Calls side by side on two streams; a captured call replayed after lengths, starts and mask have changed."""
    batches = [Batch([(900 + 50 * i, 5), (40, 9), (300, 2)], 16, 20 + i, fmt, extra_blocks=2) for i in range(3)]
    blocks = max(b.blocks for b in batches)
    dev = [b.to(DEV) for b in batches]
    for d in dev:
        d["block_tables"] = torch.nn.functional.pad(d["block_tables"], (0, blocks - d["block_tables"].shape[1]), value=-1).contiguous()
    want = [smla.sparse_mla_tree(**d, kv_format=fmt) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    got = [None] * len(dev)
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i] = smla.sparse_mla_tree(**dev[i], kv_format=fmt, stream=s)
    for s in streams:
        s.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    held = {k: v.clone() for k, v in dev[0].items()}
    rows = max(d["kv_cache"].shape[0] for d in dev)
    held["kv_cache"] = torch.zeros(rows, dev[0]["kv_cache"].shape[1], dtype=dev[0]["kv_cache"].dtype, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = smla.sparse_mla_tree(**held, kv_format=fmt)
    for i in (1, 0, 2):
        for k, v in dev[i].items():
            held[k][:v.shape[0]] = v
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    smla.sync_status()


@pytest.mark.gpu
def test_gpu_pages_past_32_bit_offsets():
    """A cache of more than 2^32 bytes, the sequence in its last pages."""
    batch = Batch([(300, 4)], 16, 16, spare=0)
    n = 2 ** 32 // (1152 * 64) + 40
    used = batch.cache.shape[0] // 64
    cache = torch.zeros((n * 64, 576), dtype=torch.bfloat16, device=DEV)
    cache[(n - used) * 64:] = batch.cache.to(DEV)
    d = batch.to(DEV)
    d["kv_cache"], d["block_tables"] = cache, d["block_tables"] + (n - used)
    out, lse = smla.sparse_mla_tree(**d)
    smla.sync_status()
    _check(batch, out.cpu(), lse.cpu())


@pytest.mark.gpu
def test_gpu_equals_the_forward_over_the_whole_list():
    """One token per sequence: the forward with every position listed."""
    batch = Batch([(500, 1), (90, 1), (1023, 1)], 16, 17)
    out, lse = _run(batch)
    lists = torch.full((3, 1024), -1, dtype=torch.int32)
    for b in range(3):
        s = torch.from_numpy(batch.slots(b))
        lists[b, :s.numel()] = s.int()
    wo, wl = smla.sparse_mla_fwd(batch.q.to(DEV), batch.cache.to(DEV), lists.to(DEV))
    smla.sync_status()
    assert (lse - wl.cpu()).abs().max().item() <= 1e-4
    v = ref.to64(batch.cache[torch.from_numpy(np.concatenate([batch.slots(b) for b in range(3)]))])
    assert (out.double() - wo.cpu().double()).abs().max().item() <= 3 * 2.0 ** -8 * np.abs(v).max()


# ----------------------------------------------------------------------------- refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    return smla.library()


def _c(lib, **kw):
    a = dict(q=0x1000, kv=0x1000, tables=0x1000, lengths=0x1000, starts=0x1000, mask=0x1000, T=4, h=8, seqs=2, blocks=3, words=1,
             num_slots=256, fmt=0, scale=0.04, out=0x1000, lse=0x1000, ws=0x1000, nws=1 << 40)
    a.update(kw)
    return lib.sparse_mla_tree(a["q"], a["kv"], a["tables"], a["lengths"], a["starts"], a["mask"], a["T"], a["h"], a["seqs"], a["blocks"],
                               a["words"], a["num_slots"], a["fmt"], a["scale"], a["out"], a["lse"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(kv=0), dict(tables=0), dict(lengths=0), dict(starts=0), dict(out=0), dict(lse=0), dict(T=-1), dict(h=0), dict(seqs=-1),
    dict(blocks=0), dict(blocks=1 << 25), dict(words=0), dict(num_slots=0), dict(num_slots=1 << 31), dict(fmt=2), dict(scale=float("nan")),
    dict(scale=float("-inf")), dict(q=0x1008), dict(kv=0x1004), dict(out=0x1002), dict(tables=0x1002), dict(lengths=0x1001),
    dict(starts=0x1002), dict(mask=0x1002), dict(lse=0x1001), dict(T=1 << 30, h=2)])
def test_the_library_refuses(lib, kw):
    assert _c(lib, **kw) == 1
    assert lib.sparse_mla_last_error().decode()


@pytest.mark.parametrize("kw", [dict(T=0), dict(seqs=0)])
def test_no_work_is_a_noop(lib, kw):
    assert _c(lib, q=0, kv=0, tables=0, lengths=0, starts=0, mask=0, out=0, lse=0, ws=0, nws=0, **kw) == 0


def test_workspace_bytes(lib):
    """Two slots of a tile's rows in groups of 32 for each of 76 CTA pairs (152 SMs assumed without a device), 16
    bytes for each tile or pair."""
    def up(x):
        return -(-x // 256) * 256

    assert smla.tree_workspace_bytes(0, 8, 1) == 0 and smla.tree_workspace_bytes(1, 8, 0) == 0
    assert smla.tree_workspace_bytes(1, 8, 1) == up(152 * 32 * 514 * 4) + 256
    assert smla.tree_workspace_bytes(512, 8, 32) == up(152 * 128 * 514 * 4) + up(64 * 16)
    assert smla.tree_workspace_bytes(512, 64, 8) == up(152 * 128 * 514 * 4) + up(76 * 16)
    assert smla.tree_workspace_bytes(5, 16, 1) == up(152 * 96 * 514 * 4) + 256


def _args():
    return dict(q=_d((3, 8, 576), torch.bfloat16), kv_cache=_d((640, 576), torch.bfloat16), block_tables=_d((2, 4), torch.int32),
                lengths=_d((2,), torch.int32), starts=_d((3,), torch.int32), mask=_d((3, 2), torch.int32))


def test_marshalling(fake, monkeypatch):
    a = _args()
    out, lse, ws = _d((3, 8, 512), torch.bfloat16), _d((3, 8), torch.float32), _d((4096,), torch.uint8)
    assert smla.sparse_mla_tree(**a, scale=0.25, out=out, lse=lse, workspace=ws) == (out, lse)
    p = {k: v.data_ptr() for k, v in a.items()}
    assert fake.lib.calls == [("sparse_mla_tree", (p["q"], p["kv_cache"], p["block_tables"], p["lengths"], p["starts"], p["mask"], 3, 8, 2, 4,
                                                   2, 640, 0, 0.25, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), 4096, STREAM))]
    assert fake.entered == [CUDA0]
    a.update(kv_cache=_d((640, 656), torch.uint8), mask=None)
    _binding._tree_workspace_bytes.cache_clear()
    smla.sparse_mla_tree(**a, out=out, lse=lse, kv_format="fp8", workspace=ws)
    name, args = fake.lib.calls[-1]
    assert args[5] is None and args[10] == 0 and args[12:14] == (1, 576 ** -0.5)


@pytest.mark.parametrize("kw", [
    dict(q=_d((3, 8, 512), torch.bfloat16)), dict(q=_d((3, 8, 576), torch.float32)), dict(q=torch.zeros(3, 8, 576, dtype=torch.bfloat16)),
    dict(kv_cache=_d((640, 656), torch.uint8)), dict(kv_cache=_d((640, 576), torch.bfloat16, 1)), dict(block_tables=_d((8,), torch.int32)),
    dict(block_tables=_d((2, 0), torch.int32)), dict(block_tables=_d((2, 4), torch.int64)), dict(block_tables=_d((3, 4), torch.int32)),
    dict(block_tables=_d((2, 4), torch.int32, 1)), dict(lengths=_d((3,), torch.int32)), dict(lengths=_d((2,), torch.int64)),
    dict(lengths=_d((2,), torch.int32, 1)), dict(starts=_d((2,), torch.int32)), dict(starts=_d((3,), torch.float32)),
    dict(starts=_d((3,), torch.int32, 1)), dict(mask=_d((2, 2), torch.int32)), dict(mask=_d((3, 0), torch.int32)),
    dict(mask=_d((3, 2), torch.int64)), dict(mask=_d((3, 2), torch.int32, 1)), dict(out=_d((3, 8, 576), torch.bfloat16)),
    dict(out=_d((3, 8, 512), torch.bfloat16, 1)), dict(lse=_d((3, 8), torch.float64)), dict(lse=torch.zeros(3, 8)),
    dict(workspace=_d((4096,), torch.float32)), dict(workspace=_d((4096,), torch.uint8, 1)), dict(kv_format="int8")])
def test_the_wrapper_refuses(fake, kw):
    a = dict(_args(), out=_d((3, 8, 512), torch.bfloat16), lse=_d((3, 8), torch.float32), workspace=_d((4096,), torch.uint8))
    a.update(kw)
    with pytest.raises(ValueError):
        smla.sparse_mla_tree(**a)
    assert fake.lib.calls == []
