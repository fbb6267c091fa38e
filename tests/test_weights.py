"""sparse_mla_weights: the attention weight that every cached row of a batch has gathered.

Tolerance, against the definition in 64 bits over the rows that the kernel multiplies (fp8 rows dequantised to
bf16) and the lse that it is given: a logit is an fp32 sum of 576 exact products, off by at most 576 * 2^-23
of their absolute sum; y = logit - lse is rounded once (2^-24 of |y|), its product with log2 e once more, and
2^ of it is off by 2^-22; a position's sum of N probabilities and its weight before are added in fp32, off by
(N + 3) * 2^-24 of the result, all terms being positive.
"""

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import batch_reference as br
from tests import step_reference as ref
from tests.batch_reference import SCALE, Batch
from tests.step_reference import CUDA0, STREAM, _d, base_fake, fake  # noqa: F401
from tests.test_tree import BATCHES

DEV = "cuda:0"


def _inputs(batch, seed=0, scale=SCALE):
    """lse of the attention (rows of no sequence: NaN) and weights gathered before (past the cached rows: NaN)."""
    lse = torch.from_numpy(br.tree(batch, scale)[1]).float()
    g = torch.Generator().manual_seed(seed)
    prev = torch.empty(len(batch.seqs), batch.blocks * 64).exponential_(1.0, generator=g)
    for b, (n, _) in enumerate(batch.seqs):
        prev[b, n:] = float("nan")
    return lse, prev


def _run(batch, lse, prev, decay, scale=SCALE, in_place=False, **kw):
    d = batch.to(DEV)
    shape = (len(batch.seqs), batch.blocks * 64)
    guard = torch.full((shape[0] + 2, shape[1]), 2.5, dtype=torch.float32, device=DEV)
    held = guard[1:shape[0] + 1]
    before = None
    if prev is not None:
        before = prev.to(DEV)
        if in_place:
            held.copy_(before)
            before = held
    out = smla.sparse_mla_weights(**d, lse=lse.to(DEV), scale=scale, weights=before, decay=decay, out=held, kv_format=batch.fmt, **kw)
    smla.sync_status()
    assert guard[0].eq(2.5).all() and guard[-1].eq(2.5).all()
    return out.cpu()


def _check(batch, out, lse, prev, decay, scale=SCALE):
    want, tol = br.weights(batch, lse, prev, decay, scale)
    got = ref.to64(out)
    assert np.all(np.abs(got - want) <= tol), float(np.nanmax(np.abs(got - want) - tol))
    assert np.isfinite(got).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_gpu_matches_the_definition(i, fmt):
    seqs, h = BATCHES[i]
    batch = Batch(seqs, h, 200 + i, fmt, pad=i % 3, lead=i % 2, extra_blocks=i % 4)
    lse, prev = _inputs(batch, i)
    _check(batch, _run(batch, lse, prev, 0.75, in_place=i % 2 == 0), lse, prev, 0.75)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("tree", ["chain", "any", "none"])
def test_gpu_masks(tree, fmt):
    batch = Batch([(0, 40), (70, 40), (63, 9), (500, 17), (0, 1), (5, 0), (300, 3)], 16, 7, fmt, tree=tree)
    lse, prev = _inputs(batch)
    _check(batch, _run(batch, lse, prev, 1.0), lse, prev, 1.0)
    _check(batch, _run(batch, lse, None, 0.5), lse, None, 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_sums_are_the_probabilities(fmt):
    """With the lse that sparse_mla_tree gives, the weights of a sequence add up to its tokens times heads."""
    batch = Batch([(700, 6), (64, 40), (0, 3)], 16, 8, fmt)
    d = batch.to(DEV)
    _, lse = smla.sparse_mla_tree(**d, kv_format=fmt)
    out = smla.sparse_mla_weights(**d, lse=lse, kv_format=fmt)
    smla.sync_status()
    want = torch.tensor([dr * 16.0 for _, dr in batch.seqs], dtype=torch.float64)
    assert torch.allclose(out.cpu().double().sum(dim=1), want, rtol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_pages_outside_the_cache_and_a_cache_that_ends_inside_a_page(fmt):
    batch = Batch([(700, 7), (64, 3)], 16, 5, fmt, spare=0)
    batch.tables[0, 2], batch.tables[0, 5] = -1, 2 ** 31 - 1
    batch.cache = batch.cache[:batch.cache.shape[0] - 33].contiguous()
    lse, prev = _inputs(batch)
    _check(batch, _run(batch, lse, prev, 0.9), lse, prev, 0.9)
    batch.tables[:] = -1
    lse = torch.full_like(lse, float("-inf"))
    _check(batch, _run(batch, lse, prev, 0.9), lse, prev, 0.9)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_drafted_rows_that_are_not_seen_may_hold_anything(fmt):
    batch, hurt = (Batch([(100, 20), (62, 5), (0, 33)], 16, 9, fmt, tree="random") for _ in range(2))
    for b, j in ((0, 19), (1, 4), (2, 32)):
        for x in (batch, hurt):  # nobody sees these, not the token itself either
            x.sees[b][:, j] = False
            x.mask = x.pack()
        hurt.cache[int(hurt.slots(b)[hurt.seqs[b][0] + j])] = float("nan") if fmt == "bf16" else 0xFF
    lse, prev = _inputs(batch)
    out = _run(hurt, lse, prev, 0.9)
    assert torch.equal(out, _run(batch, lse, prev, 0.9))
    _check(batch, out, lse, prev, 0.9)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_gpu_other_scales(scale):
    batch = Batch([(333, 3), (64, 20)], 16, 12)
    lse, prev = _inputs(batch, scale=scale)
    _check(batch, _run(batch, lse, prev, 1.5, scale), lse, prev, 1.5, scale)


@pytest.mark.gpu
def test_gpu_no_tokens_keep_the_decayed_weights():
    batch = Batch([(100, 0), (0, 0), (64, 0)], 8, 14, pad=2, extra_blocks=70)
    prev = torch.rand(3, batch.blocks * 64)
    lse = torch.zeros(2, 8)
    _check(batch, _run(batch, lse, prev, 0.5), lse, prev, 0.5)
    none = Batch([(100, 0), (0, 0), (64, 0)], 8, 14)
    assert none.T == 0
    _check(none, _run(none, torch.zeros(0, 8), prev[:, :none.blocks * 64].contiguous(), 0.5), torch.zeros(0, 8),
           prev[:, :none.blocks * 64], 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_repeated_calls_streams_and_a_graph_give_the_same_bytes(fmt):
    batches = [Batch([(3000 + i, 8), (100, 3), (777, 40), (2000, 1)], 16, 15 + i, fmt) for i in range(2)]
    dev = [b.to(DEV) for b in batches]
    ins = [[x.to(DEV) for x in _inputs(b)] for b in batches]

    def call(i, **kw):
        return smla.sparse_mla_weights(**dev[i], lse=ins[i][0], weights=ins[i][1], decay=0.9, kv_format=fmt, **kw)

    want = [call(0), call(1)]
    for _ in range(10):
        assert torch.equal(call(0), want[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [call(i, stream=s) for i, s in enumerate(streams)]
    for s in streams:
        s.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(1)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[1])
    smla.sync_status()


# ----------------------------------------------------------------------------- refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    return smla.library()


def _c(lib, **kw):
    a = dict(q=0x1000, kv=0x1000, tables=0x1000, lengths=0x1000, starts=0x1000, mask=0x1000, lse=0x1000, prev=0x1000, decay=0.5, T=4, h=8,
             seqs=2, blocks=3, words=1, num_slots=256, fmt=0, scale=0.04, out=0x1000)
    a.update(kw)
    return lib.sparse_mla_weights(a["q"], a["kv"], a["tables"], a["lengths"], a["starts"], a["mask"], a["lse"], a["prev"], a["decay"],
                                  a["T"], a["h"], a["seqs"], a["blocks"], a["words"], a["num_slots"], a["fmt"], a["scale"], a["out"], None)


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(kv=0), dict(tables=0), dict(lengths=0), dict(starts=0), dict(out=0), dict(lse=0), dict(T=-1), dict(h=0), dict(seqs=-1),
    dict(blocks=0), dict(blocks=1 << 25), dict(words=0), dict(num_slots=0), dict(num_slots=1 << 31), dict(fmt=2), dict(scale=float("nan")),
    dict(decay=float("nan")), dict(decay=float("inf")), dict(q=0x1008), dict(kv=0x1004), dict(out=0x1002), dict(tables=0x1002),
    dict(lengths=0x1001), dict(starts=0x1002), dict(mask=0x1002), dict(lse=0x1001), dict(prev=0x1001), dict(T=1 << 30, h=2)])
def test_the_library_refuses(lib, kw):
    assert _c(lib, **kw) == 1
    assert lib.sparse_mla_last_error().decode()


def test_no_sequences_is_a_noop(lib):
    assert _c(lib, seqs=0, q=0, kv=0, tables=0, lengths=0, starts=0, mask=0, lse=0, prev=0, out=0) == 0


def _args():
    return dict(q=_d((3, 8, 576), torch.bfloat16), kv_cache=_d((640, 576), torch.bfloat16), block_tables=_d((2, 4), torch.int32),
                lengths=_d((2,), torch.int32), starts=_d((3,), torch.int32), mask=_d((3, 2), torch.int32), lse=_d((3, 8), torch.float32),
                weights=_d((2, 256), torch.float32), out=_d((2, 256), torch.float32))


def test_marshalling(fake):
    a = _args()
    assert smla.sparse_mla_weights(**a, scale=0.25, decay=0.5) is a["out"]
    p = {k: v.data_ptr() for k, v in a.items()}
    assert fake.lib.calls == [("sparse_mla_weights", (
        p["q"], p["kv_cache"], p["block_tables"], p["lengths"], p["starts"], p["mask"], p["lse"], p["weights"], 0.5, 3, 8, 2, 4, 2, 640, 0,
        0.25, p["out"], STREAM))]
    assert fake.entered == [CUDA0]
    a.update(kv_cache=_d((640, 656), torch.uint8), mask=None, weights=None)
    smla.sparse_mla_weights(**a, kv_format="fp8")
    args = fake.lib.calls[-1][1]
    assert args[5] is None and args[7:9] == (None, 1.0) and args[13] == 0 and args[15:17] == (1, 576 ** -0.5)


@pytest.mark.parametrize("kw", [
    dict(q=_d((3, 8, 512), torch.bfloat16)), dict(q=torch.zeros(3, 8, 576, dtype=torch.bfloat16)), dict(kv_cache=_d((640, 656), torch.uint8)),
    dict(kv_cache=_d((640, 576), torch.bfloat16, 1)), dict(block_tables=_d((2, 0), torch.int32)), dict(lengths=_d((3,), torch.int32)),
    dict(starts=_d((2,), torch.int32)), dict(mask=_d((3, 0), torch.int32)), dict(lse=_d((3,), torch.float32)),
    dict(lse=_d((3, 8), torch.float32, 1)), dict(lse=_d((3, 8), torch.bfloat16)), dict(weights=_d((2, 255), torch.float32)),
    dict(weights=_d((2, 256), torch.float64)), dict(weights=_d((2, 256), torch.float32, 1)), dict(out=_d((2, 512), torch.float32)),
    dict(out=torch.zeros(2, 256)), dict(kv_format="int8")])
def test_the_wrapper_refuses(fake, kw):
    a = dict(_args())
    a.update(kw)
    with pytest.raises(ValueError):
        smla.sparse_mla_weights(**a)
    assert fake.lib.calls == []
