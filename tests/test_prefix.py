"""sparse_mla_prefix: attention of a whole batch over one shared prefix.

Tolerances, against the definition in 64 bits over the rows that the kernel multiplies (fp8 rows
are dequantised to bf16, as the forward does):
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
from tests import step_reference as ref
from tests.step_reference import CUDA0, STREAM, _d, base_fake, fake  # noqa: F401

DEV = "cuda:0"
SCALE = 576 ** -0.5


def _case(T, h, P, seed, fmt="bf16", *, spare=3, q_sd=0.5, rows_past_end="nan"):
    """q, cache, pages; every row that is not the prefix's holds NaN (or what rows_past_end says)."""
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(T, h, 576, generator=g) * q_sd).to(torch.bfloat16)
    used = -(-P // 64)
    n = used + spare
    pages = torch.randperm(n, generator=g)[:used].int()
    x = torch.randn(n * 64, 576, generator=g) * 0.5
    live = torch.zeros(n * 64, dtype=torch.bool)
    at = torch.arange(P)
    live[pages.long()[at // 64] * 64 + at % 64] = True
    if fmt == "bf16":
        cache = x.to(torch.bfloat16)
        cache[~live] = float("nan") if rows_past_end == "nan" else float("inf")
    else:
        from workloads import quantize_fp8_rows
        cache = quantize_fp8_rows(x)
        cache[~live] = 0x7F  # NaN codes, NaN scales (0x7F7F7F7F is a huge finite one) and rope
        cache[~live, 512:528] = 0xFF
    return q, cache, pages


def _row_values(cache, fmt):
    """fp64 values of the rows as the kernel multiplies them."""
    if fmt == "bf16":
        return ref.to64(cache)
    v = torch.from_numpy(ref.fp8_row_values(cache))  # code * scale, exact in fp64
    return v.float().to(torch.bfloat16).double().numpy()


def _check(out, lse, q, cache, pages, P, fmt, scale=SCALE):
    rows = _row_values(cache, fmt)
    want_o, want_l = ref.prefix(q, rows, pages, P, scale)
    out, lse = ref.to64(out), ref.to64(lse)
    slots = [int(pages[i // 64]) * 64 + i % 64 for i in range(P) if int(pages[i // 64]) >= 0]
    slots = [s for s in slots if s < rows.shape[0]]
    if not slots:
        assert np.all(out == 0) and np.all(np.isneginf(lse))
        return
    k, x = np.abs(rows[slots]), np.abs(ref.to64(q))
    e = 576 * 2.0 ** -23 * abs(scale) * (x @ k.T).max(axis=2)
    assert np.all(np.abs(lse - want_l) <= e + 2.0 ** -22 * np.abs(want_l) + 2.0 ** -20)
    s = (ref.to64(q) @ rows[slots].T) * scale
    p = np.exp(s - want_l[:, :, None])
    pv = p @ k[:, :512]
    tol = (2.0 ** -8 + 2 * e[:, :, None]) * pv + 2.0 ** -8 * np.abs(want_o) + 1e-30
    assert np.all(np.abs(out - want_o) <= tol), float((np.abs(out - want_o) - tol).max())


def _run(q, cache, pages, P, fmt, scale=SCALE, **kw):
    T, h, _ = q.shape
    guard_o = torch.full((T + 2, h, 512), 2.5, dtype=torch.bfloat16, device=DEV)
    guard_l = torch.full((T + 2, h), 2.5, dtype=torch.float32, device=DEV)
    need = smla.prefix_workspace_bytes(T, h, P, fmt)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN where nothing is written
    out, lse = smla.sparse_mla_prefix(q.to(DEV), cache.to(DEV), pages.to(DEV), P, scale, out=guard_o[1:T + 1],
                                      lse=guard_l[1:T + 1], kv_format=fmt, workspace=ws, **kw)
    smla.sync_status()
    assert guard_o[0].eq(2.5).all() and guard_o[T + 1].eq(2.5).all()
    assert guard_l[0].eq(2.5).all() and guard_l[T + 1].eq(2.5).all()
    assert ws[need:].eq(0xFF).all()
    return out.cpu(), lse.cpu()


SHAPES = [(1, 16, 64), (1, 1, 1), (1, 16, 63), (2, 8, 65), (1, 16, 1000), (5, 13, 129), (16, 8, 500), (17, 8, 4096), (8, 16, 128), (130, 1, 257),
          (40, 16, 777), (64, 64, 70), (100, 64, 200), (3, 128, 640), (333, 8, 320), (1300, 8, 130),
          (170, 64, 300), (450, 8, 5100)]  # the last: runs that cross from a tile into the next, three pieces a tile


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("T,h,P", SHAPES)
def test_gpu_matches_the_definition(T, h, P, fmt):
    q, cache, pages = _case(T, h, P, 10 * T + P, fmt)
    out, lse = _run(q, cache, pages, P, fmt)
    _check(out, lse, q, cache, pages, P, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
def test_gpu_running_max(order, fmt):
    """Keys sorted so that every row's max grows again and again, or never after the first block."""
    T, h, P = 9, 16, 1500
    q, cache, pages = _case(T, h, P, 77, fmt, q_sd=4.0)
    if order != "mixed":
        at = torch.arange(P)
        slots = pages.long()[at // 64] * 64 + at % 64
        rows = torch.from_numpy(_row_values(cache, fmt))[slots]
        q[:] = q[:1, :1] * torch.linspace(0.5, 1.5, T * h).reshape(T, h, 1)
        by = torch.argsort(rows @ q[0, 0].double(), descending=order == "down")
        cache[slots] = cache[slots[by]]
    out, lse = _run(q, cache, pages, P, fmt)
    _check(out, lse, q, cache, pages, P, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_pages_outside_the_cache_are_masked(fmt):
    T, h, P = 7, 16, 700
    q, cache, pages = _case(T, h, P, 5, fmt)
    pages[0], pages[3], pages[4], pages[10] = -1, cache.shape[0] // 64, 2 ** 31 - 1, -2 ** 31
    out, lse = _run(q, cache, pages, P, fmt)
    _check(out, lse, q, cache, pages, P, fmt)
    pages[:] = -1
    out, lse = _run(q, cache, pages, P, fmt)
    assert out.eq(0).all() and torch.isneginf(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("short", [1, 30, 33, 63])
def test_gpu_cache_that_ends_inside_a_page(fmt, short):
    """num_slots is no multiple of 64: the last page's missing rows are masked."""
    T, h, P = 3, 24, 512
    q, cache, pages = _case(T, h, P, 6, fmt, spare=0)
    at = torch.arange(P)
    cache = cache[:cache.shape[0] - short].contiguous()
    out, lse = _run(q, cache, pages, P, fmt)
    _check(out, lse, q, cache, pages, P, fmt)
    assert at.numel() == P


@pytest.mark.gpu
def test_gpu_rows_past_the_end_may_hold_infinities():
    T, h, P = 4, 40, 100
    q, cache, pages = _case(T, h, P, 8, rows_past_end="inf")
    out, lse = _run(q, cache, pages, P, "bf16")
    _check(out, lse, q, cache, pages, P, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_gpu_other_scales(scale):
    T, h, P = 3, 16, 333
    q, cache, pages = _case(T, h, P, 9)
    out, lse = _run(q, cache, pages, P, "bf16", scale)
    _check(out, lse, q, cache, pages, P, "bf16", scale)


@pytest.mark.gpu
def test_gpu_nan_stays_in_its_row():
    T, h, P = 4, 50, 900
    q, cache, pages = _case(T, h, P, 12)
    q[1, 3, 5] = float("nan")
    out, lse = _run(q, cache, pages, P, "bf16")
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
    q[1, 3, 5] = 0.25
    ref_o, ref_l = _run(q, cache, pages, P, "bf16")
    same = torch.ones(T, h, dtype=torch.bool)
    same[1, 3] = False
    assert torch.equal(out[same], ref_o[same]) and torch.equal(lse[same], ref_l[same])


@pytest.mark.gpu
def test_gpu_empty_prefix_and_no_tokens():
    q, cache, pages = _case(5, 8, 64, 13)
    out, lse = _run(q, cache, pages, 0, "bf16")
    assert out.eq(0).all() and torch.isneginf(lse).all()
    o, l = smla.sparse_mla_prefix(q[:0].contiguous().to(DEV), cache.to(DEV), pages.to(DEV), 64)
    assert o.shape == (0, 8, 512) and l.shape == (0, 8)
    smla.sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_repeated_calls_give_the_same_bytes(fmt):
    q, cache, pages = _case(33, 16, 3000, 14, fmt)
    d = [x.to(DEV) for x in (q, cache, pages)]
    first = smla.sparse_mla_prefix(*d, 3000, kv_format=fmt)
    for _ in range(20):
        o, l = smla.sparse_mla_prefix(*d, 3000, kv_format=fmt)
        assert torch.equal(o, first[0]) and torch.equal(l, first[1])
    smla.sync_status()


@pytest.mark.gpu
def test_gpu_streams_and_graphs_with_their_own_workspaces():
    P = 2000
    cases = [_case(20 + i, 16, P, 20 + i) for i in range(2)]
    dev = [[x.to(DEV) for x in c] for c in cases]
    want = [smla.sparse_mla_prefix(*d, P) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    got = [None, None]
    for _ in range(10):  # side by side, each with the workspace its own stream allocated
        for i, s in enumerate(streams):
            got[i] = smla.sparse_mla_prefix(*dev[i], P, stream=s)
    for s in streams:
        s.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    graphs, outs = [], []
    for d in dev:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(smla.sparse_mla_prefix(*d, P))
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for g, w in zip(outs, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    smla.sync_status()


@pytest.mark.gpu
def test_gpu_pages_past_32_bit_offsets():
    """A cache of more than 2^32 bytes, the prefix in its last pages."""
    P, n = 300, 2 ** 32 // (1152 * 64) + 40
    q, small, _ = _case(3, 16, P, 15, spare=0)
    used = small.shape[0] // 64
    cache = torch.zeros((n * 64, 576), dtype=torch.bfloat16, device=DEV)
    pages = torch.arange(n - used, n, dtype=torch.int32)
    _, _, order = _case(3, 16, P, 15, spare=0)
    for i, pg in enumerate(order):
        cache[(n - used + i) * 64:(n - used + i + 1) * 64] = small[int(pg) * 64:int(pg) * 64 + 64].to(DEV)
    o, l = smla.sparse_mla_prefix(q.to(DEV), cache, pages.to(DEV), P)
    smla.sync_status()
    _check(o.cpu(), l.cpu(), q, small, order, P, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_prefix_merged_with_each_tokens_own_part(fmt):
    """prefix + own lists through the merge = the forward over the whole lists."""
    T, h, P, own = 12, 16, 640, 96
    g = torch.Generator().manual_seed(3)
    q, cache, pages = _case(T, h, P + 64 * T * 2, 31, fmt, spare=0)
    mine = pages[P // 64:].reshape(T, -1).long()
    pick = torch.stack([torch.randperm(mine.shape[1] * 64, generator=g)[:own] for _ in range(T)])
    own_slots = (mine.gather(1, pick // 64) * 64 + pick % 64).int()
    at = torch.arange(P)
    shared = (pages.long()[at // 64] * 64 + at % 64).int()
    d = [x.to(DEV) for x in (q, cache, pages[:P // 64].contiguous(), own_slots)]
    parts_o = torch.empty(2, T, h, 512, dtype=torch.bfloat16, device=DEV)
    parts_l = torch.empty(2, T, h, dtype=torch.float32, device=DEV)
    smla.sparse_mla_prefix(d[0], d[1], d[2], P, SCALE, out=parts_o[0], lse=parts_l[0], kv_format=fmt)
    smla.sparse_mla_fwd(d[0], d[1], d[3], SCALE, out=parts_o[1], lse=parts_l[1], kv_format=fmt)
    o, l = smla.sparse_mla_merge(parts_o, parts_l)
    whole = torch.cat([shared[None].expand(T, -1), own_slots], dim=1).contiguous().to(DEV)
    wo, wl = smla.sparse_mla_fwd(d[0], d[1], whole, SCALE, kv_format=fmt)
    smla.sync_status()
    # both sides round probabilities and O to bf16; the merged one rounds each part's O as well
    v = np.abs(_row_values(cache, fmt)[:, :512]).max()
    assert (l - wl).abs().max().item() <= 1e-4
    assert (o.double() - wo.double()).abs().max().item() <= 4 * 2.0 ** -8 * v


# ----------------------------------------------------------------------------- refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    return smla.library()


def _c(lib, **kw):
    a = dict(q=0x1000, kv=0x1000, pages=0x1000, T=4, h=8, P=100, num_slots=256, fmt=0, scale=0.04, out=0x1000, lse=0x1000,
             ws=0x1000, nws=1 << 40)
    a.update(kw)
    return lib.sparse_mla_prefix(a["q"], a["kv"], a["pages"], a["T"], a["h"], a["P"], a["num_slots"], a["fmt"], a["scale"], a["out"],
                                 a["lse"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(kv=0), dict(pages=0), dict(out=0), dict(lse=0), dict(T=-1), dict(h=0), dict(P=-1), dict(P=1 << 31),
    dict(num_slots=0), dict(num_slots=1 << 31), dict(fmt=3), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=0x1008),
    dict(kv=0x1004), dict(out=0x1002), dict(pages=0x1002), dict(lse=0x1001), dict(T=1 << 30, h=2)])
def test_the_library_refuses(lib, kw):
    assert _c(lib, **kw) == 1
    assert lib.sparse_mla_last_error().decode()


def test_no_tokens_is_a_noop(lib):
    assert _c(lib, T=0, q=0, kv=0, pages=0, out=0, lse=0, ws=0, nws=0) == 0


def test_workspace_bytes(lib):
    """None where no tile is cut, else two slots of a tile's rows, in groups of 32, per CTA pair (152
    SMs assumed without a device), rounded up to 256 bytes."""

    def partials(runs, rows):
        return -(-2 * runs * (-(-rows // 32) * 32) * 514 * 4 // 256) * 256

    assert smla.prefix_workspace_bytes(0, 8, 100) == 0 and smla.prefix_workspace_bytes(1, 8, 0) == 0
    assert smla.prefix_workspace_bytes(1, 8, 128) == 0
    assert smla.prefix_workspace_bytes(16 * 76, 8, 128 * 5) == 0
    assert smla.prefix_workspace_bytes(1, 16, 129) == 0  # two blocks: not worth a merge
    assert smla.prefix_workspace_bytes(1, 16, 1000) == partials(8, 16)
    assert smla.prefix_workspace_bytes(8, 16, 8192) == partials(32, 128)  # two blocks a run
    assert smla.prefix_workspace_bytes(128, 64, 32768) == partials(76, 128)
    with pytest.raises(ValueError, match="kv_format"):
        smla.prefix_workspace_bytes(1, 8, 128, "int8")
    # an fp8 prefix also has its whole pages as bf16 rows
    assert smla.prefix_workspace_bytes(1, 8, 100, "fp8") == 128 * 1152
    assert smla.prefix_workspace_bytes(1, 16, 1000, "fp8") == partials(8, 16) + 1024 * 1152


def _args(T=3, h=8, P=130):
    return [_d((T, h, 576), torch.bfloat16), _d((640, 576), torch.bfloat16), _d((3,), torch.int32), P]


def test_marshalling(fake, monkeypatch):
    q, kv, pages, P = _args()
    out, lse, ws = _d((3, 8, 512), torch.bfloat16), _d((3, 8), torch.float32), _d((4096,), torch.uint8)
    assert smla.sparse_mla_prefix(q, kv, pages, P, 0.25, out=out, lse=lse, workspace=ws) == (out, lse)
    assert fake.lib.calls == [("sparse_mla_prefix", (q.data_ptr(), kv.data_ptr(), pages.data_ptr(), 3, 8, P, 640, 0, 0.25,
                                                     out.data_ptr(), lse.data_ptr(), ws.data_ptr(), 4096, STREAM))]
    assert fake.entered == [CUDA0]
    fp8 = _d((640, 656), torch.uint8)
    smla.sparse_mla_prefix(q, fp8, pages, P, out=out, lse=lse, kv_format="fp8")  # the stand-in asks for no workspace
    name, args = fake.lib.calls[-1]
    assert name == "sparse_mla_prefix" and args[7:9] == (1, 576 ** -0.5) and args[11:13] == (None, 0)


@pytest.mark.parametrize("i,bad", [
    (0, _d((3, 8, 512), torch.bfloat16)), (0, _d((3, 8, 576), torch.float32)), (0, torch.zeros(3, 8, 576, dtype=torch.bfloat16)),
    (1, _d((640, 656), torch.uint8)), (1, _d((640, 576), torch.bfloat16, 1)), (2, _d((2,), torch.int32)), (2, _d((3,), torch.int64)),
    (2, _d((1, 3), torch.int32)), (3, -1), (3, 193)])
def test_the_wrapper_refuses(fake, i, bad):
    a = _args()
    a[i] = bad
    with pytest.raises(ValueError):
        smla.sparse_mla_prefix(*a)
    assert fake.lib.calls == []


@pytest.mark.parametrize("kw", [
    dict(out=_d((3, 8, 576), torch.bfloat16)), dict(out=_d((3, 8, 512), torch.bfloat16, 1)), dict(lse=_d((3, 8), torch.float64)),
    dict(lse=torch.zeros(3, 8)), dict(workspace=_d((4096,), torch.float32)), dict(workspace=_d((4096,), torch.uint8, 1)),
    dict(kv_format="int8")])
def test_the_wrapper_refuses_what_it_writes(fake, kw):
    a = _args()
    kw = dict(dict(out=_d((3, 8, 512), torch.bfloat16), lse=_d((3, 8), torch.float32)), **kw)
    with pytest.raises(ValueError):
        smla.sparse_mla_prefix(*a, **kw)
    assert fake.lib.calls == []
