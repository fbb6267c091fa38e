"""sparse_mla_append: rows written into the paged latent cache.

Tolerances.  bf16 rows: the kernel computes in fp32 and rounds once, so a value is off by half a
bf16 step (2^-8 relative, counting a value at the low end of its binade) plus the fp32 error of
what it rounds.  Without the norm the latent is copied (exact).  With it, n = c * r * w has three
roundings (r's rsqrt: two units; 512 squares summed: at most a few units) -- 2^-20 covers them
sixteen times over.  A rotated value is a sum of two products: 4 * 2^-24 of their absolute sum.
fp8 rows: the code is the nearest of e4m3 (2^-4 relative of a normal code; below 2^-6 half of the
smallest step, 2^-10, each times the tile's scale) and the scale a rounded quotient.
"""

import ctypes

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import step_reference as ref
from tests.step_reference import CUDA0, STREAM, _d, base_fake, fake  # noqa: F401

DEV = "cuda:0"
F32 = 2.0 ** -20


def _case(T, num_slots, seed, *, stride=576, max_pos=300, sd=1.0):
    g = torch.Generator().manual_seed(seed)
    base = (torch.randn(max(T, 1), stride, generator=g) * sd).to(torch.bfloat16)
    kv = base[:T, :576]
    slots = torch.randperm(num_slots, generator=g)[:T].int()
    pos = torch.randint(0, max_pos, (T,), generator=g).int()
    w = (1 + 0.2 * torch.randn(512, generator=g)).to(torch.bfloat16)
    return kv, pos, slots, w, ref.cos_sin_table(max_pos)


def _empty_cache(num_slots, fmt):
    if fmt == "bf16":
        return torch.full((num_slots, 576), 7.25, dtype=torch.bfloat16)
    return torch.full((num_slots, 656), 0x5A, dtype=torch.uint8)


def _run(kv, pos, slots, cache, table, **kw):
    base = kv._base if kv._base is not None else kv
    dbase = base.to(DEV)
    dkv = dbase[:kv.shape[0], :576]
    dc = cache.to(DEV)
    w = kw.pop("norm_weight", None)
    got = smla.sparse_mla_append(dkv, pos.to(DEV), slots.to(DEV), dc, table.to(DEV),
                                 norm_weight=None if w is None else w.to(DEV), **kw)
    assert got is dc
    return dc


def _check_rows(before, after, kv, pos, slots, table, weight, eps, interleaved, fmt):
    after = after.cpu()
    want = ref.append_values(kv, pos, table, weight, eps, interleaved)
    keep = [t for t in range(len(slots)) if 0 <= int(slots[t]) < before.shape[0] and np.isfinite(want[t, 0])]
    written = {int(slots[t]) for t in keep}
    rest = [s for s in range(before.shape[0]) if s not in written]
    assert torch.equal(after[rest].view(torch.uint8), before[rest].view(torch.uint8)), "rows that no token names"
    if not keep:
        return
    rows, w64 = after[[int(slots[t]) for t in keep]], want[keep]
    x = ref.to64(kv)[keep]
    # two products of a rotated value: |a cos| + |b sin| <= |a| + |b|
    pair = np.abs(x[:, 512:])
    pair_sum = (pair + (pair.reshape(-1, 32, 2)[:, :, ::-1].reshape(-1, 64) if interleaved
                        else np.roll(pair, 32, axis=1)))
    if fmt == "bf16":
        got = ref.to64(rows)
        lat_tol = (2.0 ** -8 + F32) * np.abs(w64[:, :512]) if weight is not None else 0.0
    else:
        got = ref.fp8_row_values(rows)
        tiles = np.abs(w64[:, :512]).reshape(-1, 4, 128)
        scale = tiles.max(axis=2, keepdims=True) / 448.0
        lat_tol = np.maximum((2.0 ** -4) * tiles, 2.0 ** -10 * scale).reshape(-1, 512) * (1 + F32) + F32 * np.abs(w64[:, :512])
    assert np.all(np.abs(got[:, :512] - w64[:, :512]) <= lat_tol)
    rope_tol = 2.0 ** -8 * np.abs(w64[:, 512:]) * (1 + F32) + 4 * 2.0 ** -24 * pair_sum
    assert np.all(np.abs(got[:, 512:] - w64[:, 512:]) <= rope_tol)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("T,norm,interleaved,stride", [(1, True, True, 576), (2, False, False, 584), (3, True, False, 2112),
                                                       (31, True, True, 2112), (129, False, True, 576), (1000, True, False, 640)])
def test_gpu_rows_match_the_definition(fmt, T, norm, interleaved, stride):
    num_slots = 2 * T + 70
    kv, pos, slots, w, table = _case(T, num_slots, 100 + T, stride=stride)
    w = w if norm else None
    before = _empty_cache(num_slots, fmt)
    after = _run(kv, pos, slots, before, table, norm_weight=w, eps=1e-5, interleaved=interleaved, kv_format=fmt)
    smla.sync_status()
    _check_rows(before, after, kv, pos, slots, table, w, 1e-5, interleaved, fmt)


@pytest.mark.gpu
def test_gpu_codes_equal_the_cache_generator():
    """Without the norm the fp8 rows are what the workloads' quantiser packs, byte for byte, and the
    rows read through the forward as the same rows do."""
    from workloads import quantize_fp8_rows
    T = 200
    kv, pos, slots, _, table = _case(T, 256, 5, sd=0.5)
    pos.zero_()  # angle 0: the rope dims stay as they are
    after = _run(kv, pos, slots, torch.zeros(256, 656, dtype=torch.uint8), table, kv_format="fp8").cpu()
    smla.sync_status()
    assert torch.equal(after[slots.long()], quantize_fp8_rows(kv.float()))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_gpu_padded_batch_leaves_the_cache(fmt):
    T, num_slots = 77, 100
    kv, pos, slots, w, table = _case(T, num_slots, 9)
    slots[40:] = -1
    pos[41:] = -1  # an unused place may carry any position
    before = _empty_cache(num_slots, fmt)
    after = _run(kv, pos, slots, before, table, norm_weight=w, kv_format=fmt)
    smla.sync_status()
    _check_rows(before, after, kv, pos, slots, table, w, 1e-6, True, fmt)
    slots.fill_(-1)
    after = _run(kv, pos, slots, before, table, norm_weight=w, kv_format=fmt)
    smla.sync_status()
    assert torch.equal(after.cpu(), before)


@pytest.mark.gpu
@pytest.mark.parametrize("what,value", [("slot", 100), ("slot", -2), ("slot", 2 ** 31 - 1), ("position", 300), ("position", -1),
                                        ("position", -2 ** 31)])
def test_gpu_out_of_range_is_skipped_and_reported(what, value):
    T, num_slots = 9, 100
    kv, pos, slots, _, table = _case(T, num_slots, 11)
    (slots if what == "slot" else pos)[4] = value
    before = _empty_cache(num_slots, "bf16")
    after = _run(kv, pos, slots, before, table)
    with pytest.raises(smla.SparseMLAError) as e:
        smla.sync_status()
    assert e.value.status == 5 and "append" in str(e.value)
    smla.sync_status()  # read and cleared
    _check_rows(before, after, kv, pos, slots, table, None, 0.0, True, "bf16")


@pytest.mark.gpu
def test_gpu_special_values_in_fp8_rows():
    """A tile of zeros has scale 1 and zero codes; a NaN makes its own tile NaN and no other; an
    infinity makes its tile's scale infinite; the smallest bf16 still has a scale."""
    kv = torch.zeros(4, 576, dtype=torch.bfloat16)
    kv[1, 130], kv[1, 5] = float("nan"), 3.0
    kv[2, 300], kv[2, 400] = float("inf"), 1.0
    kv[3, 7] = torch.tensor([1], dtype=torch.int16).view(torch.bfloat16)[0]  # 2^-133
    kv[3, 200] = 1.0
    slots, pos = torch.arange(4).int(), torch.zeros(4).int()
    after = _run(kv, pos, slots, torch.full((4, 656), 0x33, dtype=torch.uint8), ref.cos_sin_table(1), kv_format="fp8").cpu()
    smla.sync_status()
    assert after[0, :512].eq(0).all() and after[0, 512:528].view(torch.float32).eq(1.0).all()
    val = ref.fp8_row_values(after)
    one = 1.0 + 2.0 ** -23  # a tile's largest value is 448 times the rounded quotient of it by 448
    assert np.isnan(val[1, 128:256]).all() and 3.0 / one <= val[1, 5] <= 3.0 * one and np.isfinite(val[1, :128]).all() and (val[1, 256:] == 0).all()
    assert np.isinf(after[2, 512:528].view(torch.float32)[2].item()) and 1 / one <= val[2, 400] <= one
    assert val[3, 7] > 0 and 1 / one <= val[3, 200] <= one


@pytest.mark.gpu
def test_gpu_rows_past_32_bit_offsets():
    """A cache of more than 2^31 elements: the last slots are written, slot 0 is not."""
    num_slots = 2 ** 32 // 1152 + 4096  # more than 2^32 bytes
    cache = torch.zeros((num_slots, 576), dtype=torch.bfloat16, device=DEV)
    kv, pos, _, w, table = _case(3, 10, 13)
    slots = torch.tensor([num_slots - 1, num_slots - 700, 2 ** 31 // 576 + 1], dtype=torch.int32)
    smla.sparse_mla_append(kv.to(DEV), pos.to(DEV), slots.to(DEV), cache, table.to(DEV), norm_weight=w.to(DEV))
    smla.sync_status()
    rows = cache[slots.long().to(DEV)].cpu()
    want = ref.append_values(kv, pos, table, w, 1e-6, True)
    assert np.all(np.abs(ref.to64(rows) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)
    assert int(torch.count_nonzero(cache).item()) == int(torch.count_nonzero(rows).item())


@pytest.mark.gpu
def test_gpu_captured_and_on_another_stream():
    T, num_slots = 40, 64
    kv, pos, slots, w, table = _case(T, num_slots, 17)
    d = [x.to(DEV) for x in (kv, pos, slots, table, w)]
    want = _run(kv, pos, slots, torch.zeros(num_slots, 576, dtype=torch.bfloat16), table, norm_weight=w)
    cache = torch.zeros(num_slots, 576, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    smla.sparse_mla_append(d[0], d[1], d[2], cache, d[3], norm_weight=d[4], stream=s)
    s.synchronize()
    assert torch.equal(cache, want)
    graph = torch.cuda.CUDAGraph()
    cache.zero_()
    with torch.cuda.graph(graph):
        smla.sparse_mla_append(d[0], d[1], d[2], cache, d[3], norm_weight=d[4])
    assert int(torch.count_nonzero(cache)) == 0
    d[0].mul_(2)  # the replay reads what the buffers hold then; the norm takes the factor out
    d[4].mul_(0.5)
    graph.replay()
    smla.sync_status()
    half = ref.append_values(kv.float().mul(2).to(torch.bfloat16), pos, table, w.mul(0.5), 1e-6, True)
    got = ref.to64(cache)[slots.long().numpy()]
    assert np.all(np.abs(got - half) <= 2.0 ** -8 * np.abs(half) + 1e-5)


# ----------------------------------------------------------------------------- refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    return smla.library()


def _c(lib, **kw):
    a = dict(kv=0x1000, stride=576, pos=0x1000, slots=0x1000, T=4, cs=0x1000, max_pos=10, inter=1, w=0, eps=1e-6,
             cache=0x1000, num_slots=64, fmt=0)
    a.update(kw)
    return lib.sparse_mla_append(a["kv"], a["stride"], a["pos"], a["slots"], a["T"], a["cs"], a["max_pos"], a["inter"],
                                 a["w"], a["eps"], a["cache"], a["num_slots"], a["fmt"], None)


@pytest.mark.parametrize("kw", [
    dict(kv=0), dict(pos=0), dict(slots=0), dict(cs=0), dict(cache=0), dict(T=-1), dict(stride=568), dict(stride=580),
    dict(stride=0), dict(stride=-576), dict(max_pos=0), dict(num_slots=0), dict(num_slots=1 << 31), dict(fmt=2),
    dict(kv=0x1008), dict(cache=0x1008), dict(w=0x1002), dict(pos=0x1002), dict(slots=0x1001), dict(cs=0x1002),
    dict(w=0x1000, eps=float("nan")), dict(w=0x1000, eps=-1.0)])
def test_the_library_refuses(lib, kw):
    assert _c(lib, **kw) == 1
    assert lib.sparse_mla_last_error().decode()


def test_no_tokens_is_a_noop(lib):
    assert _c(lib, T=0, kv=0, pos=0, slots=0, cs=0, cache=0) == 0


def _args(T=3, stride=576):
    return [_d((T, stride), torch.bfloat16), _d((T,), torch.int32), _d((T,), torch.int32), _d((50, 576), torch.bfloat16),
            _d((20, 64), torch.float32)]


def test_marshalling(fake):
    kv, pos, slots, cache, table = _args()
    w = _d((512,), torch.bfloat16)
    assert smla.sparse_mla_append(kv, pos, slots, cache, table, norm_weight=w, eps=1e-5, interleaved=False) is cache
    assert fake.lib.calls == [("sparse_mla_append", (kv.data_ptr(), 576, pos.data_ptr(), slots.data_ptr(), 3, table.data_ptr(),
                                                     20, 0, w.data_ptr(), 1e-5, cache.data_ptr(), 50, 0, STREAM))]
    assert fake.entered == [CUDA0]
    fp8 = _d((50, 656), torch.uint8)
    smla.sparse_mla_append(kv, pos, slots, fp8, table, kv_format="fp8")
    assert fake.lib.calls[1][1][7:13] == (1, None, 1e-6, fp8.data_ptr(), 50, 1)


@pytest.mark.parametrize("i,bad", [
    (0, _d((3, 512), torch.bfloat16)), (0, _d((3, 576), torch.float16)), (0, torch.zeros(3, 576, dtype=torch.bfloat16)),
    (0, _d((3, 576), torch.bfloat16, 1)), (1, _d((2,), torch.int32)), (1, _d((3,), torch.int64)), (2, _d((4,), torch.int32)),
    (2, _d((3,), torch.int64)), (2, _d((3,), torch.int32, 1)), (3, _d((50, 656), torch.uint8)), (3, _d((50, 576), torch.float32)),
    (4, _d((20, 32), torch.float32)), (4, _d((20, 64), torch.bfloat16))])
def test_the_wrapper_refuses(fake, i, bad):
    a = _args()
    a[i] = bad
    with pytest.raises(ValueError):
        smla.sparse_mla_append(*a)
    assert fake.lib.calls == []


def test_the_wrapper_refuses_rows_that_overlap_or_are_spread(fake):
    _, pos, slots, cache, table = _args()
    base = torch.zeros(10000, dtype=torch.bfloat16)
    for stride in ((0, 1), (580, 1), (568, 1), (1152, 2)):
        kv = _d((1,), torch.bfloat16)
        kv._t = torch.as_strided(base, (3, 576), stride)
        with pytest.raises(ValueError, match="rows"):
            smla.sparse_mla_append(kv, pos, slots, cache, table)
    assert fake.lib.calls == []
