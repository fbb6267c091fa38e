"""sparse_mla_q_up: the queries in the cache's space.

Tolerance: fp32 accumulation of dn products (each exact in fp32; the tensor cores' sum is off by at
most dn * 2^-23 of the absolute sum), one bf16 rounding of the result (2^-8 relative); rotated dims:
two fp32 products and a sum, one bf16 rounding.
"""

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import step_reference as ref
from tests.step_reference import CUDA0, STREAM, _d, base_fake, fake  # noqa: F401

DEV = "cuda:0"


def _case(T, h, dn, seed, max_pos=500):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(T, h, dn + 64, generator=g)).to(torch.bfloat16)
    w = (torch.randn(h, dn, 512, generator=g) * dn ** -0.5).to(torch.bfloat16)
    pos = torch.randint(0, max_pos, (T,), generator=g).int()
    return q, w, pos, ref.cos_sin_table(max_pos)


def _check(got, q, w, pos, table, interleaved):
    want = ref.q_up(q, w, pos, table, interleaved)
    dn = w.shape[1]
    absum = np.einsum("thd,hdn->thn", np.abs(ref.to64(q)[:, :, :dn]), np.abs(ref.to64(w)))
    got = ref.to64(got)
    tol = 2.0 ** -8 * np.abs(want[:, :, :512]) * (1 + 2.0 ** -10) + dn * 2.0 ** -23 * absum
    assert np.all(np.abs(got[:, :, :512] - want[:, :, :512]) <= tol)
    x = np.abs(ref.to64(q)[:, :, dn:])
    other = x.reshape(*x.shape[:2], 32, 2)[..., ::-1].reshape(x.shape) if interleaved else np.roll(x, 32, axis=-1)
    tol = 2.0 ** -8 * np.abs(want[:, :, 512:]) * (1 + 2.0 ** -10) + 4 * 2.0 ** -24 * (x + other)
    assert np.all(np.abs(got[:, :, 512:] - want[:, :, 512:]) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("T,h,dn,interleaved", [(1, 8, 128, True), (32, 8, 128, False), (127, 3, 192, True), (129, 1, 256, False),
                                                (300, 16, 192, False), (1025, 2, 128, True), (2000, 1, 256, True),
                                                (5, 64, 192, True), (700, 40, 128, True)])
def test_gpu_matches_the_definition(T, h, dn, interleaved):
    q, w, pos, table = _case(T, h, dn, T + dn)
    guard = torch.full((T + 2, h, 576), 3.5, dtype=torch.bfloat16, device=DEV)
    out = smla.sparse_mla_q_up(q.to(DEV), w.to(DEV), pos.to(DEV), table.to(DEV), interleaved=interleaved, out=guard[1:T + 1])
    smla.sync_status()
    _check(out.cpu(), q, w, pos, table, interleaved)
    assert guard[0].eq(3.5).all() and guard[T + 1].eq(3.5).all()


@pytest.mark.gpu
def test_gpu_identity_weights_are_exact():
    T, h, dn = 200, 4, 128
    q, w, pos, table = _case(T, h, dn, 3)
    w.zero_()
    for d in range(dn):
        w[:, d, 4 * d] = 1.0
    out = smla.sparse_mla_q_up(q.to(DEV), w.to(DEV), pos.to(DEV), table.to(DEV)).cpu()
    smla.sync_status()
    assert torch.equal(out[:, :, 0:512:4], q[:, :, :dn])
    assert out[:, :, 1:512:4].eq(0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("value,reported", [(-1, False), (500, True), (-2, True), (2 ** 31 - 1, True)])
def test_gpu_positions_out_of_range(value, reported):
    q, w, pos, table = _case(140, 8, 128, 5)
    pos[3], pos[133] = value, value
    out = smla.sparse_mla_q_up(q.to(DEV), w.to(DEV), pos.to(DEV), table.to(DEV)).cpu()
    if reported:
        with pytest.raises(smla.SparseMLAError) as e:
            smla.sync_status()
        assert e.value.status == 5
    smla.sync_status()
    assert out[3, :, 512:].eq(0).all() and out[133, :, 512:].eq(0).all()
    _check(out, q, w, pos, table, True)


@pytest.mark.gpu
def test_gpu_captured_and_on_another_stream():
    q, w, pos, table = _case(150, 8, 192, 7)
    d = [x.to(DEV) for x in (q, w, pos, table)]
    want = smla.sparse_mla_q_up(*d)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    smla.sparse_mla_q_up(*d, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = smla.sparse_mla_q_up(*d)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap, want)
    d[0].copy_(d[0].flip(0))  # the replay reads what the buffers hold then
    graph.replay()
    again = smla.sparse_mla_q_up(*d)
    smla.sync_status()
    assert torch.equal(cap, again) and not torch.equal(cap, want)


# ----------------------------------------------------------------------------- refusals (CPU)

@pytest.fixture(scope="module")
def lib():
    return smla.library()


def _c(lib, **kw):
    a = dict(q=0x1000, w=0x1000, pos=0x1000, T=4, h=8, dn=128, cs=0x1000, max_pos=10, out=0x1000)
    a.update(kw)
    return lib.sparse_mla_q_up(a["q"], a["w"], a["pos"], a["T"], a["h"], a["dn"], a["cs"], a["max_pos"], 1, a["out"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), 1), (dict(w=0), 1), (dict(pos=0), 1), (dict(cs=0), 1), (dict(out=0), 1), (dict(T=-1), 1), (dict(h=0), 1),
    (dict(dn=64), 2), (dict(dn=512), 2), (dict(max_pos=0), 1), (dict(q=0x1008), 1), (dict(w=0x1002), 1), (dict(out=0x1004), 1),
    (dict(pos=0x1002), 1), (dict(cs=0x1001), 1), (dict(T=1 << 30), 1)])
def test_the_library_refuses(lib, kw, status):
    assert _c(lib, **kw) == status
    assert lib.sparse_mla_last_error().decode()


def test_no_tokens_is_a_noop(lib):
    assert _c(lib, T=0, q=0, w=0, pos=0, cs=0, out=0) == 0


def _args(T=3, h=8, dn=128):
    return [_d((T, h, dn + 64), torch.bfloat16), _d((h, dn, 512), torch.bfloat16), _d((T,), torch.int32),
            _d((20, 64), torch.float32)]


def test_marshalling(fake):
    q, w, pos, table = _args()
    out = _d((3, 8, 576), torch.bfloat16)
    assert smla.sparse_mla_q_up(q, w, pos, table, interleaved=False, out=out) is out
    assert fake.lib.calls == [("sparse_mla_q_up", (q.data_ptr(), w.data_ptr(), pos.data_ptr(), 3, 8, 128, table.data_ptr(), 20, 0,
                                                   out.data_ptr(), STREAM))]
    assert fake.entered == [CUDA0]


@pytest.mark.parametrize("i,bad", [
    (0, _d((3, 8, 256), torch.bfloat16)), (0, _d((3, 8, 192), torch.float16)), (0, torch.zeros(3, 8, 192, dtype=torch.bfloat16)),
    (1, _d((8, 512, 128), torch.bfloat16)), (1, _d((8, 128, 512), torch.bfloat16, 1)), (2, _d((4,), torch.int32)),
    (2, _d((3,), torch.int64)), (3, _d((20, 64), torch.float64)), (3, _d((64, 20), torch.float32))])
def test_the_wrapper_refuses(fake, i, bad):
    a = _args()
    a[i] = bad
    with pytest.raises(ValueError):
        smla.sparse_mla_q_up(*a)
    assert fake.lib.calls == []


@pytest.mark.parametrize("bad", [_d((3, 8, 512), torch.bfloat16), _d((3, 8, 576), torch.float32), _d((3, 8, 576), torch.bfloat16, 1),
                                 torch.zeros(3, 8, 576, dtype=torch.bfloat16)])
def test_the_wrapper_refuses_out(fake, bad):
    with pytest.raises(ValueError):
        smla.sparse_mla_q_up(*_args(), out=bad)
    assert fake.lib.calls == []
