"""Tensors that a wrapper allocates for a call on another stream than the current one: they belong to
the call's stream, so that the call does not write a block which the current stream's pending work still
reads, and their use by the current stream is recorded, so that dropping them there hands their block to
nobody too early."""

from types import SimpleNamespace

import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import step_reference as ref
from tests.step_reference import CUDA0, STREAM, _d, base_fake, fake  # noqa: F401
from token_sparse_mla_gb300 import _binding

DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


# ----------------------------------------------------------------------------- CPU: where they are allocated

@pytest.fixture
def allocations(fake, monkeypatch):
    """[(stream handle, shape, handles recorded)] of what the wrappers allocate."""
    active, made = [STREAM], []

    class _On:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            active.append(self.s.cuda_stream)

        def __exit__(self, *exc):
            active.pop()
            return False

    def empty(shape, *, dtype, device):
        assert device == CUDA0
        t, recorded = _d(shape, dtype), []
        t.record_stream = lambda s: recorded.append(s.cuda_stream)
        made.append((active[-1], tuple(shape), recorded))
        return t

    monkeypatch.setattr(torch.cuda, "stream", _On)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: SimpleNamespace(cuda_stream=h, device=device))
    fake.lib.sparse_mla_prefix_workspace_bytes = lambda *a: 1024
    monkeypatch.setattr(_binding.torch, "empty", empty)
    return made


def _calls():
    T, h = 3, 8
    q, kv, idx = _d((T, h, 576), BF), _d((100, 576), BF), _d((T, 64), I32)
    pos, table = _d((T,), I32), _d((20, 64), F32)
    return {
        "fwd": (lambda **k: smla.sparse_mla_fwd(q, kv, idx, 0.1, **k), 2, 0),
        "merge": (lambda **k: smla.sparse_mla_merge(_d((2, T, h, 512), BF), _d((2, T, h), F32), **k), 2, 0),
        "v_up": (lambda **k: smla.sparse_mla_v_up(_d((T, h, 512), BF), _d((h, 128, 512), BF), **k), 1, 0),
        "topk": (lambda **k: smla.sparse_mla_topk(_d((T, 100), F32), _d((T,), I32), 8, **k), 1, 0),
        "scatter_mask": (lambda **k: smla.sparse_mla_scatter_mask(idx, 100, **k), 1, 0),
        "masked_mha": (lambda **k: smla.sparse_mla_masked_mha(_d((T, h, 192), BF), _d((40, h, 192), BF), _d((40, h, 128), BF),
                                                              _d((T, 2), I32), 0.1, **k), 2, 0),
        "q_up": (lambda **k: smla.sparse_mla_q_up(_d((T, h, 192), BF), _d((h, 128, 512), BF), pos, table, **k), 1, 0),
        "prefix": (lambda **k: smla.sparse_mla_prefix(q, kv, _d((2,), I32), 100, **k), 2, 1),
    }


@pytest.mark.parametrize("name", list(_calls()))
@pytest.mark.parametrize("given,on", [(SimpleNamespace(device=CUDA0, cuda_stream=0x77E0), 0x77E0), (0x77E0, 0x77E0), (0, 0), (1, 0)])
def test_what_a_call_on_another_stream_allocates(allocations, fake, name, given, on):
    call, results, scratch = _calls()[name]
    call(stream=given)
    assert [s for s, _, _ in allocations] == [on] * (results + scratch)
    assert [r for _, _, r in allocations] == [[STREAM]] * results + [[]] * scratch
    assert fake.lib.calls[-1][1][-1] == getattr(given, "cuda_stream", given)


@pytest.mark.parametrize("name", list(_calls()))
@pytest.mark.parametrize("given", [None, STREAM, SimpleNamespace(device=CUDA0, cuda_stream=STREAM)])
def test_what_a_call_on_the_current_stream_allocates(allocations, name, given):
    call, results, scratch = _calls()[name]
    call(stream=given)
    assert [(s, r) for s, _, r in allocations] == [(STREAM, [])] * (results + scratch)


# ----------------------------------------------------------------------------- GPU

def _prefix_case():
    g = torch.Generator().manual_seed(1)
    q = torch.randn(64, 16, 576, generator=g).to(BF).to(DEV)
    kv = (torch.randn(6 * 64, 576, generator=g) * 0.5).to(BF).to(DEV)
    pages = torch.randperm(6, generator=g).int().to(DEV)
    return lambda x, **k: smla.sparse_mla_prefix(x, kv, pages, 330, **k)[0], q


def _q_up_case():
    g = torch.Generator().manual_seed(2)
    q = torch.randn(300, 8, 192, generator=g).to(BF).to(DEV)
    w = torch.randn(8, 128, 512, generator=g).to(BF).to(DEV)
    pos, table = torch.randint(0, 50, (300,), generator=g).int().to(DEV), ref.cos_sin_table(50).to(DEV)
    return lambda x, **k: smla.sparse_mla_q_up(x, w, pos, table, **k), q


@pytest.mark.gpu
@pytest.mark.parametrize("case", [_prefix_case, _q_up_case])
def test_gpu_a_call_on_another_stream_spares_what_the_current_one_still_reads(case):
    call, q = case()
    want = call(q)
    side = torch.cuda.Stream()
    call(q, stream=side)
    torch.cuda.synchronize()
    held = torch.full_like(want, 3.0)  # of the result's size, and dropped while a copy of it is pending
    torch.cuda._sleep(100_000_000)
    copy = held.clone()
    del held
    got = call(q, stream=side)
    side.synchronize()
    assert torch.equal(got.to("cpu"), want.to("cpu"))
    torch.cuda.synchronize()
    assert copy.eq(3.0).all()
    smla.sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("case", [_prefix_case, _q_up_case])
def test_gpu_a_result_dropped_while_the_current_stream_reads_it(case):
    call, q = case()
    other = q.flip(0).contiguous()
    want = call(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    copy = got.clone()
    del got
    last = [call(other, stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
    assert all(torch.equal(x, call(other)) for x in last)
    smla.sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("case", [_prefix_case, _q_up_case])
@pytest.mark.parametrize("handle", [0, 1])
def test_gpu_the_default_stream_by_handle(case, handle):
    """Raw handles of the default stream while another stream is current."""
    call, q = case()
    want = call(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(q, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    smla.sync_status()
